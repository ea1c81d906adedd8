"""What the source of the 4-bit products for many rows has to keep that no run can show without a wait
that does not end: the warpgroups ask for no more registers than a block is launched with."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "permute_grouped_gemm_gb300", "csrc")
TEXT = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "w4_wide.cu")).read())


def number(name):
    return int(re.search(r"\b%s = (\d+)" % name, TEXT).group(1))


def test_register_shares():
    warpgroups = int(re.search(r"kThreads = (\d+) \* 128", TEXT).group(1))
    shares = [number("kFewRegs")] + 2 * [number("kUnpackRegs")] + 2 * [number("kWriteRegs")]
    assert len(shares) == warpgroups and all(r % 8 == 0 and 24 <= r <= 256 for r in shares)
    assert sum(shares) <= warpgroups * number("kLaunchRegs")
    # every warpgroup takes one of them, and the kernel has at least kLaunchRegs where it is launched
    assert sorted(re.findall(r"(?:fewer|more)_registers<(\w+)>\(\)", TEXT)) == [
        "kFewRegs", "kUnpackRegs", "kWriteRegs"]
    launch = TEXT[TEXT.index("auto kern = w4_wide_kernel<U, SPLIT>"):]
    check = launch.index("if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;")
    assert check < launch.index("launch_pdl(kern")
