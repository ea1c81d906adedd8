"""Outputs of the clipping that overlap are refused on the host: what one block reads another would
write (no GPU)."""

import pytest

import permute_grouped_gemm_gb300 as pgg
from test_block_host import CLIP, FAKE, built, name  # noqa: F401

A, B, C = FAKE, FAKE + 4096, FAKE + 8192  # 4096 bytes apart
F32, BF16 = pgg.PGG_F32, pgg.PGG_BF16


def call(grads, out, sizes, dtypes=None):
    dtypes = dtypes or [F32] * len(grads)
    return name(pgg.pgg_clip_grads(**dict(CLIP, grads=grads, out=out, sizes=sizes, dtypes=dtypes)))


@pytest.mark.parametrize("grads,out,sizes,dtypes", [
    ([A, A], [A, A], [8, 8], None),                     # one gradient twice, in place
    ([A, B, A], [A, B, A], [8, 8, 4], None),            # its beginning once more
    ([A, A + 16], [A, A + 16], [8, 8], None),           # a view into it
    ([A, B], [C, C], [8, 8], None),                     # one output for two
    ([A, B], [C, C + 12], [4, 4], [F32, BF16]),
    ([A, B], [B, C], [8, 8], None),                     # an output that is another's gradient
    ([A, B], [C, A + 28], [8, 8], None),                # or reaches into it
    ([A], [A + 4], [8], None),                          # or into its own, but for being it
    ([C, A, B], [C, A, B], [8, 1025, 8], None),         # as long as to the next, and one more
])
def test_overlapping_outputs(grads, out, sizes, dtypes):
    assert call(grads, out, sizes, dtypes) == "PGG_ERR_ATTR"


@pytest.mark.parametrize("grads,out,sizes,dtypes", [
    ([A, B], [A, B], [1024, 8], None),                  # next to each other
    ([C, A, B], [C, A, B], [8, 1024, 1024], None),
    ([A, A], [B, C], [1024, 8], None),                  # a gradient read twice, written apart
    ([A, A + 16], [B, C], [8, 8], None),
    ([A, A, 0], [A, A, 0], [8, 0, 0], None),            # nothing of it the second time
    ([A, B], [A, B], [2048, 8], [BF16, F32]),
    ([], [], [], None),
])
def test_what_is_allowed_passes_this_check(grads, out, sizes, dtypes):
    # (without a GPU the call ends where it asks for the device)
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are no tensors")
    assert call(grads, out, sizes, dtypes) == "PGG_ERR_CUDA"
