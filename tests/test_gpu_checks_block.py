"""The 4-bit products, the norms around a block and the clipping in the checked build (see
test_gpu_checks): every index that the products read from the routing tables lies within its bounds,
in each form, and the results are those of the other tests. The norms and the clipping read no tables
but the launch's own; they run here for the build's other differences."""

import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, os, sys
sys.path[:0] = [sys.argv[1], os.path.join(sys.argv[1], "tests")]
import torch
import permute_grouped_gemm_gb300 as pgg
from permute_grouped_gemm_gb300 import build as pbuild

pgg.load(pbuild.LIB_CHECKS)
import test_gpu_block_norm as norm
import test_gpu_clip as clip
import test_gpu_w4 as w4

res = {}
for name, variant in (("wide", 0), ("stream", 1), ("simt", 3)):
    for product in w4.PRODUCTS:
        pgg.pgg_debug_force_variant(variant)
        try:
            # ragged groups, an expert without a row, blocks that are not full
            s = w4.case(product, T=150, G=4, counts=(0, 140, 1, 159), K=544, N=200, group=32, rit=1)
            w4.check(s)
            x = s["x"].clone()
            x[7, 3], x[9] = float("inf"), float("nan")  # (rows that another function writes)
            _, ws = w4.call(dict(s, x=x))
            res[name + "-" + product] = pgg.status(ws)
        finally:
            pgg.pgg_debug_force_variant(-1)
for gate in ("channel", "full"):
    for H in (512, 77, 9000):
        s = norm.case(T=400, H=H, post="layer", pre="layer", gate=gate)
        norm.check_forward(s)
        norm.check_backward(s)
clip.check(clip.grads_of([40000, 1, 0, 16385, 333]), 0.5)
torch.cuda.synchronize()
print(json.dumps(res))
"""


@pytest.fixture(scope="module")
def results():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build(checks=True)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True,
                       timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("product", ["rows", "gated", "combined"])
@pytest.mark.parametrize("form", ["wide", "stream", "simt"])
def test_checked_build_runs_clean(results, form, product):
    assert results[f"{form}-{product}"] == 0
