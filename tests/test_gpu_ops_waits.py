"""Bounded waits, the checked build and the example that runs the router, the
gated product and the adapters together.

A withheld accumulator release makes a kernel's wait run out: it reports
PGG_ERR_TIMEOUT and the next call on the same context is correct.
"""

import json
import os
import subprocess
import sys

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from workloads import make_case
from workloads.moe import forward_input

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pbuild.build(checks=True)
    pgg.load()
    yield
    pgg.pgg_debug_force_variant(-1)


def runs_out_then_works(call):
    good, ws = call()
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    pgg.pgg_debug_set_wait_limit_ns(20_000_000)
    pgg.pgg_debug_set_hold_release(1)
    try:
        _, ws = call()
        torch.cuda.synchronize()
        assert pgg.STATUS[pgg.status(ws)] == "PGG_ERR_TIMEOUT"
    finally:
        pgg.pgg_debug_set_hold_release(0)
        pgg.pgg_debug_set_wait_limit_ns(0)
    again, ws = call()
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    assert torch.equal(again.view(torch.int16), good.view(torch.int16))


# (tokens, experts, K, F): more than two tiles for every CTA or pair; the wide product in tiles of
# 256 and of 512 columns, the few-row one alone and with K split over a cluster
@pytest.mark.parametrize("variant,tokens,G,K,F", [(0, 6000, 8, 1024, 1024), (0, 6000, 8, 4096, 1024),
                                                  (1, 300, 64, 256, 1024), (1, 4, 16, 7168, 1152)])
def test_gated_product(variant, tokens, G, K, F):
    inp = make_case(batch=tokens, top_k=4, G=G, K=K, N=2 * F, dtype="bf16", seed=71, device="cuda",
                    w_std=K ** -0.5)
    x = forward_input(inp)

    def call():
        pgg.pgg_debug_force_variant(variant)
        try:
            h, _, ws = pgg.swiglu(x, inp.weight, inp.expanded_row_idx, inp.group_list, tokens, 4, 0)
        finally:
            pgg.pgg_debug_force_variant(-1)
        return h, ws

    runs_out_then_works(call)


def adapter_inputs(T, K, N, R, A):
    gen = torch.Generator(device="cuda").manual_seed(72)
    rnd = lambda *s: (torch.randn(*s, generator=gen, device="cuda") * 0.1).bfloat16()  # noqa: E731
    return (rnd(T, K), rnd(K, N), rnd(A, K, R), rnd(A, N, R),
            torch.randint(-1, A, (T,), generator=gen, device="cuda"))


@pytest.mark.parametrize("T,K,N", [(8000, 256, 4096), (64, 512, 65536)])
def test_projection(T, K, N):
    args = adapter_inputs(T, K, N, 16, 4)
    runs_out_then_works(lambda: pgg.adapters(*args))


def test_factor_gradients():
    args = adapter_inputs(4000, 8192, 8192, 16, 16)
    d_y = torch.randn(4000, 8192, device="cuda").bfloat16()

    def call():
        _, d_a, _, ws = pgg.adapters_grad(d_y, *args, need_x=False)
        return d_a, ws

    runs_out_then_works(call)


CHILD = r"""
import json, sys
sys.path.insert(0, sys.argv[1])
import torch
import permute_grouped_gemm_gb300 as pgg
from permute_grouped_gemm_gb300 import build as pbuild
from workloads import make_case
from workloads.moe import forward_input

pgg.load(pbuild.LIB_CHECKS)
res = {}

def gated(name, variant, **kw):
    inp = make_case(device="cuda", dtype="bf16", **kw)
    x = forward_input(inp)
    pgg.pgg_debug_force_variant(variant)
    h, gu, ws = pgg.swiglu(x, inp.weight, inp.expanded_row_idx, inp.group_list, inp.batch,
                           inp.top_k, 0, keep=True)
    d, _, _, ws2 = pgg.swiglu_grad(h, gu, inp.expanded_row_idx, inp.top_k, 0)
    torch.cuda.synchronize()
    pgg.pgg_debug_force_variant(-1)
    F = h.shape[1]
    want = torch.nn.functional.silu(gu[:, :F].float()) * gu[:, F:].float()
    res[name] = [pgg.status(ws), pgg.status(ws2), float((h.float() - want).abs().max() / want.abs().max())]

gated("wide", 0, batch=900, top_k=4, G=7, K=400, N=320, seed=81)
gated("few", 1, batch=60, top_k=4, G=7, K=400, N=320, seed=82)
gated("pipes", 3, batch=90, top_k=4, G=7, K=100, N=58, seed=83)
for T in (30, 900):
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: (torch.randn(*s, generator=gen, device="cuda") * 0.1).bfloat16()
    x, w, a, b = rnd(T, 200), rnd(200, 136), rnd(4, 200, 16), rnd(4, 136, 16)
    ad = torch.randint(-1, 4, (T,), generator=gen, device="cuda")
    y, ws = pgg.adapters(x, w, a, b, ad)
    dx, da, db, ws2 = pgg.adapters_grad(y, x, w, a, b, ad)
    torch.cuda.synchronize()
    want = x.float() @ w.float()
    for i in range(4):
        want[ad == i] += x[ad == i].float() @ a[i].float() @ b[i].float().T
    res[f"adapters {T}"] = [pgg.status(ws), pgg.status(ws2), float((y.float() - want).abs().max() / want.abs().max())]
print(json.dumps(res))
"""


def test_checked_build_runs_clean():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True,
                       timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(res) == 5
    for name, (status, status2, off) in res.items():
        assert status == 0 and status2 == 0, (name, status, status2)
        assert off <= 2e-2, (name, off)


def test_example_runs_and_checks_itself():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_layer.py")],
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert r.stdout.strip().endswith("ok")
