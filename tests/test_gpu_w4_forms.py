"""The forms of the 4-bit products, each over sizes of its own and of the others, and at the ends of
their ranges. Bounds as in test_gpu_w4 (they hold for every form: what a row or a column brought to
16 bits by a power of two loses is below 2^-35 of its largest value, far under an fp32 sum's steps).
"""

import threading

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_w4 import PRODUCTS, built, call, case, check, want, weights  # noqa: F401

pytestmark = pytest.mark.gpu
WIDE, STREAM, SIMT, ANY = 0, 1, 3, -1


@pytest.fixture(params=[WIDE, STREAM, SIMT], ids=["wide", "stream", "simt"])
def form(request):
    pgg.pgg_debug_force_variant(request.param)
    yield request.param
    pgg.pgg_debug_force_variant(ANY)


@pytest.mark.parametrize("product", PRODUCTS)
@pytest.mark.parametrize("T,G,top_k,K,N,group,zeros,scales", [
    (1, 1, 1, 128, 64, 128, False, "bf16"),
    (3, 9, 4, 384, 96, 128, True, "bf16"),      # an odd number of groups
    (40, 3, 2, 640, 200, 128, False, "bf16"),
    (33, 4, 1, 1152, 130, 384, True, "fp32"),
    (70, 2, 2, 224, 33, 32, False, "bf16"),
    (130, 2, 1, 320, 64, 64, True, "bf16"),
    (170, 1, 1, 256, 129, 64, False, "fp32"),
    (500, 3, 2, 512, 72, 32, True, "fp32")])
def test_every_form(form, product, T, G, top_k, K, N, group, zeros, scales):
    check(case(product, T=T, G=G, top_k=top_k, K=K, N=N, group=group, zeros=zeros, scales=scales,
               seed=K + T))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype,scales", [("fp16", "fp16"), ("bf16", "fp32")])
def test_every_form_types(form, dtype, scales, zeros):
    check(case("gated", T=90, G=2, K=384, N=96, group=128, dtype=dtype, scales=scales, zeros=zeros))


def test_zeros_of_eight_bits(form):
    s = case("rows", T=60, G=2, K=512, N=96, group=64)
    s["zeros"] = torch.randint(0, 256, s["zeros"].shape, device="cuda", dtype=torch.uint8)
    s["zeros"].view(-1)[:2] = torch.tensor([0, 255], device="cuda", dtype=torch.uint8)
    check(s)


@pytest.mark.parametrize("zeros", [False, True])
def test_rows_and_columns_of_any_size(form, zeros):
    """Rows of 2^100 beside rows of 2^-100 and of zeros, columns of 2^-60 beside 2^20."""
    s = case("rows", T=48, G=3, K=512, N=128, group=128, zeros=zeros, out="fp32", scales="fp32")
    e = torch.randint(-100, 60, (48, 1), device="cuda")
    e[:3, 0] = torch.tensor([100, -100, 0], device="cuda")
    s["x"] = torch.ldexp(s["x"].float(), e).bfloat16()
    s["x"][2] = 0
    e = torch.randint(-60, 20, (3, 128, 1), device="cuda")
    s["scales"] = torch.ldexp(s["scales"], e)
    s["scales"][0, 0] = 0
    got, ws = call(s)
    y, bound = want(s)
    # the smallest results are subnormal: each of a sum's K products and K additions is rounded to a
    # multiple of 2^-149 there, off by half of that
    assert pgg.status(ws) == 0 and bool(((got.double() - y).abs() <= bound + 512 * 2.0 ** -149).all())


def test_groups_of_different_size_in_a_column(form):
    s = case("gated", T=48, G=3, K=512, N=128, group=64, zeros=False)
    e = torch.randint(-12, 3, s["scales"].shape, device="cuda")
    s["scales"] = torch.ldexp(s["scales"].float(), e).bfloat16()
    check(s)


@pytest.mark.parametrize("zeros,scales,group", [(False, "bf16", 128), (True, "bf16", 128),
                                                (False, "fp32", 128), (False, "bf16", 64),
                                                (True, "fp32", 32)])
@pytest.mark.parametrize("rows", [8, 60])
def test_weights_beyond_the_cache(rows, zeros, scales, group):
    """Codes and scales that come from memory, late and out of order: the same bits each time, and
    three experts' rows against 64 bits."""
    s = case("gated", T=rows * 16, G=32, top_k=2, K=7168, N=1024, group=group, zeros=zeros,
             scales=scales)
    got, ws = call(s)
    assert pgg.status(ws) == 0
    for _ in range(8):
        assert torch.equal(call(s)[0], got)
    for g in (0, 13, 31):
        own = s["pick"] == g
        one = dict(s, G=1, codes=s["codes"][g:g + 1], scales=s["scales"][g:g + 1],
                   zeros=s["zeros"][g:g + 1] if zeros else None)
        w = weights(one)[0]
        x = s["x"].double()[s["gather"][own] // 2]
        y, e = x @ w.T, (x.abs() @ w.abs().T) * (7168 + 8) * 2.0 ** -23
        gate, up, eg, eu = y[:, :1024], y[:, 1024:], e[:, :1024], e[:, 1024:]
        p = s["probs"].double().reshape(-1)[s["gather"]][own][:, None]
        act = torch.nn.functional.silu(gate)
        y = p * act * up
        e = p * (1.1 * eg * up.abs() + act.abs() * eu + 1.1 * eg * eu) + 2.0 ** -19 * y.abs()
        half = 2.0 ** -8
        over = (got[own].double() - y).abs() - (e * (1 + half) + half * y.abs() + 1e-38)
        assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("product", PRODUCTS)
def test_two_sizes_in_one_workspace(product):
    """Calls of different sizes and forms one after the other in a workspace that fits both."""
    many, few = case(product, T=300, G=3, K=512, N=192, group=128), \
        case(product, T=2, G=3, K=256, N=64, group=64, zeros=False, seed=1)
    a, ws = call(many)
    b, other = call(few)
    ws = max(ws, other, key=len)
    for _ in range(3):
        assert torch.equal(call(few, workspace=ws)[0], b)
        assert torch.equal(call(many, workspace=ws)[0], a)


def test_threads():
    """Calls from several threads, each on its own stream."""
    cases = [case(p, T=t, G=4, K=512, N=128, group=128, seed=i)
             for i, (p, t) in enumerate((("rows", 8), ("gated", 90), ("combined", 1), ("gated", 1)))]
    want = [call(s)[0] for s in cases]
    torch.cuda.synchronize()
    wrong = []

    def run(s, y):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                if not torch.equal(call(s)[0], y):
                    wrong.append(s["product"])

    threads = [threading.Thread(target=run, args=p) for p in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
