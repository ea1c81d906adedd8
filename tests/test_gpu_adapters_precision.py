"""The low-rank rows u = scale x a and v = scale d_y b are not rounded to 16 bits on their way into
the second product: every output of a 16-bit call is one rounding of an fp32 result.

With a projection of zeros, y = u b^T, and d_x = v a^T: nothing else hides what u and v lost. Bounds:
half a unit of the output (2^-8 of it in bf16, 2^-11 in fp16); of u and v what their sum of two values
loses, through the products' absolute values: the first is cut off (a unit, 2^-7 and 2^-10), the
second rounds the rest (2^-9 and 2^-12 of a power of two above it): 2^-16, and 2^-20 in fp16, whose
smallest numbers are in the way; fp32
sums of at most 700 terms, 2^-20 of their absolute values, each.
"""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_adapters import ROUND, TINY, expand, inputs, low_rank

pytestmark = pytest.mark.gpu

KEPT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -20}
SUM = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()
    yield
    pgg.pgg_debug_force_variant(-1)


def near(got, ref, inner, sums):
    dt = got.dtype
    bound = ROUND[dt] * ref.abs() + KEPT[dt] * inner + SUM * sums + TINY[dt]
    off = (got.double() - ref).abs()
    assert (off <= bound).all(), (off / bound).max().item()


def case(T, R, dtype, ids, N=72, K=64, A=5):
    s = inputs(T, K, N, R, A, dtype=dtype, ids=ids, seed=R + T)
    s["weight"].zero_()
    return s


# few tokens, the tokens sorted (256 and 257: either side of the rule), several row blocks
@pytest.mark.parametrize("T", [1, 40, 256, 257, 700])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward(T, R, dtype):
    for ids in ("mixed", "runs"):
        s = case(T, R, dtype, ids)
        y, ws = pgg.adapters(**s)
        torch.cuda.synchronize()
        assert pgg.status(ws) == 0
        ad, scale = s["adapter"], s["scale"]
        u = low_rank(s["x"], s["a"], ad, scale)
        sums = low_rank(s["x"].abs(), s["a"].abs(), ad, scale)
        near(y, expand(u, s["b"], ad), expand(u.abs(), s["b"].abs(), ad),
             2 * expand(sums, s["b"].abs(), ad))


# the FP32 pipes: odd widths, and tensors of which one is off a 16-byte boundary
@pytest.mark.parametrize("off", ["widths", "x", "weight", "a", "b", "out", "variant"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward_on_the_pipes(off, dtype):
    s = case(400, 16 if off != "widths" else 15, dtype, "mixed", N=72 if off != "widths" else 71)
    kw = {}
    if off in ("x", "weight", "a", "b", "out"):
        t = s[off] if off != "out" else torch.empty(400, 72, dtype=s["x"].dtype, device="cuda")
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        (kw if off == "out" else s)[off] = buf[1:].view(t.shape)
    if off == "variant":
        pgg.pgg_debug_force_variant(3)
    try:
        y, ws = pgg.adapters(**s, **kw)
    finally:
        pgg.pgg_debug_force_variant(-1)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    ad, scale = s["adapter"], s["scale"]
    u = low_rank(s["x"], s["a"], ad, scale)
    sums = low_rank(s["x"].abs(), s["a"].abs(), ad, scale)
    near(y, expand(u, s["b"], ad), expand(u.abs(), s["b"].abs(), ad),
         2 * expand(sums, s["b"].abs(), ad))


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gradients(R, dtype):
    for T, ids in ((40, "mixed"), (700, "mixed"), (700, "runs")):
        s = case(T, R, dtype, ids)
        d_y = torch.randn(T, 72, device="cuda").to(s["x"].dtype)
        d_x, d_a, d_b, ws = pgg.adapters_grad(d_y, **s)
        torch.cuda.synchronize()
        assert pgg.status(ws) == 0
        ad, scale = s["adapter"], s["scale"]
        u, v = low_rank(s["x"], s["a"], ad, scale), low_rank(d_y, s["b"], ad, scale)
        us = low_rank(s["x"].abs(), s["a"].abs(), ad, scale)
        vs = low_rank(d_y.abs(), s["b"].abs(), ad, scale)
        near(d_x, expand(v, s["a"], ad), expand(v.abs(), s["a"].abs(), ad),
             2 * expand(vs, s["a"].abs(), ad))
        for got, left, right, sums in ((d_a, s["x"].double(), v, vs), (d_b, d_y.double(), u, us)):
            for i in range(5):
                m = ad == i
                near(got[i], left[m].T @ right[m], left[m].abs().T @ right[m].abs(),
                     2 * left[m].abs().T @ sums[m])


def test_infinities_stay_infinities():
    # an infinite u, and an infinite weight behind a finite one, give infinities of the right sign
    for dtype in ("bf16", "fp16"):
        s = case(300, 16, dtype, "mixed")
        on = s["adapter"] >= 0
        big = dict(s, x=torch.full_like(s["x"], 1e3), a=torch.full_like(s["a"], 1e3),
                   b=torch.ones_like(s["b"]))
        if dtype == "bf16":
            big["scale"] = torch.full((5,), 1e38, device="cuda")
        y, _ = pgg.adapters(**big)
        assert (y[on] == float("inf")).all() and not y[~on].any()
        b = s["b"].clone()
        b[:, 3, 5] = float("inf")
        y, _ = pgg.adapters(**dict(s, b=b))
        u = low_rank(s["x"], s["a"], s["adapter"], s["scale"])
        assert torch.equal(y[on, 3].double(), torch.sign(u[on, 5]) * float("inf"))
        y2, _ = pgg.adapters(**s)
        rest = torch.arange(72, device="cuda") != 3
        assert torch.equal(y[:, rest], y2[:, rest]) and not y[~on].any()
        # values that 16 bits hold exactly are split too
        x = torch.zeros_like(s["x"])
        x[:, 0] = 1.0
        a = torch.zeros_like(s["a"])
        a[:, 0, 5] = torch.tensor([1.0, 2.0, -1.0, 0.5, 3.0], device="cuda")
        y, _ = pgg.adapters(**dict(s, x=x, a=a, b=b, scale=None))
        want = torch.sign(a[s["adapter"][on], 0, 5]) * float("inf")
        assert torch.equal(y[on, 3], want)
        y, _ = pgg.adapters(**dict(s, x=x, a=a, scale=None))
        exact = a[s["adapter"][on], 0, 5][:, None].float() * s["b"][s["adapter"][on], :, 5].float()
        assert torch.equal(y[on], exact.to(y.dtype))
