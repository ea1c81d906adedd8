"""The router's gradient against 64-bit formulas within a bound that knows the scores.

With s the scores and ds = scale * d_prob at the chosen, 0 elsewhere, an fp32 gradient is off by the
errors of its factors: an exponential (2 units of 2^-23, and its argument's |l - m| * 2^-24, below 20
here), the sum over the row and a quotient, relative 3e-6 in all, times each of the terms that are
added up. So, beside the dtype's rounding of the result:

    softmax                s_e (|ds_e| + sum |ds| s)
    softmax, renormalised  scale p_j (|d_prob_j| + sum |d_prob| p)
    sigmoid                |ds_j| s_j (1 - s_j)
    sigmoid, renormalised  scale (|d_prob_j| + sum |d_prob| p) p_j (1 - s_j)
"""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_router import DT, ROUND, TINY, grad_reference, logits_of

pytestmark = pytest.mark.gpu

FP32 = 3e-6
KINDS = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def gradient(dp, logits, experts, score, renormalize, scale):
    """(gradient, sum of its terms' sizes) by the formulas in 64 bits; what is not chosen has none
    unless the softmax is the plain one."""
    z, dp, experts = logits.double().cpu(), dp.double().cpu(), experts.cpu()
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    chosen = s.gather(1, experts)
    p = chosen / chosen.sum(1, keepdim=True)
    if score == "softmax" and not renormalize:
        ds = torch.zeros_like(z).scatter(1, experts, scale * dp)
        return (s * (ds - (ds * s).sum(1, keepdim=True)),
                s * (ds.abs() + (ds.abs() * s).sum(1, keepdim=True)))
    slope = p if score == "softmax" else (p if renormalize else chosen) * (1 - chosen)
    mean = (dp * p).sum(1, keepdim=True) if renormalize else 0.0
    size = (dp.abs() * p).sum(1, keepdim=True) if renormalize else 0.0
    zeros = torch.zeros_like(z)
    return (zeros.scatter(1, experts, scale * slope * (dp - mean)),
            zeros.scatter(1, experts, scale * slope * (dp.abs() + size)))


def check(logits, k, score, renormalize, scale=1.5, out=None):
    experts = pgg.route(logits, k, score=score)[1]
    dp = torch.randn(logits.shape[0], k, device="cuda")
    want, size = gradient(dp, logits, experts, score, renormalize, scale)
    # (the Jacobian by autograd says the same)
    auto = grad_reference(dp, logits, experts, score, renormalize, scale)
    assert (auto - want).abs().max() <= 1e-12 * size.max()
    bound = ROUND[logits.dtype] * want.abs() + TINY[logits.dtype] + FP32 * size
    got = pgg.route_grad(dp, logits, experts, score=score, renormalize=renormalize, scale=scale,
                         out=out)
    off = (got.double().cpu() - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    return experts.cpu(), want, bound


@pytest.mark.parametrize("score,renormalize", KINDS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("t,g,k", [(1, 8, 2), (31, 60, 8), (700, 257, 6), (100, 1024, 32),
                                   (50, 100, 1), (300, 512, 12), (3000, 33, 4)])
def test_gradient(t, g, k, dtype, score, renormalize):
    experts, want, bound = check(logits_of(t, g, dtype, 20 + t), k, score, renormalize)
    if (score, renormalize) == ("softmax", False):
        # the bound tells the unchosen experts' gradients from zero (fp16 has its smallest numbers
        # in the way)
        unchosen = torch.ones_like(want, dtype=torch.bool).scatter(1, experts, False)
        seen = want.abs()[unchosen] > 2 * bound[unchosen]
        assert seen.double().mean() > (0.5 if dtype == "fp16" else 0.99)
    elif k > 1:
        chosen = want.gather(1, experts).abs() > 2 * bound.gather(1, experts)
        assert chosen.double().mean() > (0.5 if dtype == "fp16" else 0.99)


@pytest.mark.parametrize("score,renormalize", KINDS)
@pytest.mark.parametrize("dtype,g", [("fp32", 60), ("bf16", 256), ("fp16", 77)])
def test_in_place(dtype, g, score, renormalize):
    l = logits_of(400, g, dtype, 31)
    experts = pgg.route(l, 6, score=score)[1]
    dp = torch.randn(400, 6, device="cuda")
    want = pgg.route_grad(dp, l, experts, score=score, renormalize=renormalize)
    got = pgg.route_grad(dp, l, experts, score=score, renormalize=renormalize, out=l)
    assert got.data_ptr() == l.data_ptr()
    assert torch.equal(got, want)
