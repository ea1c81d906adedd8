"""GPU parity of the router and its gradient against plain 64-bit formulas.

The choice and the order are compared exactly: the reference sorts the same
fp32 sums logit + bias, lowest index first among equals. Weights are fp32: the
exponent's argument carries |l - m| * 2^-24 (at most about 50 * 6e-8 here), the
exponential, sum and quotient a few units more, so 1e-5 relative. Gradients:
the same times the terms of the sum, 1e-5 of the row's largest |ds| * s,
plus the dtype's rounding.
"""

import numpy as np
import pytest
import torch

import permute_grouped_gemm_gb300 as pgg

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def reference(logits, k, rit, bias, score, renormalize, scale):
    key = logits.float().cpu().numpy()
    if bias is not None:
        key = key + bias.cpu().numpy()
    key = np.where(np.isnan(key), -np.inf, key) if not np.isnan(key).any() else key
    # NaN below -inf, +0 and -0 equal: sort by (is NaN, -key), stable
    chosen = np.stack([np.lexsort((np.arange(key.shape[1]), -np.nan_to_num(r, nan=0.0, posinf=np.inf,
                                                                           neginf=-np.inf),
                                   np.isnan(r)))[:k] for r in key])
    z = logits.double().cpu().numpy()
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = z.max(1, keepdims=True)
            s = np.where(np.isneginf(z), 0.0, np.exp(z - m))
            total = s.sum(1, keepdims=True)
            s = np.where(total == 0, 0.0, s / total)
        else:
            s = 1 / (1 + np.exp(-z))
        p = np.take_along_axis(s, chosen, 1)
        if renormalize:
            t = p.sum(1, keepdims=True)
            p = np.where(t == 0, 0.0, p / t)
    flat = chosen.reshape(-1)
    gather = np.argsort(flat, kind="stable")
    idx = gather if rit == 0 else np.argsort(gather)
    return p * scale, chosen, idx, np.bincount(flat, minlength=logits.shape[1])


def check(logits, k, rit=0, bias=None, score="softmax", renormalize=True, scale=1.0):
    probs, experts, idx, groups, ws = pgg.route(logits, k, rit, bias=bias, score=score,
                                                renormalize=renormalize, scale=scale)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    rp, re, ri, rg = reference(logits, k, rit, bias, score, renormalize, scale)
    assert np.array_equal(experts.cpu().numpy(), re)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(groups.cpu().numpy(), rg)
    np.testing.assert_allclose(probs.double().cpu().numpy(), rp, rtol=1e-5, atol=1e-30)
    return probs, experts, idx, groups


def logits_of(t, g, dtype, seed, std=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(t, g, generator=gen, device="cuda") * std).to(DT[dtype])


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True),
                                               ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("t,g,k", [(1, 8, 2), (1, 60, 8), (17, 1, 1), (5, 33, 33 - 1), (256, 64, 8),
                                   (257, 64, 8), (999, 257, 6), (3000, 1024, 12)])
def test_cases(t, g, k, dtype, score, renormalize):
    bias = torch.randn(g, device="cuda") * 0.3 if k % 2 == 0 else None
    check(logits_of(t, g, dtype, t + g), k, rit=k % 3 % 2, bias=bias, score=score,
          renormalize=renormalize, scale=1.0 if k < 8 else 2.5)


def test_ties_go_to_the_lowest_index_and_signed_zeros_are_equal():
    l = torch.zeros(300, 96, device="cuda")
    l[:, ::2] = -0.0
    l[100:200, 50] = 1.0
    check(l, 5)
    check(torch.randint(0, 3, (700, 40), device="cuda").to(torch.bfloat16), 7, rit=1)


def test_masked_experts_and_tokens():
    l = logits_of(400, 24, "fp32", 3)
    l[:, 3:20] = float("-inf")          # seven experts left, eight chosen
    l[7] = float("-inf")                # a token with nothing left
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            p, e, _, _ = check(l, 8, score=score, renormalize=renorm)
            assert not torch.isnan(p).any()
            assert torch.count_nonzero(p[7]) == 0
            assert torch.equal(e[7].cpu(), torch.arange(8))


def test_nan_logits_keep_the_order_valid():
    l = logits_of(300, 20, "fp32", 4)
    l[5, 3] = float("nan")
    l[6] = float("nan")
    l[9, 2] = float("inf")
    probs, experts, idx, groups, ws = pgg.route(l, 4, renormalize=False)
    assert torch.isnan(probs[5]).all() and torch.isnan(probs[6]).all()
    assert torch.isnan(probs[9, 0]) and int(experts[9, 0]) == 2
    assert not (experts[5] == 3).any() and torch.equal(experts[6].cpu(), torch.arange(4))
    assert torch.equal(torch.sort(idx).values.cpu(), torch.arange(1200))
    assert int(groups.sum()) == 1200
    clean = torch.ones(300, dtype=torch.bool)
    clean[[5, 6, 9]] = False
    assert not torch.isnan(probs[clean.cuda()]).any()


def test_repeats_bitwise_and_on_another_stream():
    l = logits_of(20000, 256, "bf16", 5)
    first = pgg.route(l, 8, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = pgg.route(l, 8, 1)
    torch.cuda.synchronize()
    for a, b in zip(first[:4], second[:4]):
        assert torch.equal(a, b)


def test_more_pairs_per_block_than_it_sorts_at_a_time():
    l = logits_of(250000, 40, "bf16", 7)
    probs, experts, idx, groups, _ = pgg.route(l, 6)
    flat = experts.reshape(-1)
    want = torch.sort(flat, stable=True).indices
    assert torch.equal(idx, want)
    assert torch.equal(groups, torch.bincount(flat, minlength=40))
    rows = torch.randperm(250000)[:500].cuda()
    check(l[rows].contiguous(), 6)
    assert torch.equal(experts[rows], torch.sort(l[rows].float(), dim=1, descending=True,
                                                 stable=True).indices[:, :6])


def test_the_order_is_what_the_grouped_products_take():
    l = logits_of(500, 12, "fp32", 6)
    probs, experts, idx, groups, _ = pgg.route(l, 3, 1)
    x = torch.randn(500, 64, device="cuda").bfloat16()
    w = torch.randn(12, 64, 32, device="cuda").bfloat16() * 0.1
    y, ws = pgg.fwd(x, w, idx, groups, 500, 3, 1, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    want = torch.einsum("tk,tjkn->tjn", x.float(), w.float()[experts])
    got = y[idx.reshape(500, 3)]
    assert (got - want).abs().max() <= 1e-4 * want.abs().max()


# ------------------------------------------------------------------ gradient

def grad_reference(dp, logits, experts, score, renormalize, scale):
    """sum over the chosen of d_prob times the Jacobian, in float64."""
    z = logits.double().cpu().requires_grad_()
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    p = s.gather(1, experts.cpu())
    if renormalize:
        p = p / p.sum(1, keepdim=True)
    (g,) = torch.autograd.grad((scale * p * dp.double().cpu()).sum(), z)
    return g


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True),
                                               ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("t,g,k", [(1, 8, 2), (31, 60, 8), (700, 257, 6), (100, 1024, 32)])
def test_gradient(t, g, k, dtype, score, renormalize):
    l = logits_of(t, g, dtype, 10 + t)
    _, experts, _, _, _ = pgg.route(l, k, score=score)
    dp = torch.randn(t, k, device="cuda")
    got = pgg.route_grad(dp, l, experts, score=score, renormalize=renormalize, scale=1.5)
    want = grad_reference(dp, l, experts, score, renormalize, 1.5)
    assert got.dtype == l.dtype
    scale = 1.5 * dp.abs().double().cpu().sum(1, keepdim=True)
    bound = ROUND[l.dtype] * want.abs() + 1e-5 * scale + TINY[l.dtype]
    assert ((got.double().cpu() - want).abs() <= bound).all()


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True),
                                               ("sigmoid", True)])
def test_gradient_against_differences(score, renormalize):
    # central differences of the router's own weights, h = 2^-6: truncation h^2 / 6 * |p'''|
    # (at most about 4e-5 here, |d_prob| <= 1), fp32 weights / h: 6e-8 * 64
    l = logits_of(6, 10, "fp32", 12, std=1.0)
    k, h = 3, 2.0 ** -6
    _, experts, _, _, _ = pgg.route(l, k, score=score, renormalize=renormalize)
    dp = torch.rand(6, k, device="cuda") * 2 - 1
    got = pgg.route_grad(dp, l, experts, score=score, renormalize=renormalize)

    def weights(z):  # of the same experts: a bias far above the logits holds the choice
        out = torch.empty(6, k, device="cuda")
        for t in range(6):
            bias = torch.full((10,), -100.0, device="cuda")
            bias[experts[t]] = 100.0 - 10 * torch.arange(k, device="cuda", dtype=torch.float32)
            out[t] = pgg.route(z[t:t + 1].contiguous(), k, bias=bias, score=score,
                               renormalize=renormalize)[0][0]
        return out

    for e in range(10):
        up, down = l.clone(), l.clone()
        up[:, e] += h
        down[:, e] -= h
        num = ((weights(up) - weights(down)).double() * dp.double()).sum(1) / (2 * h)
        assert (num - got[:, e].double()).abs().max() < 5e-4


def test_gradient_of_masked_rows_is_zero_and_bad_choices_are_nan():
    l = logits_of(8, 16, "fp32", 13)
    l[2] = float("-inf")
    l[3, 1:] = float("-inf")
    experts = torch.arange(4, device="cuda").repeat(8, 1)
    experts[5, 1] = 16
    experts[6] = torch.tensor([1, 2, 1, 3])
    dp = torch.randn(8, 4, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            g = pgg.route_grad(dp, l, experts, score=score, renormalize=renorm)
            assert torch.isnan(g[5]).all() and torch.isnan(g[6]).all()
            assert torch.count_nonzero(g[2]) == 0
            rest = [0, 1, 3, 4, 7]
            assert not torch.isnan(g[rest]).any()
