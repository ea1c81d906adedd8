"""The router's choice by score + bias against 64-bit formulas.

A score is an fp32 exponential, a sum and a quotient, at most 1, so its error and that of the sum
with a bias of at most 2 stay below 4e-7 (a few units of 2^-24 each; the softmax's argument carries
|l - m| * 2^-24 more, which the score itself, exp(l - m), makes small: x e^-x < 0.4). Experts whose
64-bit keys differ by more are in the order of the keys; those that differ by less may stand either
way. The weights go by the returned experts: 1e-5 relative, as for the choice by the logits.
"""

import numpy as np
import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_router import DT, logits_of

pytestmark = pytest.mark.gpu

CLOSE = 4e-7
KINDS = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def scores_of(logits, score):
    z = logits.double().cpu().numpy()
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-z))
        s = np.exp(z - z.max(1, keepdims=True))
        return s / s.sum(1, keepdims=True)


def check(logits, k, bias, rit=0, score="softmax", renormalize=True, scale=1.0):
    probs, experts, idx, groups, ws = pgg.route(logits, k, rit, bias=bias, score=score,
                                                renormalize=renormalize, scale=scale,
                                                bias_on="scores")
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    s = scores_of(logits, score)
    key = np.where(np.isneginf(logits.double().cpu().numpy()), -np.inf,
                   s + bias.double().cpu().numpy())
    e = experts.cpu().numpy()
    assert e.min() >= 0 and e.max() < logits.shape[1]
    assert all(len(set(r)) == k for r in e.tolist())
    mine = np.take_along_axis(key, e, 1)
    assert (mine[:, :-1] >= mine[:, 1:] - CLOSE).all()
    rest = key.copy()
    np.put_along_axis(rest, e, -np.inf, 1)
    assert (rest.max(1) <= mine[:, -1] + CLOSE).all()
    p = np.take_along_axis(s, e, 1)
    if renormalize:
        p = p / p.sum(1, keepdims=True)
    np.testing.assert_allclose(probs.double().cpu().numpy(), scale * p, rtol=1e-5, atol=1e-30)
    flat = e.reshape(-1)
    gather = np.argsort(flat, kind="stable")
    assert np.array_equal(idx.cpu().numpy(), gather if rit == 0 else np.argsort(gather))
    assert np.array_equal(groups.cpu().numpy(), np.bincount(flat, minlength=logits.shape[1]))
    return experts


@pytest.mark.parametrize("score,renormalize", KINDS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("t,g,k", [(1, 8, 2), (17, 60, 8), (256, 64, 8), (300, 256, 8),
                                   (3000, 256, 8), (999, 257, 6), (700, 512, 16), (5, 33, 32),
                                   (400, 1024, 32), (40, 7, 7)])
def test_cases(t, g, k, dtype, score, renormalize):
    gen = torch.Generator(device="cuda").manual_seed(t)
    # of the scores' own size, and so large that the scores hardly matter
    for size in (0.05, 1.0):
        bias = (torch.rand(g, generator=gen, device="cuda") * 2 - 1) * size
        check(logits_of(t, g, dtype, t + g), k, bias, rit=t % 2, score=score,
              renormalize=renormalize, scale=1.0 if k < 8 else 2.5)


def test_a_small_bias_moves_the_choice_of_nearly_saturated_scores():
    # sigmoid scores 0.982 + 0.05 and 0.9975: the first is chosen, though its logit is the smaller
    logits = torch.tensor([[4.0, 6.0]], device="cuda").repeat(3, 1)
    bias = torch.tensor([0.05, 0.0], device="cuda")
    by_score = pgg.route(logits, 1, bias=bias, score="sigmoid", bias_on="scores")
    by_logit = pgg.route(logits, 1, bias=bias, score="sigmoid")
    assert not by_score[1].any() and by_logit[1].all()
    p = pgg.route(logits, 1, bias=bias, score="sigmoid", renormalize=False, bias_on="scores")[0]
    np.testing.assert_allclose(p.cpu().numpy(), 1 / (1 + np.exp(-4.0)), rtol=1e-6)


@pytest.mark.parametrize("tokens", [3, 900])
def test_equal_keys_go_to_the_lowest_index(tokens):
    for score in ("softmax", "sigmoid"):
        logits = torch.zeros(tokens, 48, device="cuda")
        bias = torch.full((48,), 0.25, device="cuda")
        bias[40:] = 0.5
        e = check(logits, 6, bias, score=score)
        assert torch.equal(e[0].cpu(), torch.arange(40, 46))
        assert torch.equal(check(logits, 6, bias * 0, score=score)[-1].cpu(), torch.arange(6))
    # scores that are 1 in fp32
    logits = torch.arange(48, device="cuda").float().repeat(tokens, 1) + 40
    e = pgg.route(logits, 4, bias=bias * 0, score="sigmoid", bias_on="scores")[1]
    assert torch.equal(e[0].cpu(), torch.arange(4))


@pytest.mark.parametrize("tokens", [5, 700])
@pytest.mark.parametrize("score,renormalize", KINDS)
def test_a_bias_does_not_bring_back_a_masked_expert(tokens, score, renormalize):
    l = logits_of(tokens, 24, "fp32", 3)
    l[:, 3:20] = float("-inf")          # seven experts left, eight chosen
    l[2] = float("-inf")                # a token with nothing left
    bias = torch.zeros(24, device="cuda")
    bias[3:20] = 5.0
    p, e, idx, groups, _ = pgg.route(l, 8, bias=bias, score=score, renormalize=renormalize,
                                     bias_on="scores")
    rest = torch.ones(tokens, dtype=torch.bool, device="cuda")
    rest[2] = False
    left = torch.tensor([0, 1, 2, 20, 21, 22, 23])
    assert torch.equal(torch.sort(e[rest][:, :7], 1).values.cpu(),
                       left.expand(tokens - 1, 7))
    assert (e[rest][:, 7] == 3).all() and not p[rest][:, 7].any()
    assert torch.equal(e[2].cpu(), torch.arange(8)) and not p[2].any()
    assert not torch.isnan(p).any()
    assert int(groups.sum()) == 8 * tokens
    assert torch.equal(torch.sort(idx).values.cpu(), torch.arange(8 * tokens))


def test_nan_logits_keep_the_order_valid():
    l = logits_of(300, 20, "fp32", 4)
    l[5, 3] = float("nan")
    l[6] = float("nan")
    l[9, 2] = float("inf")
    bias = torch.rand(20, device="cuda")
    for score, renormalize in KINDS:
        p, e, idx, groups, _ = pgg.route(l, 4, bias=bias, score=score, renormalize=renormalize,
                                         bias_on="scores")
        assert all(len(set(r)) == 4 for r in e.tolist())
        assert torch.equal(torch.sort(idx).values.cpu(), torch.arange(1200))
        assert int(groups.sum()) == 1200
        assert torch.isnan(p[6]).all()
        if score == "softmax":
            assert torch.isnan(p[5]).all() and torch.isnan(p[9]).all()
        clean = torch.ones(300, dtype=torch.bool, device="cuda")
        clean[[5, 6, 9]] = False
        assert torch.isfinite(p[clean]).all()


def test_without_a_bias_the_choice_goes_by_the_logits():
    l = logits_of(600, 64, "bf16", 8)
    a, b = pgg.route(l, 6, bias_on="scores"), pgg.route(l, 6)
    for p, q in zip(a[:4], b[:4]):
        assert torch.equal(p, q)


def test_in_a_graph_and_on_unaligned_logits():
    buf = torch.empty(1000 * 100 + 1, device="cuda", dtype=torch.bfloat16)
    l = buf[1:].view(1000, 100)
    l.copy_(logits_of(1000, 100, "bf16", 9))
    bias = torch.rand(100, device="cuda") * 0.1
    check(l, 8, bias, score="sigmoid")
    first = pgg.route(l, 8, bias=bias, score="sigmoid", bias_on="scores")
    out = [torch.empty_like(t) for t in first]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pgg.route(l, 8, bias=bias, score="sigmoid", bias_on="scores", probs=out[0],
                  experts=out[1], expanded_row_idx=out[2], group_list=out[3], workspace=out[4])
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(first[:4], out[:4]):
        assert torch.equal(p, q)


# ------------------------------------------------------------------ NaN and +inf in a softmax

# every form: four tokens a warp, two, one; in one block and in several; loads of one value
@pytest.mark.parametrize("bias_on", ["logits", "scores"])
@pytest.mark.parametrize("t,g,k", [(9, 16, 4), (200, 60, 8), (600, 256, 8), (300, 255, 6),
                                   (40, 500, 12), (700, 96, 16), (30, 1024, 20), (500, 700, 32)])
def test_a_softmax_with_a_nan_gives_nan_weights(t, g, k, bias_on):
    l = logits_of(t, g, "fp32", t)
    low = l.argmin(1)  # an expert that is not chosen
    l[1, low[1]] = float("nan")
    l[4, g - 1] = l[4, 0] = float("nan")
    l[6, low[6]] = float("inf")
    l[7, low[7]] = float("-inf")
    # the +inf is not chosen: its key is NaN
    bias = torch.zeros(g, device="cuda")
    bias[low[6]] = float("-inf")
    for renormalize in (False, True):
        p, e, idx, _, _ = pgg.route(l, k, bias=bias, renormalize=renormalize, bias_on=bias_on)
        assert not (e[1] == low[1]).any() and not (e[7] == low[7]).any()
        if bias_on == "logits":
            assert not (e[6] == low[6]).any()
        assert torch.equal(torch.sort(idx).values.cpu(), torch.arange(t * k))
        odd = torch.zeros(t, dtype=torch.bool, device="cuda")
        odd[[1, 4, 6]] = True
        assert torch.isnan(p[odd]).all()
        assert torch.isfinite(p[~odd]).all()
        # without a bias too, where the +inf is chosen
        p = pgg.route(l, k, renormalize=renormalize)[0]
        assert torch.isnan(p[odd]).all() and torch.isfinite(p[~odd]).all()
    # a sigmoid of an expert that is not chosen does not matter
    p = pgg.route(l, k, score="sigmoid")[0]
    assert torch.isfinite(p).all()
