"""GPU parity of the gated expert product and of its gradient against plain
64-bit formulas.

Every output is rounded once to its dtype: |got - ref| <= r |ref| with r the
dtype's unit (2^-8, 2^-11, 2^-23), plus what the fp32 sums carry: the products
of K <= 7168 terms keep about sqrt(K) * 2^-24 of the row's scale, well below
2e-5 of the largest value; the gate multiplies two of them.
"""

import numpy as np
import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from workloads import make_case
from workloads.moe import forward_input, with_row_idx_type

pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
SUM = 2e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()
    yield
    pgg.pgg_debug_force_variant(-1)


def case(tokens, top_k, G, K, F, dtype="bf16", rit=0, seed=0, **kw):
    # make_case's weight is [G, K, N] with N = 2F
    kw.setdefault("w_std", K ** -0.5)
    inp = make_case(batch=tokens, top_k=top_k, G=G, K=K, N=2 * F, dtype=dtype, seed=seed,
                    device="cuda", **kw)
    return with_row_idx_type(inp, rit)


def probs_of(inp, seed=9):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(inp.batch, inp.top_k, generator=gen, device="cuda") + 0.01


def reference(inp, x, probs, rows=None):
    """(h, gate_up) in float64 of the given expanded rows (all of them by default)."""
    F = inp.weight.shape[2] // 2
    counts = inp.group_list.cpu()
    expert = torch.repeat_interleave(torch.arange(counts.numel()), counts)
    pos = inp.gather
    rows = torch.arange(pos.numel()) if rows is None else rows
    gu = torch.empty(rows.numel(), 2 * F, dtype=torch.double, device="cuda")
    for e in expert[rows].unique().tolist():
        at = (expert[rows] == e).nonzero().reshape(-1)
        tok = (pos[rows[at]] // inp.top_k).cuda()
        gu[at.cuda()] = x[tok].double() @ inp.weight[e].double()
    gate, up = gu[:, :F], gu[:, F:]
    h = gate / (1 + torch.exp(-gate)) * up
    if probs is not None:
        h = h * probs.double().reshape(-1)[pos[rows].cuda()][:, None]
    return h, gu


def near(got, ref, what=""):
    bound = ROUND[got.dtype] * ref.abs() + SUM * ref.abs().max() + TINY[got.dtype]
    off = (got.double() - ref).abs()
    assert (off <= bound).all(), f"{what}: off by {(off - bound).max().item():.3e} over the bound"


def run(inp, x, probs=None, keep=False, **kw):
    h, gu, ws = pgg.swiglu(x, inp.weight, inp.expanded_row_idx, inp.group_list, inp.batch,
                           inp.top_k, inp.row_idx_type, probs=probs, keep=keep, **kw)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0, pgg.STATUS.get(pgg.status(ws))
    return h, gu


def check(inp, weighted=True, keep=True, rows=None):
    x = forward_input(inp)
    probs = probs_of(inp) if weighted else None
    h, gu = run(inp, x, probs, keep)
    rh, rgu = reference(inp, x, probs, rows)
    at = slice(None) if rows is None else rows.cuda()
    near(h[at], rh, "h")
    if keep:
        near(gu[at], rgu, "gate_up")
    return h, gu


# (tokens, top_k, G, K, F): one row, few rows, ragged groups, more than a row block per group,
# tails in every dimension, sizes that are no multiple of a tile or of 8
SIZES = [(1, 1, 1, 64, 64), (1, 8, 60, 512, 128), (3, 2, 5, 72, 40), (17, 4, 9, 200, 104),
         (64, 8, 16, 256, 192), (130, 2, 3, 136, 264), (700, 3, 4, 448, 320), (33, 2, 4, 101, 37),
         (90, 3, 7, 66, 143), (600, 1, 1, 1024, 64)]


@pytest.mark.parametrize("weighted,keep", [(True, False), (False, True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", SIZES)
def test_cases(size, dtype, weighted, keep):
    check(case(*size, dtype=dtype, rit=size[0] % 2, seed=size[0]), weighted, keep)


@pytest.mark.parametrize("variant", [-1, 0, 1, 3])
@pytest.mark.parametrize("tokens,G", [(5, 8), (70, 8), (900, 8)])
def test_every_kernel_on_every_row_count(variant, tokens, G):
    pgg.pgg_debug_force_variant(variant)
    try:
        check(case(tokens, 4, G, 328, 200, seed=tokens))
    finally:
        pgg.pgg_debug_force_variant(-1)


def test_empty_experts_and_one_crowded_expert():
    check(case(400, 2, 12, 256, 128, empty=tuple(range(2, 11)), seed=3))
    inp = case(300, 1, 16, 256, 128, routing="zipf", zipf_s=3.0, zipf_zero=12, seed=4)
    assert int((inp.group_list == 0).sum()) >= 12
    check(inp)


def test_many_rows():
    # more rows than the one-launch preparation takes
    check(case(5000, 4, 10, 128, 64, seed=5, rit=1))
    check(case(5000, 4, 10, 128, 64, seed=5, rit=0))


def test_without_weights_equals_weights_of_one():
    inp = case(200, 3, 6, 256, 128, seed=6)
    x = forward_input(inp)
    h, _ = run(inp, x)
    h1, _ = run(inp, x, torch.ones(200, 3, device="cuda"))
    assert torch.equal(h, h1)


@pytest.mark.parametrize("tokens", [2, 100, 1500])
def test_repeats_bitwise_with_both_index_forms_and_a_reused_workspace(tokens):
    inp = case(tokens, 4, 8, 512, 256, seed=7)
    x, probs = forward_input(inp), probs_of(inp)
    h, gu = run(inp, x, probs, True)
    need = pgg.pgg_swiglu_workspace_size(4 * tokens, 256, 512, 8, 4 * tokens, tokens, 4, 0,
                                         pgg.PGG_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for other in (inp, with_row_idx_type(inp, 1)):
        h2, gu2 = run(other, x, probs, True, workspace=ws)
        assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
        assert torch.equal(gu.view(torch.int16), gu2.view(torch.int16))


@pytest.mark.parametrize("tokens", [4, 500])
def test_unaligned_tensors(tokens):
    inp = case(tokens, 2, 4, 128, 64, seed=8)
    x, probs = forward_input(inp), probs_of(inp)
    rh, _ = reference(inp, x, probs)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    for which in range(3):
        xs = shifted(x) if which == 0 else x
        w = shifted(inp.weight) if which == 1 else inp.weight
        out = shifted(torch.zeros(2 * tokens, 64, dtype=x.dtype, device="cuda")) if which == 2 else None
        h, _, ws = pgg.swiglu(xs, w, inp.expanded_row_idx, inp.group_list, tokens, 2, 0,
                              probs=probs, out=out)
        torch.cuda.synchronize()
        assert pgg.status(ws) == 0
        near(h, rh)


@pytest.mark.parametrize("tokens", [10, 6000])
def test_bad_routing_zeroes_the_outputs(tokens):
    inp = case(tokens, 2, 4, 64, 32, seed=9)
    x = forward_input(inp)
    M = 2 * tokens
    for name in ("PGG_ERR_NOT_PERM", "PGG_ERR_INDEX", "PGG_ERR_GROUPSUM"):
        idx, groups = inp.expanded_row_idx.clone(), inp.group_list.clone()
        if name == "PGG_ERR_NOT_PERM":
            idx[5] = idx[6]
        elif name == "PGG_ERR_INDEX":
            idx[5] = M
        else:
            groups[0] += 1
        out = torch.full((M, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        gu = torch.full((M, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        _, _, ws = pgg.swiglu(x, inp.weight, idx, groups, tokens, 2, 0, out=out, gate_up=gu,
                              keep=True)
        torch.cuda.synchronize()
        assert pgg.STATUS[pgg.status(ws)] == name
        assert torch.count_nonzero(out) == 0 and torch.count_nonzero(gu) == 0


@pytest.mark.parametrize("tokens", [3, 400])
def test_a_row_with_nan_stays_alone(tokens):
    inp = case(tokens, 2, 4, 256, 128, seed=10)
    x = forward_input(inp)
    clean, _ = run(inp, x)
    x[1, 5] = float("nan")
    h, _ = run(inp, x)
    bad = ((inp.gather // 2) == 1).cuda()
    assert torch.isnan(h[bad]).all()
    assert torch.equal(h[~bad].view(torch.int16), clean[~bad].view(torch.int16))


def test_large_gates_do_not_overflow():
    inp = case(64, 2, 4, 64, 32, seed=11, w_std=8.0)
    x = forward_input(inp) * 4  # gates in the hundreds, of both signs
    h, _ = run(inp, x)
    rh, rgu = reference(inp, x, None)
    assert rgu.abs().max() > 300
    near(h, rh)


def test_weights_beyond_32_bit_offsets():
    # 160 experts of 7168 x 4096: 4.7e9 weight elements
    inp = case(48, 8, 160, 7168, 2048, seed=12)
    rows = torch.randperm(384)[:96]
    check(inp, rows=rows, keep=False)


# ------------------------------------------------------------------ gradient

def grad_inputs(M, F, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    gu = (torch.randn(M, 2 * F, generator=gen, device="cuda") * 2).to(dtype)
    dh = torch.randn(M, F, generator=gen, device="cuda").to(dtype)
    return dh, gu


def grad_reference(dh, gu, probs, gather, rows=slice(None)):
    F = dh.shape[1]
    pos = gather.cuda()[rows]
    g, u, d = gu[rows, :F].double(), gu[rows, F:].double(), dh[rows].double()
    p = probs.double().reshape(-1)[pos][:, None] if probs is not None else 1.0
    sig = 1 / (1 + torch.exp(-g))
    act = g * sig
    return (torch.cat([p * d * u * sig * (1 + g * (1 - sig)), p * d * act], 1),
            (d * act * u).sum(1), p * act * u, pos)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("rit", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,k,F", [(1, 1, 8), (1, 8, 2048), (50, 3, 100), (333, 2, 37),
                                        (700, 4, 768)])
def test_gradient(tokens, k, F, dtype, rit, weighted):
    inp = case(tokens, k, max(k, 6), 8, 4, dtype=dtype, rit=rit, seed=20 + tokens)
    dh, gu = grad_inputs(tokens * k, F, inp.weight.dtype, tokens)
    probs = probs_of(inp) if weighted else None
    d_gu, d_p, h, ws = pgg.swiglu_grad(dh, gu, inp.expanded_row_idx, k, rit, probs=probs)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    r_gu, r_p, r_h, pos = grad_reference(dh, gu, probs, inp.gather)
    # element-wise: no sums, only the fast exponential's error (below 1e-6 relative for 16 bits)
    for got, ref in ((d_gu, r_gu), (h, r_h)):
        bound = (ROUND[got.dtype] + 2e-6) * ref.abs() + 2e-6 + TINY[got.dtype]
        assert ((got.double() - ref).abs() <= bound).all()
    if weighted:
        terms = (dh.double() * r_h).abs().sum(1) / probs.double().reshape(-1)[pos]
        assert ((d_p.reshape(-1)[pos].double() - r_p).abs() <= 4e-6 * terms + 1e-30).all()
    else:
        assert d_p is None


def test_gradient_against_differences():
    # central differences of the gated product itself with the identity as weight: h step 2^-7 in
    # fp32, truncation h^2 / 6 |f'''| < 2e-5 per element, rounding 6e-8 * |f| / h
    F, M = 16, 4
    x = torch.randn(M, 2 * F, device="cuda")
    w = torch.eye(2 * F, device="cuda")[None].contiguous()
    idx, groups = torch.arange(M, device="cuda"), torch.tensor([M], device="cuda")
    probs = torch.rand(M, 1, device="cuda") + 0.5
    dh = torch.randn(M, F, device="cuda")
    _, gu, _ = pgg.swiglu(x, w, idx, groups, M, 1, 0, probs=probs, keep=True)
    d_gu, d_p, h, _ = pgg.swiglu_grad(dh, gu, idx, 1, 0, probs=probs)

    def loss(z, p):
        out, _, _ = pgg.swiglu(z, w, idx, groups, M, 1, 0, probs=p)
        return (out.double() * dh.double()).sum(1)

    step = 2.0 ** -7
    for c in range(2 * F):
        up, down = x.clone(), x.clone()
        up[:, c] += step
        down[:, c] -= step
        num = (loss(up, probs) - loss(down, probs)) / (2 * step)
        assert (num - d_gu[:, c].double()).abs().max() < 2e-3
    num = (loss(x, probs + step) - loss(x, probs - step)) / (2 * step)
    assert (num - d_p[:, 0].double()).abs().max() < 2e-3


def test_gradient_extremes():
    gu = torch.tensor([[-200.0, 200.0, -90.0, 0.0, 3.0, 5.0, 2.0, -1.0],
                       [88.0, -88.0, -1e4, 1e4, 1.0, 1.0, 1.0, 1.0]], device="cuda")
    dh = torch.ones(2, 4, device="cuda")
    idx = torch.arange(2, device="cuda")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        d_gu, _, h, _ = pgg.swiglu_grad(dh.to(dt), gu.to(dt), idx, 1, 0)
        r_gu, _, r_h, _ = grad_reference(dh.to(dt), gu.to(dt), None, torch.arange(2))
        for got, ref in ((d_gu, r_gu), (h, r_h)):
            assert torch.isfinite(got).all()
            assert ((got.double() - ref).abs() <= 2 * ROUND[dt] * ref.abs() + 1e-6).all()


def test_gradient_bad_index_zeroes_and_misaligned_rows():
    inp = case(64, 2, 4, 8, 4, seed=30)
    dh, gu = grad_inputs(128, 64, torch.bfloat16, 31)
    probs = probs_of(inp)
    idx = inp.expanded_row_idx.clone()
    idx[3] = idx[4]
    outs = dict(d_gate_up=torch.full_like(gu, 7.0), d_probs=torch.full_like(probs, 7.0),
                h=torch.full_like(dh, 7.0))
    _, _, _, ws = pgg.swiglu_grad(dh, gu, idx, 2, 0, probs=probs, **outs)
    torch.cuda.synchronize()
    assert pgg.STATUS[pgg.status(ws)] == "PGG_ERR_NOT_PERM"
    assert all(torch.count_nonzero(o) == 0 for o in outs.values())
    want = pgg.swiglu_grad(dh, gu, inp.expanded_row_idx, 2, 0, probs=probs)
    buf = torch.empty(dh.numel() + 1, dtype=dh.dtype, device="cuda")
    buf[1:] = dh.reshape(-1)
    got = pgg.swiglu_grad(buf[1:].view(dh.shape), gu, inp.expanded_row_idx, 2, 0, probs=probs)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert (got[1] - want[1]).abs().max() <= 1e-5 * want[1].abs().max()


def test_gradient_beyond_32_bit_offsets():
    M, F = 540000, 2048  # gate_up holds 2.2e9 elements
    idx = torch.randperm(M, device="cuda")
    dh, gu = grad_inputs(1, F, torch.bfloat16, 33)
    gu = gu.expand(M, 2 * F).contiguous()
    gu[:, 0] = torch.arange(M, device="cuda").remainder(64).bfloat16() / 16
    dh = dh.expand(M, F).contiguous()
    probs = torch.rand(M, 1, device="cuda")
    d_gu, d_p, h, ws = pgg.swiglu_grad(dh, gu, idx, 1, 0, probs=probs)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    rows = torch.cat([torch.arange(64), torch.arange(M - 64, M)]).cuda()
    r_gu, r_p, r_h, pos = grad_reference(dh, gu, probs, idx, rows)
    for got, ref in ((d_gu[rows], r_gu), (h[rows], r_h)):
        assert ((got.double() - ref).abs() <= (2.0 ** -8 + 2e-6) * ref.abs() + 2e-6).all()


def test_a_whole_layer_forward_and_backward():
    """route -> swiglu -> dx (down projection and combine), and its gradients, against autograd
    in float64 with the same rounded intermediates' tolerance: bf16 stages, 2^-8 each, three in a
    row over sums of many terms: 2e-2 of the largest value."""
    T, k, G, H, F = 96, 4, 8, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std)  # noqa: E731
    x = rnd(T, H).bfloat16()
    wr = rnd(H, G, std=H ** -0.5)
    w1 = rnd(G, H, 2 * F, std=H ** -0.5).bfloat16()
    w2 = rnd(G, H, F, std=F ** -0.5).bfloat16()  # [G, K = H, N = F] of dx: out = h w2^T
    d_out = rnd(T, H).bfloat16()
    logits = x.float() @ wr
    probs, experts, idx, groups, _ = pgg.route(logits, k)
    h, gu, _ = pgg.swiglu(x, w1, idx, groups, T, k, 0, probs=probs, keep=True)
    out, _ = pgg.dx(h, w2, idx, groups, T, k, 0)
    # backward: d_h = d_out w2 in expanded order, then the gate, then x, the weights, the logits
    d_h, _ = pgg.fwd(d_out, w2, idx, groups, T, k, 0)
    d_gu, d_probs, hw, _ = pgg.swiglu_grad(d_h, gu, idx, k, 0, probs=probs)
    d_x, _ = pgg.dx(d_gu, w1, idx, groups, T, k, 0)
    d_w1, _ = pgg.dw(x, d_gu, idx, groups, T, k, 0)
    d_w2, _ = pgg.dw(d_out, hw, idx, groups, T, k, 0)
    d_logits = pgg.route_grad(d_probs, logits, experts)
    # the same in float64 by autograd
    X, L = x.double().requires_grad_(), logits.double().requires_grad_()
    W1, W2 = w1.double().requires_grad_(), w2.double().requires_grad_()
    P = torch.softmax(L, 1).gather(1, experts)
    P = P / P.sum(1, keepdim=True)
    A = torch.einsum("th,tjhf->tjf", X, W1[experts])
    Hd = torch.nn.functional.silu(A[..., :F]) * A[..., F:] * P[..., None]
    O = torch.einsum("tjf,tjhf->th", Hd, W2[experts])
    want = torch.autograd.grad((O * d_out.double()).sum(), (X, W1, W2, L))
    for got, ref in ((out, O.detach()), (d_x, want[0]), (d_w1, want[1]), (d_w2, want[2]),
                     (d_logits, want[3])):
        assert (got.double() - ref).abs().max() <= 2e-2 * ref.abs().max()
