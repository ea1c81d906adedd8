"""GPU parity of the projection with per-token adapters and of its gradient
against plain 64-bit formulas.

y is rounded once (r |y|, r the dtype's unit); the low-rank row u = scale x a is
rounded once to the dtype before the second product, which carries at most
r * (|u| |b|^T); fp32 sums keep 2e-5 of the largest value. The gradients alike:
r * (|v| |a|^T) in d_x, r * (|x|^T |v|) in d_a, r * (|d_y|^T |u|) in d_b.
"""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
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


def inputs(T, K, N, R, A, dtype="bf16", ids="mixed", seed=0, scaled=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(DT[dtype])  # noqa: E731
    if ids == "mixed":  # about one token in A + 1 without an adapter
        ad = torch.randint(-1, A, (T,), generator=gen, device="cuda")
    elif ids == "runs":
        ad = (torch.arange(T, device="cuda") * A // max(T, 1)).flip(0)
    else:
        ad = torch.full((T,), int(ids), device="cuda", dtype=torch.int64)
    return dict(x=rnd(T, K), weight=rnd(K, N, std=K ** -0.5), a=rnd(A, K, R, std=K ** -0.5),
                b=rnd(A, N, R, std=R ** -0.5), adapter=ad.contiguous(),
                scale=torch.rand(A, generator=gen, device="cuda") + 0.5 if scaled else None)


def low_rank(x, f, ad, scale):
    """scale x f[ad] in float64, zero rows without an adapter."""
    u = torch.zeros(x.shape[0], f.shape[2], dtype=torch.double, device="cuda")
    for i in ad.unique().tolist():
        if i >= 0:
            s = 1.0 if scale is None else scale[i].double()
            u[ad == i] = s * (x[ad == i].double() @ f[i].double())
    return u


def expand(u, f, ad):
    y = torch.zeros(u.shape[0], f.shape[1], dtype=torch.double, device="cuda")
    for i in ad.unique().tolist():
        if i >= 0:
            y[ad == i] = u[ad == i] @ f[i].double().T
    return y


def near(got, ref, inner):
    r = ROUND[got.dtype]
    bound = r * ref.abs() + r * inner + SUM * ref.abs().max() + TINY[got.dtype]
    off = (got.double() - ref).abs()
    assert (off <= bound).all(), f"off by {(off - bound).max().item():.3e} over the bound"


def check(s):
    y, ws = pgg.adapters(**s)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0, pgg.STATUS.get(pgg.status(ws))
    u = low_rank(s["x"], s["a"], s["adapter"], s["scale"])
    ref = s["x"].double() @ s["weight"].double() + expand(u, s["b"], s["adapter"])
    near(y, ref, expand(u.abs(), s["b"].abs(), s["adapter"]))
    return y


# (T, K, N, R, A): a single token, a decode batch, odd and ragged sizes, several row blocks
SIZES = [(1, 64, 64, 8, 1), (1, 1024, 512, 16, 8), (7, 200, 136, 16, 3), (48, 512, 264, 16, 64),
         (65, 128, 256, 64, 5), (300, 264, 520, 24, 4), (513, 192, 192, 32, 20),
         (200, 4096, 264, 16, 24), (90, 2048, 136, 72, 30), (40, 100, 50, 5, 6), (600, 321, 77, 7, 9), (33, 64, 128, 256, 4), (1000, 96, 72, 1, 1)]


@pytest.mark.parametrize("ids", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", SIZES)
def test_cases(size, dtype, ids):
    check(inputs(*size, dtype=dtype, ids=ids, seed=size[0], scaled=size[3] != 24))


@pytest.mark.parametrize("T", [1, 30, 400])
def test_no_adapter_at_all_and_one_for_all(T):
    s = inputs(T, 128, 192, 16, 4, ids="-1", seed=T)
    y = check(s)
    s["a"].fill_(float("nan"))  # nobody's adapters are not read into anything
    s["b"].fill_(float("inf"))
    assert torch.equal(pgg.adapters(**s)[0].view(torch.int16), y.view(torch.int16))
    check(inputs(T, 128, 192, 16, 4, ids="2", seed=T))


@pytest.mark.parametrize("variant", [-1, 0, 1, 3])
@pytest.mark.parametrize("T", [3, 60, 700])
def test_every_kernel_on_every_row_count(variant, T):
    pgg.pgg_debug_force_variant(variant)
    try:
        check(inputs(T, 328, 456, 40, 7, seed=T))
    finally:
        pgg.pgg_debug_force_variant(-1)


@pytest.mark.parametrize("T", [9, 64, 700])
def test_infinite_weights_of_one_adapter_stay_with_its_tokens(T):
    s = inputs(T, 256, 320, 16, 5, seed=40 + T)
    s["adapter"][0], s["adapter"][1], s["adapter"][2] = 2, 3, -1
    clean, _ = pgg.adapters(**s)
    s["a"][2, :, 3] = float("inf")
    s["b"][2] = float("nan")
    y, _ = pgg.adapters(**s)
    mine = s["adapter"] == 2
    assert torch.isnan(y[mine]).all()
    assert torch.equal(y[~mine].view(torch.int16), clean[~mine].view(torch.int16))
    s["x"][1] = float("nan")  # a token's own NaN reaches nobody else
    y2, _ = pgg.adapters(**s)
    rest = ~mine
    rest[1] = False
    assert torch.equal(y2[rest].view(torch.int16), clean[rest].view(torch.int16))


def test_more_tokens_than_one_block_or_one_cluster_sorts():
    check(inputs(17000, 64, 72, 8, 200, seed=50))
    check(inputs(20000, 64, 64, 8, 1023, seed=51))
    check(inputs(66000, 64, 72, 8, 1023, seed=55))
    check(inputs(70000, 64, 64, 8, 3, ids="runs", seed=56))


@pytest.mark.parametrize("T", [20, 900, 17000, 66000])
def test_an_unknown_adapter_zeroes_the_output(T):
    s = inputs(T, 64, 64, 8, 4, seed=52)
    for bad in (4, -2, 1 << 40):
        s["adapter"][T // 2] = bad
        out = torch.full((T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        _, ws = pgg.adapters(**s, out=out)
        torch.cuda.synchronize()
        assert pgg.STATUS[pgg.status(ws)] == "PGG_ERR_INDEX"
        assert torch.count_nonzero(out) == 0


@pytest.mark.parametrize("T", [5, 300])
def test_unaligned_tensors_and_a_reused_workspace(T):
    s = inputs(T, 128, 64, 16, 3, seed=53)
    need = pgg.pgg_adapters_workspace_size(T, 128, 64, 16, 3, pgg.PGG_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    y = check(s)
    assert torch.equal(pgg.adapters(**s, workspace=ws)[0].view(torch.int16), y.view(torch.int16))
    for name in ("x", "weight", "a", "b"):
        t = s[name]
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        check(dict(s, **{name: buf[1:].view(t.shape)}))


@pytest.mark.parametrize("T", [40, 2000])
def test_repeats_bitwise_and_on_another_stream(T):
    s = inputs(T, 512, 256, 32, 10, seed=54)
    y, _ = pgg.adapters(**s)
    g = pgg.adapters_grad(torch.ones_like(y), **s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y2, _ = pgg.adapters(**s)
        g2 = pgg.adapters_grad(torch.ones_like(y), **s)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    for p, q in zip(g[:3], g2[:3]):
        assert torch.equal(p.view(torch.int16), q.view(torch.int16))


# ------------------------------------------------------------------ gradient

def check_grad(s, seed=1, need_x=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, N = s["x"].shape[0], s["weight"].shape[1]
    d_y = torch.randn(T, N, generator=gen, device="cuda").to(s["x"].dtype)
    d_x, d_a, d_b, ws = pgg.adapters_grad(d_y, **s, need_x=need_x)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0, pgg.STATUS.get(pgg.status(ws))
    ad, x, dy = s["adapter"], s["x"].double(), d_y.double()
    u = low_rank(s["x"], s["a"], ad, s["scale"])
    v = low_rank(d_y, s["b"], ad, s["scale"])
    if need_x:
        near(d_x, dy @ s["weight"].double().T + expand(v, s["a"], ad),
             expand(v.abs(), s["a"].abs(), ad))
    else:
        assert d_x is None
    for got, left, right in ((d_a, x, v), (d_b, dy, u)):
        for i in range(s["a"].shape[0]):
            m = ad == i
            if not m.any():
                assert torch.count_nonzero(got[i]) == 0
                continue
            near(got[i], left[m].T @ right[m], left[m].abs().T @ right[m].abs())


@pytest.mark.parametrize("ids", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", SIZES)
def test_gradient(size, dtype, ids):
    check_grad(inputs(*size, dtype=dtype, ids=ids, seed=60 + size[0], scaled=size[3] != 24),
               need_x=size[1] != 200)


def test_gradient_of_many_tokens():
    check_grad(inputs(17000, 64, 72, 8, 30, seed=61))
    check_grad(inputs(66000, 64, 72, 8, 30, seed=65))


def test_gradient_against_differences():
    # the loss is bilinear in (a, b) and linear in x: central differences have no truncation error;
    # fp32 sums of 40 * 24 terms, step 2^-4
    s = inputs(40, 16, 24, 4, 3, dtype="fp32", seed=62)
    d_y = torch.randn(40, 24, device="cuda")
    d_x, d_a, d_b, _ = pgg.adapters_grad(d_y, **s)

    def loss():
        return (pgg.adapters(**s)[0].double() * d_y.double()).sum()

    step = 2.0 ** -4
    gen = torch.Generator().manual_seed(1)
    for name, grad in (("x", d_x), ("a", d_a), ("b", d_b)):
        flat = s[name].view(-1)
        for i in torch.randperm(flat.numel(), generator=gen)[:24].tolist():
            old = flat[i].clone()
            flat[i] = old + step
            hi = loss()
            flat[i] = old - step
            lo = loss()
            flat[i] = old
            assert abs(float((hi - lo) / (2 * step) - grad.view(-1)[i])) < 1e-3


@pytest.mark.parametrize("T", [150, 700])
def test_gradient_keeps_adapters_apart(T):
    # NaN in one adapter's tokens and weights changes nothing of another's gradients
    s = inputs(T, 128, 192, 16, 5, seed=63)
    d_y = torch.randn(T, 192, device="cuda").bfloat16()
    clean = pgg.adapters_grad(d_y, **s)
    mine = s["adapter"] == 2
    s["x"][mine] = float("nan")
    d_y[mine] = float("inf")
    s["a"][2] = float("nan")
    got = pgg.adapters_grad(d_y, **s)
    others = [0, 1, 3, 4]
    assert torch.equal(got[0][~mine].view(torch.int16), clean[0][~mine].view(torch.int16))
    for p, q in zip(got[1:3], clean[1:3]):
        assert torch.equal(p[others].view(torch.int16), q[others].view(torch.int16))
        assert torch.isnan(p[2]).any()


def test_gradient_with_an_unknown_adapter_is_zero():
    s = inputs(64, 64, 64, 8, 4, seed=64)
    s["adapter"][7] = 9
    d_y = torch.randn(64, 64, device="cuda").bfloat16()
    outs = dict(d_x=torch.full_like(s["x"], 7.0), d_a=torch.full_like(s["a"], 7.0),
                d_b=torch.full_like(s["b"], 7.0))
    *_, ws = pgg.adapters_grad(d_y, **s, **outs)
    torch.cuda.synchronize()
    assert pgg.STATUS[pgg.status(ws)] == "PGG_ERR_INDEX"
    assert all(torch.count_nonzero(o) == 0 for o in outs.values())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_neighbouring_and_scattered_rows_in_one_call(dtype):
    # runs of requests (copied as boxes) broken by tokens that change places, block by block
    s = inputs(1500, 264, 200, 16, 6, dtype=dtype, ids="runs", seed=66)
    ad = s["adapter"]
    ad[100:110] = -1
    ad[300], ad[301] = ad[900].clone(), ad[0].clone()
    ad[640:768] = torch.arange(128, device="cuda") % 6
    check(s)
    check_grad(s)
    s["adapter"] = ad.flip(0).contiguous()
    check(s)


# ---------------------------------------------------------------- launches that run side by side

BESIDE = [
    (300, 1024, 2048, 16, 9),
    (700, 4096, 512, 64, 33),
    (2500, 512, 1024, 32, 3),
]


@pytest.mark.parametrize("size", BESIDE)
def test_calls_in_a_row_with_one_workspace(size):
    """Forward and gradient of three inputs (one with an unknown adapter, one without any) again and
    again into one workspace without a synchronisation: each call finds its own tables, u and v."""
    T, K, N, R, A = size
    sets = [inputs(T, K, N, R, A, "bf16", ids, i) for i, ids in enumerate(["mixed", "runs", "-1"])]
    sets.append(dict(sets[0], adapter=sets[0]["adapter"].clone().fill_(A)))
    dys = [torch.randn(T, N, device="cuda").bfloat16() for _ in sets]
    forward = torch.empty(pgg.pgg_adapters_workspace_size(T, K, N, R, A, 2), dtype=torch.uint8,
                          device="cuda")
    backward = torch.empty(pgg.pgg_adapters_grad_workspace_size(T, K, N, R, A, 2),
                           dtype=torch.uint8, device="cuda")
    want = []
    for s, dy in zip(sets, dys):
        y, _ = pgg.adapters(**s)
        torch.cuda.synchronize()
        dx, da, db, _ = pgg.adapters_grad(dy, **s)
        torch.cuda.synchronize()
        want.append((y, dx, da, db))
    assert not want[3][0].any() and not want[3][1].any() and not want[3][2].any()
    for rep in range(4):
        got = []
        for s, dy in zip(sets, dys):
            y, _ = pgg.adapters(**s, workspace=forward)
            dx, da, db, _ = pgg.adapters_grad(dy, **s, workspace=backward)
            _, da2, db2, _ = pgg.adapters_grad(dy, **s, need_x=False, workspace=backward)
            got.append((y, dx, da, db, da2, db2))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w + w[2:]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("size", BESIDE[:2])
def test_in_a_graph(size):
    T, K, N, R, A = size
    s = inputs(T, K, N, R, A, "fp16", "mixed", 4)
    dy = torch.randn(T, N, device="cuda").half()
    y, fw = pgg.adapters(**s)
    dx, da, db, bw = pgg.adapters_grad(dy, **s)
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, da, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            pgg.adapters(**s, out=y, workspace=fw)
            pgg.adapters_grad(dy, **s, d_x=dx, d_a=da, d_b=db, workspace=bw)
    for _ in range(3):
        for t in (y, dx, da, db):
            t.fill_(7)
        graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip((y, dx, da, db), want):
        assert torch.equal(got, ref)
