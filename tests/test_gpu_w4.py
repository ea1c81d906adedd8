"""Products with 4-bit expert weights against their 64-bit formula.

Bounds: with u = 2^-24, a sum of K products is off by at most (K + 8) 2u sum |x w| (each addition
by half a step, twice that where an adder cuts off), products of 16-bit values and codes are exact
and a scale multiplies once more. Outputs are rounded once, by half a step of their type.
"""

import math

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def case(product, T=20, G=5, top_k=2, K=128, N=64, group=32, zeros=True, dtype="bf16",
         scales="bf16", out=None, rit=0, seed=0, counts=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    M = T * top_k
    if counts is None:
        pick = torch.rand(T, G, generator=gen, device="cuda").argsort(1)[:, :top_k].reshape(-1)
    else:
        pick = torch.repeat_interleave(torch.arange(G, device="cuda"),
                                       torch.tensor(counts, device="cuda"))
        pick = pick[torch.randperm(M, generator=gen, device="cuda")]
    gather = torch.argsort(pick, stable=True)
    C = 2 * N if product == "gated" else N
    dt = DT[dtype]
    s = dict(product=product, T=T, G=G, top_k=top_k, K=K, N=N, group=group, rit=rit, gather=gather,
             groups=torch.bincount(pick, minlength=G), pick=pick[gather])
    s["idx"] = gather if rit == 0 else torch.argsort(gather)
    rows = M if product == "combined" else T
    s["x"] = torch.randn(rows, K, generator=gen, device="cuda").to(dt)
    s["codes"] = torch.randint(0, 256, (G, C, (K + 1) // 2), generator=gen, device="cuda",
                               dtype=torch.uint8)
    ng = (K + group - 1) // group
    s["scales"] = ((torch.rand(G, C, ng, generator=gen, device="cuda") + 0.5) * 0.2
                   / math.sqrt(K)).to(DT[scales])
    s["zeros"] = torch.randint(0, 16, (G, C, ng), generator=gen, device="cuda",
                               dtype=torch.uint8) if zeros else None
    s["probs"] = torch.rand(T, top_k, generator=gen, device="cuda") if product == "gated" else None
    s["out_dtype"] = torch.float32 if product == "combined" else DT[out or dtype]
    return s


def weights(s):
    """[G, C, K] in 64 bits."""
    c = s["codes"].to(torch.int64)
    k = torch.arange(s["K"], device="cuda")
    code = (c[..., k // 2] >> (4 * (k % 2))) & 15
    zero = s["zeros"].double()[..., k // s["group"]] if s["zeros"] is not None else 8.0
    return s["scales"].double()[..., k // s["group"]] * (code.double() - zero)


def want(s):
    """(64-bit result, bound of its error)."""
    rows = torch.arange(s["idx"].numel(), device="cuda") if s["product"] == "combined" \
        else s["gather"] // s["top_k"]
    x, w = s["x"].double()[rows], weights(s)
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.double, device="cuda")
    e = torch.zeros_like(y)
    for g in range(s["G"]):  # (an infinite weight meets its own expert's rows only)
        own = s["pick"] == g
        y[own] = x[own] @ w[g].T
        e[own] = x[own].abs() @ w[g].abs().T
    e *= (s["K"] + 8) * 2 * U
    if s["product"] == "gated":
        N = s["N"]
        gate, up, eg, eu = y[:, :N], y[:, N:], e[:, :N], e[:, N:]
        p = s["probs"].double().reshape(-1)[s["gather"]][:, None]
        act = torch.nn.functional.silu(gate)
        y = p * act * up
        # |silu'| <= 1.1; the exponential, quotient and products: a few steps (32 u)
        e = p * (1.1 * eg * up.abs() + act.abs() * eu + 1.1 * eg * eu) + 32 * U * y.abs()
    if s["product"] == "combined":
        k = s["top_k"]
        back = torch.argsort(s["gather"])
        y, size = y[back].view(s["T"], k, -1), y[back].view(s["T"], k, -1).abs().sum(1)
        y, e = y.sum(1), e[back].view(s["T"], k, -1).sum(1) + k * U * size
    half = torch.finfo(s["out_dtype"]).eps / 2
    tiny = torch.finfo(s["out_dtype"]).smallest_normal * half * 2
    return y, (e + tiny) * (1 + half) + half * y.abs()


def call(s, **kw):
    args = (s["x"], s["codes"], s["scales"], s["idx"], s["groups"], s["T"], s["top_k"], s["rit"])
    kw = dict(group=s["group"], zeros=s["zeros"], **kw)
    if s["product"] == "gated":
        return pgg.swiglu_w4(*args, probs=s["probs"], **kw)
    if s["product"] == "combined":
        return pgg.down_w4(*args, **kw)
    return pgg.fwd_w4(*args, out_dtype=s["out_dtype"], **kw)


def check(s, **kw):
    got, ws = call(s, **kw)
    assert pgg.status(ws) == 0
    y, bound = want(s)
    over = (got.double() - y).abs() - bound
    assert got.dtype == s["out_dtype"] and bool((over <= 0).all()), float(over.max())
    return got


PRODUCTS = ("rows", "gated", "combined")


@pytest.mark.parametrize("product", PRODUCTS)
@pytest.mark.parametrize("dtype,scales", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                          ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("zeros", [False, True])
def test_types(product, dtype, scales, zeros):
    check(case(product, dtype=dtype, scales=scales, zeros=zeros, K=256, group=128, rit=int(zeros)))


@pytest.mark.parametrize("product", PRODUCTS)
@pytest.mark.parametrize("T,G,top_k", [(1, 1, 1), (1, 60, 8), (2, 7, 3), (9, 3, 1), (17, 2, 2),
                                       (40, 4, 4), (70, 3, 2), (150, 2, 1), (300, 3, 2)])
def test_rows(product, T, G, top_k):
    check(case(product, T=T, G=G, top_k=top_k, K=512, N=192, group=128, seed=T))


@pytest.mark.parametrize("product", PRODUCTS)
@pytest.mark.parametrize("K,N,group", [
    (1, 1, 1), (2, 3, 2), (31, 33, 7), (32, 64, 32), (65, 40, 64), (128, 8, 128), (256, 129, 64),
    (384, 96, 128), (1021, 286, 32), (1088, 200, 64), (1024, 136, 256), (640, 64, 1024),
    (992, 72, 96), (1056, 16, 32), (96, 128, 16)])
def test_sizes(product, K, N, group):
    check(case(product, K=K, N=N, group=group, seed=K))


def test_out_fp32():
    s = case("rows", out="fp32", K=512, group=128)
    a = check(s)
    s["out_dtype"] = torch.bfloat16
    assert torch.equal(check(s), a.bfloat16())  # rounded once


@pytest.mark.parametrize("counts", [(0, 40, 0, 0), (38, 0, 1, 1), (0, 0, 0, 40), (7, 8, 9, 16)])
@pytest.mark.parametrize("product", PRODUCTS)
def test_ragged_groups(product, counts):
    """Experts without a row, or with every row (one twice for a token, too)."""
    check(case(product, G=4, counts=counts, K=256, group=128, rit=1))


@pytest.mark.parametrize("product", PRODUCTS)
def test_any_alignment(product):
    s = case(product, K=256, N=64, group=128)
    y = check(s)
    for name in ("x", "codes", "scales", "zeros"):
        buf = torch.zeros(s[name].numel() + 1, dtype=s[name].dtype, device="cuda")
        buf[1:] = s[name].reshape(-1)
        check(dict(s, **{name: buf[1:].view(s[name].shape)}))
    buf = torch.full((y.numel() + 2,), 7.0, dtype=y.dtype, device="cuda")
    check(s, out=buf[1:-1].view(y.shape))
    assert float(buf[0]) == float(buf[-1]) == 7.0


@pytest.mark.parametrize("product", PRODUCTS)
def test_infinities_stay_in_their_rows(product):
    """A token's infinity or NaN, and an expert's infinite scale, reach what they belong to."""
    s = case(product, T=12, G=4, K=256, group=128, zeros=False)
    clean = call(s)[0]
    bad = dict(s, x=s["x"].clone())
    bad["x"][3] = float("inf")
    bad["x"][5] = float("nan")
    got = call(bad)[0]
    if product == "combined":
        hit = torch.tensor([3, 5], device="cuda")
        hit = (s["gather"] // 2)[hit]  # rows 3 and 5 belong to these tokens
        keep = torch.ones(12, dtype=torch.bool, device="cuda")
    else:
        keep = torch.ones(24, dtype=torch.bool, device="cuda")
        token = s["gather"] // 2
        hit = ((token == 3) | (token == 5)).nonzero().reshape(-1)
    keep[hit] = False
    assert torch.equal(got[keep], clean[keep])
    assert not bool(torch.isfinite(got[hit]).any())
    g = int(s["pick"][0])
    bad = dict(s, scales=s["scales"].clone())
    bad["scales"][g] = float("inf")
    got = call(bad)[0]
    if product == "combined":
        keep = torch.ones(12, dtype=torch.bool, device="cuda")
        keep[(s["gather"] // 2)[s["pick"] == g]] = False
    else:
        keep = s["pick"] != g
    assert torch.equal(got[keep], clean[keep]) and not bool(torch.isfinite(got[~keep]).any())


def test_unused_half_of_an_odd_row():
    s = case("rows", K=33, N=16, group=32, dtype="fp32", scales="fp32")
    a = check(s)
    s["codes"][..., -1] ^= 0xF0
    assert torch.equal(check(s), a)


@pytest.mark.parametrize("product", PRODUCTS)
@pytest.mark.parametrize("break_it,status", [
    (lambda s: s["idx"].__setitem__(0, s["idx"][1].clone()), "PGG_ERR_NOT_PERM"),
    (lambda s: s["idx"].__setitem__(2, -1), "PGG_ERR_INDEX"),
    (lambda s: s["groups"].__setitem__(0, s["groups"][0] + 1), "PGG_ERR_GROUPSUM")])
def test_bad_routing_gives_zeros(product, break_it, status):
    s = case(product, K=256, group=128)
    break_it(s)
    got, ws = call(s)
    assert pgg.STATUS[pgg.status(ws)] == status and not bool(got.any())


@pytest.mark.parametrize("product", PRODUCTS)
def test_repeatable_in_a_graph_and_on_a_stream(product):
    s = case(product, T=50, G=4, K=512, group=128, N=320)
    got = check(s)
    out, ws = torch.empty_like(got), call(s)[1]
    ws.fill_(0xAB)  # what a workspace holds does not matter
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(s, out=out, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(s, out=out, workspace=ws)
            call(s, out=out, workspace=ws)
    out.fill_(3)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)


def test_against_the_16_bit_products():
    """Weights that 16 bits hold exactly: the same layer by the framework's other products."""
    s = case("rows", K=256, N=128, group=128, zeros=False, out="fp32")
    s["scales"].fill_(2.0 ** -6)
    w = weights(s).bfloat16()
    other = pgg.fwd(s["x"], w.transpose(1, 2).contiguous(), s["idx"], s["groups"], s["T"], 2, 0,
                    out_dtype=torch.float32)[0]
    y, bound = want(s)
    assert bool(((call(s)[0].double() - other.double()).abs() <= 2 * bound).all())
    h = torch.randn(s["idx"].numel(), 256, device="cuda").bfloat16()
    s = dict(s, product="combined", x=h)
    other = pgg.dx(h, w, s["idx"], s["groups"], s["T"], 2, 0)[0]
    y, bound = want(s)
    assert bool(((call(s)[0].double() - other.double()).abs() <= 2 * bound).all())


def test_wrapper_refusals():
    s = case("rows", K=256, group=128)
    for bad in (dict(codes=s["codes"].to(torch.int16)), dict(scales=s["scales"][..., :1].contiguous()),
                dict(zeros=s["zeros"].float()), dict(idx=s["idx"].int()),
                dict(x=s["x"].t().contiguous().t())):
        with pytest.raises(ValueError):
            call(dict(s, **bad))
    for bad in (dict(group=0), dict(x=s["x"][:, :-2].contiguous()), dict(scales=s["scales"].half()),
                dict(x=s["x"][:-1].contiguous())):
        with pytest.raises(pgg.PggError):
            call(dict(s, **bad))
    with pytest.raises(pgg.PggError):
        call(s, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
