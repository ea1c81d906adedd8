"""The norms around a block, with gate and residual scale, and their gradient against 64-bit
formulas, autograd and differences.

Bounds, u = 2^-24: a row's sums run over at most 8 (long rows: H / 1024) terms a thread and 10
levels, so a mean square is off by at most 64 u of it, a mean by 64 u of the mean size; each is
multiplied through in a handful of steps. Outputs are rounded once, by half a step of their type.
"""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
PARAMS = ("post_weight", "post_bias", "pre_weight", "pre_bias")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def case(T=5, H=256, dtype="bf16", y="fp32", post="rms", pre="rms", gate="channel", params="fp32",
         bias=True, weight=True, seed=0, residual_scale=0.75, offset=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dt, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(DT[dt])

    s = dict(x=normal(T, H, dt=dtype, std=2.0), y=normal(T, H, dt=y) if y else None,
             post=post, pre=pre, residual_scale=residual_scale, weight_offset=offset, eps=1e-5)
    shape = dict(channel=(H,), token=(T, 1), full=(T, H)).get(gate)
    s["gate"] = normal(*shape, dt=params, std=0.5) if shape else None
    for side in ("post", "pre"):
        has = s[side] is not None and weight
        s[side + "_weight"] = (normal(H, dt="fp32", std=0.3) + 1 - offset).to(DT[params]) \
            if has else None
        s[side + "_bias"] = normal(H, dt=params, std=0.2) if s[side] == "layer" and bias else None
    s["d_r"] = normal(T, H, dt=dtype)
    s["d_h"] = normal(T, H, dt=y or dtype) if pre else None
    return s


def norm(kind, v, w, b, s):
    if kind is None:
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    n = v / (v.square().mean(1, keepdim=True) + s["eps"]).sqrt()
    n = n * (w + s["weight_offset"]) if w is not None else n
    return n + b if b is not None else n


def formula(s, p):
    """(r, h) in 64 bits from the tensors in p."""
    r = s["residual_scale"] * p["x"]
    if p["y"] is not None:
        n = norm(s["post"], p["y"], p["post_weight"], p["post_bias"], s)
        r = r + (p["gate"] * n if p["gate"] is not None else n)
    return r, norm(s["pre"], r, p["pre_weight"], p["pre_bias"], s)


def doubles(s, names=("x", "y", "gate") + PARAMS):
    return {n: s[n].double() if s[n] is not None else None for n in names}


def kwargs(s):
    return {n: s[n] for n in ("gate", "post", "pre", "residual_scale", "weight_offset", "eps")
            + PARAMS}


def near(got, want, slack, what):
    """Within half a step of the type and `slack` (of the values the result is a sum of)."""
    half = torch.finfo(got.dtype).eps / 2
    bound = half * want.abs() + slack * (1 + half) + torch.finfo(got.dtype).smallest_normal
    over = (got.double() - want).abs() - bound
    assert bool((over <= 0).all()), (what, float(over.max()))


def size(t, dim=1):
    """The root mean square of a row (what a row's sums are relative to), at least tiny."""
    return t.square().mean(dim, keepdim=True).sqrt() + 1e-30


def check_forward(s, **kw):
    r, h = pgg.block_norm(s["x"], s["y"], **kwargs(s), **kw)
    p = doubles(s)
    want_r, want_h = formula(s, p)
    scale = 96 * U * (want_r.abs() + (s["residual_scale"] * p["x"]).abs()
                      + 2 * size(want_r - s["residual_scale"] * p["x"])
                      + (want_r - s["residual_scale"] * p["x"]).abs())
    if s["gate"] is not None or s["post_bias"] is not None:
        # (a mean's error is of the rows' size, and the gate and weight scale it)
        n = norm(s["post"], p["y"], p["post_weight"], p["post_bias"], s) if p["y"] is not None else 0
        scale = scale + 96 * U * (1 + (p["gate"].abs() if p["gate"] is not None else 1)) * (
            4 + (n.abs() if p["y"] is not None else 0))
    near(r, want_r, scale, "r")
    if s["pre"]:
        rstd = 1 / (size(want_r) if s["pre"] == "rms"
                    else size(want_r - want_r.mean(1, keepdim=True)))
        w = p["pre_weight"].abs().max() + abs(s["weight_offset"]) if p["pre_weight"] is not None else 1
        slack = w * rstd * (scale + size(scale)) + 96 * U * (want_h.abs() + 4 * w + 1)
        near(h, want_h, slack, "h")
    else:
        assert h is None
    return r, h


KINDS = [(post, pre) for post in (None, "rms", "layer") for pre in (None, "rms", "layer")]


@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("H", [256, 77])
def test_forward_kinds(post, pre, gate, H):
    check_forward(case(post=post, pre=pre, gate=gate, H=H))


TYPES = [("bf16", "bf16", "bf16"), ("bf16", "fp32", "bf16"), ("bf16", "fp32", "fp32"),
         ("fp16", "fp16", "fp32"), ("fp16", "fp32", "fp16"), ("fp32", "fp32", "fp32")]


@pytest.mark.parametrize("dtype,y,params", TYPES)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7168), (3, 8), (4, 100), (7, 1021), (2, 2056),
                                 (3, 9000), (400, 512), (2, 20000), (2, 40000), (1, 8191)])
def test_forward_sizes(dtype, y, params, T, H):
    check_forward(case(T, H, dtype, y, params=params, post="layer", pre="layer", gate="full",
                       offset=1.0))


def test_forward_without_parts():
    check_forward(case(y=None, post=None, gate=None))
    check_forward(case(weight=False, bias=False, post="layer", pre="layer", gate=None))
    s = case(post=None, gate=None, weight=False)
    r, h = pgg.block_norm(s["x"], s["y"], **kwargs(s))
    x = s["x"].clone()
    out = pgg.block_norm(x, s["y"], r=x, **kwargs(s))  # in place
    assert out[0] is x and torch.equal(x, r) and torch.equal(out[1], h)


def test_h_is_taken_before_r_is_rounded():
    """r's rounding (2^-9 of it) must not show in an fp32-accurate h: rows of one large and many
    small values, where the rounded row has another norm."""
    s = case(T=4, H=512, dtype="bf16", post=None, gate=None, weight=False)
    s["x"].zero_()
    s["y"] = torch.full_like(s["y"], 1.0 + 2.0 ** -9)  # halfway between bf16 values
    s["y"][:, 0] = 64.0
    _, h = pgg.block_norm(s["x"], s["y"], **kwargs(s))
    want = formula(s, doubles(s))[1]
    near(h, want, 64 * U * want.abs(), "h")


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 0.0])
@pytest.mark.parametrize("H", [512, 77])
def test_special_rows(bad, H):
    """A row of zeros is finite; what one row holds does not reach another."""
    s = case(T=6, H=H, post="layer", pre="layer")
    r, h = pgg.block_norm(s["x"], s["y"], **kwargs(s))
    got, _ = pgg.block_norm_grad(s["d_r"], s["d_h"], r, s["y"], **kwargs(s))
    t = dict(s, x=s["x"].clone(), y=s["y"].clone())
    t["x"][2] = bad
    t["y"][2] = bad
    r2, h2 = pgg.block_norm(t["x"], t["y"], **kwargs(t))
    got2, _ = pgg.block_norm_grad(t["d_r"], t["d_h"], r2, t["y"], **kwargs(t))
    keep = torch.arange(6, device="cuda") != 2
    for a, b in ((r, r2), (h, h2), (got["d_x"], got2["d_x"]), (got["d_y"], got2["d_y"])):
        assert torch.equal(a[keep], b[keep])
        assert bool(torch.isfinite(b[2]).all()) == (bad == 0.0)


def check_backward(s, **kw):
    """Against autograd in 64 bits on the rounded r that the forward returned."""
    r = pgg.block_norm(s["x"], s["y"], **kwargs(s))[0]
    got, ws = pgg.block_norm_grad(s["d_r"], s["d_h"], r if s["pre"] else None, s["y"], **kwargs(s),
                                  **kw)
    assert pgg.status(ws) == 0
    p = doubles(s, ("y", "gate") + PARAMS)
    T, H = s["x"].shape
    p = {n: t.requires_grad_() if t is not None else None for n, t in p.items()}
    p["x"] = torch.zeros(T, H, dtype=torch.double, device="cuda")
    out, _ = formula(s, p)
    p["x"] = ((r.double() - out.detach()) / s["residual_scale"]).requires_grad_()
    out, h = formula(s, p)
    loss = (out * s["d_r"].double()).sum() if s["d_r"] is not None else 0
    loss = loss + ((h * s["d_h"].double()).sum() if s["pre"] else 0)
    names = [n for n, t in p.items() if t is not None]
    want = dict(zip(names, torch.autograd.grad(loss, [p[n] for n in names])))
    # magnitudes that the sums are relative to
    with torch.no_grad():
        g_parts = (s["d_r"].double().abs() if s["d_r"] is not None else 0) + 0 * r.double()
        if s["pre"]:
            v = r.double() - (r.double().mean(1, keepdim=True) if s["pre"] == "layer" else 0)
            rstd = 1 / (v.square().mean(1, keepdim=True) + s["eps"]).sqrt()
            f = (p["pre_weight"] + s["weight_offset"]).abs() if p["pre_weight"] is not None else 1
            u = s["d_h"].double().abs() * f
            vh = (v * rstd).abs()
            g_parts = g_parts + rstd * (u + (1 + vh) * (u.mean(1, keepdim=True)
                                                        + (u * (1 + vh)).mean(1, keepdim=True)))
            dw = s["d_h"].double().abs() * (1 + vh)
        tol = 256 * U
        near(got["d_x"], want["x"], tol * s["residual_scale"] * g_parts, "d_x")
        if s["pre_weight"] is not None:
            near(got["d_pre_weight"], want["pre_weight"], tol * dw.sum(0), "d_pre_weight")
        if s["pre_bias"] is not None:
            near(got["d_pre_bias"], want["pre_bias"], tol * dw.sum(0), "d_pre_bias")
        if s["y"] is None:
            assert got["d_y"] is None
            return got
        y = p["y"]
        gate = p["gate"].abs() if p["gate"] is not None else 1
        f = (p["post_weight"] + s["weight_offset"]).abs() if p["post_weight"] is not None else 1
        b = p["post_bias"].abs() if p["post_bias"] is not None else 0
        if s["post"]:
            v = y - (y.mean(1, keepdim=True) if s["post"] == "layer" else 0)
            rstd = 1 / (v.square().mean(1, keepdim=True) + s["eps"]).sqrt()
            vh = (v * rstd).abs() + 1
            u = g_parts * gate * f
            dy = rstd * (u + vh * (u.mean(1, keepdim=True) + (u * vh).mean(1, keepdim=True)))
        else:
            vh = y.abs()
            dy = g_parts * gate
        near(got["d_y"], want["y"], tol * dy, "d_y")
        if s["gate"] is not None:
            whole = g_parts * (vh * f + b)
            for shape, dim in (((H,), 0), ((T, 1), 1)):
                if tuple(s["gate"].shape) == shape != (T, H):
                    whole = whole.sum(dim, keepdim=dim == 1)
            assert got["d_gate"].shape == s["gate"].shape
            near(got["d_gate"], want["gate"], tol * whole, "d_gate")
        if s["post_weight"] is not None:
            near(got["d_post_weight"], want["post_weight"], tol * (g_parts * gate * vh).sum(0),
                 "d_post_weight")
        if s["post_bias"] is not None:
            near(got["d_post_bias"], want["post_bias"], tol * (g_parts * gate * vh).sum(0),
                 "d_post_bias")
    return got


@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("H", [256, 77])
def test_backward_kinds(post, pre, gate, H):
    check_backward(case(post=post, pre=pre, gate=gate, H=H))


@pytest.mark.parametrize("dtype,y,params", TYPES)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7168), (3, 8), (4, 100), (7, 1021), (2, 2056),
                                 (3, 9000), (700, 512), (2, 20000), (310, 65), (1, 8191),
                                 (2, 17000)])
def test_backward_sizes(dtype, y, params, T, H):
    check_backward(case(T, H, dtype, y, params=params, post="layer", pre="layer", gate="channel",
                        offset=1.0))
    check_backward(case(T, H, dtype, y, params=params, gate="full"))


def test_backward_without_parts():
    check_backward(case(y=None, post=None, gate=None))
    check_backward(dict(case(), d_r=None))
    check_backward(case(weight=False, bias=False, post="layer", pre="layer", gate="token"))
    s = case()
    r = pgg.block_norm(s["x"], s["y"], **kwargs(s))[0]
    want, _ = pgg.block_norm_grad(s["d_r"], s["d_h"], r, s["y"], **kwargs(s))
    d = s["d_r"].clone()
    got, _ = pgg.block_norm_grad(d, s["d_h"], r, s["y"], d_x=d, **kwargs(s))  # in place
    assert got["d_x"] is d and all(torch.equal(got[n], want[n]) for n in got if want[n] is not None)


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
def test_differences(gate):
    """d(loss) along random directions from the kernel's gradients and from 64-bit differences of
    the formula: quadratic in the step, so 1e-6 of the values is left; fp32 gradients give 1e-4."""
    s = case(T=3, H=40, dtype="fp32", post="layer", pre="rms", gate=gate)
    got = check_backward(s)
    p = doubles(s)
    r0 = pgg.block_norm(s["x"], s["y"], **kwargs(s))[0].double()
    p["x"] = p["x"] + (r0 - formula(s, p)[0]) / s["residual_scale"]

    def loss(p):
        r, h = formula(s, p)
        return (r * s["d_r"].double()).sum() + (h * s["d_h"].double()).sum()

    gen = torch.Generator(device="cuda").manual_seed(3)
    for name in ("x", "y", "gate") + PARAMS:
        if p[name] is None:
            continue
        d = torch.randn(p[name].shape, generator=gen, device="cuda", dtype=torch.double)
        step = 1e-4
        slope = (loss(dict(p, **{name: p[name] + step * d}))
                 - loss(dict(p, **{name: p[name] - step * d}))) / (2 * step)
        along = (got["d_" + name].double() * d).sum()
        size = (got["d_" + name].double() * d).abs().sum()
        assert abs(float(slope - along)) <= 1e-4 * float(size), name


def test_repeatable_in_a_graph_and_any_alignment():
    s = case(T=350, H=512, post="layer", pre="layer")
    r, h = pgg.block_norm(s["x"], s["y"], **kwargs(s))
    want, ws = pgg.block_norm_grad(s["d_r"], s["d_h"], r, s["y"], **kwargs(s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws.fill_(0xFF)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r2, h2 = pgg.block_norm(s["x"], s["y"], **kwargs(s))
            got, _ = pgg.block_norm_grad(s["d_r"], s["d_h"], r2, s["y"], workspace=ws, **kwargs(s))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, r2) and torch.equal(h, h2)
    assert all(torch.equal(got[n], want[n]) for n in want)
    for name in ("x", "y", "gate", "d_r", "d_h") + PARAMS:
        buf = torch.zeros(s[name].numel() + 1, dtype=s[name].dtype, device="cuda")
        buf[1:] = s[name].reshape(-1)
        t = dict(s, **{name: buf[1:].view(s[name].shape)})
        check_forward(t)
        check_backward(t)


def test_more_rows_than_an_offset_of_32_bits_holds():
    """T H past 2^32: the last rows are right."""
    T, H = 2**19 + 3, 8192
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, H, device="cuda").bfloat16()
    r, h = pgg.block_norm(x, residual_scale=0.5)
    assert torch.equal(r[-5:], x[-5:] * 0.5)
    small, hs = pgg.block_norm(x[-5:].clone(), residual_scale=0.5)
    assert torch.equal(h[-5:], hs) and not bool(h[:100].any())
    got, _ = pgg.block_norm_grad(None, h, r)
    few, _ = pgg.block_norm_grad(None, hs, small)
    assert torch.equal(got["d_x"][-5:], few["d_x"])


def test_wrapper_refusals():
    s = case()
    for bad in (dict(gate=s["gate"][:-1].contiguous()), dict(post="l2"), dict(pre=7),
                dict(post_weight=s["post_weight"].half()), dict(gate=s["gate"].double())):
        with pytest.raises((ValueError, pgg.PggError)):
            pgg.block_norm(s["x"], s["y"], **dict(kwargs(s), **bad))
    with pytest.raises(pgg.PggError):
        pgg.block_norm(s["x"], s["y"].half(), **kwargs(s))
    with pytest.raises(pgg.PggError):
        pgg.block_norm(s["x"], s["y"][:-1].contiguous(), **kwargs(s))
    with pytest.raises(pgg.PggError):
        pgg.block_norm(s["x"], None, **kwargs(s))
    with pytest.raises(pgg.PggError):
        pgg.block_norm_grad(None, None, s["x"], s["y"], **kwargs(s))
    with pytest.raises(pgg.PggError):
        pgg.block_norm_grad(s["d_r"], s["d_h"], s["x"], s["y"],
                            workspace=s["x"].view(torch.uint8)[:1].reshape(-1)[:256], **kwargs(s))
