"""Layer norms of rows whose first elements lie far from the row's mean, to the precision of fp32 and
whatever the row's length and alignment are: outputs of 16 bits would hide what is looked for.

Bounds, u = 2^-24, v^ a normalised element. A block's sum of squares is off by at most 24 u of it (16
terms a thread, 10 levels of exchanges, each square's own rounding). Squares about a number within two
deviations of the mean are at most five times the variance, so that is off by at most 120 u, 1 /
deviation by 60 u. A sum of v - k is off by 24 u of the sum of |v - k|, at most sqrt(5) deviations: a
mean by 54 u of the deviation. So v^ is off by at most u (60 |v^| + 54 + 2 |mean| / deviation + 4 (1 +
|v^|)), the last from a handful of steps on the way.
"""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_block_norm import DT, built  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


def rows(T, H, dtype, gen, first):
    """Rows about 0 or 5 that begin with an outlier (every other one with two), or with eight."""
    v = torch.randn(T, H, generator=gen, device="cuda")
    v[::3] += 5.0
    if first == "one":
        v[:, 0] = 200.0
        v[1::2, min(1, H - 1)] = -150.0
    else:
        v[:, :8] += torch.linspace(1.5, 30.0, T, device="cuda")[:, None]
    return v.to(DT[dtype])


def norm(v):
    """(v^, bound of its error) in 64 bits."""
    v = v.double()
    mean = v.mean(1, keepdim=True)
    dev = ((v - mean).square().mean(1, keepdim=True) + EPS).sqrt()
    n = (v - mean) / dev
    return n, U * (64 * n.abs() + 58 + 2 * mean.abs() / dev)


def within(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    over = (got.double() - want).abs() - (bound * (1 + half) + half * want.abs())
    assert bool((over <= 0).all()), (what, float((over / bound).max()))


SIZES = [40, 64, 1021, 1028, 4096, 4099, 7168, 7200, 8192, 8196]


@pytest.mark.parametrize("first", ["one", "moved"])
@pytest.mark.parametrize("H", SIZES)
def test_forward(H, first):
    T = 40 if H > 64 else 3000
    gen = torch.Generator(device="cuda").manual_seed(H)
    x, y = (rows(T, H, "fp32", gen, first) for _ in range(2))
    r, h = pgg.block_norm(x, y, post="layer", pre="layer", eps=EPS)
    n, bound = norm(y)
    want = x.double() + n
    bound = bound + 2 * U * (n.abs() + want.abs())
    within(r, want, bound, "r")
    want_h, own = norm(want)
    mean = want.mean(1, keepdim=True)
    rstd = 1 / ((want - mean).square().mean(1, keepdim=True) + EPS).sqrt()
    size = bound.square().mean(1, keepdim=True).sqrt()
    within(h, want_h, own + rstd * (bound + size * (1 + want_h.abs())), "h")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("first", ["one", "moved"])
@pytest.mark.parametrize("side", ["pre", "post"])
@pytest.mark.parametrize("H", SIZES)
def test_gradient(H, side, first, dtype):
    """One norm at a time. A weight's gradient sums d v^ over the rows (30 u of the terms' sizes for
    the sum); with d of one sign in a column the errors of v^ do not cancel. An input's gradient has
    three terms, rstd (u - v^ mean(u v^) - mean(u)); with A = mean |u v^| and C = mean |u| the errors
    of rstd (64 u of each term), v^ (64 |v^| + 64) and the means (24 u of A + 4 C, 60 u of A for its
    rstd) are at most 224 u (|u| + (1 + |v^|) (A + C)) rstd together."""
    T = 40 if H > 64 else 1500
    gen = torch.Generator(device="cuda").manual_seed(H)
    v = rows(T, H, dtype, gen, first)
    d = torch.randn(T, H, generator=gen, device="cuda")
    d[:, ::5] = d[:, ::5].abs()
    d = d.to(DT[dtype])
    w = 1 + 0.2 * torch.randn(H, generator=gen, device="cuda")
    b = torch.zeros(H, device="cuda")
    if side == "pre":
        got, _ = pgg.block_norm_grad(None, d, v, pre="layer", pre_weight=w, pre_bias=b, eps=EPS)
        d_v = got["d_x"]
    else:
        got, _ = pgg.block_norm_grad(d, None, None, v, post="layer", post_weight=w, post_bias=b,
                                     pre=None, eps=EPS)
        d_v = got["d_y"]
    n, bound = norm(v)
    d = d.double()
    within(got[f"d_{side}_weight"], (d * n).sum(0), (d.abs() * (bound + 30 * U * n.abs())).sum(0),
           "weight")
    u = d * w.double()
    rstd = 1 / ((v.double() - v.double().mean(1, keepdim=True)).square().mean(1, keepdim=True)
                + EPS).sqrt()
    want = rstd * (u - n * (u * n).mean(1, keepdim=True) - u.mean(1, keepdim=True))
    a, c = (u * n).abs().mean(1, keepdim=True), u.abs().mean(1, keepdim=True)
    far = 2 * v.double().mean(1, keepdim=True).abs() * rstd  # (v^'s error for rows away from zero)
    within(d_v, want, U * rstd * (224 * (u.abs() + (1 + n.abs()) * (a + c)) + far * (a + c)), "input")


@pytest.mark.parametrize("gate", ["token", "full"])
def test_gates_of_a_row(gate):
    """The same gradients wherever in the row the outlier lies (a layer norm does not see it)."""
    T, H = 200, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(T, H, generator=gen, device="cuda")
    y[:, 0] = 64.0
    # permuted, the outlier lies in the middle
    order = torch.arange(H, device="cuda").roll(H // 2)
    d = torch.randn(T, H, generator=gen, device="cuda")
    w = 1 + 0.2 * torch.randn(H, generator=gen, device="cuda")
    g = torch.randn(T, H if gate == "full" else 1, generator=gen, device="cuda")
    first, _ = pgg.block_norm_grad(d, None, None, y, gate=g, post="layer", post_weight=w, pre=None)
    moved = g[:, order].contiguous() if gate == "full" else g
    second, _ = pgg.block_norm_grad(d[:, order].contiguous(), None, None, y[:, order].contiguous(),
                                    gate=moved, post="layer", post_weight=w[order], pre=None)
    n = norm(y)[0]
    for name in ("d_x", "d_y", "d_gate", "d_post_weight"):
        a, b = first[name], second[name]
        a = a[..., order] if a.shape[-1] == H else a
        n_at = n[:, order].abs()
        # each within 224 u of its terms, as above; |d g w| is at most 40, |v^| its own
        size = 40 * (1 + n_at)
        if name == "d_post_weight":
            size = size.sum(0)
        if name == "d_gate" and gate == "token":
            size = size.sum(1, keepdim=True)
        assert bool(((a.double() - b.double()).abs() <= 2 * 224 * U * size).all()), name


@pytest.mark.parametrize("many", [4, 8, 64])
@pytest.mark.parametrize("H", [4096, 8192])
def test_rows_with_and_without_outliers_in_turn(H, many):
    """Rows that need their sums once more beside rows that do not, in every order."""
    T = 700
    gen = torch.Generator(device="cuda").manual_seed(H)
    y = torch.randn(T, H, generator=gen, device="cuda")
    y[torch.rand(T, generator=gen, device="cuda") < 0.5, :many] += 50.0
    r, _ = pgg.block_norm(torch.zeros_like(y), y, post="layer", pre=None, eps=EPS)
    n, bound = norm(y)
    within(r, n, bound, "r")
    w = torch.ones(H, device="cuda")
    d = torch.ones_like(y)
    got, _ = pgg.block_norm_grad(d, None, None, y, post="layer", post_weight=w, pre=None, eps=EPS)
    within(got["d_post_weight"], n.sum(0), (bound + 30 * U * n.abs()).sum(0), "weight")
