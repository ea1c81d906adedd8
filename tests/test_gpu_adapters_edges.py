"""Edges of the adapters' calls that the parity tests' sizes and tensors do not reach."""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_adapters import expand, inputs, low_rank, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def shifted(shape, dtype, by, value=7.0):
    """(buffer, view of it that starts `by` elements into it)."""
    n = 1
    for d in shape:
        n *= d
    buf = torch.full((n + by + 8,), value, dtype=dtype, device="cuda")
    assert buf.data_ptr() % 16 == 0
    return buf, buf[by:by + n].view(shape)


# every form that a call may take: one token, blocks of 16, 32 and 64 tokens, several blocks, the
# tokens sorted, the FP32 pipes (an odd width, fp32)
@pytest.mark.parametrize("by", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("T,K,N,R,dtype", [
    (1, 256, 128, 16, "bf16"), (16, 256, 136, 8, "fp16"), (30, 512, 264, 16, "bf16"),
    (64, 256, 128, 32, "bf16"), (200, 256, 192, 16, "bf16"), (700, 256, 192, 16, "fp16"),
    (20, 100, 51, 5, "bf16"), (20, 64, 64, 8, "fp32")])
def test_an_output_at_any_element(T, K, N, R, dtype, by):
    # y may start at any element; whatever width a form writes, nothing around it changes
    s = inputs(T, K, N, R, 3, dtype=dtype, seed=T + by)
    buf, y = shifted((T, N), s["x"].dtype, by)
    _, ws = pgg.adapters(**s, out=y)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    assert (buf[:by] == 7.0).all() and (buf[by + T * N:] == 7.0).all()
    u = low_rank(s["x"], s["a"], s["adapter"], s["scale"])
    ref = s["x"].double() @ s["weight"].double() + expand(u, s["b"], s["adapter"])
    near(y, ref, expand(u.abs(), s["b"].abs(), s["adapter"]))


@pytest.mark.parametrize("T", [200, 700])
@pytest.mark.parametrize("name", ["d_x", "d_a", "d_b"])
def test_a_gradient_at_any_element(T, name):
    s = inputs(T, 256, 192, 16, 3, seed=T)
    d_y = torch.randn(T, 192, device="cuda").bfloat16()
    d_x, d_a, d_b, _ = pgg.adapters_grad(d_y, **s)
    want = dict(d_x=d_x, d_a=d_a, d_b=d_b)
    for by in (1, 2, 4):
        buf, view = shifted(tuple(want[name].shape), torch.bfloat16, by)
        got = pgg.adapters_grad(d_y, **s, **{name: view})
        torch.cuda.synchronize()
        n = view.numel()
        assert (buf[:by] == 7.0).all() and (buf[by + n:] == 7.0).all()
        # each side rounds the sum and the low-rank row once
        for g, w in zip(got[:3], want.values()):
            assert (g.double() - w.double()).abs().max() <= 3 * 2.0 ** -8 * w.double().abs().max()


# ------------------------------------------------------- infinities at an adapter's last token

COUNTS = (1, 127, 128, 129, 300)


def with_counts(order, dtype, K=64, N=72, R=16):
    """Inputs whose adapters have COUNTS tokens, in runs or mixed, and each one's last token."""
    T = sum(COUNTS)
    s = inputs(T, K, N, R, len(COUNTS), dtype=dtype, seed=91)
    ids = torch.repeat_interleave(torch.arange(len(COUNTS)), torch.tensor(COUNTS))
    if order == "mixed":
        ids = ids[torch.randperm(T, generator=torch.Generator().manual_seed(3))]
    s["adapter"] = ids.cuda()
    last = [int((ids == i).nonzero().max()) for i in range(len(COUNTS))]
    return s, last


# on the tensor cores; with an odd rank (the weight-gradient kernel that gathers both operands); with
# an output off a 16-byte boundary; on the FP32 pipes
@pytest.mark.parametrize("form", ["tensor", "rank 10", "unaligned", "pipes", "fp32"])
@pytest.mark.parametrize("order", ["runs", "mixed"])
def test_an_infinity_at_an_adapters_last_token_stays_one(order, form):
    dtype = {"tensor": "bf16", "fp32": "fp32"}.get(form, "fp16")
    s, last = with_counts(order, dtype, R=10 if form == "rank 10" else 16)
    T, N, R = s["x"].shape[0], s["weight"].shape[1], s["a"].shape[2]
    d_y = torch.randn(T, N, device="cuda").to(s["x"].dtype)
    out = {}
    if form == "unaligned":
        out = dict(d_a=shifted(tuple(s["a"].shape), s["a"].dtype, 4)[1],
                   d_b=shifted(tuple(s["b"].shape), s["b"].dtype, 4)[1])

    def grads(s, d_y):
        if form == "pipes":
            pgg.pgg_debug_force_variant(3)
        try:
            got = pgg.adapters_grad(d_y, **s, **out)
        finally:
            pgg.pgg_debug_force_variant(-1)
        torch.cuda.synchronize()
        assert pgg.status(got[3]) == 0
        return got[0], got[1].clone(), got[2].clone()

    _, d_a, d_b = grads(s, d_y)
    assert torch.isfinite(d_a).all() and torch.isfinite(d_b).all()
    v = low_rank(d_y, s["b"], s["adapter"], s["scale"])
    u = low_rank(s["x"], s["a"], s["adapter"], s["scale"])
    for i, t in enumerate(last):
        x2, dy2 = s["x"].clone(), d_y.clone()
        x2[t, 5] = float("inf")
        dy2[t, 7] = float("-inf")
        # x^T v: the column of the infinity is infinite with v's signs, the others are as before
        _, got, _ = grads(dict(s, x=x2), d_y)
        assert torch.equal(got[i, 5].double(), torch.sign(v[t]) * float("inf"))
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[i, 5] = False
        assert torch.equal(got[rest], d_a[rest])
        # d_y^T u alike
        _, _, got = grads(s, dy2)
        assert torch.equal(got[i, 7].double(), torch.sign(u[t]) * float("-inf"))
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[i, 7] = False
        assert torch.equal(got[rest], d_b[rest])
