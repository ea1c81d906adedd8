"""The norms around a block over many rows a block of threads, with rows on their way in shared
memory, and layer norms whose rows lie far from zero or begin with an outlier. Bounds as in
test_gpu_block_norm.
"""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_block_norm import (built, case, check_backward, check_forward,  # noqa: F401
                                 kwargs)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("post,pre,gate,bias", [
    ("rms", "rms", "channel", False), ("rms", "rms", None, False), (None, "rms", "channel", False),
    ("rms", None, "channel", False), ("layer", "layer", "channel", True),
    ("layer", "rms", "token", True), ("rms", "layer", "full", True), (None, "layer", "token", True),
    ("layer", None, "full", False)])
@pytest.mark.parametrize("T,H", [(700, 64), (1300, 1032), (640, 4096), (460, 7168), (310, 8192)])
def test_many_rows(post, pre, gate, bias, T, H):
    s = case(T=T, H=H, post=post, pre=pre, gate=gate, bias=bias, params="bf16", seed=H)
    check_forward(s)
    check_backward(s)


@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "channel"), ("layer", "layer", "full"),
                                           ("layer", "rms", "token")])
@pytest.mark.parametrize("dtype,y,params,H", [
    ("bf16", "bf16", "fp32", 7168), ("bf16", "fp32", "fp32", 2056), ("fp16", "fp32", "fp16", 520),
    ("fp32", "fp32", "fp32", 7168), ("fp32", "fp32", "fp32", 7200), ("fp32", "fp32", "fp32", 1028),
    ("bf16", "fp32", "bf16", 8200), ("fp16", "fp16", "fp16", 16392)])
def test_many_rows_types(dtype, y, params, H, post, pre, gate):
    s = case(T=340, H=H, dtype=dtype, y=y, params=params, post=post, pre=pre, gate=gate, seed=H)
    check_forward(s)
    check_backward(s)


@pytest.mark.parametrize("H", [64, 1021, 4096])
def test_rows_that_begin_with_an_outlier(H):
    """A layer norm's sums are taken about the mean of the row's first vector: with an element of
    200 deviations in it, that lies up to sqrt(H / 8) deviations from the row's mean, which costs at
    most H / 8 steps of 2^-24 of the variance, twice that for its second use: 2^-15 of the result
    at H = 4096, less than an eighth of the output's half step."""
    s = case(T=320, H=H, post="layer", pre="layer", gate=None, weight=False, bias=False, y="bf16")
    s["y"][:, 0] = 200.0
    s["x"][::2, 1] = -150.0
    for t in range(0, 320, 2):
        s["y"][t] += 8.0  # (rows away from zero)
    r, h = pgg.block_norm(s["x"], s["y"], **kwargs(s))
    y = s["y"].double()

    def norm(v):
        v = v - v.mean(1, keepdim=True)
        return v / (v.square().mean(1, keepdim=True) + 1e-5).sqrt()

    want = s["residual_scale"] * s["x"].double() + norm(y)
    # (an element is as far off as its own rounding, the mean's and the deviation's)
    off = (r.double() - want).abs() / (want.abs() + norm(y).abs() + 1)
    assert float(off.max()) <= 2.0 ** -8 + 2.0 ** -14
    off = (h.double() - norm(want)).abs() / (norm(want).abs() + 1)
    assert float(off.max()) <= 2.0 ** -8 + 2.0 ** -13


@pytest.mark.parametrize("gate,post", [("channel", "rms"), ("full", "layer"), ("token", "layer")])
@pytest.mark.parametrize("y", ["fp32", "bf16"])
def test_the_same_bits_each_time(gate, post, y):
    s = case(T=3000, H=7168, post=post, pre=post, gate=gate, params="bf16", y=y)
    r, h = pgg.block_norm(s["x"], s["y"], **kwargs(s))
    args = (s["d_r"], s["d_h"], r, s["y"])
    first = pgg.block_norm_grad(*args, **kwargs(s))[0]
    for _ in range(8):
        r2, h2 = pgg.block_norm(s["x"], s["y"], **kwargs(s))
        assert torch.equal(r, r2) and torch.equal(h, h2)
        again = pgg.block_norm_grad(*args, **kwargs(s))[0]
        for name, g in first.items():
            assert (g is None and again[name] is None) or torch.equal(g, again[name]), name


@pytest.mark.parametrize("gate", ["channel", "full"])
def test_in_place(gate):
    s = case(T=500, H=4096, gate=gate, params="bf16")
    r, h = pgg.block_norm(s["x"], s["y"], **kwargs(s))
    x = s["x"].clone()
    r2, h2 = pgg.block_norm(x, s["y"], r=x, **kwargs(s))
    assert torch.equal(r, x) and torch.equal(h, h2) and r2.data_ptr() == x.data_ptr()
    want = pgg.block_norm_grad(s["d_r"], s["d_h"], r, s["y"], **kwargs(s))[0]
    d = s["d_r"].clone()
    got = pgg.block_norm_grad(d, s["d_h"], r, s["y"], d_x=d, **kwargs(s))[0]
    for name, g in want.items():
        assert g is None or torch.equal(g, got[name]), name


@pytest.mark.parametrize("post,pre,gate,bias", [("rms", "rms", "channel", False),
                                                ("layer", "layer", "full", True),
                                                ("layer", "rms", "token", True)])
@pytest.mark.parametrize("dtype,y,H", [("bf16", "fp32", 3001), ("bf16", "bf16", 6998),
                                       ("fp16", "fp32", 8191), ("fp32", "fp32", 5003),
                                       ("bf16", "fp32", 8193), ("fp16", "fp16", 16382),
                                       ("bf16", "bf16", 16386)])
def test_long_rows_of_odd_lengths(dtype, y, H, post, pre, gate, bias):
    s = case(T=170, H=H, dtype=dtype, y=y, params=dtype, post=post, pre=pre, gate=gate, bias=bias,
             seed=H)
    check_forward(s)
    check_backward(s)
