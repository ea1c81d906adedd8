"""How many bits the 4-bit products keep where the worst case of a long sum, which bounds the other
tests, would hide a loss: root mean squares at real lengths, and groups of small scales by themselves.

u = 2^-24.
"""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_w4 import built, call, case, want, weights  # noqa: F401
from test_gpu_w4_forms import form  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("zeros,dtype,scales,group", [
    (False, "bf16", "bf16", 128), (True, "bf16", "bf16", 128), (False, "bf16", "fp32", 64),
    (True, "fp16", "fp16", 32), (False, "fp16", "fp32", 128)])
def test_root_mean_square_of_long_sums(form, zeros, dtype, scales, group):  # noqa: F811
    """An adder that cuts off is off by half a step (u of the sum so far) on average, towards zero; a
    random sum's size grows with the root of its length, 2/3 of the last on average over the steps,
    which are at most 2 K / 16 (two products of each 16 of k): K u / 12 of the result. (Weights of 11
    bits, half of a pair of products, would be off by 2^-12 / sqrt(3), 2400 u: 600 are allowed.)"""
    K = 7168
    s = case("rows", T=60, G=2, top_k=1, K=K, N=128, group=group, zeros=zeros, dtype=dtype,
             scales=scales, out="fp32", seed=group)
    got, ws = call(s)
    y, _ = want(s)
    assert pgg.status(ws) == 0
    off = float((got.double() - y).square().mean().sqrt() / y.square().mean().sqrt())
    assert off <= K * U / 12, off / U


@pytest.mark.parametrize("down", [0, -8, -16, -24])
@pytest.mark.parametrize("zeros", [None, 15, 255])
@pytest.mark.parametrize("dtype,scales", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp32")])
def test_a_group_of_small_scales_by_itself(form, dtype, scales, zeros, down):  # noqa: F811
    """x meets only a group whose scales are 2^down of their columns' largest. A weight is off by at
    most 2^-22 of it and by |code - zero| + 1 times 2^-35 of the column's largest scale (2^-31 where
    zeros go up to 255): many rows an expert bring a column to fp16 by one power of two. (Few rows and
    the FP32 pipes keep all of a scale.)"""
    group, K = 64, 512
    s = case("rows", T=48, G=2, top_k=1, K=K, N=96, group=group, zeros=zeros is not None, dtype=dtype,
             scales=scales, out="fp32", seed=7)
    if zeros is not None:
        s["zeros"] = torch.randint(0, zeros + 1, s["zeros"].shape, device="cuda", dtype=torch.uint8)
        s["zeros"][..., 0] = zeros
    s["scales"][..., 3] = torch.ldexp(s["scales"][..., 3].float(), torch.tensor(down)).to(
        s["scales"].dtype)
    s["x"][:, :3 * group] = 0
    s["x"][:, 4 * group:] = 0
    got, ws = call(s)
    y, bound = want(s)
    assert pgg.status(ws) == 0
    w = weights(s)
    largest = s["scales"].double().abs().amax(2, keepdim=True)
    steps = w.abs() / s["scales"].double()[..., 3:4].abs()  # |code - zero| of the group's
    off = w.abs() * 2.0 ** -22 + (steps + 1) * largest * 2.0 ** (-31 if zeros == 255 else -35)
    x = s["x"].double()[s["gather"]].abs()
    more = torch.stack([x[i] @ off[int(s["pick"][i])].T for i in range(x.shape[0])])
    assert bool(((got.double() - y).abs() <= bound + more).all())


@pytest.mark.parametrize("zeros,dtype,scales", [(False, "bf16", "bf16"), (True, "bf16", "fp32"),
                                                (False, "fp16", "fp32"), (True, "fp16", "fp16")])
@pytest.mark.parametrize("product", ["rows", "combined"])
@pytest.mark.parametrize("K", [2048, 7168])
def test_fp32_results_keep_fp32_bits(form, product, zeros, dtype, scales, K):  # noqa: F811
    """Sums that are cut off at every step would lose more the longer they are. Where at most 64 steps
    go into one, each off by u of it on average towards zero (2/3 of its last size on average), that is
    43 u of the result, K / 1024 sums to add K / 1024 u; sums that are rounded K times are off by
    0.58 u at each, at random: 0.58 sqrt(K / 2) u, 35 u."""
    s = case(product, T=60, G=2, top_k=1, K=K, N=128, group=128, zeros=zeros, dtype=dtype,
             scales=scales, out="fp32", seed=K)
    got, ws = call(s)
    y, _ = want(s)
    assert pgg.status(ws) == 0
    off = float((got.double() - y).square().mean().sqrt() / y.square().mean().sqrt())
    assert off <= 50 * U, off / U
