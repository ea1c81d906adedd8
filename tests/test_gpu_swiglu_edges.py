"""Edges of the gated product's gradient: the fp32 gradient of the routing weights from 16-bit rows."""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_swiglu import grad_inputs, grad_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("F", [8, 6])  # 16 bytes a load, an element a load
def test_the_weights_gradient_is_a_32_bit_one(F, dtype):
    # one term a row, d_h silu(gate) up: the exponential within 2 units of 2^-23, its sum with 1 and
    # the three products half a unit, the reciprocal one: 6e-7 relative
    gates = torch.cat([-torch.arange(1, 81, dtype=torch.float32),
                       torch.arange(0, 81, dtype=torch.float32) / 4]).cuda()
    M = gates.numel()
    dh, gu = grad_inputs(M, F, dtype, 40)
    gu[:, :F] = (gates[:, None] * (1 + torch.rand(M, F, device="cuda") / 64)).to(dtype)
    dh[:, 1:] = 0
    idx = torch.randperm(M, device="cuda")
    probs = torch.rand(M, 1, device="cuda") + 0.1
    _, d_p, _, ws = pgg.swiglu_grad(dh, gu, idx, 1, 0, probs=probs)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    _, want, _, pos = grad_reference(dh, gu, None, idx)
    assert ((d_p[pos, 0].double() - want).abs() <= 7e-7 * want.abs() + 2.0 ** -126).all()


def test_the_weights_gradient_beyond_32_bit_offsets():
    # gate_up holds 2.2e9 elements; every row's own first gate tells it from its neighbours
    M, F = 540000, 2048
    idx = torch.randperm(M, device="cuda")
    dh, gu = grad_inputs(1, F, torch.bfloat16, 33)
    gu = gu.expand(M, 2 * F).contiguous()
    gu[:, 0] = torch.arange(M, device="cuda").remainder(64).bfloat16()
    dh = dh.expand(M, F).contiguous()
    dh[:, 0] = 64
    probs = torch.rand(M, 1, device="cuda")
    _, d_p, _, ws = pgg.swiglu_grad(dh, gu, idx, 1, 0, probs=probs)
    torch.cuda.synchronize()
    assert pgg.status(ws) == 0
    rows = torch.cat([torch.arange(64), torch.arange(M - 64, M)]).cuda()
    _, want, h, pos = grad_reference(dh, gu, None, idx, rows)
    # 64 terms a lane and a sum over 32 lanes: 75 roundings of 2^-24
    bound = 75 * 2.0 ** -24 * (dh[rows].double() * h).abs().sum(1)
    off = (d_p[pos, 0].double() - want).abs()
    assert (off <= bound).all()
    # rows that stand for each other would be seen
    assert ((want[:63] - want[1:64]).abs() > 4 * bound[:63]).all()
