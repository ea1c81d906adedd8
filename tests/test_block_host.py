"""The 4-bit experts, the norms around a block and the clipping of gradients refuse bad arguments
on the host, before any CUDA call (no GPU)."""

import ctypes

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from permute_grouped_gemm_gb300 import build as pbuild

FAKE = 1 << 20  # an aligned address that is never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def built():
    pbuild.build()
    pgg.load()


def name(rc):
    return pgg.STATUS[rc]


W4 = dict(product=pgg.PGG_W4_GATED, x=FAKE, codes=FAKE, scales=FAKE, zeros=FAKE,
          expandedRowIdx=FAKE, groupList=FAKE, probs=FAKE, M=48, N=32, K=64, G=4, L=48, batch=24,
          topK=2, rowIdxType=0, groupSize=32, dtype=pgg.PGG_BF16, scale_dtype=pgg.PGG_F32,
          out_dtype=pgg.PGG_BF16, workspace=FAKE, workspace_bytes=1 << 30, out=FAKE, stream=None)
ROWS, COMBINED = pgg.PGG_W4_ROWS, pgg.PGG_W4_COMBINED


@pytest.mark.parametrize("change,want", [
    (dict(x=0), "NULL"), (dict(codes=0), "NULL"), (dict(scales=0), "NULL"), (dict(out=0), "NULL"),
    (dict(expandedRowIdx=0), "NULL"), (dict(groupList=0), "NULL"), (dict(workspace=0), "NULL"),
    (dict(product=3), "ATTR"), (dict(groupSize=0), "ATTR"), (dict(groupSize=-1), "ATTR"),
    (dict(topK=0), "ATTR"), (dict(batch=0), "ATTR"), (dict(rowIdxType=2), "ATTR"),
    (dict(product=ROWS), "ATTR"),  # probs belong to the gated product
    (dict(dtype=3), "DTYPE"), (dict(scale_dtype=pgg.PGG_F16), "DTYPE"),
    (dict(out_dtype=pgg.PGG_F32), "DTYPE"),
    (dict(product=COMBINED, probs=0), "DTYPE"),  # (its output is fp32)
    (dict(product=ROWS, probs=0, out_dtype=pgg.PGG_F16), "DTYPE"),
    (dict(M=0), "SHAPE"), (dict(N=0), "SHAPE"), (dict(K=0), "SHAPE"), (dict(G=0), "SHAPE"),
    (dict(L=47), "SHAPE"), (dict(batch=23), "SHAPE"), (dict(M=2**31, L=2**31, batch=2**30), "SHAPE"),
    (dict(N=2**30), "SHAPE"), (dict(groupSize=2**31), "SHAPE"),
    (dict(x=FAKE + 1), "ALIGN"), (dict(scales=FAKE + 2), "ALIGN"), (dict(out=FAKE + 1), "ALIGN"),
    (dict(probs=FAKE + 2), "ALIGN"), (dict(expandedRowIdx=FAKE + 4), "ALIGN"),
    (dict(groupList=FAKE + 4), "ALIGN"), (dict(workspace=FAKE + 64), "ALIGN"),
    (dict(workspace_bytes=255), "WORKSPACE"),
])
def test_w4_refusals(change, want):
    assert name(pgg.pgg_w4_execute(**dict(W4, **change))) == "PGG_ERR_" + want


def test_w4_workspace():
    sizes = dict(M=48, N=32, K=64, G=4, L=48, batch=24, topK=2, rowIdxType=0, groupSize=32,
                 dtype=pgg.PGG_BF16)
    rows = pgg.pgg_w4_workspace_size(product=ROWS, **sizes)
    combined = pgg.pgg_w4_workspace_size(product=COMBINED, **sizes)
    assert rows % 256 == 0 and combined >= rows + 4 * 48 * 32
    assert name(pgg.pgg_w4_execute(**dict(W4, workspace_bytes=pgg.pgg_w4_workspace_size(
        product=pgg.PGG_W4_GATED, **sizes) - 1))) == "PGG_ERR_WORKSPACE"
    with pytest.raises(pgg.PggError):
        pgg.pgg_w4_workspace_size(product=ROWS, **dict(sizes, K=0))


NORM = dict(x=FAKE, y=FAKE, gate=FAKE, post_weight=FAKE, post_bias=FAKE, pre_weight=FAKE,
            pre_bias=FAKE, T=5, H=64, dtype=pgg.PGG_BF16, y_dtype=pgg.PGG_F32,
            param_dtype=pgg.PGG_F32, post=pgg.PGG_NORM_LAYER, pre=pgg.PGG_NORM_LAYER,
            gate_kind=pgg.PGG_GATE_CHANNEL, residual_scale=1.0, weight_offset=0.0, eps=1e-6,
            r=FAKE, h=FAKE, stream=None)
NORM_BAD = [
    (dict(y=0), "NULL"), (dict(gate=0), "NULL"),
    (dict(gate_kind=pgg.PGG_GATE_NONE), "NULL"), (dict(gate_kind=4), "ATTR"),
    (dict(post=3), "ATTR"), (dict(pre=-1), "ATTR"), (dict(T=0), "ATTR"),
    (dict(post=pgg.PGG_NORM_RMS), "ATTR"), (dict(pre=pgg.PGG_NORM_RMS), "ATTR"),  # with a bias
    (dict(post=pgg.PGG_NORM_NONE, post_bias=0), "ATTR"),
    (dict(dtype=7), "DTYPE"), (dict(y_dtype=pgg.PGG_F16), "DTYPE"),
    (dict(param_dtype=pgg.PGG_F16), "DTYPE"), (dict(H=0), "SHAPE"), (dict(H=2**31), "SHAPE"),
    (dict(T=2**31), "SHAPE"), (dict(y=FAKE + 2), "ALIGN"), (dict(gate=FAKE + 2), "ALIGN"),
    (dict(post_weight=FAKE + 1), "ALIGN"), (dict(pre_bias=FAKE + 2), "ALIGN"),
]


@pytest.mark.parametrize("change,want", NORM_BAD + [
    (dict(x=0), "NULL"), (dict(r=0, h=0), "NULL"), (dict(h=0), "NULL"),
    (dict(pre=pgg.PGG_NORM_NONE, pre_weight=0, pre_bias=0), "NULL"),  # h without its norm
    (dict(x=FAKE + 1), "ALIGN"), (dict(h=FAKE + 1), "ALIGN"),
])
def test_norm_refusals(change, want):
    assert name(pgg.pgg_block_norm(**dict(NORM, **change))) == "PGG_ERR_" + want


GRAD = dict({k: v for k, v in NORM.items() if k not in ("x", "r", "h")}, d_r=FAKE, d_h=FAKE,
            r=FAKE, dh_dtype=pgg.PGG_F32, workspace=FAKE, workspace_bytes=1 << 30, d_x=FAKE,
            d_y=FAKE, d_gate=FAKE, d_post_weight=FAKE, d_post_bias=FAKE, d_pre_weight=FAKE,
            d_pre_bias=FAKE)


@pytest.mark.parametrize("change,want", NORM_BAD[2:] + [
    (dict(d_x=0), "NULL"), (dict(d_r=0, d_h=0), "NULL"), (dict(d_h=0), "NULL"), (dict(r=0), "NULL"),
    (dict(d_y=0), "NULL"), (dict(y=0), "NULL"), (dict(d_gate=0), "NULL"), (dict(gate=0), "NULL"),
    (dict(post_weight=0), "NULL"), (dict(pre_bias=0), "NULL"), (dict(workspace=0), "NULL"),
    (dict(dh_dtype=pgg.PGG_F16), "DTYPE"), (dict(d_gate=FAKE + 2), "ALIGN"),
    (dict(d_pre_weight=FAKE + 2), "ALIGN"), (dict(workspace=FAKE + 16), "ALIGN"),
    (dict(workspace_bytes=4096), "WORKSPACE"),
])
def test_norm_grad_refusals(change, want):
    assert name(pgg.pgg_block_norm_grad(**dict(GRAD, **change))) == "PGG_ERR_" + want


CLIP = dict(grads=[FAKE, FAKE], sizes=[5, 7], dtypes=[pgg.PGG_F32, pgg.PGG_BF16], max_norm=1.0,
            eps=1e-6, scale=1.0, workspace=FAKE, workspace_bytes=1 << 20, norm=FAKE,
            out=[FAKE, FAKE], stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(workspace=0), "NULL"), (dict(norm=0), "NULL"), (dict(grads=[FAKE, 0]), "NULL"),
    (dict(out=[0, FAKE]), "NULL"), (dict(dtypes=[0, 5]), "DTYPE"), (dict(sizes=[5, -1]), "SHAPE"),
    (dict(sizes=[2**47, 1]), "SHAPE"), (dict(max_norm=-1.0), "ATTR"),
    (dict(max_norm=float("nan")), "ATTR"), (dict(eps=-1.0), "ATTR"),
    (dict(grads=[FAKE + 2, FAKE]), "ALIGN"), (dict(out=[FAKE, FAKE + 1]), "ALIGN"),
    (dict(norm=FAKE + 2), "ALIGN"), (dict(workspace=FAKE + 8), "ALIGN"),
    (dict(workspace_bytes=256), "WORKSPACE"),
])
def test_clip_refusals(change, want):
    assert name(pgg.pgg_clip_grads(**dict(CLIP, **change))) == "PGG_ERR_" + want


def test_clip_workspace_grows_with_the_launches():
    assert pgg.pgg_clip_workspace_size(0) == pgg.pgg_clip_workspace_size(512)
    assert pgg.pgg_clip_workspace_size(513) > pgg.pgg_clip_workspace_size(512)
    size = ctypes.c_size_t()
    assert name(pgg.load().pgg_clip_workspace_size(-1, ctypes.byref(size))) == "PGG_ERR_ATTR"


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int64)
    codes, scales = torch.zeros(2, 8, 32, dtype=torch.uint8), torch.zeros(2, 8, 1)
    for call in (pgg.fwd_w4, pgg.swiglu_w4, pgg.down_w4):
        with pytest.raises(ValueError):
            call(x, codes, scales, i, i[:2], 4, 1, 0)
    with pytest.raises(ValueError):
        pgg.block_norm(x)
    with pytest.raises(ValueError):
        pgg.block_norm_grad(x, x, x)
    with pytest.raises(ValueError):
        pgg.clip_grads([x], 1.0)
    with pytest.raises(ValueError):
        pgg.grad_norm([x])
    with pytest.raises(ValueError):
        pgg.grad_norm([])
