"""Refusals and sizes of the router, the gated product and the adapters: host
checks come before any CUDA call, so they run without a GPU."""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from permute_grouped_gemm_gb300 import build as pbuild

FAKE = 1 << 20  # aligned non-null address, never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def lib():
    pbuild.build()
    return pgg.load()


def name_of(call, base, **over):
    return pgg.STATUS[call(**dict(base, **over))]


def refused(call, *args):
    with pytest.raises(pgg.PggError) as e:
        call(*args)
    return pgg.STATUS[e.value.code]


def test_route_refusals():
    need = pgg.pgg_route_workspace_size(100, 60, 8)
    base = dict(logits=FAKE, bias=FAKE, batch=100, G=60, topK=8, rowIdxType=0, dtype=pgg.PGG_BF16,
                score=0, renormalize=1, scale=1.0, workspace=FAKE, workspace_bytes=need,
                probs=FAKE, experts=FAKE, expandedRowIdx=FAKE, groupList=FAKE, stream=None)

    def code(**o):
        return name_of(pgg.pgg_route_execute, base, **o)

    for p in ("logits", "workspace", "probs", "experts", "expandedRowIdx", "groupList"):
        assert code(**{p: 0}) == "PGG_ERR_NULL", p
    assert code(dtype=3) == "PGG_ERR_DTYPE"
    assert code(score=2) == code(rowIdxType=2) == code(batch=0) == code(topK=0) == "PGG_ERR_ATTR"
    assert code(topK=61) == code(G=1025) == code(topK=33) == "PGG_ERR_SHAPE"
    assert code(batch=2 ** 30) == "PGG_ERR_SHAPE"
    assert code(workspace_bytes=need - 1) == "PGG_ERR_WORKSPACE"
    assert code(logits=FAKE + 1) == code(bias=FAKE + 2) == code(experts=FAKE + 4) == "PGG_ERR_ALIGN"
    assert code(workspace=FAKE + 64) == "PGG_ERR_ALIGN"
    assert refused(pgg.pgg_route_workspace_size, 0, 60, 8) == "PGG_ERR_ATTR"
    # counters and four bytes a pair
    assert pgg.pgg_route_workspace_size(1 << 20, 1024, 8) < (8 << 20) * 4 + (4 << 20)


def test_route_grad_refusals():
    base = dict(d_probs=FAKE, logits=FAKE, experts=FAKE, batch=10, G=60, topK=8,
                dtype=pgg.PGG_F32, score=1, renormalize=0, scale=1.0, d_logits=FAKE, stream=None)

    def code(**o):
        return name_of(pgg.pgg_route_grad, base, **o)

    assert code(d_probs=0) == code(d_logits=0) == "PGG_ERR_NULL"
    assert code(dtype=-1) == "PGG_ERR_DTYPE"
    assert code(score=-1) == "PGG_ERR_ATTR"
    assert code(G=7) == "PGG_ERR_SHAPE"
    assert code(d_logits=FAKE + 2) == "PGG_ERR_ALIGN"


def test_swiglu_refusals():
    sizes = dict(M=800, F=256, K=512, G=16, L=800, batch=100, topK=8, rowIdxType=0,
                 dtype=pgg.PGG_BF16)
    need = pgg.pgg_swiglu_workspace_size(**sizes)
    base = dict(sizes, x=FAKE, weight=FAKE, expandedRowIdx=FAKE, groupList=FAKE, probs=FAKE,
                workspace=FAKE, workspace_bytes=need, h=FAKE, gate_up=FAKE, stream=None)

    def code(**o):
        return name_of(pgg.pgg_swiglu_execute, base, **o)

    for p in ("x", "weight", "expandedRowIdx", "groupList", "workspace", "h"):
        assert code(**{p: 0}) == "PGG_ERR_NULL", p
    assert code(dtype=7) == "PGG_ERR_DTYPE"
    assert code(batch=0) == code(rowIdxType=-1) == "PGG_ERR_ATTR"
    assert code(L=799) == code(batch=99) == code(F=0) == code(K=0) == code(G=0) == "PGG_ERR_SHAPE"
    assert code(M=2 ** 31, L=2 ** 31, batch=2 ** 28) == "PGG_ERR_SHAPE"
    assert code(F=2 ** 30) == "PGG_ERR_SHAPE"
    assert code(workspace_bytes=need - 1) == "PGG_ERR_WORKSPACE"
    assert code(x=FAKE + 1) == code(probs=FAKE + 2) == code(groupList=FAKE + 4) == "PGG_ERR_ALIGN"
    assert code(gate_up=FAKE + 1) == code(workspace=FAKE + 128) == "PGG_ERR_ALIGN"
    # the pages' scale: a few bytes per row, never an [M, F] array
    assert pgg.pgg_swiglu_workspace_size(108000, 2048, 7168, 60, 108000, 13500, 8, 0,
                                         pgg.PGG_BF16) < 4 << 20


def test_swiglu_grad_refusals():
    need = pgg.pgg_swiglu_grad_workspace_size(800, 100, 8)
    base = dict(d_h=FAKE, gate_up=FAKE, probs=FAKE, expandedRowIdx=FAKE, M=800, F=256, batch=100,
                topK=8, rowIdxType=1, dtype=pgg.PGG_F16, workspace=FAKE, workspace_bytes=need,
                d_gate_up=FAKE, d_probs=FAKE, h=FAKE, stream=None)

    def code(**o):
        return name_of(pgg.pgg_swiglu_grad, base, **o)

    assert code(d_h=0) == code(d_gate_up=0) == code(probs=0) == "PGG_ERR_NULL"
    assert code(dtype=5) == "PGG_ERR_DTYPE"
    assert code(rowIdxType=3) == "PGG_ERR_ATTR"
    assert code(M=801) == code(F=0) == "PGG_ERR_SHAPE"
    assert code(workspace_bytes=need - 1) == "PGG_ERR_WORKSPACE"
    assert code(h=FAKE + 1) == code(d_probs=FAKE + 2) == "PGG_ERR_ALIGN"


def test_adapters_refusals():
    sizes = dict(T=100, K=512, N=256, R=16, A=8, dtype=pgg.PGG_BF16)
    need = pgg.pgg_adapters_workspace_size(**sizes)
    base = dict(sizes, x=FAKE, weight=FAKE, a=FAKE, b=FAKE, adapter=FAKE, scale=FAKE,
                workspace=FAKE, workspace_bytes=need, y=FAKE, stream=None)

    def code(**o):
        return name_of(pgg.pgg_adapters_execute, base, **o)

    for p in ("x", "weight", "a", "b", "adapter", "workspace", "y"):
        assert code(**{p: 0}) == "PGG_ERR_NULL", p
    assert code(dtype=9) == "PGG_ERR_DTYPE"
    assert code(T=0) == "PGG_ERR_ATTR"
    assert code(K=0) == code(N=0) == code(R=0) == code(A=0) == "PGG_ERR_SHAPE"
    assert code(R=257) == code(A=1024) == code(T=2 ** 30) == "PGG_ERR_SHAPE"
    assert code(workspace_bytes=need - 1) == "PGG_ERR_WORKSPACE"
    assert code(b=FAKE + 1) == code(scale=FAKE + 2) == code(adapter=FAKE + 4) == "PGG_ERR_ALIGN"
    grad_need = pgg.pgg_adapters_grad_workspace_size(**sizes)
    grad = dict(sizes, d_y=FAKE, x=FAKE, weight=FAKE, a=FAKE, b=FAKE, adapter=FAKE, scale=0,
                workspace=FAKE, workspace_bytes=grad_need, d_x=FAKE, d_a=FAKE, d_b=FAKE,
                stream=None)
    for p in ("d_y", "d_a", "d_b", "adapter"):
        assert name_of(pgg.pgg_adapters_grad, grad, **{p: 0}) == "PGG_ERR_NULL", p
    assert name_of(pgg.pgg_adapters_grad, grad, workspace_bytes=need) == "PGG_ERR_WORKSPACE"
    assert name_of(pgg.pgg_adapters_grad, grad, d_x=FAKE + 1) == "PGG_ERR_ALIGN"
    assert refused(pgg.pgg_adapters_grad_workspace_size, 0, 1, 1, 1, 1, 0) == "PGG_ERR_ATTR"


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        pgg.route(x, 2)
    with pytest.raises(ValueError):
        pgg.swiglu(x, torch.zeros(2, 8, 4), torch.arange(4), torch.tensor([2, 2]), 4, 1, 0)
    with pytest.raises(ValueError):
        pgg.adapters(x, torch.zeros(8, 4), torch.zeros(1, 8, 2), torch.zeros(1, 4, 2),
                     torch.zeros(4, dtype=torch.int64))


def test_plans():
    def gated(tokens, k, G, K, F, dt):
        return pgg.pgg_swiglu_plan(tokens * k, F, K, G, tokens * k, tokens, k, 0, dt)

    p = gated(13500, 8, 60, 7168, 2048, pgg.PGG_BF16)
    assert p["variant"] == 0 and p["rows_per_block"] == 256 and p["cta_pair"] == 1
    p = gated(1, 8, 60, 7168, 2048, pgg.PGG_BF16)       # one row an expert
    assert p["variant"] == 1 and p["rows_per_block"] == 16
    p = gated(256, 8, 256, 7168, 2048, pgg.PGG_F16)     # eight on average
    assert p["variant"] == 1 and p["rows_per_block"] == 16
    p = gated(700, 8, 60, 7168, 2048, pgg.PGG_BF16)     # 93 on average
    assert p["variant"] == 1 and p["rows_per_block"] == 128
    assert gated(900, 8, 60, 7168, 2048, pgg.PGG_BF16)["variant"] == 0
    for K, F, dt in ((7168, 2048, pgg.PGG_F32), (7167, 2048, pgg.PGG_BF16), (64, 36, pgg.PGG_F16)):
        assert gated(64, 4, 8, K, F, dt)["variant"] == 3

    def adapters(T, K=4096, N=4096, R=16, A=8, dt=pgg.PGG_BF16):
        return pgg.pgg_adapters_plan(T, K, N, R, A, dt)

    assert [adapters(T)["rows_per_block"] for T in (1, 16, 17, 33, 256, 257)] == \
        [16, 16, 32, 64, 64, 256]
    assert adapters(256)["variant"] == 1 and adapters(257)["variant"] == 0
    assert adapters(256, N=5120)["variant"] == 0 and adapters(256, R=64)["variant"] == 0
    for kw in (dict(R=12), dict(K=100), dict(N=77), dict(dt=pgg.PGG_F32)):
        assert adapters(64, **kw)["variant"] == 3
    assert refused(pgg.pgg_adapters_plan, 1, 1, 1, 1, 0, 0) == "PGG_ERR_SHAPE"
