"""Refusals of the router's choice by score + bias: before any CUDA call."""

import permute_grouped_gemm_gb300 as pgg
from test_ops_host import FAKE, lib, name_of  # noqa: F401 (lib: the module's fixture)


def test_route_codes():
    need = pgg.pgg_route_workspace_size(100, 60, 8)
    base = dict(logits=FAKE, bias=FAKE, batch=100, G=60, topK=8, rowIdxType=0, dtype=pgg.PGG_BF16,
                score=0, renormalize=1, scale=1.0, workspace=FAKE, workspace_bytes=need - 1,
                probs=FAKE, experts=FAKE, expandedRowIdx=FAKE, groupList=FAKE, stream=None)

    def code(score, **o):
        return name_of(pgg.pgg_route_execute, base, score=score, **o)

    # accepted, with a bias or without (the workspace is what is refused here)
    for kind in (pgg.PGG_SCORE_SOFTMAX, pgg.PGG_SCORE_SIGMOID):
        assert code(kind + pgg.PGG_BIAS_ON_SCORE) == "PGG_ERR_WORKSPACE"
        assert code(kind + pgg.PGG_BIAS_ON_SCORE, bias=0) == "PGG_ERR_WORKSPACE"
    for bad in (2, 8, 18, 32, 33, -1):
        assert code(bad) == "PGG_ERR_ATTR", bad
    # the gradient knows no bias
    grad = dict(d_probs=FAKE, logits=FAKE, experts=FAKE, batch=10, G=60, topK=8,
                dtype=pgg.PGG_F32, score=pgg.PGG_BIAS_ON_SCORE, renormalize=0, scale=1.0,
                d_logits=FAKE, stream=None)
    assert name_of(pgg.pgg_route_grad, grad) == "PGG_ERR_ATTR"
