"""Tensors that the wrappers of the router, the gated product and the adapters refuse: every one
of a call's tensors has to be contiguous and on the same GPU, since the kernels take addresses."""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def on(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


T, K, N, R, A, G, TOPK, F = 6, 64, 32, 8, 3, 4, 2, 16
I64, F32 = torch.int64, torch.float32


def calls():
    idx = torch.arange(T * TOPK, device="cuda")
    groups = torch.full((G,), T * TOPK // G, device="cuda")
    size = 1 << 20  # of every workspace here
    ws = on(size, torch.uint8)
    yield pgg.route, dict(logits=on((T, G), F32), top_k=TOPK, bias=on(G, F32),
                          probs=on((T, TOPK), F32), experts=on((T, TOPK), I64),
                          expanded_row_idx=on(T * TOPK, I64), group_list=on(G, I64), workspace=ws)
    yield pgg.route_grad, dict(d_probs=on((T, TOPK), F32), logits=on((T, G), F32),
                               experts=idx[:TOPK].repeat(T, 1), out=on((T, G), F32))
    yield pgg.swiglu, dict(x=on((T, K)), weight=on((G, K, 2 * F)), expanded_row_idx=idx,
                           group_list=groups, batch=T, top_k=TOPK, row_idx_type=0,
                           probs=on((T, TOPK), F32), out=on((T * TOPK, F)),
                           gate_up=on((T * TOPK, 2 * F)), workspace=ws)
    yield pgg.swiglu_grad, dict(d_h=on((T * TOPK, F)), gate_up=on((T * TOPK, 2 * F)),
                                expanded_row_idx=idx, top_k=TOPK, row_idx_type=0,
                                probs=on((T, TOPK), F32), d_gate_up=on((T * TOPK, 2 * F)),
                                d_probs=on((T, TOPK), F32), h=on((T * TOPK, F)), workspace=ws)
    low = dict(x=on((T, K)), weight=on((K, N)), a=on((A, K, R)), b=on((A, N, R)),
               adapter=on(T, I64), scale=on(A, F32), workspace=ws)
    yield pgg.adapters, dict(low, out=on((T, N)))
    yield pgg.adapters_grad, dict(low, d_y=on((T, N)), d_x=on((T, K)), d_a=on((A, K, R)),
                                  d_b=on((A, N, R)))


def test_tensors_of_the_host_and_strided_ones_are_refused():
    for call, args in calls():
        call(**args)  # as it is, it runs
        torch.cuda.synchronize()
        for name, t in args.items():
            if not isinstance(t, torch.Tensor):
                continue
            with pytest.raises(ValueError):
                call(**dict(args, **{name: t.cpu()}))
            # (one element over and over: the bytes that it says it has are not there)
            with pytest.raises(ValueError):
                call(**dict(args, **{name: t.reshape(-1)[:1].expand(t.numel()).view_as(t)
                                     if t.dim() == 1 else t.mT.contiguous().mT}))


def test_a_workspace_that_is_too_small_is_refused():
    for call, args in calls():
        if "workspace" in args:
            with pytest.raises(pgg.PggError) as e:
                call(**dict(args, workspace=args["workspace"][:256]))
            assert pgg.STATUS[e.value.code] == "PGG_ERR_WORKSPACE"
