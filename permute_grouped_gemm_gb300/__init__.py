"""GB300 (sm_103a) fused MoE permute + grouped-matmul backward, input gradient.

    d_x[b, k] = sum_{i : batch(i) = b} sum_n grad_y[i, n] * weight[g(i), k, n]

("MoeInitRoutingGroupedMatmulGrad design", section "数学定义和公式".) The work
runs in libpgg.so (include/pgg.h); this package is its thin binding. PyTorch
supplies device memory and the current stream only.
"""

from __future__ import annotations

from ._lib import (  # noqa: F401
    CODES, PGG_BF16, PGG_BIAS_ON_SCORE, PGG_F16, PGG_F32, PGG_SCORE_SIGMOID, PGG_SCORE_SOFTMAX, STATUS, PggError,
    load, pgg_adapters_execute, pgg_adapters_grad, pgg_adapters_grad_workspace_size,
    pgg_adapters_plan, pgg_adapters_workspace_size, pgg_route_execute, pgg_route_grad, pgg_route_workspace_size,
    pgg_swiglu_execute, pgg_swiglu_grad, pgg_swiglu_grad_workspace_size,
    pgg_swiglu_plan, pgg_swiglu_workspace_size,
    pgg_debug_force_variant, pgg_debug_set_band_k_blocks, pgg_debug_set_hold_release,
    pgg_debug_set_ticket_bias, pgg_debug_set_wait_limit_ns,
    pgg_dw_execute, pgg_dw_grouped_gemm, pgg_dw_plan, pgg_dw_workspace_size,
    pgg_fwd_execute, pgg_fwd_grouped_gemm, pgg_fwd_plan, pgg_fwd_route_prep,
    pgg_fwd_workspace_size, pgg_unpermute_grad, pgg_unpermute_grad_apply,
    pgg_unpermute_grad_prep, pgg_unpermute_grad_workspace_size,
    pgg_dx_execute, pgg_dx_execute_static_scratch, pgg_dx_grouped_gemm, pgg_dx_plan,
    pgg_dx_route_prep,
    pgg_dx_workspace_size, pgg_status_string,
)

_DT = None


def dtype_code(torch_dtype) -> int:
    global _DT
    if _DT is None:
        import torch
        _DT = {torch.float32: PGG_F32, torch.float16: PGG_F16, torch.bfloat16: PGG_BF16}
    if torch_dtype not in _DT:
        raise PggError(CODES["PGG_ERR_DTYPE"], "dtype_code")
    return _DT[torch_dtype]


def _args(grad_y, weight, expanded_row_idx, group_list, batch, top_k):
    M, N = grad_y.shape
    G, K, _ = weight.shape
    return M, N, K, G, expanded_row_idx.shape[0], batch, top_k


def workspace_bytes(grad_y, weight, expanded_row_idx, group_list, batch, top_k,
                    row_idx_type) -> int:
    sizes = _args(grad_y, weight, expanded_row_idx, group_list, batch, top_k)
    return pgg_dx_workspace_size(*sizes, row_idx_type, dtype_code(grad_y.dtype))


def dx(grad_y, weight, expanded_row_idx, group_list, batch: int, top_k: int,
       row_idx_type: int, out=None, workspace=None, stream=None):
    """d_x [batch, K] fp32 on grad_y's device (torch tensors, contiguous, CUDA).

    Allocates ``out`` and the workspace through torch when not given. The call
    is asynchronous on ``stream`` (default: torch's current stream); the
    device-detected status is the first int32 of the workspace.
    Returns (out, workspace).
    """
    import torch
    for t in (grad_y, weight, expanded_row_idx, group_list):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if expanded_row_idx.dtype != torch.int64 or group_list.dtype != torch.int64:
        raise ValueError("expandedRowIdx and groupList must be int64")
    sizes = _args(grad_y, weight, expanded_row_idx, group_list, batch, top_k)
    dt = dtype_code(grad_y.dtype)
    if weight.dtype != grad_y.dtype:
        raise PggError(CODES["PGG_ERR_DTYPE"], "dx")
    need = pgg_dx_workspace_size(*sizes, row_idx_type, dt)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=grad_y.device)
    if out is None:
        out = torch.empty(batch, sizes[2], dtype=torch.float32, device=grad_y.device)
    if stream is None:
        stream = torch.cuda.current_stream(grad_y.device)
    rc = pgg_dx_execute(grad_y.data_ptr(), weight.data_ptr(), expanded_row_idx.data_ptr(),
                        group_list.data_ptr(), *sizes, row_idx_type, dt, workspace.data_ptr(),
                        workspace.numel() * workspace.element_size(), out.data_ptr(),
                        stream.cuda_stream)
    if rc != 0:
        raise PggError(rc, "pgg_dx_execute")
    return out, workspace


def dw(x, grad_y, expanded_row_idx, group_list, batch: int, top_k: int, row_idx_type: int,
       G: int | None = None, out_dtype=None, out=None, workspace=None, stream=None):
    """d_weight [G, K, N] (``out_dtype``: grad_y's dtype by default, or
    torch.float32) from the forward input x [batch, K] and grad_y [M, N].
    G defaults to len(group_list). Returns (out, workspace)."""
    import torch
    for t in (x, grad_y, expanded_row_idx, group_list):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if expanded_row_idx.dtype != torch.int64 or group_list.dtype != torch.int64:
        raise ValueError("expandedRowIdx and groupList must be int64")
    if x.dtype != grad_y.dtype:
        raise PggError(CODES["PGG_ERR_DTYPE"], "dw")
    M, N = grad_y.shape
    _, K = x.shape
    G = group_list.shape[0] if G is None else G
    sizes = (M, N, K, G, expanded_row_idx.shape[0], batch, top_k)
    dt = dtype_code(grad_y.dtype)
    out_dtype = grad_y.dtype if out_dtype is None else out_dtype
    odt = dtype_code(out_dtype)
    need = pgg_dw_workspace_size(*sizes, row_idx_type, dt)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=grad_y.device)
    if out is None:
        out = torch.empty(G, K, N, dtype=out_dtype, device=grad_y.device)
    if stream is None:
        stream = torch.cuda.current_stream(grad_y.device)
    rc = pgg_dw_execute(x.data_ptr(), grad_y.data_ptr(), expanded_row_idx.data_ptr(),
                        group_list.data_ptr(), *sizes, row_idx_type, dt, odt,
                        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        out.data_ptr(), stream.cuda_stream)
    if rc != 0:
        raise PggError(rc, "pgg_dw_execute")
    return out, workspace


def fwd(x, weight, expanded_row_idx, group_list, batch: int, top_k: int, row_idx_type: int,
        out_dtype=None, out=None, workspace=None, stream=None):
    """Forward y [M, N] (expanded order; ``out_dtype``: x's dtype by default, or
    torch.float32) from x [batch, K] and weight [G, K, N]. Returns (y, workspace)."""
    import torch
    for t in (x, weight, expanded_row_idx, group_list):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if expanded_row_idx.dtype != torch.int64 or group_list.dtype != torch.int64:
        raise ValueError("expandedRowIdx and groupList must be int64")
    if x.dtype != weight.dtype:
        raise PggError(CODES["PGG_ERR_DTYPE"], "fwd")
    G, K, N = weight.shape
    M = expanded_row_idx.shape[0]
    sizes = (M, N, K, G, M, batch, top_k)
    dt = dtype_code(x.dtype)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    odt = dtype_code(out_dtype)
    need = pgg_fwd_workspace_size(*sizes, row_idx_type, dt)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    rc = pgg_fwd_execute(x.data_ptr(), weight.data_ptr(), expanded_row_idx.data_ptr(),
                         group_list.data_ptr(), *sizes, row_idx_type, dt, odt,
                         workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         out.data_ptr(), stream.cuda_stream)
    if rc != 0:
        raise PggError(rc, "pgg_fwd_execute")
    return out, workspace


def unpermute_grad(permuted, d_out, probs, expanded_row_idx, top_k: int, row_idx_type: int,
                   probs_grad_dtype=None, perm_grad=None, probs_grad=None, workspace=None,
                   stream=None):
    """(perm_grad [M, H], probs_grad [batch, topK] or None, workspace) of the
    probs-weighted unpermute (probs None: plain scatter copy)."""
    import torch
    for t in (d_out, expanded_row_idx) + ((permuted, probs) if probs is not None else ()):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    batch, H = d_out.shape
    M = expanded_row_idx.shape[0]
    dt = dtype_code(d_out.dtype)
    pdt = d_out.dtype if probs_grad_dtype is None else probs_grad_dtype
    need = pgg_unpermute_grad_workspace_size(M, batch, top_k)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=d_out.device)
    if perm_grad is None:
        perm_grad = torch.empty(M, H, dtype=d_out.dtype, device=d_out.device)
    if probs is not None and probs_grad is None:
        probs_grad = torch.empty(batch, top_k, dtype=pdt, device=d_out.device)
    if stream is None:
        stream = torch.cuda.current_stream(d_out.device)
    rc = pgg_unpermute_grad(permuted.data_ptr() if probs is not None else 0, d_out.data_ptr(),
                            probs.data_ptr() if probs is not None else 0,
                            expanded_row_idx.data_ptr(), M, H, batch, top_k, row_idx_type, dt,
                            dtype_code(pdt), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), perm_grad.data_ptr(),
                            probs_grad.data_ptr() if probs is not None else 0,
                            stream.cuda_stream)
    if rc != 0:
        raise PggError(rc, "pgg_unpermute_grad")
    return perm_grad, (probs_grad if probs is not None else None), workspace


_SCORES = {"softmax": PGG_SCORE_SOFTMAX, "sigmoid": PGG_SCORE_SIGMOID}


def _score_code(score: str) -> int:
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    return _SCORES[score]


_BIAS_ON = {"logits": 0, "scores": PGG_BIAS_ON_SCORE}


def _stream_of(stream, device) -> int:
    """Address of ``stream``, or of torch's current stream on ``device``."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _dense(first, *others):
    """Every given tensor is contiguous and on the first one's GPU (a kernel takes addresses)."""
    device = first.get_device()  # -1 on the host
    for t in (first, *others):
        if t is not None and (t.get_device() != device or device < 0 or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors of one device")


def _is(what: str, t, shape, dtype):
    """An optional tensor of the given shape and dtype."""
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")


def route(logits, top_k: int, row_idx_type: int = 0, bias=None, score: str = "softmax",
          renormalize: bool = True, scale: float = 1.0, probs=None, experts=None,
          expanded_row_idx=None, group_list=None, workspace=None, stream=None,
          bias_on: str = "logits"):
    """Top-k routing of logits [batch, G]: (probs [batch, top_k] fp32, experts [batch, top_k]
    int64, expanded_row_idx [batch * top_k] int64, group_list [G] int64, workspace).

    The choice goes by logits + bias (fp32 [G], optional), or with ``bias_on="scores"`` by
    scores + bias, which is what a selection bias learnt for the scores needs (routers that
    balance their experts' load by a bias have such); the lowest index first among equals.
    probs are the chosen experts' softmax or sigmoid scores without the bias, divided by their
    sum with ``renormalize``, times ``scale``. Outputs are allocated when not given.
    """
    import torch
    _dense(logits, bias, probs, experts, expanded_row_idx, group_list, workspace)
    batch, G = logits.shape
    M, dev = batch * top_k, logits.device
    if bias_on not in _BIAS_ON:
        raise ValueError("bias_on must be 'logits' or 'scores'")
    _is("bias", bias, (G,), torch.float32)
    _is("probs", probs, (batch, top_k), torch.float32)
    _is("experts", experts, (batch, top_k), torch.int64)
    _is("expanded_row_idx", expanded_row_idx, (M,), torch.int64)
    _is("group_list", group_list, (G,), torch.int64)
    if workspace is None:
        workspace = torch.empty(pgg_route_workspace_size(batch, G, top_k),
                                dtype=torch.uint8, device=dev)
    if probs is None:
        probs = torch.empty(batch, top_k, dtype=torch.float32, device=dev)
    if experts is None:
        experts = torch.empty(batch, top_k, dtype=torch.int64, device=dev)
    if expanded_row_idx is None:
        expanded_row_idx = torch.empty(M, dtype=torch.int64, device=dev)
    if group_list is None:
        group_list = torch.empty(G, dtype=torch.int64, device=dev)
    stream = _stream_of(stream, dev)
    rc = pgg_route_execute(logits.data_ptr(), bias.data_ptr() if bias is not None else 0, batch, G,
                           top_k, row_idx_type, dtype_code(logits.dtype),
                           _score_code(score) + _BIAS_ON[bias_on], int(renormalize), scale,
                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                           probs.data_ptr(), experts.data_ptr(), expanded_row_idx.data_ptr(),
                           group_list.data_ptr(), stream)
    if rc != 0:
        raise PggError(rc, "pgg_route_execute")
    return probs, experts, expanded_row_idx, group_list, workspace


def route_grad(d_probs, logits, experts, score: str = "softmax", renormalize: bool = True,
               scale: float = 1.0, out=None, stream=None):
    """d_logits [batch, G] (logits' dtype) from d_probs [batch, top_k] fp32 and the ``experts``
    that ``route`` chose from ``logits`` with the same score, renormalize and scale. ``out`` may
    be ``logits``."""
    import torch
    _dense(d_probs, logits, experts, out)
    batch, G = logits.shape
    top_k = experts.shape[1]
    _is("d_probs", d_probs, (batch, top_k), torch.float32)
    _is("experts", experts, (batch, top_k), torch.int64)
    _is("out", out, (batch, G), logits.dtype)
    if out is None:
        out = torch.empty_like(logits)
    stream = _stream_of(stream, logits.device)
    rc = pgg_route_grad(d_probs.data_ptr(), logits.data_ptr(), experts.data_ptr(), batch, G, top_k,
                        dtype_code(logits.dtype), _score_code(score), int(renormalize), scale,
                        out.data_ptr(), stream)
    if rc != 0:
        raise PggError(rc, "pgg_route_grad")
    return out


def swiglu(x, weight, expanded_row_idx, group_list, batch: int, top_k: int, row_idx_type: int,
           probs=None, keep: bool = False, out=None, gate_up=None, workspace=None, stream=None):
    """Gated expert product: (h [M, F], gate_up [M, 2F] or None, workspace), expanded order.

    [gate | up] = x[token] weight[expert] for x [batch, K] and weight [G, K, 2F];
    h = prob * silu(gate) * up, with probs [batch, top_k] fp32 (1 when None). ``keep``
    also returns the pre-activations, which ``swiglu_grad`` reads.
    """
    import torch
    _dense(x, weight, expanded_row_idx, group_list, probs, out, gate_up, workspace)
    if expanded_row_idx.dtype != torch.int64 or group_list.dtype != torch.int64:
        raise ValueError("expandedRowIdx and groupList must be int64")
    if x.dtype != weight.dtype:
        raise PggError(CODES["PGG_ERR_DTYPE"], "swiglu")
    G, K, F2 = weight.shape
    if F2 % 2 or x.shape != (batch, K) or group_list.shape != (G,):
        raise PggError(CODES["PGG_ERR_SHAPE"], "swiglu")
    M, F, dev = expanded_row_idx.shape[0], F2 // 2, x.device
    _is("probs", probs, (batch, top_k), torch.float32)
    _is("out", out, (M, F), x.dtype)
    _is("gate_up", gate_up, (M, F2), x.dtype)
    dt = dtype_code(x.dtype)
    if workspace is None:
        need = pgg_swiglu_workspace_size(M, F, K, G, M, batch, top_k, row_idx_type, dt)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(M, F, dtype=x.dtype, device=dev)
    if keep and gate_up is None:
        gate_up = torch.empty(M, F2, dtype=x.dtype, device=dev)
    stream = _stream_of(stream, dev)
    rc = pgg_swiglu_execute(x.data_ptr(), weight.data_ptr(), expanded_row_idx.data_ptr(),
                            group_list.data_ptr(), probs.data_ptr() if probs is not None else 0,
                            M, F, K, G, M, batch, top_k, row_idx_type, dt, workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), out.data_ptr(),
                            gate_up.data_ptr() if gate_up is not None else 0, stream)
    if rc != 0:
        raise PggError(rc, "pgg_swiglu_execute")
    return out, gate_up, workspace


def swiglu_grad(d_h, gate_up, expanded_row_idx, top_k: int, row_idx_type: int, probs=None,
                d_gate_up=None, d_probs=None, h=None, workspace=None, stream=None):
    """(d_gate_up [M, 2F], d_probs [batch, top_k] fp32 or None without probs, h [M, F],
    workspace) from d_h [M, F] and the gate_up that ``swiglu`` kept. d_gate_up is the grad_y of
    ``dx`` and ``dw`` for the gated weight; h (weighted) is the grad_y of ``dw`` for the down
    projection."""
    import torch
    _dense(d_h, gate_up, expanded_row_idx, probs, d_gate_up, d_probs, h, workspace)
    if expanded_row_idx.dtype != torch.int64:
        raise ValueError("expandedRowIdx must be int64")
    if d_h.dtype != gate_up.dtype:
        raise PggError(CODES["PGG_ERR_DTYPE"], "swiglu_grad")
    M, F = d_h.shape
    if gate_up.shape != (M, 2 * F) or expanded_row_idx.shape != (M,) or top_k <= 0 \
            or M % top_k:
        raise PggError(CODES["PGG_ERR_SHAPE"], "swiglu_grad")
    batch, dev = M // top_k, d_h.device
    _is("probs", probs, (batch, top_k), torch.float32)
    _is("d_gate_up", d_gate_up, (M, 2 * F), d_h.dtype)
    _is("d_probs", d_probs, (batch, top_k), torch.float32)
    _is("h", h, (M, F), d_h.dtype)
    if workspace is None:
        workspace = torch.empty(pgg_swiglu_grad_workspace_size(M, batch, top_k),
                                dtype=torch.uint8, device=dev)
    if d_gate_up is None:
        d_gate_up = torch.empty_like(gate_up)
    if probs is not None and d_probs is None:
        d_probs = torch.empty_like(probs)
    if h is None:
        h = torch.empty_like(d_h)
    stream = _stream_of(stream, dev)
    rc = pgg_swiglu_grad(d_h.data_ptr(), gate_up.data_ptr(),
                         probs.data_ptr() if probs is not None else 0,
                         expanded_row_idx.data_ptr(), M, F, batch, top_k, row_idx_type,
                         dtype_code(d_h.dtype), workspace.data_ptr(),
                         workspace.numel() * workspace.element_size(), d_gate_up.data_ptr(),
                         d_probs.data_ptr() if probs is not None else 0, h.data_ptr(),
                         stream)
    if rc != 0:
        raise PggError(rc, "pgg_swiglu_grad")
    return d_gate_up, (d_probs if probs is not None else None), h, workspace


def _adapter_sizes(where, x, weight, a, b, adapter, scale):
    """(T, K, N, R, A) of an adapter call whose tensors agree with each other."""
    import torch
    T, K = x.shape
    N = weight.shape[1]
    A, _, R = a.shape
    if weight.shape != (K, N) or a.shape != (A, K, R) or b.shape != (A, N, R) \
            or adapter.shape != (T,):
        raise PggError(CODES["PGG_ERR_SHAPE"], where)
    if not x.dtype == weight.dtype == a.dtype == b.dtype:
        raise PggError(CODES["PGG_ERR_DTYPE"], where)
    if adapter.dtype != torch.int64:
        raise ValueError("adapter must be int64")
    _is("scale", scale, (A,), torch.float32)
    return T, K, N, R, A


def adapters(x, weight, a, b, adapter, scale=None, out=None, workspace=None, stream=None):
    """(y [T, N], workspace) of a shared projection with one low-rank adapter per token:
    y[t] = x[t] weight + scale[ad] (x[t] a[ad]) b[ad]^T with ad = adapter[t], -1 for none.

    x [T, K], weight [K, N], a [A, K, R], b [A, N, R] of one dtype; adapter [T] int64;
    scale [A] fp32 (1 when None). Tokens may be in any order.
    """
    import torch
    _dense(x, weight, a, b, adapter, scale, out, workspace)
    T, K, N, R, A = _adapter_sizes("adapters", x, weight, a, b, adapter, scale)
    _is("out", out, (T, N), x.dtype)
    dt, dev = dtype_code(x.dtype), x.device
    if workspace is None:
        workspace = torch.empty(pgg_adapters_workspace_size(T, K, N, R, A, dt),
                                dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(T, N, dtype=x.dtype, device=dev)
    stream = _stream_of(stream, dev)
    rc = pgg_adapters_execute(x.data_ptr(), weight.data_ptr(), a.data_ptr(), b.data_ptr(),
                              adapter.data_ptr(), scale.data_ptr() if scale is not None else 0,
                              T, K, N, R, A, dt, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), out.data_ptr(),
                              stream)
    if rc != 0:
        raise PggError(rc, "pgg_adapters_execute")
    return out, workspace


def adapters_grad(d_y, x, weight, a, b, adapter, scale=None, need_x: bool = True, d_x=None,
                  d_a=None, d_b=None, workspace=None, stream=None):
    """(d_x [T, K] or None, d_a [A, K, R], d_b [A, N, R], workspace) of ``adapters`` from d_y
    [T, N], with the projection frozen. ``need_x`` False leaves d_x out."""
    import torch
    _dense(d_y, x, weight, a, b, adapter, scale, d_x, d_a, d_b, workspace)
    T, K, N, R, A = _adapter_sizes("adapters_grad", x, weight, a, b, adapter, scale)
    _is("d_y", d_y, (T, N), x.dtype)
    _is("d_x", d_x, (T, K), x.dtype)
    _is("d_a", d_a, (A, K, R), x.dtype)
    _is("d_b", d_b, (A, N, R), x.dtype)
    dt = dtype_code(x.dtype)
    if workspace is None:
        workspace = torch.empty(pgg_adapters_grad_workspace_size(T, K, N, R, A, dt),
                                dtype=torch.uint8, device=x.device)
    if need_x and d_x is None:
        d_x = torch.empty_like(x)
    if d_a is None:
        d_a = torch.empty_like(a)
    if d_b is None:
        d_b = torch.empty_like(b)
    stream = _stream_of(stream, x.device)
    rc = pgg_adapters_grad(d_y.data_ptr(), x.data_ptr(), weight.data_ptr(), a.data_ptr(),
                           b.data_ptr(), adapter.data_ptr(),
                           scale.data_ptr() if scale is not None else 0, T, K, N, R, A, dt,
                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                           d_x.data_ptr() if need_x else 0, d_a.data_ptr(), d_b.data_ptr(),
                           stream)
    if rc != 0:
        raise PggError(rc, "pgg_adapters_grad")
    return (d_x if need_x else None), d_a, d_b, workspace


def status(workspace) -> int:
    """Device-detected status word of a finished call (synchronises)."""
    import torch
    return int(workspace[:4].view(torch.int32).item())
