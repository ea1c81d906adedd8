"""GB300 (sm_103a) fused MoE permute + grouped-matmul backward, input gradient.

    d_x[b, k] = sum_{i : batch(i) = b} sum_n grad_y[i, n] * weight[g(i), k, n]

("MoeInitRoutingGroupedMatmulGrad design", section "数学定义和公式".) The work
runs in libpgg.so (include/pgg.h); this package is its thin binding. PyTorch
supplies device memory and the current stream only.
"""

from __future__ import annotations

from ._lib import (  # noqa: F401
    CODES, PGG_BF16, PGG_BIAS_ON_SCORE, PGG_F16, PGG_F32, PGG_SCORE_SIGMOID, PGG_SCORE_SOFTMAX, STATUS, PggError,
    PGG_GATE_CHANNEL, PGG_GATE_FULL, PGG_GATE_NONE, PGG_GATE_TOKEN, PGG_NORM_LAYER, PGG_NORM_NONE,
    PGG_NORM_RMS, PGG_W4_COMBINED, PGG_W4_GATED, PGG_W4_ROWS, pgg_block_norm, pgg_block_norm_grad,
    pgg_block_norm_grad_workspace_size, pgg_clip_grads, pgg_clip_workspace_size, pgg_grad_norm,
    pgg_w4_execute, pgg_w4_workspace_size,
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


def _w4(where, product, x, codes, scales, expanded_row_idx, group_list, batch, top_k, row_idx_type,
        group, zeros, probs, out_dtype, out, workspace, stream):
    """One of the products with 4-bit weights: (out, workspace)."""
    import torch
    _dense(x, codes, scales, expanded_row_idx, group_list, zeros, probs, out, workspace)
    if expanded_row_idx.dtype != torch.int64 or group_list.dtype != torch.int64:
        raise ValueError("expandedRowIdx and groupList must be int64")
    if codes.dtype != torch.uint8:
        raise ValueError("codes must be uint8")
    if group <= 0:
        raise PggError(CODES["PGG_ERR_ATTR"], where)
    G, C, row_bytes = codes.shape
    rows, K = x.shape
    M, dev = expanded_row_idx.shape[0], x.device
    combined, gated = product == PGG_W4_COMBINED, product == PGG_W4_GATED
    if rows != (M if combined else batch) or group_list.shape != (G,) or (gated and C % 2) \
            or row_bytes != (K + 1) // 2:
        raise PggError(CODES["PGG_ERR_SHAPE"], where)
    if scales.dtype not in (x.dtype, torch.float32):
        raise PggError(CODES["PGG_ERR_DTYPE"], where)
    N = C // 2 if gated else C
    shape = (G, C, (K + group - 1) // group)
    _is("scales", scales, shape, scales.dtype)
    _is("zeros", zeros, shape, torch.uint8)
    _is("probs", probs, (batch, top_k), torch.float32)
    out_shape = (batch if combined else M, N)
    _is("out", out, out_shape, out_dtype)
    dt = dtype_code(x.dtype)
    if workspace is None:
        need = pgg_w4_workspace_size(product, M, N, K, G, M, batch, top_k, row_idx_type, group, dt)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(out_shape, dtype=out_dtype, device=dev)
    stream = _stream_of(stream, dev)
    rc = pgg_w4_execute(product, x.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                        zeros.data_ptr() if zeros is not None else 0, expanded_row_idx.data_ptr(),
                        group_list.data_ptr(), probs.data_ptr() if probs is not None else 0, M, N,
                        K, G, M, batch, top_k, row_idx_type, group, dt, dtype_code(scales.dtype),
                        dtype_code(out_dtype), workspace.data_ptr(),
                        workspace.numel() * workspace.element_size(), out.data_ptr(), stream)
    if rc != 0:
        raise PggError(rc, "pgg_w4_execute")
    return out, workspace


def fwd_w4(x, codes, scales, expanded_row_idx, group_list, batch: int, top_k: int,
           row_idx_type: int, group: int = 128, zeros=None, out_dtype=None, out=None,
           workspace=None, stream=None):
    """Forward with 4-bit expert weights: (y [M, N] in expanded order, workspace).

    y[i] = sum_k x[token, k] w[expert, :, k], w = scale (code - zero), for x [batch, K], codes
    uint8 [G, N, ceil(K / 2)] (two codes a byte along K, the lower half first), scales
    [G, N, ceil(K / group)] (x's dtype or fp32) and zeros uint8 of the same shape (8 when None).
    ``out_dtype``: x's dtype by default, or torch.float32.
    """
    return _w4("fwd_w4", PGG_W4_ROWS, x, codes, scales, expanded_row_idx, group_list, batch, top_k,
               row_idx_type, group, zeros, None, x.dtype if out_dtype is None else out_dtype, out,
               workspace, stream)


def swiglu_w4(x, codes, scales, expanded_row_idx, group_list, batch: int, top_k: int,
              row_idx_type: int, group: int = 128, zeros=None, probs=None, out=None,
              workspace=None, stream=None):
    """``swiglu`` with 4-bit expert weights: (h [M, F], workspace). codes [G, 2F, ceil(K / 2)]
    hold F gate columns, then F up columns; scales and zeros as for ``fwd_w4``."""
    return _w4("swiglu_w4", PGG_W4_GATED, x, codes, scales, expanded_row_idx, group_list, batch,
               top_k, row_idx_type, group, zeros, probs, x.dtype, out, workspace, stream)


def down_w4(h, codes, scales, expanded_row_idx, group_list, batch: int, top_k: int,
            row_idx_type: int, group: int = 128, zeros=None, out=None, workspace=None,
            stream=None):
    """Down projection with 4-bit expert weights, summed over each token's experts:
    (out [batch, N] fp32, workspace), for h [M, K] in expanded order and codes
    [G, N, ceil(K / 2)]; what ``dx`` computes with 16-bit weights [G, N, K]."""
    import torch
    return _w4("down_w4", PGG_W4_COMBINED, h, codes, scales, expanded_row_idx, group_list, batch,
               top_k, row_idx_type, group, zeros, None, torch.float32, out, workspace, stream)


_NORMS = {None: PGG_NORM_NONE, "rms": PGG_NORM_RMS, "layer": PGG_NORM_LAYER}


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


def _norm_setup(where, T, H, dtype, y, gate, post, post_weight, post_bias, pre, pre_weight,
                pre_bias):
    """Codes (y_dtype, param_dtype, post, pre, gate_kind) of a norm call whose tensors agree."""
    if post not in _NORMS or pre not in _NORMS:
        raise ValueError("post and pre must be None, 'rms' or 'layer'")
    params = {"post_weight": post_weight, "post_bias": post_bias, "pre_weight": pre_weight,
              "pre_bias": pre_bias}
    given = [t for t in (gate, *params.values()) if t is not None]
    pdt = given[0].dtype if given else dtype
    code = dtype_code(dtype)
    if dtype_code(pdt) not in (code, PGG_F32):
        raise PggError(CODES["PGG_ERR_DTYPE"], where)
    for name, t in params.items():
        _is(name, t, (H,), pdt)
    kind = PGG_GATE_NONE
    if gate is not None:
        shape = tuple(gate.shape)
        if shape == (T, H):
            kind = PGG_GATE_FULL
        elif shape == (T, 1):
            kind = PGG_GATE_TOKEN
        elif shape == (H,):
            kind = PGG_GATE_CHANNEL
        else:
            raise ValueError(f"gate must be [{H}], [{T}, 1] or [{T}, {H}], got {list(shape)}")
        _is("gate", gate, shape, pdt)
    ydt = code
    if y is not None:
        ydt = dtype_code(y.dtype)
        if y.shape != (T, H):
            raise PggError(CODES["PGG_ERR_SHAPE"], where)
        if ydt not in (code, PGG_F32):
            raise PggError(CODES["PGG_ERR_DTYPE"], where)
    return ydt, dtype_code(pdt), _NORMS[post], _NORMS[pre], kind


def block_norm(x, y=None, gate=None, post=None, post_weight=None, post_bias=None, pre="rms",
               pre_weight=None, pre_bias=None, residual_scale: float = 1.0,
               weight_offset: float = 0.0, eps: float = 1e-6, r=None, h=None, stream=None):
    """What stands between two blocks, in one pass: (r [T, H], h [T, H] or None without ``pre``).

        r = residual_scale x + gate N_post(y),  h = N_pre(r)

    x [T, H]: the residual stream; y [T, H] (x's dtype or fp32): the block's output, or None.
    ``post`` and ``pre`` are None, "rms" or "layer"; a norm's factor is weight_offset + weight (1
    without a weight), a layer norm may have a bias. gate: [H], [T, 1] or [T, H]. All parameters
    and the gate are of one dtype, x's or fp32. h is taken from r before r is rounded. ``r`` may
    be ``x``.
    """
    import torch
    _dense(x, y, gate, post_weight, post_bias, pre_weight, pre_bias, r, h)
    T, H = x.shape
    codes = _norm_setup("block_norm", T, H, x.dtype, y, gate, post, post_weight, post_bias, pre,
                        pre_weight, pre_bias)
    _is("r", r, (T, H), x.dtype)
    _is("h", h, (T, H), x.dtype)
    if r is None:
        r = torch.empty_like(x)
    if pre is not None and h is None:
        h = torch.empty_like(x)
    rc = pgg_block_norm(x.data_ptr(), _ptr(y), _ptr(gate), _ptr(post_weight), _ptr(post_bias),
                        _ptr(pre_weight), _ptr(pre_bias), T, H, dtype_code(x.dtype), *codes,
                        residual_scale, weight_offset, eps, r.data_ptr(), _ptr(h),
                        _stream_of(stream, x.device))
    if rc != 0:
        raise PggError(rc, "pgg_block_norm")
    return r, h


def block_norm_grad(d_r, d_h, r, y=None, gate=None, post=None, post_weight=None, post_bias=None,
                    pre="rms", pre_weight=None, pre_bias=None, residual_scale: float = 1.0,
                    weight_offset: float = 0.0, eps: float = 1e-6, d_x=None, d_y=None,
                    workspace=None, stream=None):
    """Gradients of ``block_norm`` from d_r (r's later uses; None: 0) and d_h (r's dtype or fp32),
    the r that it returned and its y: (a dict, workspace). The dict holds d_x, d_y [T, H] in r's
    dtype, d_gate (the gate's shape; fp32, a [T, H] gate's in its dtype) and fp32 d_post_weight,
    d_post_bias, d_pre_weight, d_pre_bias [H], None for what is not there. ``d_x`` may be ``d_r``.
    Without ``pre``, d_h is None and r is not read.
    """
    import torch
    base = r if r is not None else d_r
    if base is None:
        raise PggError(CODES["PGG_ERR_NULL"], "block_norm_grad")
    _dense(base, d_r, d_h, y, gate, post_weight, post_bias, pre_weight, pre_bias, d_x, d_y,
           workspace)
    T, H = base.shape
    dtype, dev = base.dtype, base.device
    ydt, pdt, post_code, pre_code, kind = _norm_setup(
        "block_norm_grad", T, H, dtype, y, gate, post, post_weight, post_bias, pre, pre_weight,
        pre_bias)
    _is("d_r", d_r, (T, H), dtype)
    for name, t in (("d_x", d_x), ("d_y", d_y)):
        _is(name, t, (T, H), dtype)
    dhdt = dtype_code(dtype)
    if d_h is not None:
        dhdt = dtype_code(d_h.dtype)
        _is("d_h", d_h, (T, H), d_h.dtype)
    if d_x is None:
        d_x = torch.empty_like(base)
    if y is not None and d_y is None:
        d_y = torch.empty(T, H, dtype=dtype, device=dev)
    d_gate = None if gate is None else torch.empty(
        gate.shape, dtype=gate.dtype if kind == PGG_GATE_FULL else torch.float32, device=dev)
    d_params = [None if p is None else torch.empty(H, dtype=torch.float32, device=dev)
                for p in (post_weight, post_bias, pre_weight, pre_bias)]
    if workspace is None:
        workspace = torch.empty(pgg_block_norm_grad_workspace_size(T, H), dtype=torch.uint8,
                                device=dev)
    rc = pgg_block_norm_grad(
        _ptr(d_r), _ptr(d_h), _ptr(r) if pre is not None else 0, _ptr(y), _ptr(gate),
        _ptr(post_weight), _ptr(post_bias), _ptr(pre_weight), _ptr(pre_bias), T, H,
        dtype_code(dtype), ydt, dhdt, pdt, post_code, pre_code, kind, residual_scale,
        weight_offset, eps, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        d_x.data_ptr(), _ptr(d_y), _ptr(d_gate), *(_ptr(p) for p in d_params),
        _stream_of(stream, dev))
    if rc != 0:
        raise PggError(rc, "pgg_block_norm_grad")
    names = ("d_post_weight", "d_post_bias", "d_pre_weight", "d_pre_bias")
    return dict(zip(names, d_params), d_x=d_x, d_y=d_y, d_gate=d_gate), workspace


def _addresses(tensors, device):
    """Addresses of dense tensors on the GPU of that index."""
    for t in tensors:
        if t.get_device() != device or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors of one device")
    return [t.data_ptr() for t in tensors]


def _grad_list(grads, workspace, norm):
    """(addresses, sizes, dtype codes, device, workspace, norm) of a list of gradients."""
    import torch
    given = [t for t in (workspace, norm) if t is not None]
    if not grads and not given:
        raise ValueError("an empty list needs a workspace or norm to tell the device")
    dev = (grads[0] if grads else given[0]).device
    if dev.type != "cuda":
        raise ValueError("tensors must be contiguous CUDA tensors of one device")
    _addresses(given, dev.index)
    _is("norm", norm, (), torch.float32)
    if workspace is None:
        workspace = torch.empty(pgg_clip_workspace_size(len(grads)), dtype=torch.uint8, device=dev)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=dev)
    dtypes = [t.dtype for t in grads]
    codes = {d: dtype_code(d) for d in set(dtypes)}
    return (_addresses(grads, dev.index), [t.numel() for t in grads], [codes[d] for d in dtypes],
            dev, workspace, norm)


def grad_norm(grads, scale: float = 1.0, norm=None, workspace=None, stream=None):
    """(norm, workspace): the fp32 scalar |scale| sqrt(sum of all squares) over the tensors."""
    ptrs, sizes, dtypes, dev, workspace, norm = _grad_list(grads, workspace, norm)
    rc = pgg_grad_norm(ptrs, sizes, dtypes, scale, workspace.data_ptr(),
                       workspace.numel() * workspace.element_size(), norm.data_ptr(),
                       _stream_of(stream, dev))
    if rc != 0:
        raise PggError(rc, "pgg_grad_norm")
    return norm, workspace


def clip_grads(grads, max_norm: float, eps: float = 1e-6, scale: float = 1.0, out=None, norm=None,
               workspace=None, stream=None):
    """Clips gradients by their global norm: (norm, out, workspace).

    norm = |scale| sqrt(sum of all squares); out[i] = grads[i] scale min(1, max_norm / (norm +
    eps)), in place when ``out`` (a list of like tensors) is None. No output may overlap another, or
    another's gradient: a tensor that is shared is listed once. A norm that is not finite clips
    nothing (out = grads scale): look at it before the step.
    """
    out = grads if out is None else out
    ptrs, sizes, dtypes, dev, workspace, norm = _grad_list(grads, workspace, norm)
    to = ptrs
    if out is not grads:
        if len(out) != len(grads):
            raise PggError(CODES["PGG_ERR_SHAPE"], "clip_grads")
        to = _addresses(out, dev.index)
        for g, o in zip(grads, out):
            if g.dtype != o.dtype or g.shape != o.shape:
                raise ValueError("out must hold tensors like the gradients")
    rc = pgg_clip_grads(ptrs, sizes, dtypes, max_norm, eps, scale, workspace.data_ptr(),
                        workspace.numel() * workspace.element_size(), norm.data_ptr(),
                        to, _stream_of(stream, dev))
    if rc != 0:
        raise PggError(rc, "pgg_clip_grads")
    return norm, out, workspace


def status(workspace) -> int:
    """Device-detected status word of a finished call (synchronises)."""
    import torch
    return int(workspace[:4].view(torch.int32).item())
