"""A mixture-of-experts layer with a shared projection, from the library's operators.

    logits = x w_router
    probs, order = route(logits)                          top-k choice and expanded order
    h = swiglu(x, w_gate_up, order, probs)                gated expert product, weighted
    y = dx(h, w_down, order)                              down projection and combination
    y += adapters(x, w_shared, a, b, adapter)             shared projection, one adapter a token

dx, the framework's fused input gradient, is the down projection here: with w_down
[experts, hidden, inner] it computes sum over a token's experts of h w_down^T. The backward pass
uses the same operators the other way round. The routing is computed once and serves them all.

    python examples/moe_layer.py            one training step and one decode step, checked
"""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import permute_grouped_gemm_gb300 as pgg  # noqa: E402


class MoELayer:
    """Weights of one layer on the GPU, in ``dtype``; the router's in fp32."""

    def __init__(self, hidden, inner, experts, top_k, adapters, rank, dtype=torch.bfloat16,
                 seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

        self.top_k = top_k
        self.w_router = normal(hidden, experts, std=hidden ** -0.5).float()
        self.w_gate_up = normal(experts, hidden, 2 * inner, std=hidden ** -0.5)
        self.w_down = normal(experts, hidden, inner, std=inner ** -0.5)
        self.w_shared = normal(hidden, hidden, std=hidden ** -0.5)
        self.a = normal(adapters, hidden, rank, std=hidden ** -0.5)
        self.b = normal(adapters, hidden, rank, std=0.5 * rank ** -0.5)
        self.scale = torch.full((adapters,), 2.0, device="cuda")

    def forward(self, x, adapter, keep=False):
        """y [tokens, hidden] fp32, and what ``backward`` needs when ``keep``."""
        tokens = x.shape[0]
        logits = x.float() @ self.w_router
        probs, experts, idx, groups, _ = pgg.route(logits, self.top_k)
        h, gate_up, _ = pgg.swiglu(x, self.w_gate_up, idx, groups, tokens, self.top_k, 0,
                                   probs=probs, keep=keep)
        y, _ = pgg.dx(h, self.w_down, idx, groups, tokens, self.top_k, 0)
        shared, _ = pgg.adapters(x, self.w_shared, self.a, self.b, adapter, scale=self.scale)
        y += shared
        return y, (x, adapter, logits, probs, experts, idx, groups, gate_up) if keep else None

    def backward(self, d_y, kept):
        """Gradients of x, the expert weights, the router's weight and the adapters (the shared
        projection is frozen) from d_y [tokens, hidden] in the layer's dtype."""
        x, adapter, logits, probs, experts, idx, groups, gate_up = kept
        tokens, k = x.shape[0], self.top_k
        d_h, _ = pgg.fwd(d_y, self.w_down, idx, groups, tokens, k, 0)
        d_gate_up, d_probs, h, _ = pgg.swiglu_grad(d_h, gate_up, idx, k, 0, probs=probs)
        d_x, _ = pgg.dx(d_gate_up, self.w_gate_up, idx, groups, tokens, k, 0)
        d_w_gate_up, _ = pgg.dw(x, d_gate_up, idx, groups, tokens, k, 0)
        d_w_down, _ = pgg.dw(d_y, h, idx, groups, tokens, k, 0)
        d_logits = pgg.route_grad(d_probs, logits, experts)
        d_x_shared, d_a, d_b, _ = pgg.adapters_grad(d_y, x, self.w_shared, self.a, self.b, adapter,
                                                    scale=self.scale)
        d_x += d_x_shared
        d_x += d_logits @ self.w_router.T
        return dict(x=d_x, w_gate_up=d_w_gate_up, w_down=d_w_down,
                    w_router=x.float().T @ d_logits, a=d_a, b=d_b)


def reference(layer, x, adapter, d_y):
    """y and the same gradients by autograd in float64, with dense loops over nothing: every token
    gathers its experts' weights (small sizes only)."""
    names = ("w_gate_up", "w_down", "w_router", "a", "b")
    w = {n: getattr(layer, n).double().requires_grad_() for n in names}
    xd = x.double().requires_grad_()
    logits = xd @ w["w_router"]
    # the choice is the layer's own: rounding may order two nearly equal logits otherwise
    experts = pgg.route((x.float() @ layer.w_router), layer.top_k)[1]
    p = torch.softmax(logits, 1).gather(1, experts)
    p = p / p.sum(1, keepdim=True)
    inner = layer.w_down.shape[2]
    gu = torch.einsum("th,tjhf->tjf", xd, w["w_gate_up"][experts])
    h = torch.nn.functional.silu(gu[..., :inner]) * gu[..., inner:] * p[..., None]
    y = torch.einsum("tjf,tjhf->th", h, w["w_down"][experts])
    y = y + xd @ layer.w_shared.double()
    on = (adapter >= 0).nonzero().reshape(-1)
    ad = adapter[on]
    low = torch.einsum("th,thr->tr", xd[on], w["a"][ad]) * layer.scale.double()[ad][:, None]
    y = y.index_add(0, on, torch.einsum("tr,tnr->tn", low, w["b"][ad]))
    grads = torch.autograd.grad((y * d_y.double()).sum(), [xd] + [w[n] for n in names])
    return y.detach(), dict(zip(("x",) + names, grads))


def main():
    gen = torch.Generator(device="cuda").manual_seed(1)
    layer = MoELayer(hidden=256, inner=128, experts=16, top_k=4, adapters=5, rank=16)
    for tokens in (300, 1):
        x = torch.randn(tokens, 256, generator=gen, device="cuda").bfloat16()
        d_y = torch.randn(tokens, 256, generator=gen, device="cuda").bfloat16()
        adapter = torch.randint(-1, 5, (tokens,), generator=gen, device="cuda")
        y, kept = layer.forward(x, adapter, keep=True)
        grads = layer.backward(d_y, kept)
        want, want_grads = reference(layer, x, adapter, d_y)
        worst = float((y.double() - want).abs().max() / want.abs().max())
        print(f"{tokens} tokens: y off by {worst:.1e} of its largest value")
        for name, g in grads.items():
            off = float((g.double() - want_grads[name]).abs().max())
            off /= max(float(want_grads[name].abs().max()), 1e-30)
            worst = max(worst, off)
            print(f"    gradient of {name}: {off:.1e}")
        # bf16 operands, intermediates and outputs: a few units of 2^-8 of the largest values
        if not worst <= 3e-2:
            raise SystemExit("further from the float64 values than the dtype explains")
    print("ok")


if __name__ == "__main__":
    from permute_grouped_gemm_gb300 import build
    build.build()
    main()
