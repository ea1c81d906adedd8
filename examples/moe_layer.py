"""A mixture-of-experts layer with a shared projection, from the library's operators.

    logits = x w_router
    probs, order = route(logits)                          top-k choice and expanded order
    h = swiglu(x, w_gate_up, order, probs)                gated expert product, weighted
    y = dx(h, w_down, order)                              down projection and combination
    y += adapters(x, w_shared, a, b, adapter)             shared projection, one adapter a token

dx, the framework's fused input gradient, is the down projection here: with w_down
[experts, hidden, inner] it computes sum over a token's experts of h w_down^T. The backward pass
uses the same operators the other way round. The routing is computed once and serves them all.

Around the layer stands a block of a decoder,

    r, h = block_norm(x, pre="rms")                       the norm before the layer
    r, h = block_norm(r, layer(h), gate, post="rms", pre="rms")
                                                          its output's norm, gate and sum with the
                                                          residual stream, the next block's norm

whose gradients are clipped by their global norm; for serving, the experts' weights are brought to
4 bits with a scale a group and run by swiglu_w4 and down_w4.

    python examples/moe_layer.py            one training step and one decode step, checked, of the
                                            layer and of the block, and one with 4-bit experts
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

        self.w4 = None

    def quantise(self, group=64):
        """4-bit experts from here on, for serving; the weights that they stand for."""
        gate_up = to_4_bits(self.w_gate_up.transpose(1, 2), group)
        down = to_4_bits(self.w_down, group)
        self.w4 = group, gate_up[:2], down[:2]
        return gate_up[2].transpose(1, 2).contiguous(), down[2]

    def forward(self, x, adapter, keep=False):
        """y [tokens, hidden] fp32, and what ``backward`` needs when ``keep``."""
        tokens = x.shape[0]
        logits = x.float() @ self.w_router
        probs, experts, idx, groups, _ = pgg.route(logits, self.top_k)
        if self.w4 is None:
            h, gate_up, _ = pgg.swiglu(x, self.w_gate_up, idx, groups, tokens, self.top_k, 0,
                                       probs=probs, keep=keep)
            y, _ = pgg.dx(h, self.w_down, idx, groups, tokens, self.top_k, 0)
        else:
            group, up, down = self.w4
            h, _ = pgg.swiglu_w4(x, *up, idx, groups, tokens, self.top_k, 0, group, probs=probs)
            y, _ = pgg.down_w4(h, *down, idx, groups, tokens, self.top_k, 0, group)
            gate_up = None
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


def to_4_bits(w, group):
    """(codes, scales, what they stand for) of w [experts, columns, k]: two codes a byte, one scale
    of w's dtype a group of k, and no zero points (8 stands for 0)."""
    g, n, k = w.shape
    parts = w.float().contiguous().reshape(g, n, k // group, group)
    scales = (parts.abs().amax(3) / 7).clamp_min(1e-8).to(w.dtype)
    codes = (parts / scales.float()[..., None]).round().clamp(-8, 7).reshape(g, n, k) + 8
    value = (codes - 8).reshape(parts.shape).double() * scales.double()[..., None]
    codes = codes.to(torch.uint8)
    return codes[..., ::2] | codes[..., 1::2] << 4, scales, value.reshape(g, n, k)


class Block:
    """The layer in a decoder's residual stream, with the norm of the block behind it."""

    def __init__(self, layer, hidden, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layer = layer
        self.w_in, self.w_post, self.w_next, self.gate = (
            (torch.randn(hidden, generator=gen, device="cuda") * 0.2 + 1).to(layer.w_down.dtype)
            for _ in range(4))

    def _around(self):
        return dict(gate=self.gate, post="rms", post_weight=self.w_post, pre="rms",
                    pre_weight=self.w_next, residual_scale=0.9)

    def forward(self, x, adapter, keep=False):
        """(the residual stream, the next block's input), and what ``backward`` needs."""
        r0, h0 = pgg.block_norm(x, pre="rms", pre_weight=self.w_in)
        y, kept = self.layer.forward(h0, adapter, keep=keep)
        r, h = pgg.block_norm(r0, y, **self._around())
        return r, h, (r0, y, r, kept) if keep else None

    def backward(self, d_r, d_h, kept, max_norm):
        """The gradient of x, and the parameters' gradients clipped by their global norm."""
        r0, y, r, kept = kept
        out, _ = pgg.block_norm_grad(d_r, d_h, r, y, **self._around())
        grads = self.layer.backward(out["d_y"], kept)
        first, _ = pgg.block_norm_grad(out["d_x"], grads.pop("x"), r0, pre="rms",
                                       pre_weight=self.w_in)
        grads.update(w_in=first["d_pre_weight"], w_post=out["d_post_weight"],
                     w_next=out["d_pre_weight"], gate=out["d_gate"])
        norm, _, _ = pgg.clip_grads(list(grads.values()), max_norm)
        return first["d_x"], grads, norm


def block_reference(block, x, adapter, d_r, d_h, max_norm):
    """(r, h), and the same gradients by autograd in float64."""
    names = ("w_in", "w_post", "w_next", "gate")
    p = {n: getattr(block, n).double().requires_grad_() for n in names}

    def rms(v, w):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w

    xd = x.double().requires_grad_()
    # the experts are those of the norm that the layer reads, which is rounded
    h0 = pgg.block_norm(x, pre="rms", pre_weight=block.w_in)[1]
    y, w = reference(block.layer, h0, adapter, x=rms(xd, p["w_in"]))
    r = 0.9 * xd + p["gate"] * rms(y, p["w_post"])
    h = rms(r, p["w_next"])
    w.update(p)
    grads = torch.autograd.grad((r * d_r.double()).sum() + (h * d_h.double()).sum(),
                                [xd] + list(w.values()))
    d_x, grads = grads[0], dict(zip(w, grads[1:]))
    norm = sum(g.square().sum() for g in grads.values()).sqrt()
    factor = min(1.0, max_norm / (float(norm) + 1e-6))
    return r.detach(), h.detach(), d_x, {n: g * factor for n, g in grads.items()}, norm


def reference(layer, h, adapter, d_y=None, x=None):
    """y and the same gradients by autograd in float64, with dense loops over nothing: every token
    gathers its experts' weights (small sizes only). With x, h in float64, instead of d_y: y and the
    weights that it depends on."""
    names = ("w_gate_up", "w_down", "w_router", "a", "b")
    w = {n: getattr(layer, n).double().requires_grad_() for n in names}
    xd = h.double().requires_grad_() if x is None else x
    logits = xd @ w["w_router"]
    # the choice is the layer's own: rounding may order two nearly equal logits otherwise
    experts = pgg.route((h.float() @ layer.w_router), layer.top_k)[1]
    p = torch.softmax(logits, 1).gather(1, experts)
    p = p / p.sum(1, keepdim=True)
    inner = layer.w_down.shape[2]
    gu = torch.einsum("th,tjhf->tjf", xd, w["w_gate_up"][experts])
    act = torch.nn.functional.silu(gu[..., :inner]) * gu[..., inner:] * p[..., None]
    y = torch.einsum("tjf,tjhf->th", act, w["w_down"][experts])
    y = y + xd @ layer.w_shared.double()
    on = (adapter >= 0).nonzero().reshape(-1)
    ad = adapter[on]
    low = torch.einsum("th,thr->tr", xd[on], w["a"][ad]) * layer.scale.double()[ad][:, None]
    y = y.index_add(0, on, torch.einsum("tr,tnr->tn", low, w["b"][ad]))
    if x is not None:
        return y, w
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
    block = Block(layer, 256)
    for tokens in (300, 1):
        x, d_r, d_h = (torch.randn(tokens, 256, generator=gen, device="cuda").bfloat16()
                       for _ in range(3))
        adapter = torch.randint(-1, 5, (tokens,), generator=gen, device="cuda")
        r, h, kept = block.forward(x, adapter, keep=True)
        d_x, grads, norm = block.backward(d_r, d_h, kept, max_norm=1.0)
        want = block_reference(block, x, adapter, d_r, d_h, max_norm=1.0)
        got = dict(r=(r, want[0]), h=(h, want[1]), d_x=(d_x, want[2]), norm=(norm, want[4]),
                   **{n: (g, want[3][n]) for n, g in grads.items()})
        off = {n: float((a.double() - b).abs().max()) / max(float(b.abs().max()), 1e-30)
               for n, (a, b) in got.items()}
        print(f"block, {tokens} tokens: off by at most {max(off.values()):.1e}")
        if not max(off.values()) <= 3e-2:
            raise SystemExit(f"further from the float64 values than the dtype explains: {off}")
    layer.w_gate_up, layer.w_down = layer.quantise()  # (what the codes stand for, for the check)
    for tokens in (300, 1):
        x = torch.randn(tokens, 256, generator=gen, device="cuda").bfloat16()
        adapter = torch.randint(-1, 5, (tokens,), generator=gen, device="cuda")
        y, _ = layer.forward(x, adapter)
        want, _ = reference(layer, x, adapter, torch.zeros_like(x))
        off = float((y.double() - want).abs().max() / want.abs().max())
        print(f"4-bit experts, {tokens} tokens: y off by {off:.1e}")
        if not off <= 3e-2:
            raise SystemExit("further from the float64 values than the dtype explains")
    print("ok")


if __name__ == "__main__":
    from permute_grouped_gemm_gb300 import build
    build.build()
    main()
