"""Cases, plain forms and exact values of the operators of a whole mixture-of-experts block.

w4           products with 4-bit expert weights and group scales over ragged groups of rows:
             "rows" y = x w[g], "gated" h = prob silu(x w_gate[g]) (x w_up[g]), and "combined",
             the down projection summed over a token's experts
block_norm   the norms around a block with its gate and residual scale,
             r = residual_scale x + gate N_post(y), h = N_pre(r); its gradient
clip         the global norm of a list of gradients, and the gradients clipped to it

`run` computes them in plain torch operations in 32 bits (own = False) or through
permute_grouped_gemm_gb300 (own = True).
"""

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # decoding one token: eight experts' gate and up weights are streamed for one row each
        dict(name="w4-token", op="w4", product="gated", tokens=1, experts=60, top_k=8, k=7168,
             n=2048, group=128, zeros=False, dtype="bf16", scales="bf16", out="bf16", skew=0.0,
             row_idx_type=0),
        # its down projection with the sum over the token's experts
        dict(name="w4-down", op="w4", product="combined", tokens=1, experts=60, top_k=8, k=2048,
             n=7168, group=128, zeros=False, dtype="bf16", scales="bf16", out="fp32", skew=0.0,
             row_idx_type=0),
        # decoding a batch over many experts, about eight rows each, weights with zero points
        dict(name="w4-batch", op="w4", product="gated", tokens=256, experts=256, top_k=8, k=7168,
             n=2048, group=128, zeros=True, dtype="bf16", scales="bf16", out="bf16", skew=0.0,
             row_idx_type=0),
        # a prefill: hundreds of rows an expert, the products bound it
        dict(name="w4-prefill", op="w4", product="gated", tokens=2048, experts=60, top_k=8, k=7168,
             n=2048, group=128, zeros=False, dtype="bf16", scales="bf16", out="bf16", skew=0.0,
             row_idx_type=1),
        # full precision, odd widths, rows of 511 bytes, a last group that is cut short
        dict(name="w4-odd", op="w4", product="rows", tokens=150, experts=7, top_k=3, k=1021, n=286,
             group=32, zeros=True, dtype="fp32", scales="fp32", out="fp32", skew=0.8,
             row_idx_type=1),
        # one decoded token between two blocks
        dict(name="norm-token", op="block_norm", tokens=1, hidden=7168, dtype="bf16", y="fp32",
             post="rms", pre="rms", gate="channel", params="bf16", bias=False),
        # a training step's forward at the largest size, y as the experts' products leave it
        dict(name="norm-train", op="block_norm", tokens=13500, hidden=7168, dtype="bf16", y="fp32",
             post="rms", pre="rms", gate="channel", params="bf16", bias=False),
        # its backward pass
        dict(name="norm-grad", op="block_norm_grad", tokens=13500, hidden=7168, dtype="bf16",
             y="fp32", post="rms", pre="rms", gate="channel", params="bf16", bias=False),
        # full precision, an odd width, norms with mean and bias, a gate of one number a token
        dict(name="norm-odd", op="block_norm_grad", tokens=1500, hidden=1021, dtype="fp32",
             y="fp32", post="layer", pre="layer", gate="token", params="fp32", bias=True),
        # the gradients of a few adapters
        dict(name="clip-adapters", op="clip", sizes="adapters", tensors=14, numel=1 << 20,
             dtype="fp16", max_norm=1.0, scale=1 / 1024.0),
        # the gradients of a layer of 60 experts, small tensors beside very large ones
        dict(name="clip-experts", op="clip", sizes="mixed", tensors=40, numel=1 << 29,
             dtype="bf16", max_norm=1.0, scale=1.0),
        # the norm alone, of the gradients of a whole model in many tensors
        dict(name="grad-norm", op="grad_norm", sizes="mixed", tensors=300, numel=400_000_003,
             dtype="mixed", max_norm=1.0, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_WIDTHS = (512, 1024, 1408, 2048, 2560, 3584, 4096, 5120, 7168)


def draw(rng):
    op = rng.choice(("w4", "w4", "w4", "block_norm", "block_norm", "block_norm_grad",
                     "block_norm_grad", "clip", "clip", "grad_norm"))
    if op == "w4":
        odd = rng.random() < 0.2  # any type and width
        dtype = rng.choice(("fp32", "bf16", "fp16") if odd else ("bf16", "bf16", "fp16"))
        product = rng.choice(("rows", "gated", "gated", "combined"))
        return dict(op=op, product=product, tokens=_log_int(rng, 1, 150 if odd else 1500),
                    experts=_log_int(rng, 8, 16 if odd else 96), top_k=rng.randint(1, 8),
                    k=rng.randint(65, 1100) if odd else rng.choice(_WIDTHS),
                    n=rng.randint(33, 400) if odd else rng.choice(_WIDTHS[:6]),
                    group=rng.choice((32, 64, 128, 128)), zeros=rng.random() < 0.4, dtype=dtype,
                    scales=rng.choice((dtype, dtype, "fp32")),
                    out="fp32" if product == "combined" or (product == "rows" and
                                                            rng.random() < 0.4) else dtype,
                    skew=rng.choice((0.0, 0.0, 0.6)), row_idx_type=rng.randint(0, 1))
    if op in ("block_norm", "block_norm_grad"):
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        return dict(op=op, tokens=_log_int(rng, 1, 12000 if dtype != "fp32" else 6000),
                    hidden=rng.choice(_WIDTHS) if rng.random() < 0.75 else rng.randint(33, 7000),
                    dtype=dtype, y=rng.choice((dtype, "fp32")),
                    post=rng.choice(("rms", "rms", "layer", "none")),
                    pre=rng.choice(("rms", "rms", "layer")),
                    gate=rng.choice(("none", "channel", "token", "full")),
                    params=rng.choice((dtype, "fp32")), bias=rng.random() < 0.5)
    return dict(op=op, sizes=rng.choice(("mixed", "mixed", "adapters")),
                tensors=_log_int(rng, 1, 60 if op == "clip" else 300),
                numel=_log_int(rng, 20_000, 250_000_000),
                dtype=rng.choice(("bf16", "fp16", "fp32", "mixed")),
                max_norm=rng.choice((0.5, 1.0, 1e9)), scale=rng.choice((1.0, 1.0, 1 / 1024.0)))


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(gen, shape, dtype, std=1.0):
    """N(0, std^2) drawn in fp32 slice by slice of the first axis, rounded to `dtype`."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    rows = max(1, (1 << 28) // max(1, t[0].numel()))
    for i in range(0, shape[0], rows):
        s = t[i:i + rows]
        s.copy_(torch.randn(s.shape, generator=gen, device="cuda") * std)
    return t


def _routing(gen, case):
    """(expandedRowIdx, groupList, gather): top_k distinct experts a token, popularity r^-skew over
    the experts in a random order, rows sorted by (expert, original position)."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    rank = torch.randperm(e, generator=gen, device="cuda").float() + 1
    u = torch.rand(t, e, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    pick = (-case["skew"] * rank.log() - (-u.log()).log()).topk(k, dim=1).indices.reshape(-1)
    gather = torch.argsort(pick, stable=True)
    counts = torch.bincount(pick, minlength=e)
    if case["row_idx_type"] == 0:
        return gather, counts, gather
    scatter = torch.empty_like(gather)
    scatter[gather] = torch.arange(gather.numel(), device="cuda")
    return scatter, counts, gather


def _prepare_w4(gen, case):
    t, k = case["tokens"], case["k"]
    columns = case["n"] * (2 if case["product"] == "gated" else 1)
    s = dict(case=case)
    s["idx"], s["groups"], gather = _routing(gen, case)
    rows = gather.numel() if case["product"] == "combined" else t
    s["x"] = _normal(gen, (rows, k), DTYPES[case["dtype"]])
    # the bytes of quantised weights: nearly all codes are used; an odd width leaves the last byte's
    # upper half, which belongs to no weight, as it comes
    shape = (case["experts"], columns)
    s["codes"] = torch.randint(0, 256, shape + ((k + 1) // 2,), generator=gen, device="cuda",
                               dtype=torch.uint8)
    groups = (k + case["group"] - 1) // case["group"]
    scales = torch.rand(shape + (groups,), generator=gen, device="cuda") + 0.5
    s["scales"] = (scales * (0.2 / math.sqrt(k))).to(DTYPES[case["scales"]])
    s["zeros"] = torch.randint(5, 11, shape + (groups,), generator=gen, device="cuda",
                               dtype=torch.uint8) if case["zeros"] else None
    s["probs"] = None
    if case["product"] == "gated":
        p = torch.rand(t, case["top_k"], generator=gen, device="cuda") + 1e-3
        s["probs"] = p / p.sum(1, keepdim=True)
    return s


def _prepare_norm(gen, case):
    t, h = case["tokens"], case["hidden"]
    dt, pt = DTYPES[case["dtype"]], DTYPES[case["params"]]
    s = dict(case=case, residual_scale=0.75)
    s["x"] = _normal(gen, (t, h), dt, 2.0)
    s["y"] = _normal(gen, (t, h), DTYPES[case["y"]], 0.7)
    shape = {"none": None, "channel": (h,), "token": (t, 1), "full": (t, h)}[case["gate"]]
    s["gate"] = _normal(gen, shape, pt, 0.5) if shape else None
    for side in ("post", "pre"):
        s[side + "_weight"] = None if case[side] == "none" else (
            1 + 0.2 * torch.randn(h, generator=gen, device="cuda")).to(pt)
        s[side + "_bias"] = _normal(gen, (h,), pt, 0.1) \
            if case[side] == "layer" and case["bias"] else None
    if case["op"] == "block_norm_grad":
        s["r"] = s.pop("x")  # (the forward's output: what is kept for the backward)
        s["d_r"] = _normal(gen, (t, h), dt)
        s["d_h"] = _normal(gen, (t, h), DTYPES[case["y"]])  # (what the experts' gradient leaves)
    return s


def _numels(case):
    """Sizes of the tensors: alike, or a few large ones that hold nearly everything."""
    n, total = case["tensors"], case["numel"]
    if case["sizes"] == "adapters":
        return [max(1, total // n)] * n
    part = [math.exp(-12 * (i * 0.618034 % 1)) for i in range(n)]
    return [max(1, int(p / sum(part) * total)) for p in part]


def _prepare_clip(gen, case):
    kinds = ("bf16", "fp32", "fp16") if case["dtype"] == "mixed" else (case["dtype"],)
    s = dict(case=case)
    s["grads"] = [_normal(gen, (n,), DTYPES[kinds[i % len(kinds)]], 0.02 / case["scale"])
                  for i, n in enumerate(_numels(case))]
    s["out"] = [torch.empty_like(g) for g in s["grads"]] if case["op"] == "clip" else None
    return s


def prepare(case, seed):
    make = {"w4": _prepare_w4, "block_norm": _prepare_norm, "block_norm_grad": _prepare_norm,
            "clip": _prepare_clip, "grad_norm": _prepare_clip}
    return make[case["op"]](_generator(seed), case)


# ---------------------------------------------------------------- plain forms

def _positions(s):
    """Original position of every expanded row."""
    if s["case"]["row_idx_type"] == 0:
        return s["idx"]
    pos = torch.empty_like(s["idx"])
    pos[s["idx"]] = torch.arange(s["idx"].numel(), device="cuda")
    return pos


def _padded(counts):
    """The non-empty groups, and each row's place (group, slot) in an array padded to the longest."""
    live = counts.nonzero().reshape(-1)
    counts = counts[live]
    start = counts.cumsum(0) - counts
    group = torch.repeat_interleave(torch.arange(live.numel(), device="cuda"), counts)
    slot = torch.arange(group.numel(), device="cuda") - start[group]
    return live, group, slot, int(counts.max())


def _plain_weights(s, live):
    """scale (code - zero) of the live experts, [live, columns, k] in 32 bits."""
    k, group = s["case"]["k"], s["case"]["group"]
    codes = s["codes"][live]
    w = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:2], -1)[..., :k].float()
    at = torch.arange(k, device="cuda") // group
    w -= s["zeros"][live][..., at] if s["zeros"] is not None else 8
    w *= s["scales"][live].float()[..., at]
    return w


def _plain_w4(s):
    c = s["case"]
    pos = _positions(s)
    live, group, slot, most = _padded(s["groups"])
    x = torch.zeros(live.numel(), most, c["k"], device="cuda")
    x[group, slot] = (s["x"] if c["product"] == "combined" else s["x"][pos // c["top_k"]]).float()
    y = torch.bmm(x, _plain_weights(s, live).transpose(1, 2))[group, slot]
    if c["product"] == "gated":
        gate, up = y[:, :c["n"]], y[:, c["n"]:]
        y = gate / (1 + (-gate).exp()) * up * s["probs"].reshape(-1)[pos][:, None]
    if c["product"] == "combined":
        by_token = torch.empty_like(y)
        by_token[pos] = y
        y = by_token.reshape(c["tokens"], c["top_k"], c["n"]).sum(1)
    return y.to(DTYPES[c["out"]])


def _plain_norm_parts(v, kind):
    """The normalised rows and 1 / their deviation."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rstd = 1 / ((v * v).mean(1, keepdim=True) + EPS).sqrt()
    return v * rstd, rstd


def _plain_norm_of(s, side, v):
    if s["case"][side] == "none":
        return v
    n, _ = _plain_norm_parts(v, s["case"][side])
    n = n * s[side + "_weight"].float()
    return n if s[side + "_bias"] is None else n + s[side + "_bias"].float()


def _gate_of(s):
    """The gate, in a shape that broadcasts over [tokens, hidden]."""
    return 1.0 if s["gate"] is None else s["gate"].float()


def _plain_block_norm(s):
    dt = s["x"].dtype
    r = s["residual_scale"] * s["x"].float() + _gate_of(s) * _plain_norm_of(s, "post", s["y"].float())
    return dict(r=r.to(dt), h=_plain_norm_of(s, "pre", r).to(dt))


def _plain_norm_back(s, side, v, d, got):
    """The gradient of v through one norm; the weight's and the bias's go into `got`."""
    kind = s["case"][side]
    if kind == "none":
        return d
    n, rstd = _plain_norm_parts(v, kind)
    got[f"d_{side}_weight"] = (d * n).sum(0)
    if s[side + "_bias"] is not None:
        got[f"d_{side}_bias"] = d.sum(0)
    d = d * s[side + "_weight"].float()
    d = d - n * (d * n).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if kind == "layer" else 0)
    return d * rstd


def _plain_block_norm_grad(s):
    dt, got = s["r"].dtype, {}
    g = s["d_r"].float() + _plain_norm_back(s, "pre", s["r"].float(), s["d_h"].float(), got)
    got["d_x"] = (s["residual_scale"] * g).to(dt)
    y = s["y"].float()
    kind = s["case"]["gate"]
    if kind != "none":
        d_gate = g * _plain_norm_of(s, "post", y)
        got["d_gate"] = (d_gate.sum(0) if kind == "channel" else d_gate.sum(1, keepdim=True) if kind == "token"
                         else d_gate.to(s["gate"].dtype))
    got["d_y"] = _plain_norm_back(s, "post", y, g * _gate_of(s), got).to(dt)
    return got


def _plain_grad_norm(s):
    squares = [(g.float() * g.float()).sum(dtype=torch.float64) for g in s["grads"]]
    return (torch.stack(squares).sum().sqrt() * s["case"]["scale"]).float()


def _plain_clip(s):
    norm = _plain_grad_norm(s)
    by = s["case"]["scale"] * (s["case"]["max_norm"] / (norm + 1e-6)).clamp(max=1)
    return dict(norm=norm, grads=[(g.float() * by).to(g.dtype) for g in s["grads"]])


# ---------------------------------------------------------------- the framework's calls

def _own_w4(s):
    import permute_grouped_gemm_gb300 as pgg
    c = s["case"]
    common = (s["x"], s["codes"], s["scales"], s["idx"], s["groups"], c["tokens"], c["top_k"],
              c["row_idx_type"])
    if c["product"] == "gated":
        return pgg.swiglu_w4(*common, group=c["group"], zeros=s["zeros"], probs=s["probs"])[0]
    if c["product"] == "combined":
        return pgg.down_w4(*common, group=c["group"], zeros=s["zeros"])[0]
    return pgg.fwd_w4(*common, group=c["group"], zeros=s["zeros"], out_dtype=DTYPES[c["out"]])[0]


def _norm_args(s):
    kinds = {side: None if s["case"][side] == "none" else s["case"][side] for side in ("post", "pre")}
    return dict(kinds, gate=s["gate"], post_weight=s["post_weight"], post_bias=s["post_bias"],
                pre_weight=s["pre_weight"], residual_scale=s["residual_scale"], eps=EPS)


def _own_block_norm(s):
    import permute_grouped_gemm_gb300 as pgg
    r, h = pgg.block_norm(s["x"], s["y"], pre_bias=s["pre_bias"], **_norm_args(s))
    return dict(r=r, h=h)


def _own_block_norm_grad(s):
    import permute_grouped_gemm_gb300 as pgg
    got, _ = pgg.block_norm_grad(s["d_r"], s["d_h"], s["r"], s["y"], pre_bias=s["pre_bias"],
                                 **_norm_args(s))
    return {name: t for name, t in got.items() if t is not None}


def _own_grad_norm(s):
    import permute_grouped_gemm_gb300 as pgg
    return pgg.grad_norm(s["grads"], scale=s["case"]["scale"])[0]


def _own_clip(s):
    import permute_grouped_gemm_gb300 as pgg
    norm, grads, _ = pgg.clip_grads(s["grads"], s["case"]["max_norm"], scale=s["case"]["scale"],
                                    out=s["out"])
    return dict(norm=norm, grads=grads)


_PLAIN = dict(w4=_plain_w4, block_norm=_plain_block_norm, block_norm_grad=_plain_block_norm_grad,
              clip=_plain_clip, grad_norm=_plain_grad_norm)
_OWN = dict(w4=_own_w4, block_norm=_own_block_norm, block_norm_grad=_own_block_norm_grad,
            clip=_own_clip, grad_norm=_own_grad_norm)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

_BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}


def work(case):
    op = case["op"]
    if op == "w4":
        t, k, n, e, m = (case[x] for x in ("tokens", "k", "n", "experts", "top_k"))
        m *= t
        columns = n * (2 if case["product"] == "gated" else 1)
        live = e * (1 - (1 - case["top_k"] / e) ** t)
        groups = (k + case["group"] - 1) // case["group"]
        weights = (k + 1) // 2 + groups * (_BYTES[case["scales"]] + (1 if case["zeros"] else 0))
        combined = case["product"] == "combined"
        return dict(bytes=live * columns * weights + (m if combined else t) * k * _BYTES[case["dtype"]]
                    + (t if combined else m) * n * _BYTES[case["out"]] + 8 * m + 8 * e
                    + (4 * m if case["product"] == "gated" else 0), flops=2 * m * k * columns)
    if op in ("block_norm", "block_norm_grad"):
        t, h, es, ys = case["tokens"], case["hidden"], _BYTES[case["dtype"]], _BYTES[case["y"]]
        gate = {"none": 0, "channel": h, "token": t, "full": t * h}[case["gate"]]
        params = sum(case[side] != "none" for side in ("post", "pre"))
        params += sum(case[side] == "layer" and case["bias"] for side in ("post", "pre"))
        once = (gate + params * h) * _BYTES[case["params"]]
        if op == "block_norm":
            return dict(bytes=t * h * (3 * es + ys) + once, flops=14 * t * h)
        back = params * h * 4 + gate * (_BYTES[case["params"]] if case["gate"] == "full" else 4)
        return dict(bytes=t * h * (4 * es + 2 * ys) + once + back, flops=34 * t * h)
    size = 8 / 3 if case["dtype"] == "mixed" else _BYTES[case["dtype"]]
    return dict(bytes=case["numel"] * size * (2 if op == "clip" else 1),
                flops=case["numel"] * (3 if op == "clip" else 2))


# ---------------------------------------------------------------- exact values

def _exact_w4(s):
    c = s["case"]
    k, n = c["k"], c["n"]
    idx = s["idx"].cpu()
    pos = (idx if c["row_idx_type"] == 0 else torch.argsort(idx)).cuda()
    column = torch.arange(k, device="cuda")
    parts, at = [], 0
    for g, rows in enumerate(s["groups"].tolist()):
        if rows == 0:
            continue
        take = torch.arange(at, at + rows, device="cuda")
        x = s["x"][take if c["product"] == "combined" else pos[take] // c["top_k"]].double()
        # sixteen to the power of k mod 2 divides the byte's upper half down
        code = (s["codes"][g][:, column // 2].to(torch.int32) // 16 ** (column % 2).to(torch.int32)) % 16
        zero = 8.0 if s["zeros"] is None else s["zeros"][g].double()[:, column // c["group"]]
        w = s["scales"][g].double()[:, column // c["group"]] * (code.double() - zero)
        parts.append(x @ w.T)
        at += rows
    y = torch.cat(parts)
    if c["product"] == "gated":
        y = torch.nn.functional.silu(y[:, :n]) * y[:, n:]
        y = y * s["probs"].double().reshape(-1)[pos][:, None]
    if c["product"] == "combined":
        y = torch.zeros(c["tokens"], n, dtype=torch.double, device="cuda").index_add_(
            0, pos // c["top_k"], y)
    return y


def _exact_forward(s, p):
    """r and h from the tensors in `p`, by torch's own norms in 64 bits."""
    c = s["case"]
    width = (c["hidden"],)

    def norm(side, v):
        if c[side] == "layer":
            return torch.nn.functional.layer_norm(v, width, p[side + "_weight"], p.get(side + "_bias"),
                                                  EPS)
        return v if c[side] == "none" else torch.nn.functional.rms_norm(v, width, p[side + "_weight"],
                                                                        EPS)

    n = norm("post", p["y"])
    if "gate" in p:
        n = p["gate"] * n
    r = s["residual_scale"] * p["x"] + n
    return r, norm("pre", r)


def _exact_block_norm(s):
    parts, step = [], 2048
    for i in range(0, s["case"]["tokens"], step):  # slices of rows: 64 bits of everything are large
        p = _exact_inputs(s, i, i + step, ("x", "y"))
        parts.append(_exact_forward(s, p))
    return dict(r=torch.cat([r for r, _ in parts]), h=torch.cat([h for _, h in parts]))


def _exact_inputs(s, begin, end, rows):
    p = {n: s[n][begin:end].double() for n in rows}
    for n in ("gate", "post_weight", "post_bias", "pre_weight", "pre_bias"):
        if s[n] is not None:
            by_row = n == "gate" and s["case"]["gate"] != "channel"
            p[n] = (s[n][begin:end] if by_row else s[n]).double()
    return p


def _exact_block_norm_grad(s):
    """By differentiation: x is what gives the kept r, in 64 bits."""
    by_row, summed, step = {}, {}, 2048
    for i in range(0, s["case"]["tokens"], step):
        p = _exact_inputs(s, i, i + step, ("r", "y"))
        with torch.enable_grad():
            r = p.pop("r")
            p["x"] = torch.zeros_like(r)
            p = {n: t.requires_grad_() for n, t in p.items()}
            out, _ = _exact_forward(s, p)
            p["x"] = ((r - out) / s["residual_scale"]).detach().requires_grad_()
            out, h = _exact_forward(s, p)
            loss = (out * s["d_r"][i:i + step].double()).sum() \
                + (h * s["d_h"][i:i + step].double()).sum()
            grads = dict(zip(p, torch.autograd.grad(loss, list(p.values()))))
        for n, d in grads.items():
            if n in ("x", "y") or (n == "gate" and s["case"]["gate"] != "channel"):
                by_row.setdefault("d_" + n, []).append(d)
            else:
                summed["d_" + n] = summed.get("d_" + n, 0) + d
    return dict({n: torch.cat(d) for n, d in by_row.items()}, **summed)


def _exact_norm(s):
    # slices: 64 bits of a very large tensor are large
    return abs(s["case"]["scale"]) * math.sqrt(math.fsum(
        float(torch.linalg.vector_norm(part.double())) ** 2
        for g in s["grads"] for part in g.split(1 << 27)))


def _exact_clip(s):
    c, norm = s["case"], _exact_norm(s)
    factor = c["scale"] * min(1.0, c["max_norm"] / (norm + 1e-6))
    return dict(norm=torch.tensor(norm, dtype=torch.double),
                grads=[g.double() * factor for g in s["grads"]])


_EXACT = dict(w4=_exact_w4, block_norm=_exact_block_norm, block_norm_grad=_exact_block_norm_grad,
              clip=_exact_clip,
              grad_norm=lambda s: torch.tensor(_exact_norm(s), dtype=torch.double))


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
