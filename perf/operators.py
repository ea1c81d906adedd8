"""Cases, plain forms and exact values of the operators around the grouped expert products.

Three operators, each with its gradient:

route      top-k expert choice from router logits, the routing weights, and the expanded order
           (expandedRowIdx, groupList) that the grouped products read
swiglu     the gated product of the experts, h = prob * silu(x w_gate[g]) * (x w_up[g]), over
           ragged groups of rows; its gradient from d_h and the kept pre-activations
adapters   a shared projection with one low-rank adapter per token,
           y = x W + scale[ad] (x a[ad]) b[ad]^T; its gradient for x, a and b

`run` computes them in plain torch operations in 32 bits (own = False) or through
permute_grouped_gemm_gb300 (own = True).
"""

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the router of one decoded token: latency only
        dict(name="route-token", op="route", tokens=1, experts=60, top_k=8, dtype="fp32",
             score="softmax", renormalize=True, bias=False, row_idx_type=0),
        # the router of a long prefill over many experts, with a selection bias
        dict(name="route-prefill", op="route", tokens=65536, experts=256, top_k=8, dtype="bf16",
             score="sigmoid", renormalize=True, bias=True, row_idx_type=1),
        # the router's backward pass in a training step
        dict(name="route-train", op="route_grad", tokens=13500, experts=60, top_k=8, dtype="fp32",
             score="softmax", renormalize=False, bias=False, row_idx_type=0),
        # decoding one token: eight experts' weights are streamed for one row each
        dict(name="swiglu-token", op="swiglu", tokens=1, experts=60, top_k=8, hidden=7168,
             inner=2048, dtype="bf16", keep=False, weighted=True, skew=0.0, row_idx_type=0),
        # decoding a batch over many experts: all weights are streamed, about eight rows each
        dict(name="swiglu-batch", op="swiglu", tokens=256, experts=256, top_k=8, hidden=7168,
             inner=2048, dtype="bf16", keep=False, weighted=True, skew=0.0, row_idx_type=0),
        # a training step's forward at the largest size: gate and up are kept for the backward
        dict(name="swiglu-train", op="swiglu", tokens=13500, experts=60, top_k=8, hidden=7168,
             inner=2048, dtype="bf16", keep=True, weighted=True, skew=0.0, row_idx_type=0),
        # full precision, ragged groups, an odd hidden size and rows of 1144 bytes
        dict(name="swiglu-odd", op="swiglu", tokens=1500, experts=7, top_k=3, hidden=1021,
             inner=286, dtype="fp32", keep=False, weighted=False, skew=0.8, row_idx_type=1),
        # the backward of the gate at the training step's size
        dict(name="swiglu-grad", op="swiglu_grad", tokens=13500, experts=60, top_k=8, inner=2048,
             dtype="bf16", weighted=True, skew=0.0, row_idx_type=0),
        # one decoded token of one request
        dict(name="adapters-token", op="adapters", tokens=1, hidden=7168, out=2048, rank=16,
             adapters=8, spread="mixed", dtype="bf16"),
        # a decode batch in which nearly every request has its own adapter
        dict(name="adapters-batch", op="adapters", tokens=48, hidden=7168, out=4096, rank=16,
             adapters=64, spread="mixed", dtype="bf16"),
        # a prefill of several requests, their tokens one after another
        dict(name="adapters-prefill", op="adapters", tokens=8191, hidden=4096, out=4096, rank=32,
             adapters=24, spread="runs", dtype="bf16"),
        # training a handful of adapters on one frozen projection
        dict(name="adapters-train", op="adapters_grad", tokens=8192, hidden=4096, out=2048,
             rank=32, adapters=6, spread="runs", dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_WIDTHS = (512, 1000, 1024, 2048, 2560, 3584, 4096, 5120, 7168)


def draw(rng):
    op = rng.choice(("route", "route_grad", "swiglu", "swiglu", "swiglu_grad", "adapters",
                     "adapters", "adapters_grad"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op in ("route", "route_grad"):
        experts = _log_int(rng, 8, 512)
        return dict(op=op, tokens=_log_int(rng, 1, 60000), experts=experts,
                    top_k=rng.randint(1, min(12, experts)), dtype=rng.choice(("fp32", "bf16")),
                    score=rng.choice(("softmax", "softmax", "sigmoid")),
                    renormalize=rng.random() < 0.6, bias=rng.random() < 0.4,
                    row_idx_type=rng.randint(0, 1))
    if op == "swiglu_grad":
        return dict(op=op, tokens=_log_int(rng, 1, 12000), experts=_log_int(rng, 8, 128),
                    top_k=rng.randint(1, 8),
                    inner=rng.choice((256, 512, 768, 1024, 1408, 2048)) + rng.choice((0, 0, 8, 3)),
                    dtype=rng.choice((dtype, dtype, "fp32")), weighted=rng.random() < 0.7,
                    skew=rng.choice((0.0, 0.6)), row_idx_type=rng.randint(0, 1))
    if op == "swiglu":
        odd = rng.random() < 0.15  # full precision, any width
        tokens = _log_int(rng, 1, 400) if odd else _log_int(rng, 1, 8000)
        hidden = rng.randint(65, 700) if odd else rng.choice(_WIDTHS)
        inner = rng.randint(33, 400) if odd else rng.choice((256, 512, 768, 1024, 1408, 2048))
        return dict(op=op, tokens=tokens, experts=_log_int(rng, 8, 16 if odd else 96),
                    top_k=rng.randint(1, 8), hidden=hidden, inner=inner,
                    dtype="fp32" if odd else dtype, keep=rng.random() < 0.3,
                    weighted=rng.random() < 0.6, skew=rng.choice((0.0, 0.0, 0.6)),
                    row_idx_type=rng.randint(0, 1))
    lo = 1 if op == "adapters" else 512
    return dict(op=op, tokens=_log_int(rng, lo, 6000), hidden=rng.choice(_WIDTHS[:7]),
                out=rng.choice(_WIDTHS[:7]), rank=rng.choice((8, 16, 16, 24, 32, 64)),
                adapters=_log_int(rng, 1, 64), spread=rng.choice(("runs", "mixed")), dtype=dtype)


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


def _probs(gen, t, k):
    p = torch.rand(t, k, generator=gen, device="cuda") + 1e-3
    return p / p.sum(1, keepdim=True)


def prepare(case, seed):
    gen = _generator(seed)
    dt = DTYPES[case["dtype"]]
    op, t = case["op"], case["tokens"]
    s = dict(case=case)
    if op in ("route", "route_grad"):
        e, k = case["experts"], case["top_k"]
        liked = torch.randn(e, generator=gen, device="cuda") * 0.5
        s["logits"] = (torch.randn(t, e, generator=gen, device="cuda") * 1.5 + liked).to(dt)
        s["bias"] = torch.randn(e, generator=gen, device="cuda") * 0.2 if case["bias"] else None
        if op == "route_grad":
            biased = s["logits"].float() + (s["bias"] if case["bias"] else 0.0)
            s["experts"] = torch.argsort(biased, dim=1, descending=True, stable=True)[:, :k].contiguous()
            s["d_probs"] = torch.randn(t, k, generator=gen, device="cuda")
        return s
    if op in ("swiglu", "swiglu_grad"):
        s["idx"], s["groups"], gather = _routing(gen, case)
        m, f = gather.numel(), case["inner"]
        s["probs"] = _probs(gen, t, case["top_k"]) if case["weighted"] else None
        if op == "swiglu":
            s["x"] = _normal(gen, (t, case["hidden"]), dt)
            s["weight"] = _normal(gen, (case["experts"], case["hidden"], 2 * f), dt,
                                  1 / math.sqrt(case["hidden"]))
        else:
            s["gate_up"] = _normal(gen, (m, 2 * f), dt)
            s["d_h"] = _normal(gen, (m, f), dt)
        return s
    k, n, r, a = case["hidden"], case["out"], case["rank"], case["adapters"]
    if case["spread"] == "runs":  # requests one after another, of unequal lengths
        cuts = torch.rand(a, generator=gen, device="cuda")
        ends = (cuts.cumsum(0) / cuts.sum() * t).round()
        ids = torch.bucketize(torch.arange(t, device="cuda", dtype=torch.float32) + 0.5, ends)
        ids = torch.randperm(a, generator=gen, device="cuda")[ids.clamp_(max=a - 1)]
    else:
        ids = torch.randint(0, a, (t,), generator=gen, device="cuda")
    # one request in eight has no adapter
    plain = torch.rand(a, generator=gen, device="cuda") < 0.125
    s["adapter"] = torch.where(plain[ids] & (a > 1), -1, ids)
    s["x"] = _normal(gen, (t, k), dt)
    s["weight"] = _normal(gen, (k, n), dt, 1 / math.sqrt(k))
    s["a"] = _normal(gen, (a, k, r), dt, 1 / math.sqrt(k))
    s["b"] = _normal(gen, (a, n, r), dt, 0.3 / math.sqrt(r))
    s["scale"] = torch.rand(a, generator=gen, device="cuda") + 0.5
    if op == "adapters_grad":
        s["d_y"] = _normal(gen, (t, n), dt)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_route(s):
    c = s["case"]
    e, k = c["experts"], c["top_k"]
    logits = s["logits"].float()
    keyed = logits if s["bias"] is None else logits + s["bias"]
    experts = torch.sort(keyed, dim=1, descending=True, stable=True).indices[:, :k]
    if c["score"] == "softmax":
        score = (logits - logits.amax(1, keepdim=True)).exp()
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + (-logits).exp())
    probs = score.gather(1, experts)
    if c["renormalize"]:
        probs = probs / probs.sum(1, keepdim=True)
    flat = experts.reshape(-1)
    gather = torch.sort(flat, stable=True).indices
    groups = torch.zeros_like(flat[:1]).expand(e).scatter_add(0, flat, torch.ones_like(flat))
    if c["row_idx_type"] == 1:
        idx = torch.empty_like(gather)
        idx[gather] = torch.arange(gather.numel(), device="cuda")
    else:
        idx = gather
    return dict(probs=probs, experts=experts, idx=idx, groups=groups)


def _plain_route_grad(s):
    c = s["case"]
    logits, experts, dp = s["logits"].float(), s["experts"], s["d_probs"]
    if c["score"] == "softmax":
        score = (logits - logits.amax(1, keepdim=True)).exp()
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + (-logits).exp())
    chosen = score.gather(1, experts)
    if c["renormalize"]:
        total = chosen.sum(1, keepdim=True)
        dp = (dp - (dp * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(score).scatter(1, experts, dp)
    if c["score"] == "softmax":
        d = score * (ds - (ds * score).sum(1, keepdim=True))
    else:
        d = ds * score * (1 - score)
    return d.to(s["logits"].dtype)


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
    return live, group, slot, int(counts.max()) if live.numel() else 0


def _plain_swiglu(s):
    c = s["case"]
    dt, f = s["x"].dtype, c["inner"]
    pos = _positions(s)
    live, group, slot, most = _padded(s["groups"])
    x = torch.zeros(live.numel(), most, c["hidden"], device="cuda")
    x[group, slot] = s["x"][pos // c["top_k"]].float()
    gu = torch.bmm(x, s["weight"][live].float())[group, slot]
    gate, up = gu[:, :f], gu[:, f:]
    h = gate / (1 + (-gate).exp()) * up
    if s["probs"] is not None:
        h = h * s["probs"].reshape(-1)[pos][:, None]
    return dict(h=h.to(dt), gate_up=gu.to(dt)) if c["keep"] else dict(h=h.to(dt))


def _plain_swiglu_grad(s):
    c = s["case"]
    dt, f = s["d_h"].dtype, c["inner"]
    pos = _positions(s)
    gate, up, dh = s["gate_up"][:, :f].float(), s["gate_up"][:, f:].float(), s["d_h"].float()
    sig = 1 / (1 + (-gate).exp())
    act = gate * sig
    p = s["probs"].reshape(-1)[pos][:, None] if s["probs"] is not None else 1.0
    d_gate = p * dh * up * sig * (1 + gate * (1 - sig))
    d_up = p * dh * act
    got = dict(d_gate_up=torch.cat([d_gate, d_up], 1).to(dt), h=(p * act * up).to(dt))
    if s["probs"] is not None:
        d_probs = torch.empty_like(s["probs"]).reshape(-1)
        d_probs[pos] = (dh * act * up).sum(1)
        got["d_probs"] = d_probs.reshape(s["probs"].shape)
    return got


def _by_adapter(s):
    """Tokens that have an adapter, in the adapters' order, and their places in a padded array."""
    ad = s["adapter"]
    order = torch.sort(ad, stable=True).indices
    order = order[ad[order] >= 0]
    counts = (ad[:, None] == torch.arange(s["case"]["adapters"], device="cuda")).sum(0)
    return (order,) + _padded(counts)


def _pad(t, order, group, slot, groups, most):
    p = torch.zeros(groups, most, t.shape[1], device="cuda")
    p[group, slot] = t[order].float()
    return p


def _plain_adapters(s):
    order, live, group, slot, most = _by_adapter(s)
    y = s["x"].float() @ s["weight"].float()
    u = torch.bmm(_pad(s["x"], order, group, slot, live.numel(), most), s["a"][live].float())
    low = torch.bmm(u, s["b"][live].float().transpose(1, 2)) * s["scale"][live][:, None, None]
    y[order] += low[group, slot]
    return y.to(s["x"].dtype)


def _plain_adapters_grad(s):
    dt = s["x"].dtype
    order, live, group, slot, most = _by_adapter(s)
    a, b = s["a"][live].float(), s["b"][live].float()
    x = _pad(s["x"], order, group, slot, live.numel(), most)
    dy = _pad(s["d_y"], order, group, slot, live.numel(), most) * s["scale"][live][:, None, None]
    v = torch.bmm(dy, b)
    d_x = s["d_y"].float() @ s["weight"].float().T
    d_x[order] += torch.bmm(v, a.transpose(1, 2))[group, slot]
    d_a, d_b = torch.zeros_like(s["a"]), torch.zeros_like(s["b"])
    d_a[live] = torch.bmm(x.transpose(1, 2), v).to(dt)
    d_b[live] = torch.bmm(dy.transpose(1, 2), torch.bmm(x, a)).to(dt)
    return dict(d_x=d_x.to(dt), d_a=d_a, d_b=d_b)


# ---------------------------------------------------------------- the framework's calls

def _own_route(s):
    import permute_grouped_gemm_gb300 as pgg
    c = s["case"]
    probs, experts, idx, groups, _ = pgg.route(
        s["logits"], c["top_k"], c["row_idx_type"], bias=s["bias"], score=c["score"],
        renormalize=c["renormalize"])
    return dict(probs=probs, experts=experts, idx=idx, groups=groups)


def _own_route_grad(s):
    import permute_grouped_gemm_gb300 as pgg
    c = s["case"]
    return pgg.route_grad(s["d_probs"], s["logits"], s["experts"], score=c["score"],
                          renormalize=c["renormalize"])


def _own_swiglu(s):
    import permute_grouped_gemm_gb300 as pgg
    c = s["case"]
    h, gate_up, _ = pgg.swiglu(s["x"], s["weight"], s["idx"], s["groups"], c["tokens"], c["top_k"],
                               c["row_idx_type"], probs=s["probs"], keep=c["keep"])
    return dict(h=h, gate_up=gate_up) if c["keep"] else dict(h=h)


def _own_swiglu_grad(s):
    import permute_grouped_gemm_gb300 as pgg
    c = s["case"]
    d_gate_up, d_probs, h, _ = pgg.swiglu_grad(s["d_h"], s["gate_up"], s["idx"], c["top_k"],
                                               c["row_idx_type"], probs=s["probs"])
    got = dict(d_gate_up=d_gate_up, h=h)
    return dict(got, d_probs=d_probs) if s["probs"] is not None else got


def _own_adapters(s):
    import permute_grouped_gemm_gb300 as pgg
    y, _ = pgg.adapters(s["x"], s["weight"], s["a"], s["b"], s["adapter"], scale=s["scale"])
    return y


def _own_adapters_grad(s):
    import permute_grouped_gemm_gb300 as pgg
    d_x, d_a, d_b, _ = pgg.adapters_grad(s["d_y"], s["x"], s["weight"], s["a"], s["b"],
                                         s["adapter"], scale=s["scale"])
    return dict(d_x=d_x, d_a=d_a, d_b=d_b)


_PLAIN = dict(route=_plain_route, route_grad=_plain_route_grad, swiglu=_plain_swiglu,
              swiglu_grad=_plain_swiglu_grad, adapters=_plain_adapters,
              adapters_grad=_plain_adapters_grad)
_OWN = dict(route=_own_route, route_grad=_own_route_grad, swiglu=_own_swiglu,
            swiglu_grad=_own_swiglu_grad, adapters=_own_adapters,
            adapters_grad=_own_adapters_grad)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

def _live(draws, among):
    """Expected number of distinct values among `draws` even draws of `among`."""
    return among * (1 - (1 - 1 / among) ** draws)


def work(case):
    op, t = case["op"], case["tokens"]
    es = 4 if case["dtype"] == "fp32" else 2
    if op in ("route", "route_grad"):
        e, m = case["experts"], t * case["top_k"]
        if op == "route":
            return dict(bytes=t * e * es + (4 * e if case["bias"] else 0) + m * 20 + 8 * e,
                        flops=6 * t * e)
        # what is not chosen has no gradient when the weights are renormalised or sigmoids
        read = t * e if case["score"] == "softmax" and not case["renormalize"] else m
        return dict(bytes=(read + t * e) * es + m * 12, flops=8 * t * e)
    if op == "swiglu":
        m, k, f, e = t * case["top_k"], case["hidden"], case["inner"], case["experts"]
        live = e * (1 - (1 - case["top_k"] / e) ** t)
        return dict(bytes=(t * k + live * k * 2 * f + m * f * (3 if case["keep"] else 1)) * es
                    + 8 * m + 8 * e + (4 * m if case["weighted"] else 0),
                    flops=2 * m * k * 2 * f + 6 * m * f)
    if op == "swiglu_grad":
        m, f = t * case["top_k"], case["inner"]
        return dict(bytes=6 * m * f * es + 8 * m + (8 * m if case["weighted"] else 0),
                    flops=16 * m * f)
    k, n, r = case["hidden"], case["out"], case["rank"]
    live = _live(t, case["adapters"]) if case["spread"] == "mixed" else min(t, case["adapters"])
    if op == "adapters":
        return dict(bytes=(t * (k + n) + k * n + live * r * (k + n)) * es + 8 * t + 4 * live,
                    flops=2 * t * k * n + 2 * t * r * (k + n))
    return dict(bytes=(t * (2 * k + n) + k * n + (live + case["adapters"]) * r * (k + n)) * es
                + 8 * t + 4 * live, flops=2 * t * k * n + 6 * t * r * (k + n))


# ---------------------------------------------------------------- exact values

def _exact_score(logits, kind):
    return torch.softmax(logits, 1) if kind == "softmax" else torch.sigmoid(logits)


def _exact_route(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    # the order of choice is that of the 32-bit sums logit + bias, lowest index first among equals
    key = s["logits"].float()
    key = (key + s["bias"] if c["bias"] else key).double().cpu()
    chosen = torch.argsort(-key, dim=1, stable=True)[:, :k]
    p = torch.gather(_exact_score(s["logits"].double().cpu(), c["score"]), 1, chosen)
    if c["renormalize"]:
        p = p / p.sum(1, keepdim=True)
    flat = chosen.reshape(-1)
    by_expert = torch.argsort(flat * (t * k) + torch.arange(t * k))
    idx = by_expert if c["row_idx_type"] == 0 else torch.argsort(by_expert)
    return dict(probs=p, experts=chosen, idx=idx, groups=torch.bincount(flat, minlength=e))


def _exact_route_grad(s):
    """The gradient by its definition: sum over the chosen of d_prob times the Jacobian."""
    c = s["case"]
    with torch.enable_grad():
        z = s["logits"].double().requires_grad_()
        p = _exact_score(z, c["score"]).gather(1, s["experts"])
        if c["renormalize"]:
            p = p / p.sum(1, keepdim=True)
        return torch.autograd.grad((p * s["d_probs"].double()).sum(), z)[0]


def _exact_rows(s):
    """(token, position) of every expanded row, on the host."""
    idx = s["idx"].cpu()
    pos = idx if s["case"]["row_idx_type"] == 0 else torch.argsort(idx)
    return pos // s["case"]["top_k"], pos


def _exact_swiglu(s):
    f = s["case"]["inner"]
    token, pos = _exact_rows(s)
    parts, at = [], 0
    for g, n in enumerate(s["groups"].tolist()):
        if n:
            rows = s["x"][token[at:at + n].cuda()].double()
            parts.append(rows @ s["weight"][g].double())
            at += n
    gu = torch.cat(parts)
    h = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
    if s["probs"] is not None:
        h *= s["probs"].double().reshape(-1)[pos.cuda()][:, None]
    return dict(h=h, gate_up=gu) if s["case"]["keep"] else dict(h=h)


def _exact_swiglu_grad(s):
    f, parts = s["case"]["inner"], []
    _, pos = _exact_rows(s)
    d_probs = None if s["probs"] is None else torch.zeros(pos.numel(), dtype=torch.double,
                                                          device="cuda")
    step = 16384
    for i in range(0, pos.numel(), step):  # slices of rows: 64 bits of everything are large
        at = pos[i:i + step].cuda()
        with torch.enable_grad():
            gu = s["gate_up"][i:i + step].double().requires_grad_()
            p = (torch.ones(at.numel(), dtype=torch.double, device="cuda") if s["probs"] is None
                 else s["probs"].double().reshape(-1)[at]).requires_grad_()
            h = p[:, None] * torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
            d = torch.autograd.grad((h * s["d_h"][i:i + step].double()).sum(), (gu, p))
        parts.append((d[0], h.detach()))
        if d_probs is not None:
            d_probs[at] = d[1]
    got = dict(d_gate_up=torch.cat([d for d, _ in parts]), h=torch.cat([h for _, h in parts]))
    if d_probs is not None:
        got["d_probs"] = d_probs.reshape(s["probs"].shape)
    return got


def _exact_adapters(s, grad=False):
    x, w = s["x"].double(), s["weight"].double()
    dy = s["d_y"].double() if grad else None
    y = dy @ w.T if grad else x @ w
    d_a, d_b = torch.zeros_like(s["a"], dtype=torch.double), torch.zeros_like(s["b"], dtype=torch.double)
    for i in range(s["case"]["adapters"]):
        rows = (s["adapter"] == i).nonzero().reshape(-1)
        if rows.numel() == 0:
            continue
        a, b, scale = s["a"][i].double(), s["b"][i].double(), s["scale"][i].double()
        u = x[rows] @ a
        if not grad:
            y[rows] += scale * (u @ b.T)
            continue
        v = dy[rows] @ b
        y[rows] += scale * (v @ a.T)
        d_a[i] = scale * (x[rows].T @ v)
        d_b[i] = scale * (dy[rows].T @ u)
    return dict(d_x=y, d_a=d_a, d_b=d_b) if grad else y


_EXACT = dict(route=_exact_route, route_grad=_exact_route_grad, swiglu=_exact_swiglu,
              swiglu_grad=_exact_swiglu_grad, adapters=_exact_adapters,
              adapters_grad=lambda s: _exact_adapters(s, True))


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
