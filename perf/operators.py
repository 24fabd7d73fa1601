"""The decode-side MoE operators at the sizes they are used at: the router, products with
4-bit weights, and a whole MoE layer for a few tokens.

  route        router scores [n, E] to top-k expert ids and weights (the inputs of ep_layout
               and ep_combine), and the gradient of the scores
  w4_linear    y[n, N] = x[n, K] . W^T with 4-bit weights and one fp32 scale per group of a row
  moe_layer    x and router scores to the MoE layer's output: top-k, each chosen expert's gated
               product, its down product, and the weighted sum back to the tokens; expert
               weights in bf16 or in the 4-bit form

Each case is a dict; `prepare` makes its inputs from a seed, `run` is one pass: in the plain
form (elementary torch operations in fp32, rounded once at the end) or, with `own` set, through
the package's entry points.  `exact` computes the same in 64 bits.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a 64-expert decode step: nothing but latency
        dict(name="route_one", op="route", n=1, experts=64, topk=8, dtype="fp32",
             score="softmax", renorm=True, scale=1.0, masked=0.0, grad=False),
        # a prefill batch of 8 x 4096 tokens over 256 experts
        dict(name="route_prefill", op="route", n=32768, experts=256, topk=8, dtype="fp32",
             score="softmax", renorm=True, scale=1.0, masked=0.0, grad=False),
        # a training step's router: sigmoid scores, bf16 logits, forward and gradient
        dict(name="route_train_sigmoid", op="route", n=16384, experts=128, topk=6, dtype="bf16",
             score="sigmoid", renorm=True, scale=2.5, masked=0.0, grad=True),
        # odd sizes, some experts masked out for some tokens, weights not renormalised (the
        # gradient then reaches every expert)
        dict(name="route_train_masked", op="route", n=8191, experts=250, topk=7, dtype="fp32",
             score="softmax", renorm=False, scale=1.0, masked=0.3, grad=True),
        # the smallest projection, one token
        dict(name="w4_small", op="w4", n=1, rows=1024, cols=1024, group=32, out="bf16"),
        # a square projection of a hidden size of 7168, one token
        dict(name="w4_decode", op="w4", n=1, rows=7168, cols=7168, group=128, out="bf16"),
        # an odd number of sequences and of output rows (a vocabulary's slice)
        dict(name="w4_odd", op="w4", n=13, rows=20011, cols=4096, group=64, out="bf16"),
        # a long contraction for a decode batch of 32
        dict(name="w4_batch", op="w4", n=32, rows=4096, cols=14336, group=128, out="bf16"),
        # a small layer, four tokens
        dict(name="moe_tiny", op="moe", n=4, hidden=1024, inter=512, experts=32, topk=4,
             weights="bf16", group=0, score="softmax", renorm=True),
        # one token of the 64-expert decode configuration: eight experts' weights are read
        dict(name="moe_one", op="moe", n=1, hidden=7168, inter=2048, experts=64, topk=8,
             weights="bf16", group=0, score="softmax", renorm=True),
        # eight tokens, 4-bit experts, an odd number of channel tiles
        dict(name="moe_w4", op="moe", n=8, hidden=4096, inter=1408, experts=128, topk=6,
             weights="int4", group=128, score="sigmoid", renorm=True),
        # a full decode batch: every expert is active, several tokens on each
        dict(name="moe_batch", op="moe", n=64, hidden=7168, inter=2048, experts=64, topk=8,
             weights="bf16", group=0, score="softmax", renorm=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "w4", "moe"])
    if op == "route":
        e = _log_int(rng, 8, 512)
        return dict(op="route", n=_log_int(rng, 1, 32768), experts=e,
                    topk=rng.randint(1, min(e, 16)), dtype=rng.choice(["fp32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.2, 0.9]),
                    grad=rng.random() < 0.5)
    if op == "w4":
        g = rng.choice([32, 64, 128])
        return dict(op="w4", n=_log_int(rng, 1, 64), rows=_log_int(rng, 257, 20011),
                    cols=g * _log_int(rng, max(1, 512 // g), 14336 // g), group=g,
                    out=rng.choice(["bf16", "bf16", "fp32"]))
    w = rng.choice(["bf16", "int4"])
    g = rng.choice([32, 64, 128]) if w == "int4" else 0
    step = g if g else 8
    e = rng.choice([8, 16, 32, 60, 64, 128])
    h = step * _log_int(rng, max(1, 512 // step), 7168 // step)
    # at most a billion and a half expert parameters in all
    i = step * _log_int(rng, max(1, 128 // step), max(1, min(8192, (3 << 29) // (3 * e * h)) // step))
    return dict(op="moe", n=_log_int(rng, 1, 64), hidden=h, inter=i, experts=e,
                topk=rng.randint(1, min(8, e)), weights=w, group=g,
                score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7)


# ---------------------------------------------------------------- inputs

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _normal(shape, g, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _int4(lead, rows, cols, group, g):
    """Packed 4-bit weights uint8 [..., rows, cols / 2] (low nibble: the even column; value
    nibble - 8) and their scales fp32 [..., rows, cols / group]; the products have unit size."""
    q = torch.randint(0, 256, (*lead, rows, cols // 2), dtype=torch.uint8, device="cuda",
                      generator=g)
    s = torch.rand((*lead, rows, cols // group), device="cuda", generator=g) + 0.5
    return q, s * (1.0 / (4.6 * math.sqrt(cols)))


def _inputs(c, seed):
    g = _gen(seed)
    if c["op"] == "route":
        n, e, k = c["n"], c["experts"], c["topk"]
        # router scores: N(0, 1) per token plus a popularity of each expert
        logits = _normal((n, e), g, torch.float32) + 0.5 * _normal((1, e), g, torch.float32)
        if c["masked"] > 0:
            m = torch.rand((n, e), device="cuda", generator=g) < c["masked"]
            logits = logits.masked_fill(m, -math.inf)
        s = dict(logits=logits.to(_DT[c["dtype"]]))
        if c["grad"]:
            s["grad_weights"] = _normal((n, k), g, torch.float32)
        return s
    if c["op"] == "w4":
        x = _normal((c["n"], c["cols"]), g, torch.bfloat16)
        q, s = _int4((), c["rows"], c["cols"], c["group"], g)
        return dict(x=x, q=q, scales=s)
    n, h, i, e = c["n"], c["hidden"], c["inter"], c["experts"]
    s = dict(x=_normal((n, h), g, torch.bfloat16), logits=_normal((n, e), g, torch.float32))
    if c["weights"] == "int4":
        s["w13"], s["w13_scales"] = _int4((e,), 2 * i, h, c["group"], g)
        s["w2"], s["w2_scales"] = _int4((e,), h, i, c["group"], g)
    else:
        s["w13"] = _normal((e, 2 * i, h), g, torch.bfloat16, h ** -0.5)
        s["w2"] = _normal((e, h, i), g, torch.bfloat16, i ** -0.5)
        s["w13_scales"] = s["w2_scales"] = None
    return s


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if not own:
        return s
    import combine_ep_layout_gb300 as ep
    c, dev = case, "cuda"
    if c["op"] == "w4":
        s["out"] = torch.empty((c["n"], c["rows"]), dtype=_DT[c["out"]], device=dev)
        return s
    n, e, k = c["n"], c["experts"], c["topk"]
    s["topk_idx"] = torch.empty((n, k), dtype=torch.int64, device=dev)
    s["topk_weights"] = torch.empty((n, k), dtype=torch.float32, device=dev)
    s["route_cfg"] = ep.make_route_cfg(e, k, c["score"], c["renorm"], c.get("scale", 1.0))
    if c["op"] == "route":
        if c["grad"]:
            s["grad_logits"] = torch.empty_like(s["logits"])
        return s
    s["moe"] = ep.EpMoe(ep.make_moe_cfg(c["hidden"], c["inter"], e, k, max_tokens=n,
                                        weight_dtype=c["weights"], group_size=c["group"]))
    s["weights"] = ep.EpMoeWeights(s["w13"], s["w2"], s["w13_scales"], s["w2_scales"])
    s["out"] = torch.empty((n, c["hidden"]), dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(s):
    import combine_ep_layout_gb300 as ep
    op = s["case"]["op"]
    if op == "w4":
        ep.ep_w4_linear(s["x"], s["q"], s["scales"], s["out"])
        return dict(y=s["out"])
    if op == "route":
        ep.ep_route(s["route_cfg"], s["logits"], s["topk_idx"], s["topk_weights"])
        r = dict(topk_idx=s["topk_idx"], topk_weights=s["topk_weights"])
        if s["case"]["grad"]:
            ep.ep_route_backward(s["route_cfg"], s["logits"], s["topk_idx"], s["grad_weights"],
                                 s["grad_logits"])
            r["grad_logits"] = s["grad_logits"]
        return r
    s["moe"].layer(s["route_cfg"], s["x"], s["logits"], s["weights"], s["topk_idx"],
                   s["topk_weights"], s["out"])
    return dict(y=s["out"], topk_idx=s["topk_idx"], topk_weights=s["topk_weights"])


def _pick(c, logits):
    """The k largest scores of each row, ties to the lowest index; -1 where none is left.
    Returns ids, which of them count, and the chosen scores (0 in place of the others)."""
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :c["topk"]], idx[:, :c["topk"]]
    ok = top > -math.inf
    return torch.where(ok, idx, -1), ok, torch.where(ok, top, 0.0)


def _plain_route(s):
    c, logits = s["case"], s["logits"].float()
    scale = c.get("scale", 1.0)
    idx, ok, top = _pick(c, logits)
    if c["score"] == "softmax":
        peak = torch.where(ok[:, :1], top[:, :1], 0.0)
        e = torch.exp(logits - peak)
        whole = e.sum(1, keepdim=True)
        score = torch.where(ok, torch.exp(top - peak), 0.0)
        if not c["renorm"]:
            score = score / whole.clamp_min(1e-30)
    else:
        score = torch.where(ok, 1.0 / (1.0 + torch.exp(-top)), 0.0)
    sig = score
    if c["renorm"]:
        score = score / score.sum(1, keepdim=True).clamp_min(1e-30)
    r = dict(topk_idx=idx, topk_weights=score * scale)
    if c.get("grad"):
        g = torch.where(ok, s["grad_weights"], 0.0) * scale
        mean = (g * score).sum(1, keepdim=True)
        if c["score"] == "softmax":
            chosen = score * (g - mean) if c["renorm"] else score * g
        else:
            chosen = score * (g - mean if c["renorm"] else g) * (1.0 - sig)
        d = torch.zeros_like(logits) if c["renorm"] or c["score"] == "sigmoid" else \
            -mean * e / whole.clamp_min(1e-30)
        d = d.scatter_add(1, idx.clamp_min(0), torch.where(ok, chosen, 0.0))
        r["grad_logits"] = d.to(s["logits"].dtype)
    return r


def _plain_weights(q, scales, group):
    """fp32 weights of the packed 4-bit form."""
    if scales is None:
        return q.float()
    v = torch.stack((q & 15, q >> 4), dim=-1).to(torch.float32) - 8.0
    return (v.reshape(*scales.shape, group) * scales[..., None]).flatten(-2)


def _plain_w4(s):
    c = s["case"]
    w = _plain_weights(s["q"], s["scales"], c["group"])
    return dict(y=(s["x"].float() @ w.T).to(_DT[c["out"]]))


def _plain_moe(s):
    c, x = s["case"], s["x"].float()
    n, e, k, i = c["n"], c["experts"], c["topk"], c["inter"]
    r = _plain_route(s)
    idx, w = r["topk_idx"], r["topk_weights"]
    if n * k < e:    # the chosen experts' weights, gathered for every (token, choice)
        at = idx.flatten()
        part = lambda t: None if t is None else t[at]                            # noqa: E731
        a = x.repeat_interleave(k, 0)[:, None]
        share = w.reshape(n, k, 1)
    else:            # every expert on every token
        part = lambda t: t                                                       # noqa: E731
        a = x.expand(e, n, -1)
        share = torch.zeros((n, e), device=x.device).scatter_add(1, idx, w).T[..., None]
    h = a @ _plain_weights(part(s["w13"]), part(s["w13_scales"]), c["group"]).transpose(1, 2)
    gate, up = h[..., :i], h[..., i:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = h @ _plain_weights(part(s["w2"]), part(s["w2_scales"]), c["group"]).transpose(1, 2)
    y = (y.reshape(n, k, -1) * share).sum(1) if n * k < e else (y * share).sum(0)
    return dict(r, y=y.to(torch.bfloat16))


_PLAIN = {"route": _plain_route, "w4": _plain_w4, "moe": _plain_moe}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "route":
        b = 4 if c["dtype"] == "fp32" else 2
        n, e, k = c["n"], c["experts"], c["topk"]
        byts, flops = n * e * b + n * k * 12, 4 * n * e
        if c["grad"]:    # the scores in once, the gradient of the weights in, that of the scores out
            byts += n * e * b + n * k * 4
            flops += 3 * n * e
        return dict(bytes=byts, flops=flops)
    if c["op"] == "w4":
        n, r, k, g = c["n"], c["rows"], c["cols"], c["group"]
        return dict(bytes=r * k // 2 + r * (k // g) * 4 + n * k * 2 +
                    n * r * (2 if c["out"] == "bf16" else 4), flops=2 * n * r * k)
    n, h, i, e, k = c["n"], c["hidden"], c["inter"], c["experts"], c["topk"]
    per = 2.0 if c["weights"] == "bf16" else 0.5 + 4.0 / c["group"]
    active = e * (1.0 - (1.0 - k / e) ** n)      # distinct experts that n tokens choose, on average
    return dict(bytes=active * 3 * h * i * per + n * (4 * h + 4 * e + 12 * k),
                flops=n * k * 6 * h * i)


# ---------------------------------------------------------------- 64 bits

def _exact_route(c, s):
    z = s["logits"].double()
    n, e, k = c["n"], c["experts"], c["topk"]
    scale = c.get("scale", 1.0)
    order = torch.argsort(-z, dim=1, stable=True)[:, :k]
    member = torch.zeros((n, e), dtype=torch.bool, device=z.device).scatter_(1, order, True)
    member &= torch.isfinite(z)
    live = torch.isfinite(z)
    f = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
    f = torch.where(live, f, 0.0)
    v = f * member
    tot = v.sum(1, keepdim=True)
    p = v / torch.where(tot > 0, tot, 1.0) if c["renorm"] else v
    wts = scale * torch.gather(p, 1, order)
    ids = torch.where(torch.gather(member, 1, order), order, -1)
    r = dict(topk_idx=ids, topk_weights=wts)
    if c.get("grad"):
        gw = torch.zeros((n, e), dtype=torch.float64, device=z.device)
        gw.scatter_(1, order, s["grad_weights"].double())
        gw = scale * gw * member
        if c["renorm"]:                                       # through v / sum(v)
            gw = member * (gw - (gw * p).sum(1, keepdim=True)) / torch.where(tot > 0, tot, 1.0)
        if c["score"] == "softmax":
            d = f * (gw - (gw * f).sum(1, keepdim=True))
        else:
            d = gw * f * (1.0 - f)
        r["grad_logits"] = torch.where(live, d, 0.0)
    return r


def _exact_matrix(q, scales):
    if scales is None:
        return q.double()
    rows, half = q.shape
    w = torch.empty((rows, 2 * half), dtype=torch.float64, device=q.device)
    w[:, 0::2] = (q.int() % 16 - 8).double()
    w[:, 1::2] = (q.int() // 16 - 8).double()
    return w * scales.double().repeat_interleave(2 * half // scales.shape[1], 1)


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "w4":
        out = torch.empty((c["n"], c["rows"]), dtype=torch.float64, device="cuda")
        for r0 in range(0, c["rows"], 4096):
            w = _exact_matrix(s["q"][r0:r0 + 4096], s["scales"][r0:r0 + 4096])
            out[:, r0:r0 + 4096] = s["x"].double() @ w.T
        return dict(y=out)
    r = _exact_route(c, s)
    x = s["x"].double()
    y = torch.zeros((c["n"], c["hidden"]), dtype=torch.float64, device="cuda")
    one = lambda t, e: None if t is None else t[e]                               # noqa: E731
    for e in r["topk_idx"].unique().tolist():
        t, k = (r["topk_idx"] == e).nonzero(as_tuple=True)
        u = x[t] @ _exact_matrix(s["w13"][e], one(s["w13_scales"], e)).T
        gate, up = u[:, :c["inter"]], u[:, c["inter"]:]
        u = gate * torch.sigmoid(gate) * up
        u = u @ _exact_matrix(s["w2"][e], one(s["w2_scales"], e)).T
        y.index_add_(0, t, u * r["topk_weights"][t, k][:, None])
    return dict(r, y=y)
