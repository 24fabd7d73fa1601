"""The router's training losses and the 8-bit path around the experts, at the sizes they are used at.

  balance   the load-balance and z losses of the router's scores, with each expert's token count,
            and the gradient of the scores
  quantize  rows to int8 with one fp32 scale each; or straight to the receive rows of a routing
  linear    y[n, rows] = x . W^T, both int8, a scale for each token and each channel; plain or
            gated (gate rows, then up rows: act(gate) * up)
  experts   the same for the receive rows of a routing, each expert's rows with its own weights

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
        # a small batch's losses alone (a validation step): nothing but latency
        dict(name="balance_small", op="balance", n=64, experts=64, topk=8, score="softmax", dtype="fp32",
             sequences=1, ragged=False, masked=0.0, grad=False),
        # a training step of 8 sequences of 4096 tokens over 256 experts, with the gradient
        dict(name="balance_train", op="balance", n=32768, experts=256, topk=8, score="softmax", dtype="fp32",
             sequences=8, ragged=False, masked=0.0, grad=True),
        # packed documents of every length, empty ones too, sigmoid scores in bf16, some experts
        # masked and some tokens padding, tokens behind the last document
        dict(name="balance_packed", op="balance", n=8191, experts=250, topk=7, score="sigmoid", dtype="bf16",
             sequences=37, ragged=True, masked=0.2, grad=True),
        # an odd batch of fp32 activations
        dict(name="quantize_odd", op="quantize", n=1001, cols=14336, dtype="fp32", experts=0, topk=0, align=1,
             masked=0.0),
        # a batch of 4096 tokens to its 8 experts each
        dict(name="quantize_dispatch", op="quantize", n=4096, cols=7168, dtype="bf16", experts=256, topk=8,
             align=128, masked=0.0),
        # one token of a decode step
        dict(name="linear_one", op="linear", n=1, rows=7168, cols=7168, out="bf16", act=""),
        # an odd number of sequences and of output rows (a vocabulary's slice), fp32 scores
        dict(name="linear_odd", op="linear", n=45, rows=20011, cols=4096, out="fp32", act=""),
        # a gated projection of a short prompt
        dict(name="linear_gated", op="linear", n=333, rows=11008, cols=4096, out="bf16", act="silu"),
        # a prefill batch through a square projection
        dict(name="linear_prefill", op="linear", n=8192, rows=7168, cols=7168, out="bf16", act=""),
        # a decode batch: every expert's gate and up rows are read for a few tokens each
        dict(name="experts_decode", op="experts", n=64, experts=64, topk=8, align=16, rows=4096, cols=7168,
             out="bf16", act="silu", skew=0.5, masked=0.0),
        # the down product of a training batch's skewed routing, with padding tokens
        dict(name="experts_down", op="experts", n=4095, experts=60, topk=4, align=8, rows=2048, cols=1408,
             out="bf16", act="", skew=1.5, masked=0.1),
        # a prefill batch's gate and up products over 128 experts
        dict(name="experts_prefill", op="experts", n=8192, experts=128, topk=6, align=128, rows=2816, cols=4096,
             out="bf16", act="silu", skew=0.5, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "quantize", "linear", "experts"])
    if op == "balance":
        n, e = _log_int(rng, 1, 32768), _log_int(rng, 8, 256)
        return dict(op=op, n=n, experts=e, topk=rng.randint(1, min(e, 8)), score=rng.choice(["softmax", "sigmoid"]),
                    dtype=rng.choice(["fp32", "bf16"]), sequences=_log_int(rng, 1, max(1, min(64, n))),
                    ragged=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.2, 0.6]), grad=rng.random() < 0.7)
    if op == "quantize":
        cols = 16 * _log_int(rng, 16, 896)
        e = rng.choice([0, 16, 64, 250, 256])
        n = _log_int(rng, 1, 2048 if e else 8192)
        return dict(op=op, n=n, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp32"]), experts=e,
                    topk=rng.randint(1, 8) if e else 0, align=rng.choice([1, 8, 16, 128]) if e else 1,
                    masked=rng.choice([0.0, 0.3]) if e else 0.0)
    act = rng.choice(["", "silu", "gelu_tanh"])
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "linear":
        cols = 16 * _log_int(rng, 16, 896)
        rows = 2 * _log_int(rng, 129, 10005) - (0 if act else rng.randint(0, 1))
        n = _log_int(rng, 1, max(1, min(8192, (7168 * 7168 * 8192) // (rows * cols))))
        return dict(op=op, n=n, rows=rows, cols=cols, out=out, act=act)
    e = rng.choice([8, 16, 32, 60, 64, 128])
    cols = 16 * _log_int(rng, 32, 448)
    # at most 1.8 G expert parameters
    rows = 2 * _log_int(rng, 128, max(128, min(4096, (9 << 27) // (e * cols)) // 2))
    k = rng.randint(1, min(8, e))
    n = _log_int(rng, 1, max(1, min(8192, (8192 * 6 * 2816 * 4096) // (rows * cols * k))))
    return dict(op=op, n=n, experts=e, topk=k, align=rng.choice([1, 8, 16, 128]), rows=rows, cols=cols, out=out,
                act=act, skew=rng.choice([0.0, 0.5, 1.5]), masked=rng.choice([0.0, 0.0, 0.3]))


# ---------------------------------------------------------------- inputs

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _normal(shape, g, dtype=torch.float32, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _int8(shape, g):
    """Rows of a quantised normal distribution: the largest of a row is about 4 deviations."""
    return _normal(shape, g, torch.bfloat16, 31.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, g, size):
    return (torch.rand(shape, device="cuda", generator=g) + 0.5) * (size / 31.0)


def _routing(c, g):
    """topk_idx int64 [n, K] of distinct experts, some of them -1, by scores with popular experts."""
    n, e, k = c["n"], c["experts"], c["topk"]
    z = _normal((n, e), g) + c.get("skew", 0.5) * _normal((1, e), g)
    idx = torch.topk(z, k, dim=1).indices
    if c["masked"] > 0:
        idx = idx.masked_fill(torch.rand((n, 1), device="cuda", generator=g) < c["masked"], -1)
    return idx


def _plan(c, idx):
    """The expand layout of a routing: each (token, choice)'s receive row (-1: none), each expert's
    first row and count, and the number of receive rows that any routing fits in."""
    e, a = c["experts"], c["align"]
    flat = idx.flatten()
    count = torch.bincount(flat[flat >= 0], minlength=e)
    start = torch.cumsum((count + a - 1) // a * a, 0) - (count + a - 1) // a * a
    order = torch.argsort(torch.where(flat >= 0, flat, e), stable=True)
    first = torch.cumsum(count, 0) - count
    of = flat[order].clamp_min(0)
    rank = torch.arange(flat.numel(), device=flat.device) - first[of]
    slot = torch.empty_like(flat)
    slot[order] = torch.where(flat[order] >= 0, start[of] + rank, -1)
    w = _world(e)
    per = -(-c["n"] // w)
    return dict(slot=slot.view_as(idx), count=count, start=start, most=int(count.max()),
                capacity=w * per * c["topk"] + e * (a - 1), world=w, per=per)


def _world(e):
    return 8 if e % 8 == 0 else 1


def _inputs(c, seed):
    g = _gen(seed)
    if c["op"] == "balance":
        n, e, k, m = c["n"], c["experts"], c["topk"], c["sequences"]
        z = _normal((n, e), g) + 0.5 * _normal((1, e), g)
        if c["masked"] > 0:
            z = z.masked_fill(torch.rand((n, e), device="cuda", generator=g) < c["masked"], -math.inf)
        z = z.to(_DT[c["dtype"]])
        top, idx = torch.topk(z.float(), k, dim=1)
        idx = idx.masked_fill(top == -math.inf, -1)
        if c["masked"] > 0:      # padding tokens
            idx = idx.masked_fill(torch.rand((n, 1), device="cuda", generator=g) < 0.1, -1)
        if c["ragged"]:          # cuts anywhere, the last one before the end
            cuts = torch.sort(torch.randint(0, n + 1, (m,), device="cuda", generator=g)).values
            offsets = torch.cat([torch.zeros_like(cuts[:1]), cuts])
        else:
            offsets = torch.arange(m + 1, device="cuda") * n // m
        return dict(logits=z, topk_idx=idx, offsets=offsets.int(),
                    grad_loss=torch.rand(2, device="cuda", generator=g) * 0.01 + 0.001)
    if c["op"] == "quantize":
        x = _normal((c["n"], c["cols"]), g)
        # rows of different sizes, some channels far larger than the rest
        x = x * torch.exp(_normal((c["n"], 1), g)) * torch.exp(1.5 * _normal((1, c["cols"]), g))
        s = dict(x=x.to(_DT[c["dtype"]]))
        if c["experts"]:
            s["topk_idx"] = _routing(c, g)
            s["plan"] = _plan(c, s["topk_idx"])
        return s
    if c["op"] == "linear":
        return dict(x=_int8((c["n"], c["cols"]), g), x_scales=_scales((c["n"],), g, 1.0),
                    w=_int8((c["rows"], c["cols"]), g), w_scales=_scales((c["rows"],), g, c["cols"] ** -0.5))
    idx = _routing(c, g)
    plan = _plan(c, idx)
    e, cap = c["experts"], plan["capacity"]
    return dict(topk_idx=idx, plan=plan, x=_int8((cap, c["cols"]), g), x_scales=_scales((cap,), g, 1.0),
                w=_int8((e, c["rows"], c["cols"]), g),
                w_scales=_scales((e, c["rows"]), g, c["cols"] ** -0.5))


def prepare(case, seed):
    c, dev = case, "cuda"
    s = dict(_inputs(c, seed), case=c)
    if c["op"] == "balance":
        s["grad_logits"] = torch.zeros_like(s["logits"])      # rows outside every sequence stay as they are
    elif c["op"] == "quantize":
        rows = s["plan"]["capacity"] if c["experts"] else c["n"]
        s["q"] = torch.zeros((rows, c["cols"]), dtype=torch.int8, device=dev)
        s["scales"] = torch.zeros((rows,), dtype=torch.float32, device=dev)
    else:
        rows = c["n"] if c["op"] == "linear" else s["plan"]["capacity"]
        s["out"] = torch.zeros((rows, c["rows"] // 2 if c["act"] else c["rows"]), dtype=_DT[c["out"]], device=dev)
    if not own:
        return s
    import combine_ep_layout_gb300 as ep
    if c["op"] == "balance":
        m, e = c["sequences"], c["experts"]
        s["balance"] = ep.EpBalance(ep.make_route_cfg(e, c["topk"], c["score"]), max_tokens=c["n"], max_sequences=m)
        s["counts"] = torch.empty((m, e), dtype=torch.int32, device=dev)
        s["prob_sums"] = torch.empty((m, e), dtype=torch.float32, device=dev)
        s["tokens"] = torch.empty((m + 1,), dtype=torch.int32, device=dev)
        s["loss"] = torch.empty((2,), dtype=torch.float32, device=dev)
    elif c.get("experts"):
        p = s["plan"]
        s["handle"] = ep.EpHandle(ep.make_cfg(p["world"], c["cols"], p["per"], c["experts"] // p["world"], c["topk"],
                                              c["align"], "bf16", True))
        s["handle"].layout(s["topk_idx"])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(s):
    import combine_ep_layout_gb300 as ep
    c = s["case"]
    if c["op"] == "balance":
        b = s["balance"]
        b.forward(s["logits"], s["topk_idx"], s["counts"], s["prob_sums"], s["tokens"], s["loss"],
                  seq_offsets=s["offsets"])
        r = dict(counts=s["counts"], prob_sums=s["prob_sums"], tokens=s["tokens"], loss=s["loss"])
        if c["grad"]:
            b.backward(s["logits"], s["topk_idx"], s["counts"], s["tokens"], s["grad_loss"], s["grad_logits"],
                       seq_offsets=s["offsets"])
            r["grad_logits"] = s["grad_logits"]
        return r
    if c["op"] == "quantize":
        if c["experts"]:
            ep.ep_i8_dispatch(s["handle"], s["x"], s["q"], s["scales"])
        else:
            ep.ep_i8_quantize(s["x"], s["q"], s["scales"])
        return dict(q=s["q"], scales=s["scales"])
    if c["op"] == "linear":
        ep.ep_i8_linear(s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"], activation=c["act"] or None)
    else:
        ep.ep_i8_grouped(s["handle"], s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"],
                         activation=c["act"] or None)
    return dict(y=s["out"])


def _plain_balance(s):
    c, z, idx = s["case"], s["logits"].float(), s["topk_idx"]
    n, e, k, m = c["n"], c["experts"], c["topk"], c["sequences"]
    offsets = s["offsets"].long()
    of = torch.searchsorted(offsets, torch.arange(n, device=z.device), right=True) - 1    # the token's sequence
    inside = of < m
    of = of.clamp(0, m - 1)
    live = ((idx >= 0).any(1) & inside)[:, None]
    unmasked = z > -math.inf
    peak = z.amax(1, keepdim=True)
    peak = torch.where(peak > -math.inf, peak, 0.0)
    ez = torch.where(unmasked, torch.exp(z - peak), 0.0)
    whole = ez.sum(1, keepdim=True).clamp_min(1e-30)
    soft = ez / whole
    lse = torch.where(live, peak + torch.log(whole), 0.0)
    sig = torch.where(unmasked, 1.0 / (1.0 + torch.exp(-z)), 0.0)
    p = soft if c["score"] == "softmax" else sig / sig.sum(1, keepdim=True).clamp_min(1e-30)
    chosen = torch.zeros((n, e + 1), dtype=torch.int32, device=z.device)
    chosen = chosen.scatter_add(1, torch.where(idx >= 0, idx, e), torch.ones_like(idx, dtype=torch.int32))[:, :e]
    counts = torch.zeros((m, e), dtype=torch.int32, device=z.device).index_add(0, of, chosen * live.int())
    prob_sums = torch.zeros((m, e), device=z.device).index_add(0, of, torch.where(live, p, 0.0))
    tokens = torch.zeros((m,), dtype=torch.int32, device=z.device).index_add(0, of, live[:, 0].int())
    total = tokens.sum().float()
    t = tokens.float().clamp_min(1.0)[:, None]
    share = e / (k * m * t * t)
    loss = torch.stack([(counts * prob_sums * share).sum(), lse.square().sum() / total.clamp_min(1.0)])
    r = dict(counts=counts, prob_sums=prob_sums, tokens=torch.cat([tokens, tokens.sum()[None].int()]), loss=loss)
    if c["grad"]:
        mean = k * t / e                           # any constant may be taken from the counts: sum p = 1
        cnt = (counts.float() - mean)[of]
        d = p * (cnt - (cnt * p).sum(1, keepdim=True)) * share[of]
        if c["score"] == "sigmoid":
            d = d / (1.0 + torch.exp(z))           # 1 - s
        d = s["grad_loss"][0] * d + s["grad_loss"][1] * (2.0 / total.clamp_min(1.0)) * lse * soft
        r["grad_logits"] = torch.where(live & unmasked, d, 0.0).to(s["logits"].dtype)
    return r


def _plain_quantize(s):
    c, x = s["case"], s["x"].float()
    amax = x.abs().amax(1, keepdim=True)
    scales = amax / torch.full_like(amax, 127.0)
    q = torch.where(scales > 0, x / scales, 0.0).round().clamp(-127, 127).to(torch.int8)
    if not c["experts"]:
        return dict(q=q, scales=scales[:, 0])
    slot, rows = s["plan"]["slot"].flatten(), s["plan"]["capacity"]
    to = torch.where(slot >= 0, slot, rows)        # a row behind the last takes what has no place
    of = torch.arange(c["n"], device=x.device).repeat_interleave(c["topk"])
    out = torch.zeros((rows + 1, c["cols"]), dtype=torch.int8, device=x.device).index_copy(0, to, q[of])
    sc = torch.zeros((rows + 1,), device=x.device).index_copy(0, to, scales[of, 0])
    return dict(q=out[:rows], scales=sc[:rows])


def _act(name, v):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))


def _gated(c, y):
    if not c["act"]:
        return y
    half = c["rows"] // 2
    return _act(c["act"], y[..., :half]) * y[..., half:]


def _plain_linear(s):
    c = s["case"]
    y = (s["x"].float() @ s["w"].float().T) * s["w_scales"] * s["x_scales"][:, None]
    return dict(y=_gated(c, y).to(_DT[c["out"]]))


def _plain_experts(s):
    c, p = s["case"], s["plan"]
    # each expert's rows, padded to the most that one has
    at = torch.arange(p["most"], device=s["x"].device)
    row = p["start"][:, None] + at
    ok = at < p["count"][:, None]
    row = torch.where(ok, row, p["capacity"])
    src = row.clamp_max(p["capacity"] - 1)
    y = torch.bmm(s["x"][src].float(), s["w"].float().transpose(1, 2))
    y = _gated(c, y * s["w_scales"][:, None] * s["x_scales"][src][..., None]).to(_DT[c["out"]])
    out = torch.zeros((p["capacity"] + 1, y.shape[-1]), dtype=y.dtype, device=y.device)
    return dict(y=out.index_copy(0, row.flatten(), y.flatten(0, 1))[:-1])


_PLAIN = {"balance": _plain_balance, "quantize": _plain_quantize, "linear": _plain_linear,
          "experts": _plain_experts}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "balance":
        n, e, k, m = c["n"], c["experts"], c["topk"], c["sequences"]
        b = 4 if c["dtype"] == "fp32" else 2
        byts, flops = n * e * b + n * k * 8 + m * e * 8, 6 * n * e
        if c["grad"]:
            byts, flops = byts + n * e * b, flops + 8 * n * e
        return dict(bytes=byts, flops=flops)
    if c["op"] == "quantize":
        n, h = c["n"], c["cols"]
        to = n * c["topk"] * (1.0 - c["masked"]) if c["experts"] else n
        return dict(bytes=n * h * (2 if c["dtype"] == "bf16" else 4) + to * (h + 4), flops=3 * n * h)
    b = 2 if c["out"] == "bf16" else 4
    r, k = c["rows"], c["cols"]
    y = r // 2 if c["act"] else r
    if c["op"] == "linear":
        n = c["n"]
        return dict(bytes=r * k + 4 * r + n * (k + 4) + n * y * b, flops=2 * n * r * k)
    n, e = c["n"] * (1.0 - c["masked"]), c["experts"]
    active = e * (1.0 - (1.0 - c["topk"] / e) ** n)      # distinct experts that n tokens choose, on average
    rows = n * c["topk"]
    return dict(bytes=active * (r * k + 4 * r) + rows * (k + 4 + y * b), flops=2 * rows * r * k)


# ---------------------------------------------------------------- 64 bits

def _exact_balance(c, s):
    z, idx, o = s["logits"].double(), s["topk_idx"], s["offsets"].tolist()
    n, e, k, m = c["n"], c["experts"], c["topk"], c["sequences"]
    live = (idx >= 0).any(1)
    soft = torch.nan_to_num(torch.softmax(z, 1))
    lse = torch.where(live, torch.logsumexp(z, 1), 0.0)
    sig = torch.sigmoid(z)
    p = soft if c["score"] == "softmax" else torch.nan_to_num(sig / sig.sum(1, keepdim=True))
    counts = torch.zeros((m, e), dtype=torch.int32, device=z.device)
    sums = torch.zeros((m, e), dtype=torch.float64, device=z.device)
    tokens = torch.zeros((m + 1,), dtype=torch.int32, device=z.device)
    grad = torch.zeros_like(z)
    inside = torch.zeros_like(live)
    loss = torch.zeros((2,), dtype=torch.float64, device=z.device)
    gb, gz = s["grad_loss"].double()
    for i in range(m):
        a, b = o[i], o[i + 1]
        if b <= a:
            continue
        inside[a:b] = live[a:b]
        ids = idx[a:b].flatten()
        counts[i] = torch.bincount(ids[ids >= 0], minlength=e).int()
        lv = live[a:b, None].double()
        pp = p[a:b] * lv
        t = int(live[a:b].sum())
        sums[i], tokens[i] = pp.sum(0), t
        if t == 0:
            continue
        w = e / (k * m * t * t)
        cnt = counts[i].double()
        loss[0] += w * (cnt * sums[i]).sum()
        d = pp * (cnt - (cnt * pp).sum(1, keepdim=True))
        grad[a:b] = gb * w * (d if c["score"] == "softmax" else d * torch.sigmoid(-z[a:b]))
    total = max(1, int(inside.sum()))
    tokens[m] = int(inside.sum())
    lse = lse * inside
    loss[1] = lse.square().sum() / total
    grad += gz * (2.0 / total) * lse[:, None] * torch.where(inside[:, None], soft, 0.0)
    r = dict(counts=counts, prob_sums=sums, tokens=tokens, loss=loss)
    if c["grad"]:
        r["grad_logits"] = torch.where(z > -math.inf, grad, 0.0)
    return r


def _exact_quantize(c, s):
    sc = s["x"].double().abs().amax(1) / 127.0
    if c["experts"]:
        slot = s["plan"]["slot"]
        out = torch.zeros((s["plan"]["capacity"],), dtype=torch.float64, device=sc.device)
        for k in range(c["topk"]):
            t = (slot[:, k] >= 0).nonzero()[:, 0]
            out[slot[t, k]] = sc[t]
        sc = out
    return dict(q=None, scales=sc)       # whole numbers, equal or not


def _exact_product(c, x, xs, w, ws):
    y = (x.double() @ w.double().T) * ws.double() * xs.double()[:, None]
    if not c["act"]:
        return y
    gate, up = y.chunk(2, dim=1)
    if c["act"] == "silu":
        return gate * torch.sigmoid(gate) * up
    return torch.nn.functional.gelu(gate, approximate="tanh") * up


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "balance":
        return _exact_balance(c, s)
    if c["op"] == "quantize":
        return _exact_quantize(c, s)
    if c["op"] == "linear":
        return dict(y=_exact_product(c, s["x"], s["x_scales"], s["w"], s["w_scales"]))
    p = s["plan"]
    out = torch.zeros((p["capacity"], c["rows"] // 2 if c["act"] else c["rows"]), dtype=torch.float64, device="cuda")
    for e, (a, t) in enumerate(zip(p["start"].tolist(), p["count"].tolist())):
        out[a:a + t] = _exact_product(c, s["x"][a:a + t], s["x_scales"][a:a + t], s["w"][e], s["w_scales"][e])
    return dict(y=out)
