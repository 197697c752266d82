"""Cases of the decode step's operators around the block-format products, with plain forms and exact values.

Three operators:

* ``add_rmsnorm``: the residual's addition and the root-mean-square norm that stand before every product.
  It reads a product's output x and the residual stream r and gives
  h = x + r (stored in the stream's type), y = h / sqrt(mean(h^2) + eps) * weight as float16 or bfloat16 and,
  where asked for, y in 8 bits (e4m3) with one float32 scale = max|y| / 448 per group of a row.
* ``moe``: a whole mixture-of-experts layer for a few tokens: the router's product, its top choices, and the
  chosen experts' gated MLPs, whose weights are packed ROCmFP4 blocks.
* ``logprobs``: from a head's logits, the log probability of a given token per row, the entropy of the row
  and its most probable tokens (ties go to the lowest index).

``own`` selects who computes: false, elementary torch operations in 32 bits; true, this repository's entry points.
"""
import math

import torch

own = False

FP8_MAX = 448.0
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "": 0}
ROUTES = ("softmax", "softmax_topk", "sigmoid")
CODES = (0, 1, 2, 3, 4, 6, 8, 10, 0, -1, -2, -3, -4, -6, -8, -10)


def listed():
    def norm(name, rows, d, x, res, y, group, pad=0):
        return {"name": name, "op": "add_rmsnorm", "rows": rows, "d": d, "x": x, "residual": res, "y": y, "group": group, "pad": pad}

    def moe(name, m, e, k, d, i, layout, act, route):
        return {"name": name, "op": "moe", "m": m, "experts": e, "top_k": k, "d": d, "i": i, "layout": layout, "act": act, "route": route}

    def lp(name, rows, v, t, n, masked, scale=1.0):
        return {"name": name, "op": "logprobs", "rows": rows, "v": v, "type": t, "top_n": n, "masked": masked, "scale": scale}

    return [
        # one token between two products of a decode step
        norm("norm decode 1x5120", 1, 5120, "f32", "bf16", "f16", 0),
        # a few ragged sequences, an odd width, strided rows, and an 8-bit output for a product that takes one
        norm("norm ragged 37x2049 q8", 37, 2049, "bf16", "f32", "bf16", 64, 7),
        # a prompt of 4096 tokens with an 8-bit output by groups of 128 only
        norm("norm prompt 4096x5120 q8", 4096, 5120, "bf16", "bf16", "", 128),
        # the longest prompt of the benchmark: products' float32 outputs into a bfloat16 stream
        norm("norm prompt 23552x5120", 23552, 5120, "f32", "bf16", "bf16", 0),
        # one token through many small experts, dual-scale
        moe("moe 1 token 128x768", 1, 128, 8, 2048, 768, "dual", "f16", "softmax_topk"),
        # eight sequences decoded together over the same experts
        moe("moe 8 tokens 128x768", 8, 128, 8, 2048, 768, "dual", "bf16", "softmax_topk"),
        # a wider layer in the single-scale layout, a short draft of tokens to verify
        moe("moe 4 tokens 64x1536 fast", 4, 64, 6, 5120, 1536, "fast", "f16", "sigmoid"),
        # sizes that are no multiple of a tile, more tokens than experts
        moe("moe 13 tokens 10x352 odd", 13, 10, 3, 1056, 352, "dual", "bf16", "softmax"),
        # the sampled token of one sequence from the head's float32 logits
        lp("logprobs 1x152064", 1, 152064, "f32", 5, 0.0),
        # eight sequences under a grammar that masks most tokens, at a temperature
        lp("logprobs 8x152064 masked", 8, 152064, "f32", 20, 0.9, 1.25),
        # a small vocabulary of odd size, half-precision logits with many ties, no alternatives asked for
        lp("logprobs 333x32001 f16", 333, 32001, "f16", 0, 0.0),
        # scoring a prompt
        lp("logprobs 1024x152064 bf16", 1024, 152064, "bf16", 8, 0.0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("add_rmsnorm", "moe", "logprobs"))
    if op == "add_rmsnorm":
        d = _log_uniform(rng, 64, 16384)
        if rng.random() < 0.6:
            d = (d + 31) // 32 * 32
        rows = _log_uniform(rng, 1, max(1, min(23552, 23552 * 5120 // d)))
        group = rng.choice((0, 0, 32, 64, 128, -1))
        y = rng.choice(("f16", "bf16", "")) if group else rng.choice(("f16", "bf16"))
        return {"op": op, "rows": rows, "d": d, "x": rng.choice(("f32", "f16", "bf16")), "residual": rng.choice(("", "f32", "f16", "bf16", "bf16")),
                "y": y, "group": group, "pad": rng.choice((0, 0, 1, 8))}
    if op == "moe":
        layout = rng.choice(("dual", "fast"))
        unit = rng.choice((32, 256, 512))
        d = max(unit, _log_uniform(rng, 128, 7168) // unit * unit)
        i = max(unit, _log_uniform(rng, 64, 2048) // unit * unit)
        e = _log_uniform(rng, 4, 256)
        while e * i * d > 1 << 28:
            e = max(4, e // 2)
            i = i if e > 4 else max(unit, i // 2 // unit * unit)
        k = rng.randint(1, min(8, e))
        m = _log_uniform(rng, 1, 32)
        m = max(1, min(m, int(2.4e8 / (k * i * d))))
        return {"op": op, "m": m, "experts": e, "top_k": k, "d": d, "i": i, "layout": layout, "act": rng.choice(("f16", "bf16")), "route": rng.choice(ROUTES)}
    v = _log_uniform(rng, 50, 200000)
    t = rng.choice(("f32", "f16", "bf16"))
    rows = _log_uniform(rng, 1, max(1, min(4096, 1024 * 152064 // v // (2 if t == "f32" else 1))))
    return {"op": op, "rows": rows, "v": v, "type": t, "top_n": rng.choice((0, 1, 5, 20, 32)), "masked": rng.choice((0.0, 0.0, 0.5, 0.95)),
            "scale": rng.choice((1.0, 1.0, 1.4285714626312256, 0.5))}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 40) + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _strided(t, dtype, pad):
    """t as rows of a wider buffer: a view whose rows are pad values apart beyond its width."""
    buf = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=dtype, device="cuda")
    view = buf[:, : t.shape[1]]
    view.copy_(t)
    return view


def _blocks(g, rows, k, layout):
    """Packed blocks of rows x k weights: uniform codes, scale bytes of the magnitude that trained weights have."""
    nb, bb = k // 32, 18 if layout == "dual" else 17
    w = torch.randint(0, 256, (rows, nb, bb), generator=g, device="cuda", dtype=torch.uint8)
    e = 1 + w[..., 16:] % 2
    m = (w[..., 16:] >> 4) & 7
    w[..., 16:] = e * 8 + m
    return w.view(rows * nb * bb)


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    if c["op"] == "add_rmsnorm":
        rows, d = c["rows"], c["d"]
        # products' outputs and a residual stream with a few large channels, as trained networks have them
        loud = torch.ones(d, device="cuda")
        loud[torch.randint(0, d, (max(1, d // 512),), generator=g, device="cuda")] = 20.0
        c["xt"] = _strided(_normal(g, rows, d) * 2.0, TYPES[c["x"]], c["pad"])
        c["rt"] = _strided(_normal(g, rows, d) * loud, TYPES[c["residual"]], c["pad"]) if c["residual"] else None
        c["wt"] = (1.0 + 0.2 * _normal(g, d)).to(torch.bfloat16)
        c["eps"] = 1e-6
        c["yt"] = torch.empty(rows, d, dtype=TYPES[c["y"]], device="cuda") if c["y"] else None
        c["ht"] = torch.empty(rows, d, dtype=TYPES[c["residual"]], device="cuda") if c["residual"] else None
        c["qt"] = c["st"] = None
        if c["group"]:
            size = d if c["group"] < 0 else c["group"]
            c["qt"] = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
            c["st"] = torch.empty(rows, -(-d // size), dtype=torch.float32, device="cuda")
    elif c["op"] == "moe":
        m, e, k, d, i = c["m"], c["experts"], c["top_k"], c["d"], c["i"]
        c["xt"] = _normal(g, m, d).to(TYPES[c["act"]])
        c["router"] = (_normal(g, e, d) * (2.0 / math.sqrt(d))).to(torch.bfloat16)
        c["wgu"] = _blocks(g, e * 2 * i, d, c["layout"])
        c["wd"] = _blocks(g, e * d, i, c["layout"])
        c["yt"] = torch.empty(m, d, dtype=torch.float32, device="cuda")
        c["ids"] = torch.empty(m, k, dtype=torch.int32, device="cuda")
        c["probs"] = torch.empty(m, k, dtype=torch.float32, device="cuda")
    else:
        rows, v, n = c["rows"], c["v"], min(c["top_n"], c["v"])
        z = torch.empty(rows, v, dtype=TYPES[c["type"]], device="cuda")
        # a head's logits: a wide bulk and, in each row, some tokens that stand out
        z.normal_(0.0, 2.5, generator=g)
        out = torch.randperm(v, generator=g, device="cuda")[:min(v, 40)] + 7 * torch.arange(rows, device="cuda")[:, None]
        out = out % v  # no token twice in a row
        z.scatter_add_(1, out, (_normal(g, rows, out.shape[1]).abs() * 5.0).to(z.dtype))
        if c["masked"]:
            keep = torch.rand(1, v, generator=g, device="cuda") >= c["masked"]
            keep[0, out[1:, 0]] = True  # the given tokens are legal ones, but perhaps the first row's
            z.masked_fill_(~keep, -math.inf)
            if rows >= 4:  # a row whose mask leaves nothing, and one masked with the type's lowest value
                z[1] = -math.inf
                z[2].clamp_(min=torch.finfo(z.dtype).min)
        c["zt"] = z
        c["targets"] = out[:, 0].to(torch.int32).contiguous()
        c["lp"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        c["ent"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        c["tid"] = torch.empty(rows, n, dtype=torch.int32, device="cuda")
        c["tlp"] = torch.empty(rows, n, dtype=torch.float32, device="cuda")
    return c


def run(state):
    return {"add_rmsnorm": _norm_own if own else _norm_plain, "moe": _moe_own if own else _moe_plain,
            "logprobs": _logprobs_own if own else _logprobs_plain}[state["op"]](state)


# ---- this repository's entry points ------------------------------------------------------------------------------------

def _norm_own(s):
    import gemm_rocmfp4_dequant_gb300 as rf4
    o = rf4.add_rmsnorm(s["xt"], s["wt"], residual=s["rt"], eps=s["eps"], y=s["yt"], residual_out=s["ht"], q=s["qt"], scales=s["st"],
                        group=s["group"])
    return {"y": o.y, "residual": o.residual, "q": o.q, "scales": o.scales}


def _moe_own(s):
    import gemm_rocmfp4_dequant_gb300 as rf4
    y, ids, probs = rf4.moe(s["xt"], s["router"], s["wgu"], s["wd"], s["i"], s["top_k"], rf4.DUAL if s["layout"] == "dual" else rf4.FAST,
                            ROUTES.index(s["route"]), Y=s["yt"], ids=s["ids"], probs=s["probs"])
    return {"y": y, "ids": ids, "probs": probs}


def _logprobs_own(s):
    import gemm_rocmfp4_dequant_gb300 as rf4
    lp, ent, ids, top = rf4.logprobs(s["zt"], s["targets"], top_n=s["tid"].shape[1], scale=s["scale"], logprob=s["lp"], entropy=s["ent"],
                                     top_ids=s["tid"], top_logprobs=s["tlp"])
    return {"logprob": lp, "entropy": ent, "top_ids": ids, "top_logprobs": top}


# ---- plain forms: elementary torch operations in 32 bits -----------------------------------------------------------------

def _norm_plain(s):
    h = s["xt"].float()
    if s["rt"] is not None:
        h = h + s["rt"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["wt"].float()
    got = {"y": None if s["yt"] is None else y.to(s["yt"].dtype), "residual": None if s["rt"] is None else h.to(s["rt"].dtype), "q": None, "scales": None}
    if s["group"]:
        rows, d = y.shape
        size = d if s["group"] < 0 else s["group"]
        n = -(-d // size)
        wide = torch.zeros(rows, n * size, dtype=torch.float32, device=y.device)
        wide[:, :d] = y
        wide = wide.view(rows, n, size)
        scale = wide.abs().amax(-1) / FP8_MAX
        q = torch.where(scale[..., None] > 0, wide / scale[..., None], torch.zeros_like(wide)).clamp(-FP8_MAX, FP8_MAX)
        got["q"] = q.view(rows, n * size)[:, :d].contiguous().to(torch.float8_e4m3fn)
        got["scales"] = scale
    return got


def _decode_plain(w, layout):
    """Blocks (..., blocks, 17 or 18 bytes) to float32 weights (..., blocks * 32)."""
    qs = w[..., :16]
    codes = torch.cat((qs & 15, qs >> 4), -1)
    table = torch.tensor(CODES, dtype=torch.float32, device=w.device)
    v = table[codes.int()]
    b = w[..., 16:].int()
    ex, mant = (b >> 3) & 15, (b & 7).float()
    scale = torch.where(ex > 0, (1.0 + mant / 8.0) * torch.exp2(ex.float() - 8.0), mant / 1024.0)
    scale = scale.repeat_interleave(16 if layout == "dual" else 32, -1)
    return (v * scale).flatten(-2)


def _moe_plain(s):
    m, e, k, d, i = s["m"], s["experts"], s["top_k"], s["d"], s["i"]
    bb = 18 if s["layout"] == "dual" else 17
    x = s["xt"].float()
    logits = x @ s["router"].float().T
    ranked, order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids, best = order[:, :k].contiguous(), ranked[:, :k]
    if s["route"] == "softmax":
        full = torch.exp(logits - ranked[:, :1])
        p = torch.exp(best - ranked[:, :1]) / full.sum(-1, keepdim=True)
    elif s["route"] == "softmax_topk":
        p = torch.exp(best - ranked[:, :1])
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-best))
        p = p / p.sum(-1, keepdim=True)
    gu = _decode_plain(s["wgu"].view(e, 2 * i, d // 32, bb)[ids], s["layout"])  # tokens, choices, 2i, d
    gu = (gu @ x[:, None, :, None]).squeeze(-1)
    gate, up = gu[..., :i], gu[..., i:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    wd = _decode_plain(s["wd"].view(e, d, i // 32, bb)[ids], s["layout"])
    out = (wd @ h[..., None]).squeeze(-1)
    return {"y": (out * p[..., None]).sum(1), "ids": ids.int(), "probs": p}


def _logprobs_plain(s):
    z = s["zt"].float()
    v, n = z.shape[1], s["tid"].shape[1]
    zs = z * s["scale"]
    top = zs.amax(-1, keepdim=True)
    empty = top == -math.inf
    top = torch.where(empty, torch.zeros_like(top), top)
    e = torch.exp(zs - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    minus = torch.full_like(zs[:, :1], -math.inf)
    lp = torch.where(empty, minus, zs.gather(1, s["targets"].long()[:, None]) - lse)
    ent = torch.log(total) - torch.where(e > 0, e * (zs - top), torch.zeros_like(e)).sum(-1, keepdim=True) / total
    ent = torch.where(empty, torch.zeros_like(ent), ent)
    ids = torch.sort(z, dim=-1, descending=True, stable=True)[1][:, :n].contiguous() if n else s["targets"].long()[:, None][:, :0]
    tlp = torch.where(empty, minus, zs.gather(1, ids) - lse)
    return {"logprob": lp[:, 0], "entropy": ent[:, 0], "top_ids": ids.int(), "top_logprobs": tlp}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "add_rmsnorm":
        n = c["rows"] * c["d"]
        groups = 0 if not c["group"] else 1 if c["group"] < 0 else -(-c["d"] // c["group"])
        per = SIZE[c["x"]] + 2 * SIZE[c["residual"]] + SIZE[c["y"]] + (1 if c["group"] else 0)
        return {"bytes": n * per + 2 * c["d"] + 4 * groups * c["rows"], "flops": 6 * n}
    if c["op"] == "moe":
        m, e, k, d, i = c["m"], c["experts"], c["top_k"], c["d"], c["i"]
        reached = e * (1.0 - (1.0 - k / e) ** m)  # experts that some token chooses, where the router spreads them evenly
        blocks = 3 * i * d // 32 * (18 if c["layout"] == "dual" else 17)
        return {"bytes": reached * blocks + 2 * e * d + 6 * m * d + 8 * m * k, "flops": 2 * m * d * (e + 3 * k * i)}
    n = c["rows"] * c["v"]
    return {"bytes": n * SIZE[c["type"]] + c["rows"] * (12 + 8 * min(c["top_n"], c["v"])), "flops": 6 * n}


# ---- exact values, from the definitions in 64 bits -------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"add_rmsnorm": _norm_exact, "moe": _moe_exact, "logprobs": _logprobs_exact}[s["op"]](s)


def _to_e4m3(t):
    """The nearest e4m3 value, ties to even mantissas, of |t| <= 448."""
    a = t.abs()
    _, ex = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), torch.clamp(ex - 1, min=-6) - 3)
    return torch.sign(t) * torch.round(a / step) * step


def _norm_exact(s):
    y, h, q, sc = [], [], [], []
    w = s["wt"].double()
    for a in range(0, s["rows"], 2048):
        v = s["xt"][a:a + 2048].double()
        if s["rt"] is not None:
            v += s["rt"][a:a + 2048].double()
            h.append(v.clone())
        v /= torch.sqrt(torch.einsum("rd,rd->r", v, v)[:, None] / s["d"] + s["eps"])
        v *= w
        if s["yt"] is not None:
            y.append(v)
        if s["group"]:
            parts = [v] if s["group"] < 0 else list(v.split(s["group"], dim=1))
            amax = [p.abs().max(dim=1).values / FP8_MAX for p in parts]
            q.append(torch.cat([_to_e4m3(p / t.clamp(min=1e-300)[:, None]) for p, t in zip(parts, amax)], 1))
            sc.append(torch.stack(amax, 1))
    whole = lambda p: torch.cat(p) if p else None  # noqa: E731
    return {"y": whole(y), "residual": whole(h), "q": whole(q), "scales": whole(sc)}


def _expert_exact(w, rows, k, layout):
    """One matrix of packed blocks in 64 bits."""
    bb = 18 if layout == "dual" else 17
    w = w.view(rows, k // 32, bb).long()
    sign = lambda q: torch.where(q >= 8, -1.0, 1.0).double()  # noqa: E731
    size = lambda q: torch.where(q % 8 <= 4, q % 8, 2 * (q % 8) - 4).double()  # noqa: E731
    out = torch.empty(rows, k // 32, 32, dtype=torch.float64, device=w.device)
    for half in (0, 1):
        q = (w[..., :16] // (16 if half else 1)) % 16
        e = w[..., 16 + (half if layout == "dual" else 0)]
        field, mant = e // 8 % 16, e % 8
        hs = torch.where(field > 0, torch.ldexp((8 + mant).double(), field - 11), torch.ldexp(mant.double(), torch.full_like(field, -10)))
        out[..., 16 * half:16 * half + 16] = sign(q) * size(q) * hs[..., None]
    return out.view(rows, k)


def _moe_exact(s):
    m, e, k, d, i = s["m"], s["experts"], s["top_k"], s["d"], s["i"]
    x = s["xt"].double()
    logits = torch.einsum("md,ed->me", x, s["router"].double())
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    chosen = torch.gather(logits, 1, ids)
    if s["route"] == "softmax":
        p = torch.exp(chosen - torch.logsumexp(logits, 1, keepdim=True))
    elif s["route"] == "softmax_topk":
        p = torch.exp(chosen - torch.logsumexp(chosen, 1, keepdim=True))
    else:
        p = torch.sigmoid(chosen)
        p = p / p.sum(1, keepdim=True)
    wgu, wd = s["wgu"].view(e, -1), s["wd"].view(e, -1)
    y = torch.zeros(m, d, dtype=torch.float64, device=x.device)
    for expert in torch.unique(ids).tolist():
        token, place = torch.nonzero(ids == expert, as_tuple=True)
        both = x[token] @ _expert_exact(wgu[expert], 2 * i, d, s["layout"]).T
        h = both[:, :i] * torch.sigmoid(both[:, :i]) * both[:, i:]
        y.index_add_(0, token, p[token, place][:, None] * (h @ _expert_exact(wd[expert], d, i, s["layout"]).T))
    return {"y": y, "ids": ids.int(), "probs": p}


def _logprobs_exact(s):
    n, parts = s["tid"].shape[1], []
    for a in range(0, s["rows"], 128):
        raw = s["zt"][a:a + 128].double()
        z = raw * float(s["scale"])
        z = torch.where(z < -torch.finfo(torch.float32).max, -math.inf, z)  # below the least float32
        lse = torch.logsumexp(z, 1, keepdim=True)
        none = torch.isinf(lse) & (lse < 0)
        logp = torch.where(none, lse, z - lse)
        p = torch.exp(logp)
        ent = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
        order = torch.argsort(raw, dim=1, descending=True, stable=True)[:, :n]
        parts.append((logp.gather(1, s["targets"][a:a + 128].long()[:, None])[:, 0], ent, order.int(), logp.gather(1, order)))
    lp, ent, ids, top = (torch.cat(p) for p in zip(*parts))
    return {"logprob": lp, "entropy": ent, "top_ids": ids, "top_logprobs": top}
