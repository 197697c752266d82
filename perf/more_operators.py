"""Cases of a paged ROCmFP4 K/V cache and the attention that reads it, with plain forms and exact values.

Four operators:

* ``rope_append``: takes the rows of a fused QKV product, turns the heads of q and k by their positions' angles, gives q
  as float16 or bfloat16 and packs k and v as ROCmFP4 blocks into the pages of their sequences;
* ``cache_read``: the pages' values of the last tokens of every sequence, as dense rows;
* ``paged_attention`` of a chunk of new tokens (one or many) of every sequence over its pages: causal, causal with a
  window, or over all of the tokens (a cross attention to an encoder's states);
* ``rotary``: the same turn of q alone, without a cache (a cross attention's or an uncached layer's queries).

A cache is ``pages`` x KV heads x ``page`` rows of D / 32 blocks.  Sequence b holds ``lens[b]`` tokens; token t lies in
page ``table[b][t / page]``.  Rows ``cu[b] .. cu[b + 1] - 1`` of q, k, v and the outputs are the last tokens of sequence
b (the queries of a cross attention, whose count is their own); rows at or behind ``cu[B]`` are padding.

``own`` selects who computes: false, elementary torch operations in 32 bits; true, this repository's entry points.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CODES = (0, 1, 2, 3, 4, 6, 8, 10, 0, -1, -2, -3, -4, -6, -8, -10)
MIDDLES = (0.5, 1.5, 2.5, 3.5, 5.0, 7.0, 9.0)


def listed():
    def append(name, b, n, t, h, hkv, d, page, layout, x, act, rot, style, stretch=1.0, pad=0, ragged=False):
        return {"name": name, "op": "append", "b": b, "n": n, "t": t, "h": h, "hkv": hkv, "d": d, "page": page, "layout": layout, "x": x, "act": act,
                "rot": rot, "style": style, "stretch": stretch, "pad": pad, "ragged": ragged}

    def read(name, b, t, hkv, d, page, layout, out, ragged=False):
        return {"name": name, "op": "read", "b": b, "n": t, "t": t, "hkv": hkv, "d": d, "page": page, "layout": layout, "out": out, "ragged": ragged}

    def attend(name, b, n, t, h, hkv, d, page, layout, act, causal=True, window=0, pad=0, ragged=False):
        return {"name": name, "op": "attention", "b": b, "n": n, "t": t, "h": h, "hkv": hkv, "d": d, "page": page, "layout": layout, "act": act,
                "causal": causal, "window": window, "pad": pad, "ragged": ragged}

    return [
        # the new token of one sequence, from the float32 output of the layer's QKV product
        append("append 1 token 40/8x128", 1, 1, 4096, 40, 8, 128, 64, "dual", "f32", "f16", 128, "half"),
        # short pieces of seven sequences in a padded batch, a part of each head turned, in pages of 16
        append("append 7 pieces 16/4x64 part", 7, 61, 777, 16, 4, 64, 16, "fast", "bf16", "bf16", 24, "interleaved", 1.0, 5, True),
        # a prompt of 4096 tokens behind a long context whose positions are stretched
        append("append 4096 tokens stretched", 1, 4096, 131072, 40, 8, 128, 64, "dual", "f32", "bf16", 128, "half", 8.0),
        # the queries of 512 tokens alone
        {"name": "rotary 512x40x128", "op": "rotary", "rows": 512, "h": 40, "d": 128, "x": "f32", "act": "f16", "rot": 128, "style": "half", "stretch": 1.0, "first": 70000},
        # the queries of one token's 16 heads, a part of each turned
        {"name": "rotary 3x16x64 part", "op": "rotary", "rows": 3, "h": 16, "d": 64, "x": "f16", "act": "bf16", "rot": 20, "style": "interleaved", "stretch": 4.0, "first": 9},
        # a few short sequences read back to be moved elsewhere, odd lengths
        read("read 5 sequences x 700", 5, 700, 4, 64, 48, "fast", "f32", True),
        # sixteen sequences of 4096 tokens read back whole
        read("read 16x4096", 16, 4096, 8, 128, 64, "dual", "bf16"),
        # one sequence's next token over a long context
        attend("attend 1x32768", 1, 1, 32768, 40, 8, 128, 64, "dual", "f16"),
        # sixteen sequences decoded together
        attend("attend 16x4096", 16, 1, 4096, 40, 8, 128, 32, "fast", "bf16"),
        # drafts of up to five tokens of nine sequences to verify, with a window, in a padded batch of small pages
        attend("attend 9 drafts x 5, window", 9, 5, 3001, 16, 4, 64, 16, "dual", "f16", True, 1024, 3, True),
        # queries of a decoder over the states of an encoder, of another length, no heads shared
        attend("cross 4x333 over 1500", 4, 333, 1500, 16, 16, 64, 32, "fast", "f16", False, 0, 0, True),
        # a prompt of 4096 tokens
        attend("attend prompt 4096", 1, 4096, 4096, 40, 8, 128, 64, "dual", "bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "rotary", "read", "attention", "attention", "attention"))
    d = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 8, 8, 16))
    group = rng.choice((1, 2, 3, 4, 5, 8, 12))
    h = hkv * group if hkv * group <= 64 else hkv
    page = rng.choice((16, 16, 32, 48, 64, 64, 128, 256))
    layout = rng.choice(("dual", "dual", "fast"))
    act = rng.choice(("f16", "bf16"))
    b = _log_uniform(rng, 1, 48)
    ragged = b > 1 and rng.random() < 0.7
    pad = rng.choice((0, 0, 1, 7))
    turn = {"rot": rng.choice((d, d, d // 2, 2 * rng.randint(1, d // 2))), "style": rng.choice(("half", "interleaved")), "stretch": rng.choice((1.0, 1.0, 4.0, 32.0))}
    x = rng.choice(("f32", "f32", "f16", "bf16"))
    if op == "rotary":
        return {"op": op, "rows": _log_uniform(rng, 1, min(8192, 2 ** 24 // (h * d))), "h": h, "d": d, "x": x, "act": act, "first": rng.choice((0, 1000, 1000000)), **turn}
    if op == "append":
        n = _log_uniform(rng, 1, max(1, min(4096, 2 ** 24 // (b * (h + 2 * hkv) * d))))
        t = n + _log_uniform(rng, 1, 65536 // b) - 1
        return {"op": op, "b": b, "n": n, "t": t, "h": h, "hkv": hkv, "d": d, "page": page, "layout": layout, "x": x, "act": act, "pad": pad, "ragged": ragged, **turn}
    if op == "read":
        t = _log_uniform(rng, 1, min(65536, 2 ** 26 // (b * hkv * d)))
        return {"op": op, "b": b, "n": t, "t": t, "hkv": hkv, "d": d, "page": page, "layout": layout, "out": rng.choice(("f32", "f16", "bf16")), "ragged": ragged}
    t = _log_uniform(rng, 1, 65536 // max(1, b // 4))
    n = rng.choice((1, 1, rng.randint(2, 16), _log_uniform(rng, 1, 4096)))
    causal = rng.random() < 0.8
    while b * n * t * h * d > 1 << 35 or b * t * hkv * d > 1 << 29 or b * n * h * d > 1 << 26:
        n, t, b = max(1, n // 2), max(1, t // 2), max(1, b - b // 4)
    if causal:
        n = min(n, t)
    ragged = ragged and b > 1
    return {"op": op, "b": b, "n": n, "t": t, "h": h, "hkv": hkv, "d": d, "page": page, "layout": layout, "act": act, "causal": causal,
            "window": rng.choice((0, 0, 1 + t // 3)) if causal else 0, "pad": pad, "ragged": ragged}


def _lengths(c):
    """(new rows, tokens) of every sequence: the case's own n and t, or up to them where the batch is ragged."""
    b, n, t = c["b"], c["n"], c["t"]
    if not c["ragged"]:
        return [n] * b, [t] * b
    r = random.Random(1000003 * n + 1009 * t + b)
    ts = [t] + [r.randint(1, t) for _ in range(b - 1)]
    ns = [n] + [r.randint(1, n) for _ in range(b - 1)]
    if c["op"] == "read":
        ns = list(ts)
    elif c["op"] == "append" or c["causal"]:
        ns = [min(a, e) for a, e in zip(ns, ts)]
    if b > 2 and c["op"] != "read":
        ns[1] = 0  # a sequence that waits
    return ns, ts


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 40) + 29)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _frequencies(rot, stretch):
    """One frequency per pair; a stretched context leaves the fast pairs as they are and slows the slow ones by `stretch`."""
    half = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = 1.0e6 ** (-2.0 * half / rot)
    keep = ((8192.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return (f * (keep + (1.0 - keep) / stretch)).float(), 0.1 * math.log(stretch) + 1.0


def _table(g, c, ts):
    """Page numbers in no order, each page of one sequence; entries behind a sequence's last page are -1."""
    page, b = c["page"], c["b"]
    width = -(-max(ts) // page)
    count = torch.tensor([-(-t // page) for t in ts], device="cuda")
    used = torch.arange(width, device="cuda")[None, :] < count[:, None]
    spare = 3
    order = torch.randperm(int(sum(-(-t // page) for t in ts)) + spare, generator=g, device="cuda")
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    table[used] = order[:order.numel() - spare].int()
    return table, order.numel()


def _block_rows(g, c, pages):
    """Valid blocks everywhere: uniform codes, scales for values of about unit size."""
    nb, bb = c["d"] // 32, 18 if c["layout"] == "dual" else 17
    w = torch.randint(0, 256, (pages, c["hkv"], c["page"], nb, bb), generator=g, device="cuda", dtype=torch.uint8)
    w[..., 16:] = 32 + w[..., 16:] % 16
    return w.view(-1)


def _spoil_rest(c, s):
    """Rows behind a sequence's last token hold no blocks: scale bytes that are no numbers."""
    page, width = c["page"], s["table"].shape[1]
    t = torch.arange(width * page, device="cuda")
    b, t = torch.nonzero((t[None, :] >= s["lens"][:, None]) & (s["table"].long().repeat_interleave(page, 1) >= 0), as_tuple=True)
    rows = s["table"].long()[b, t // page]
    for name in ("K", "V"):
        s[name].view(-1, c["hkv"], page, s[name].numel() // (s["pages"] * c["hkv"] * page))[rows, :, t % page] = 255


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    c = s
    if c["op"] == "rotary":
        m, h, d = c["rows"], c["h"], c["d"]
        s["q"] = _normal(g, m, h, d).to(TYPES[c["x"]])
        s["positions"] = (c["first"] + torch.randperm(m, generator=g, device="cuda")).int()
        s["freq"], s["amplitude"] = _frequencies(c["rot"], c["stretch"])
        s["q_out"] = torch.zeros(m, h, d, dtype=TYPES[c["act"]], device="cuda")
        return s
    ns, ts = _lengths(c)
    s["table"], s["pages"] = _table(g, c, ts)
    s["lens"] = torch.tensor(ts, dtype=torch.int32, device="cuda")
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["longest"] = max(ns)
    m, d = cu[-1] + c.get("pad", 0), c["d"]
    s["K"], s["V"] = _block_rows(g, c, s["pages"]), _block_rows(g, c, s["pages"])
    if c["op"] == "append":
        # a product's rows: some channels of k louder than the others, as trained networks have them
        h, hkv = c["h"], c["hkv"]
        loud = torch.ones(h + 2 * hkv, d, device="cuda")
        loud[h:h + hkv, torch.randint(0, d, (3,), generator=g, device="cuda")] = 8.0
        qkv = (_normal(g, m, h + 2 * hkv, d) * loud).to(TYPES[c["x"]])
        s["q"], s["k"], s["v"] = qkv.split((h, hkv, hkv), dim=1)  # views of the product's rows
        s["freq"], s["amplitude"] = _frequencies(c["rot"], c["stretch"])
        s["q_out"] = torch.zeros(m, h, d, dtype=TYPES[c["act"]], device="cuda")
        s["k_out"], s["v_out"] = (torch.zeros(m, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    elif c["op"] == "read":
        s["k_out"], s["v_out"] = (torch.zeros(m, c["hkv"], d, dtype=TYPES[c["out"]], device="cuda") for _ in range(2))
    else:
        _spoil_rest(c, s)
        s["q"] = (2.0 * _normal(g, m, c["h"], d)).to(TYPES[c["act"]])
        s["scale"] = d ** -0.5
        s["out"] = torch.zeros(m, c["h"], d, dtype=TYPES[c["act"]], device="cuda")
    return s


def run(state):
    if own:
        return _own(state)
    return {"append": _append_plain, "rotary": _rotary_plain, "read": _read_plain, "attention": _attention_plain}[state["op"]](state)


# ---- this repository's entry points ------------------------------------------------------------------------------------

def _own(s):
    import gemm_rocmfp4_dequant_gb300 as rf4
    if s["op"] == "rotary":
        return {"q": rf4.rotary(s["q"], s["freq"], s["positions"], interleaved=s["style"] == "interleaved", amplitude=s["amplitude"], out=s["q_out"])}
    cache = s.get("cache")
    if cache is None:  # a program makes this once and keeps it
        cache = s["cache"] = rf4.PagedCache(s["K"], s["V"], s["table"], s["lens"], s["cu"], kv_heads=s["hkv"], head=s["d"], page_size=s["page"],
                                            variant=rf4.DUAL if s["layout"] == "dual" else rf4.FAST)
    if s["op"] == "read":
        k, v = rf4.cache_read(cache, k_out=s["k_out"], v_out=s["v_out"])
        return {"k": k, "v": v}
    if s["op"] == "append":
        q = rf4.rope_append(cache, s["q"], s["k"], s["v"], s["freq"], interleaved=s["style"] == "interleaved", amplitude=s["amplitude"], q_out=s["q_out"])
        k, v = rf4.cache_read(cache, k_out=s["k_out"], v_out=s["v_out"])
        return {"q": q, "k": k, "v": v}
    return {"out": rf4.paged_attention(s["q"], cache, s["scale"], causal=s["causal"], window=s["window"], out=s["out"])}


# ---- plain forms: elementary torch operations in 32 bits -----------------------------------------------------------------

def _rows_of(s):
    """For each row of the batch but the padding: its sequence and the token that it is."""
    cu = s["cu"].long()
    row = torch.arange(sum(_lengths(s)[0]), device=cu.device)  # their count is known to the program without a look at the GPU
    b = torch.searchsorted(cu[1:], row, right=True)
    return b, s["lens"].long()[b] - (cu[b + 1] - row)


def _turn(x, angle, s):
    """The first `rot` values of each head turned by their pairs' angles (64 bits), in 32 bits."""
    rot, amp = s["rot"], s["amplitude"]
    cos, sin = (torch.cos(angle) * amp).float()[:, None, :], (torch.sin(angle) * amp).float()[:, None, :]
    x = x.float()
    if s["style"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., rot:]), -1)


def _rotary_plain(s):
    angle = s["positions"].double()[:, None] * s["freq"].double()
    return {"q": _turn(s["q"], angle, s).to(s["q_out"].dtype)}


def _e4m3_table(device):
    e = torch.arange(127, device=device)
    return torch.where(e >= 8, (8.0 + (e % 8)) * torch.exp2((e // 8).float() - 10.0), (e % 8) * 2.0 ** -9)


def _pack(x, layout):
    """Values (..., D) in 32 bits to blocks (..., D / 32, 17 or 18): the least scale that covers a group, the nearest codes."""
    group = 16 if layout == "dual" else 32
    v = x.unflatten(-1, (-1, group))
    table = _e4m3_table(x.device)
    e = torch.searchsorted(5.0 * table, v.abs().amax(-1)).clamp(max=126)
    a = v.abs()
    hs = 0.5 * table[e][..., None]
    code = torch.zeros_like(a, dtype=torch.int32)
    for m in MIDDLES:
        code += a > m * hs
    code = torch.where((v < 0) & (code > 0), code + 8, code).flatten(-2).unflatten(-1, (-1, 2, 16))
    qs = code[..., 0, :] + 16 * code[..., 1, :]
    return torch.cat((qs, e.unflatten(-1, (-1, 32 // group))), -1).to(torch.uint8)


def _unpack(w, layout):
    """Blocks (..., blocks, 17 or 18 bytes) to float32 values (..., blocks * 32)."""
    codes = torch.cat((w[..., :16] & 15, w[..., :16] >> 4), -1)
    v = torch.tensor(CODES, dtype=torch.float32, device=w.device)[codes.int()]
    scale = 0.5 * torch.cat((_e4m3_table(w.device), torch.zeros(129, device=w.device)))[w[..., 16:].int()]
    return (v * scale.repeat_interleave(16 if layout == "dual" else 32, -1)).flatten(-2)


def _pages(s, name):
    bb = 18 if s["layout"] == "dual" else 17
    return s[name].view(s["pages"], s["hkv"], s["page"], s["d"] // 32, bb)


def _append_plain(s):
    b, t = _rows_of(s)
    m = b.numel()
    angle = t.double()[:, None] * s["freq"].double()
    s["q_out"][:m] = _turn(s["q"][:m], angle, s).to(s["q_out"].dtype)
    page = s["table"].long()[b, t // s["page"]]
    at = t % s["page"]
    _pages(s, "K")[page, :, at] = _pack(_turn(s["k"][:m], angle, s), s["layout"])
    _pages(s, "V")[page, :, at] = _pack(s["v"][:m].float(), s["layout"])
    return {"q": s["q_out"], **_read_plain(s)}


def _read_plain(s):
    b, t = _rows_of(s)
    page, at = s["table"].long()[b, t // s["page"]], t % s["page"]
    for name in ("K", "V"):
        out = s[name.lower() + "_out"]
        out[:b.numel()] = _unpack(_pages(s, name)[page, :, at], s["layout"]).to(out.dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _attention_plain(s):
    """All sequences padded to the longest one's queries and tokens."""
    page, h, hkv, d, n = s["page"], s["h"], s["hkv"], s["d"], s["longest"]
    table = s["table"].long().clamp(min=0)
    B, T = table.shape[0], table.shape[1] * page
    K, V = (_unpack(_pages(s, name)[table], s["layout"]).transpose(1, 2).reshape(B, hkv, T, d) for name in ("K", "V"))
    lens, cu = s["lens"].long(), s["cu"].long()
    count = cu[1:] - cu[:-1]
    i, t = torch.arange(n, device=table.device), torch.arange(T, device=table.device)
    V = torch.where(t[None, None, :, None] < lens[:, None, None, None], V, torch.zeros_like(V[:1, :1, :1, :1]))
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, n, hkv, h // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, h // hkv * n, d)
    x = (q @ K.transpose(2, 3)).mul_(s["scale"]).view(B, hkv, h // hkv, n, T)
    keep = (t < lens[:, None, None]).expand(B, n, T)
    if s["causal"]:
        last = (lens[:, None] - count[:, None] + i)[:, :, None]
        keep = keep & (t <= last)
        if s["window"]:
            keep = keep & (t > last - s["window"])
    x.masked_fill_(~keep[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    y = (x.view(B, hkv, -1, T) @ V).view(B, hkv, h // hkv, n, d) / torch.where(total > 0, total, torch.ones_like(total))
    real = i[None, :] < count[:, None]
    s["out"][rows[real]] = y.permute(0, 3, 1, 2, 4).reshape(B, n, h, d)[real].to(s["out"].dtype)
    return {"out": s["out"]}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["rows"] * c["h"] * c["d"]
        return {"bytes": n * (SIZE[c["x"]] + SIZE[c["act"]]), "flops": 3 * n}
    ns, ts = _lengths(c)
    row = c["d"] // 32 * (18 if c["layout"] == "dual" else 17)
    m = sum(ns)
    if c["op"] == "append":  # the rows in, q and the blocks out, and the blocks read back
        rows = m * c["hkv"]
        return {"bytes": m * c["d"] * ((c["h"] + 2 * c["hkv"]) * SIZE[c["x"]] + c["h"] * SIZE[c["act"]]) + rows * 2 * (2 * row + 2 * c["d"]),
                "flops": m * c["d"] * (3 * c["h"] + 20 * c["hkv"])}
    if c["op"] == "read":
        return {"bytes": m * c["hkv"] * 2 * (row + c["d"] * SIZE[c["out"]]), "flops": 2 * m * c["hkv"] * c["d"]}
    seen, pairs = 0, 0
    for n, t in zip(ns, ts):
        if not n:
            continue
        if not c["causal"]:
            seen, pairs = seen + t, pairs + n * t
            continue
        w = c["window"] or t
        seen += t - max(0, t - n + 1 - w)
        pairs += sum(min(w, t - n + 1 + i) for i in range(n))
    return {"bytes": seen * c["hkv"] * 2 * row + 4 * m * c["h"] * c["d"], "flops": 4 * c["d"] * c["h"] * pairs}


# ---- exact values, from the definitions in 64 bits -------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append_exact, "rotary": _rotary_exact, "read": _read_exact, "attention": _attention_exact}[s["op"]](s)


def _turn_exact(x, position, s):
    """A complex product per pair."""
    rot = s["rot"]
    f = s["freq"].double() * position.double()[:, None]
    z = torch.polar(torch.full_like(f, s["amplitude"]), f)[:, None, :]
    x = x.double()
    if s["style"] == "half":
        p = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        return torch.cat((p.real, p.imag, x[..., rot:]), -1)
    p = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z
    return torch.cat((torch.view_as_real(p).flatten(-2), x[..., rot:]), -1)


def _rotary_exact(s):
    return {"q": _turn_exact(s["q"], s["positions"], s)}


def _quantised_exact(x, layout):
    """The values that the blocks of x stand for: of all scales the least that covers, of all magnitudes the nearest."""
    g = x.unflatten(-1, (-1, 16 if layout == "dual" else 32))
    scales = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=x.device)
    amax = g.abs().amax(-1, keepdim=True)
    least = (5 * scales < amax).sum(-1, keepdim=True).clamp(max=126)
    hs = scales[least] / 2
    best, gap = torch.zeros_like(g), g.abs()
    for m in (1, 2, 3, 4, 6, 8, 10):
        away = (g.abs() - m * hs).abs()
        best, gap = torch.where(away < gap, m * hs, best), torch.minimum(away, gap)
    return (torch.sign(g) * best).flatten(-2)


def _exact_rows(s):
    ns, ts = _lengths(s)
    b = [i for i, n in enumerate(ns) for _ in range(n)]
    t = [e - n + i for n, e in zip(ns, ts) for i in range(n)]
    dev = s["lens"].device
    return torch.tensor(b, device=dev, dtype=torch.int64), torch.tensor(t, device=dev, dtype=torch.int64)


def _filled(values, like):
    out = torch.zeros(like.shape, dtype=torch.float64, device=like.device)
    out[:values.shape[0]] = values
    return out


def _append_exact(s):
    _, t = _exact_rows(s)
    m = t.numel()
    return {"q": _filled(_turn_exact(s["q"][:m], t, s), s["q_out"]),
            "k": _filled(_quantised_exact(_turn_exact(s["k"][:m], t, s), s["layout"]), s["k_out"]),
            "v": _filled(_quantised_exact(s["v"][:m].double(), s["layout"]), s["v_out"])}


def _values_exact(w, layout):
    """Rows of blocks (rows, blocks, bytes) in 64 bits."""
    w = w.long()
    size = lambda q: torch.where(q % 8 <= 4, q % 8, 2 * (q % 8) - 4).double() * torch.where(q >= 8, -1.0, 1.0).double()  # noqa: E731
    out = torch.empty(*w.shape[:-1], 32, dtype=torch.float64, device=w.device)
    for half in (0, 1):
        e = w[..., 16 + (half if layout == "dual" else 0)]
        field, mant = e // 8 % 16, e % 8
        hs = torch.where(field > 0, torch.ldexp((8 + mant).double(), field - 11), torch.ldexp(mant.double(), torch.full_like(field, -10)))
        out[..., 16 * half:16 * half + 16] = size((w[..., :16] // (16 if half else 1)) % 16) * hs[..., None]
    return out.flatten(-2)


def _tokens_exact(s, name, b, t):
    bb = 18 if s["layout"] == "dual" else 17
    rows = s[name].view(s["pages"], s["hkv"], s["page"], s["d"] // 32, bb)
    return _values_exact(rows[s["table"].long()[b, torch.div(t, s["page"], rounding_mode="floor")], :, t % s["page"]], s["layout"])


def _read_exact(s):
    b, t = _exact_rows(s)
    return {n.lower(): _filled(_tokens_exact(s, n, b, t), s[n.lower() + "_out"]) for n in ("K", "V")}


def _attention_exact(s):
    ns, ts = _lengths(s)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    group, at = s["h"] // s["hkv"], 0
    for b, (n, t) in enumerate(zip(ns, ts)):
        if not n:
            continue
        tok = torch.arange(t, device="cuda")
        where = torch.full_like(tok, b)
        K, V = (_tokens_exact(s, name, where, tok) for name in ("K", "V"))
        for kv in range(s["hkv"]):
            q = s["q"][at:at + n, kv * group:(kv + 1) * group].double()
            z = torch.einsum("ngd,td->ngt", q, K[:, kv]) * s["scale"]
            if s["causal"]:
                last = (t - n + torch.arange(n, device="cuda"))[:, None, None]
                z = torch.where(tok > last, -math.inf, z)
                if s["window"]:
                    z = torch.where(tok <= last - s["window"], -math.inf, z)
            out[at:at + n, kv * group:(kv + 1) * group] = torch.einsum("ngt,td->ngd", torch.softmax(z, -1), V[:, kv])
        at += n
    return {"out": out}
