"""The paged cache's operators together, as a model's layer calls them: rotary
positions with packing, attention over the pages, reading back; a prompt in
pieces, then single tokens, captured once and replayed as the sequences grow."""
import math

import pytest
import torch

import gemm_rocmfp4_dequant_gb300 as rf4

pytestmark = pytest.mark.gpu

H, HKV, D, PAGE = 8, 2, 64, 16


def _angles(freq, positions):
    return positions.double()[:, None] * freq.double()[None, :]


def _turned(x, angle):
    """x [T][heads][D], halves paired, in 64 bits."""
    half = D // 2
    a, b = x[..., :half], x[..., half:]
    c, s = angle.cos()[:, None, :], angle.sin()[:, None, :]
    return torch.cat((a * c - b * s, b * c + a * s), dim=-1)


def _attend(q, k, v, first, scale):
    """Rows first, first + 1, ... of a sequence over its keys and values, in 64 bits."""
    g = H // HKV
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    w = torch.einsum("mhd,thd->hmt", q, k) * scale
    seen = torch.arange(k.shape[0], device=q.device)[None, :] <= first + torch.arange(q.shape[0], device=q.device)[:, None]
    p = torch.softmax(w.masked_fill(~seen[None], -math.inf), dim=-1)
    return torch.einsum("hmt,thd->mhd", p, v)


@pytest.mark.parametrize("variant,act", [(rf4.DUAL, torch.float16), (rf4.FAST, torch.bfloat16)])
def test_prompt_in_pieces_then_tokens(variant, act):
    g = torch.Generator(device="cuda").manual_seed(11)
    prompts, steps, cut = (37, 1, 130), 5, 20
    B = len(prompts)
    total = [n + steps for n in prompts]
    width = -(-max(total) // PAGE)
    pages = sum(-(-t // PAGE) for t in total) + 2
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, t in enumerate(total):
        n = -(-t // PAGE)
        table[b, :n] = order[at:at + n]
        at += n
    bb = D // 32 * (18 if variant == rf4.DUAL else 17)
    K, V = (torch.full((pages * HKV * PAGE * bb,), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    freq, _ = rf4.rotary_frequencies(D, 10000.0)
    x = [torch.randn(t, H + 2 * HKV, D, generator=g, device="cuda") for t in total]
    scale = D ** -0.5
    eps = torch.finfo(act).eps / 2
    got_q, got_o = [[] for _ in range(B)], [[] for _ in range(B)]

    def pieces(lens, cu):
        return rf4.PagedCache(K, V, table, lens, cu, kv_heads=HKV, head=D, page_size=PAGE, variant=variant)

    def step(cache, rows, q_out=None, out=None):
        q, k, v = rows.split((H, HKV, HKV), dim=1)
        q_out = rf4.rope_append(cache, q, k, v, freq, dtype=act, q_out=q_out)
        return q_out, rf4.paged_attention(q_out, cache, scale, out=out)

    done = [0] * B
    while any(d < n for d, n in zip(done, prompts)):
        ns = [min(cut * (b + 1), prompts[b] - done[b]) for b in range(B)]
        cu = [0]
        for n in ns:
            cu.append(cu[-1] + n)
        rows = torch.cat([x[b][done[b]:done[b] + ns[b]] for b in range(B)])
        done = [d + n for d, n in zip(done, ns)]
        q, o = step(pieces(torch.tensor(done, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")), rows)
        for b in range(B):
            got_q[b].append(q[cu[b]:cu[b + 1]])
            got_o[b].append(o[cu[b]:cu[b + 1]])

    # single tokens: one capture, the lengths grow in place
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cache = pieces(lens, torch.arange(B + 1, dtype=torch.int32, device="cuda"))
    rows = torch.zeros(B, H + 2 * HKV, D, device="cuda")
    q_out = torch.empty(B, H, D, dtype=act, device="cuda")
    out = torch.empty_like(q_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        step(cache, rows, q_out, out)
    for i in range(steps):
        rows.copy_(torch.stack([x[b][prompts[b] + i] for b in range(B)]))
        graph.replay()
        for b in range(B):
            got_q[b].append(q_out[b:b + 1].clone())
            got_o[b].append(out[b:b + 1].clone())

    # what the pages hold, read back whole
    cu = [0]
    for t in total:
        cu.append(cu[-1] + t)
    whole = pieces(torch.tensor(total, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda"))
    k_all, v_all = (torch.empty(cu[-1], HKV, D, dtype=torch.float32, device="cuda") for _ in range(2))
    rf4.cache_read(whole, k_out=k_all, v_out=v_all)
    assert rf4.device_error_bits() == 0
    for b in range(B):
        q, o = torch.cat(got_q[b]), torch.cat(got_o[b])
        xd, angle = x[b].double(), _angles(freq, torch.arange(total[b], device="cuda"))
        qe = _turned(xd[:, :H], angle)
        # one rounding, and fp32's of the sine, the cosine and two products (8 half steps of the pair's length at most)
        bound = eps * qe.abs() + 8 * 2.0 ** -24 * (xd[:, :H].abs() + xd[:, :H].roll(D // 2, -1).abs()) + 2.0 ** -25
        assert bool(((q.double() - qe).abs() <= bound).all())
        # K and V: the codes are 0, 1, 2, 3, 4, 6, 8, 10 half scales, so a value is off by one half scale at most; ten of them
        # are the group's largest value, rounded up to the next E4M3 (an eighth more, or 2^-9 of a subnormal one)
        for got, want in ((k_all[cu[b]:cu[b + 1]].double(), _turned(xd[:, H:H + HKV], angle)), (v_all[cu[b]:cu[b + 1]].double(), xd[:, H + HKV:])):
            blocks = want.abs().reshape(total[b], HKV, D // 32, 32).amax(-1, keepdim=True)
            assert bool(((got - want).abs().reshape(total[b], HKV, D // 32, 32) <= blocks * 0.1125 + 2.0 ** -10 + 1e-5).all())
        # attention over what the pages hold, by the rounded queries
        oe = _attend(q.double(), k_all[cu[b]:cu[b + 1]].double(), v_all[cu[b]:cu[b + 1]].double(), 0, scale)
        # the output's rounding; P's, 2^-11 of a weighted mean; scores of 64 products in fp32, which move P by their error
        vmax = v_all[cu[b]:cu[b + 1]].abs().amax().double()
        smax = (q.double().abs().amax() * k_all[cu[b]:cu[b + 1]].abs().amax().double()) * D * scale
        assert bool(((o.double() - oe).abs() <= eps * oe.abs() + (2.0 ** -11 + 4 * 64 * 2.0 ** -24 * smax) * vmax + 2.0 ** -24).all())
