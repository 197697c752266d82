"""GPU tests of attention over a paged cache, against its definition in 64 bits.

Bound of an output, from the arithmetic (paged_util.Paged.attention): the decoded K and V are exact, so a score is off by
its fp32 accumulation, dx = (16 + D / 16) * 2^-23 * scale * max_t sum_d |q_d k_td| and 2^-20 for the exponent's
argument; a weight is off by 2 dx (its own and the sum's) and by fp16's half step, 2^-11; the weighted sum by its
fp32 accumulation, (T / 16 + 16) * 2^-23; all of them relative to sum_t p_t |V_t|.  The output adds half a step of its type."""
import math

import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import torch

pytestmark = pytest.mark.gpu
if torch().cuda.is_available():
    import paged_util as pu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    assert rf4.device_error_bits() == 0


def check(p, q, causal=True, window=0, scale=None, out=None):
    t = torch()
    scale = p.d ** -0.5 if scale is None else scale
    pad = q.shape[0] - p.m
    if out is None:
        out = t.full((q.shape[0], q.shape[1], p.d), 3.0, dtype=q.dtype, device="cuda")
    rf4.paged_attention(q, p.cache, scale, causal=causal, window=window, out=out)
    want, tol = p.attention(q[:p.m], scale, causal, window)
    bad = (out[:p.m].double() - want).abs() > tol + pu.rounding(want, q.dtype) * (1 + 2.0 ** -6)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"
    assert pad == 0 or bool((out[p.m:] == 3.0).all())
    return out


ACTS = ["f16", "bf16"]


def act(name):
    return {"f16": torch().float16, "bf16": torch().bfloat16}[name]


@pytest.mark.parametrize("variant", [rf4.DUAL, rf4.FAST])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,hkv,page", [(1, 1, 16), (10, 2, 64), (8, 8, 48), (12, 1, 32), (16, 2, 128)])
def test_single_tokens(variant, name, D, H, hkv, page):
    """Decode: lengths of zero, one, around the tiles' and pages' borders, and a few long ones."""
    ts = [0, 1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 255, 257, 700, 2049]
    p = pu.Paged([1] * len(ts), ts, hkv, D, page, variant, seed=D + H, extra=5)
    check(p, p.queries(H, act(name)))


@pytest.mark.parametrize("variant", [rf4.DUAL, rf4.FAST])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,hkv,page", [(5, 1, 64), (4, 4, 16), (16, 2, 48), (20, 4, 32)])
def test_chunks(variant, name, D, H, hkv, page):
    """Chunks of any number of rows in one batch: none, more than the sequence has tokens, all of it, a few of many."""
    ns = [1, 0, 5, 3, 130, 64, 17, 300, 2]
    ts = [1, 40, 3, 3, 130, 500, 1000, 301, 0]
    p = pu.Paged(ns, ts, hkv, D, page, variant, seed=D + H + page)
    check(p, p.queries(H, act(name), pad=3))


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 5000])
@pytest.mark.parametrize("D,variant,name", [(64, rf4.FAST, "bf16"), (128, rf4.DUAL, "f16")])
def test_windows(window, D, variant, name):
    p = pu.Paged([1, 7, 200, 1, 33, 4], [1, 300, 640, 777, 33, 2], 2, D, 32, variant, seed=window)
    check(p, p.queries(6, act(name)), window=window)


@pytest.mark.parametrize("D,H,hkv,variant,name", [(64, 4, 4, rf4.DUAL, "f16"), (128, 6, 2, rf4.FAST, "bf16")])
def test_cross(D, H, hkv, variant, name):
    """Queries of any number over another's states: more queries than states, no states, no queries."""
    p = pu.Paged([7, 333, 0, 1, 5, 90], [900, 100, 50, 129, 0, 1], hkv, D, 16, variant, seed=D)
    check(p, p.queries(H, act(name), pad=1), causal=False)


@pytest.mark.parametrize("ns,ts", [([1], [20000]), ([3], [30001]), ([40], [9000]), ([700], [700]), ([1, 1000], [4000, 5000])])
def test_long_contexts_are_split(ns, ts):
    """Work split along the tokens and joined."""
    p = pu.Paged(ns, ts, 2, 128, 64, rf4.DUAL, seed=len(ns))
    q = p.queries(10, torch().float16)
    out = check(p, q)
    again = rf4.paged_attention(q, p.cache, p.d ** -0.5)
    assert torch().equal(out, again)  # bitwise repeatable


def test_peaked_and_growing_scores():
    """One token that outweighs all others, early, late, and scores that grow along the tokens, so that maxima move on."""
    t = torch()
    p = pu.Paged([1, 4, 150, 1], [3000, 3000, 900, 513], 1, 64, 32, rf4.DUAL, seed=9)
    for b, T in enumerate(p.ts):
        i = t.arange(T, device="cuda")
        page, at = p.table.long()[b, i // 32], i % 32
        p.K[page, 0, at, :, 16:] = (8 + i * 56 // T).to(t.uint8)[:, None, None]  # scales from 2^-6 to 2^1
        p.K[page, 0, at, :, :16] = 0x77  # all of one sign
    p.K[int(p.table[0, 3]), 0, 5, :, 16:] = 72
    q = p.queries(3, t.float16, scale=0.5).abs()
    check(p, q)
    check(p, -q)
    check(p, q, scale=4.0)


def test_strided_rows_and_views():
    t = torch()
    p = pu.Paged([3, 20], [60, 20], 2, 64, 16, rf4.DUAL, seed=2)
    check(p, p.queries(4, t.float16, stride=24))
    wide = p.queries(9, t.bfloat16)
    check(p, wide[:, 2:6])


def test_shared_pages_and_contiguous_cache():
    """Two sequences with one beginning; and a contiguous cache as decode_attention takes it, with equal results to its bound."""
    t = torch()
    p = pu.Paged([2, 2], [64, 70], 2, 128, 32, rf4.DUAL, seed=5)
    p.table[1, :2] = p.table[0, :2]
    check(p, p.queries(8, t.float16))
    B, hkv, T, D, H = 3, 2, 96, 128, 10
    c = pu.Paged([1] * B, [96, 41, 0], hkv, D, T, rf4.DUAL, seed=6, spare=1, width=1)
    c.table.copy_(t.arange(B, dtype=t.int32).view(B, 1))
    c.K.copy_(c._blocks())  # valid blocks again where the pages' owners changed
    c.V.copy_(c._blocks())
    c.spoil()
    q = c.queries(H, t.float16)
    out = check(c, q)
    dense = rf4.decode_attention(q, c.K[:B].reshape(-1), c.V[:B].reshape(-1), c.lens, hkv, T, D ** -0.5)
    assert float((out.double() - dense.double()).abs().max()) <= 2.0 ** -9 * float(dense.abs().max())


def test_bad_pages_are_no_tokens():
    t = torch()
    for ns in ([1, 1], [40, 3]):
        p = pu.Paged(ns, [200, 90], 2, 64, 16, rf4.DUAL, seed=3)
        p.table[0, 4], p.table[0, 12], p.table[1, 0] = p.pages, -1, 2 ** 31 - 1
        check(p, p.queries(4, t.float16))
        assert rf4.device_error_bits() == 2
    p = pu.Paged([1], [64], 1, 64, 16, rf4.DUAL)
    p.table.fill_(-1)
    q = p.queries(2, t.float16)
    assert bool((rf4.paged_attention(q, p.cache, 0.1) == 0).all())
    assert rf4.device_error_bits() == 2


def test_queries_that_are_no_numbers_stay_in_their_rows():
    t = torch()
    p = pu.Paged([3, 140], [50, 200], 2, 64, 16, rf4.FAST, seed=8)
    q = p.queries(4, t.float16)
    clean = rf4.paged_attention(q, p.cache, 0.125)
    q[1, 2, 5], q[70, 0, 0] = math.nan, math.inf
    out = rf4.paged_attention(q, p.cache, 0.125)
    hit = t.zeros(p.m, 4, dtype=t.bool, device="cuda")
    hit[1, 2] = hit[70, 0] = True
    assert bool(out[1, 2].isnan().all()) and t.equal(out[~hit], clean[~hit])


def test_captured_and_replayed_with_other_batches():
    """A captured call follows lens, cu and table as they are at each replay."""
    t = torch()
    p = pu.Paged([1, 1, 1, 1], [300, 300, 300, 300], 2, 128, 32, rf4.DUAL, seed=4)
    q = p.queries(10, t.bfloat16)
    out = rf4.paged_attention(q, p.cache, 0.1)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        rf4.paged_attention(q, p.cache, 0.1, out=out)
    valid = p._blocks()
    p.K.copy_(valid)
    p.V.copy_(valid.flip(0))
    for ns, ts in (([1, 1, 1, 1], [1, 300, 17, 0]), ([4, 0, 0, 0], [299, 5, 5, 5]), ([0, 2, 1, 0], [3, 200, 64, 128])):
        p.ns, p.ts, p.m = ns, ts, sum(ns)
        p.lens.copy_(t.tensor(ts, dtype=t.int32))
        p.cu.copy_(t.tensor([0] + [sum(ns[:i + 1]) for i in range(4)], dtype=t.int32))
        out.fill_(3.0)
        g.replay()
        want, tol = p.attention(q[:p.m], 0.1)
        assert bool(((out[:p.m].double() - want).abs() <= tol + pu.rounding(want, q.dtype) * (1 + 2.0 ** -6)).all())
        assert bool((out[p.m:] == 3.0).all())


def test_on_another_stream():
    t = torch()
    p = pu.Paged([5, 1], [500, 800], 2, 64, 16, rf4.DUAL, seed=1)
    q = p.queries(8, t.float16)
    want = rf4.paged_attention(q, p.cache, 0.125)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    got = rf4.paged_attention(q, p.cache, 0.125, stream=s)
    t.cuda.current_stream().wait_stream(s)
    assert t.equal(got, want)


def test_refusals_and_empty():
    t = torch()
    p = pu.Paged([2], [5], 2, 64, 16, rf4.DUAL)
    q = p.queries(4, t.float16)
    for f in (lambda: rf4.paged_attention(q.float(), p.cache, 0.1), lambda: rf4.paged_attention(q.cpu(), p.cache, 0.1),
              lambda: rf4.paged_attention(q[..., :32], p.cache, 0.1), lambda: rf4.paged_attention(q, p.cache, 0.1, out=q.bfloat16()),
              lambda: rf4.paged_attention(q.transpose(0, 1), p.cache, 0.1)):
        with pytest.raises((ValueError, TypeError)):
            f()
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=0.1, window=-1), dict(scale=0.1, causal=False, window=4)):
        with pytest.raises(rf4.RocmFP4Error):
            rf4.paged_attention(q, p.cache, **kw)
    with pytest.raises(rf4.RocmFP4Error):
        rf4.paged_attention(q[:, :3], p.cache, 0.1)  # three heads over two
    assert rf4.paged_attention(q[:0], p.cache, 0.1).shape == (0, 4, 64)


@pytest.mark.parametrize("ns,ts,H,hkv,D,variant,name", [([1], [32768], 40, 8, 128, rf4.DUAL, "f16"), ([1] * 16, [4000 + 7 * i for i in range(16)], 40, 8, 128, rf4.FAST, "bf16"),
                                                        ([1] * 40, [1500 + 11 * i for i in range(40)], 16, 16, 64, rf4.DUAL, "bf16"), ([60] * 3, [6000, 9001, 12345], 16, 8, 64, rf4.FAST, "f16")])
def test_many_token_tiles_a_block(ns, ts, H, hkv, D, variant, name):
    """Stretches of more token tiles than any ring holds, over caches that are not in the L2, launch after launch: every one alike."""
    t = torch()
    p = pu.Paged(ns, ts, hkv, D, 32, variant, seed=H)
    q = p.queries(H, act(name))
    flush = t.empty(200 << 20, dtype=t.uint8, device="cuda")
    out = check(p, q)
    for _ in range(10):
        flush.fill_(1)
        assert t.equal(rf4.paged_attention(q, p.cache, D ** -0.5), out)
    for _ in range(10):
        again = rf4.paged_attention(q, p.cache, D ** -0.5)
    assert t.equal(again, out)
