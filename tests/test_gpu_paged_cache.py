"""GPU tests of rotary positions, of packing new tokens into a paged cache and of reading it back, against the definitions
in 64 bits.

A turned value is off by at most `turned`'s bound, from the fp32 sine, cosine, product and sum; q adds half a step of its
type.  A packed value has to be a right answer of the quantiser's rule for some value within that bound: its scale byte
lies between those of the group's largest magnitude less and more the bound, and no magnitude of that scale is nearer by
more than twice the bound.  Without a turn the bound is zero, and the blocks are those of rf4.quantize, byte by byte."""
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


def dtype_of(name):
    return {"f32": torch().float32, "f16": torch().float16, "bf16": torch().bfloat16}[name]


def check_rotary(y, x, pos, freq, interleaved, amplitude):
    want, tol = pu.turned(x, pos, freq, interleaved, amplitude)
    assert bool(((y.double() - want).abs() <= tol + pu.rounding(want, y.dtype) + tol * 2.0 ** -7).all())


@pytest.mark.parametrize("x,act", [("f32", "f16"), ("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 128, True), (64, 24, False), (64, 20, True), (96, 50, False), (32, 2, False),
                                               (256, 256, False), (64, 6, True)])
def test_rotary(x, act, D, rot, interleaved):
    t = torch()
    t.manual_seed(D + rot)
    for M, H in ((1, 1), (3, 5), (33, 7)):
        v = t.randn(M, H, D, device="cuda").to(dtype_of(x))
        freq, amp = rf4.rotary_frequencies(rot, 1e6)
        pos = t.randint(-50, 100000, (M,), dtype=t.int32, device="cuda")
        check_rotary(rf4.rotary(v, freq, pos, interleaved=interleaved, amplitude=1.25, dtype=dtype_of(act)), v, pos, freq, interleaved, 1.25)


def test_rotary_far_positions():
    """Angles of positions up to the type's limits: the fastest pair turns 2^31 / 2 pi times."""
    t = torch()
    pos = t.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=t.int32, device="cuda")
    x = t.randn(7, 2, 64, device="cuda")
    freq = t.cat((rf4.rotary_frequencies(56)[0], t.tensor([0.0, -0.75, 7.5, 1e-9], device="cuda")))
    check_rotary(rf4.rotary(x, freq, pos, dtype=t.float16), x, pos, freq, False, 1.0)


def test_rotary_passes_what_it_does_not_turn():
    """Infinities and NaN of a pair stay in it; values behind rot are rounded alone."""
    t = torch()
    x = t.randn(2, 3, 64, device="cuda")
    x[0, 0, 5], x[1, 2, 40] = math.inf, math.nan
    freq, _ = rf4.rotary_frequencies(16)
    y = rf4.rotary(x, freq, t.tensor([3, 4], dtype=t.int32, device="cuda"))
    odd = ~y.isfinite()
    assert odd[0, 0, 5] and odd[0, 0, 13] and odd[1, 2, 40] and int(odd.sum()) == 3
    assert t.equal(y[..., 16:][~odd[..., 16:]], x[..., 16:].half()[~odd[..., 16:]])


def test_rotary_of_parts_of_rows_and_empty():
    t = torch()
    rows = t.randn(5, 9, 64, device="cuda")
    freq, _ = rf4.rotary_frequencies(64)
    pos = t.arange(5, dtype=t.int32, device="cuda")
    assert t.equal(rf4.rotary(rows[:, 3:7], freq, pos), rf4.rotary(rows[:, 3:7].contiguous(), freq, pos))
    assert rf4.rotary(rows[:0], freq, pos[:0]).shape == (0, 9, 64)


def quantised_ok(blocks, x, tol, variant):
    """Whether blocks (rows, hkv, D / 32, bytes) are a right quantisation of values within tol of x (rows, hkv, D)."""
    t = torch()
    group = 16 if variant == rf4.DUAL else 32
    got = pu.decode(blocks, variant).unflatten(-1, (-1, group))
    x, tol = x.unflatten(-1, (-1, group)), tol.unflatten(-1, (-1, group))
    e = blocks[..., 16:].flatten(-2).long()  # one per group, in order
    values = pu.e4m3_values(x.device)[:127]
    amax, slack = x.abs().amax(-1), tol.amax(-1)
    least = t.searchsorted(5 * values, (amax - slack).clamp(min=0.0)).clamp(max=126)
    most = t.searchsorted(5 * values, amax + slack).clamp(max=126)
    assert bool(((e >= least) & (e <= most)).all())
    hs = 0.5 * values[e][..., None]
    gaps = t.stack([(x.abs() - m * hs).abs() for m in pu.MAGNITUDES], -1).amin(-1)
    assert bool(((got - x).abs() <= gaps + 2 * tol).all())


def appended(p, which):
    """The blocks (rows, hkv, D / 32, bytes) of the batch's rows that are tokens, and the rows."""
    t = torch()
    w = p.K if which == "K" else p.V
    rows, out, at = [], [], 0
    for b, (n, T) in enumerate(zip(p.ns, p.ts)):
        for i in range(n):
            tok = T - n + i
            if tok >= 0:
                rows.append(at + i)
                out.append(w[int(p.table[b, tok // p.page]), :, tok % p.page])
        at += n
    return t.stack(out), t.tensor(rows, device="cuda")


def places(p):
    return torch().tensor([T - n + i for n, T in zip(p.ns, p.ts) for i in range(n)], dtype=torch().int32, device="cuda")


@pytest.mark.parametrize("variant", [rf4.DUAL, rf4.FAST])
@pytest.mark.parametrize("x,act", [("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("D,rot,interleaved,page,hkv,H", [(128, 128, False, 64, 2, 10), (64, 24, True, 16, 4, 4), (64, 14, False, 48, 1, 3), (96, 96, False, 32, 3, 6)])
def test_append(variant, x, act, D, rot, interleaved, page, hkv, H):
    t = torch()
    p = pu.Paged([3, 0, 1, 20, 5], [3, 9, 40, 97, 2], hkv, D, page, variant, seed=D + rot, extra=3)
    before = p.K.clone(), p.V.clone()
    pad = 2
    rows = (t.randn(p.m + pad, H + 2 * hkv, D, generator=p.g, device="cuda") * 3).to(dtype_of(x))
    q, k, v = rows.split((H, hkv, hkv), 1)
    freq, _ = rf4.rotary_frequencies(rot, 1e5)
    out = t.full((p.m + pad, H, D), 7.0, dtype=dtype_of(act), device="cuda")
    got = rf4.rope_append(p.cache, q, k, v, freq, interleaved=interleaved, amplitude=0.875, q_out=out)
    assert got is out and bool((out[p.m:] == 7.0).all())
    pos = places(p)
    check_rotary(out[:p.m], q[:p.m], pos, freq, interleaved, 0.875)
    blocks, real = appended(p, "K")
    want, tol = pu.turned(k[:p.m], pos, freq, interleaved, 0.875)
    quantised_ok(blocks, want[real], tol[real], variant)
    blocks, real = appended(p, "V")
    quantised_ok(blocks, v[real].double(), t.zeros_like(v[real].double()), variant)
    # nothing else changed
    for w, old in zip((p.K, p.V), before):
        changed = (w != old).flatten(3).any(-1)
        allowed = t.zeros_like(changed)
        at = 0
        for b, (n, T) in enumerate(zip(p.ns, p.ts)):
            for i in range(max(0, T - n), T):
                allowed[int(p.table[b, i // page]), :, i % page] = True
        assert not bool((changed & ~allowed).any())
    # and the rows read back are the blocks' values; the first rows of the last sequence are no tokens
    for dt in (t.float32, t.float16, t.bfloat16):
        ko, vo = rf4.cache_read(p.cache, k_out=t.full((p.m + pad, hkv, D), 5.0, dtype=dt, device="cuda"), v_out=t.full((p.m + pad, hkv, D), 5.0, dtype=dt, device="cuda"))
        for o, which in ((ko, "K"), (vo, "V")):
            blocks, real = appended(p, which)
            full = t.zeros(p.m, hkv, D, dtype=t.float64, device="cuda")
            full[real] = pu.decode(blocks, variant)
            assert t.equal(o[:p.m].double(), full) and bool((o[p.m:] == 5.0).all())
    ko, none = rf4.cache_read(p.cache, k_out=t.empty_like(ko))
    assert none is None and t.equal(ko[:p.m].double(), rf4.cache_read(p.cache, p.m, dtype=t.float32)[0].double())


@pytest.mark.parametrize("variant", [rf4.DUAL, rf4.FAST])
@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_append_without_turn_is_the_quantiser(variant, x):
    """freq None: the blocks of rf4.quantize, over magnitudes from subnormal to saturating, zeros, infinities and NaN among them."""
    t = torch()
    p = pu.Paged([50, 14], [50, 31], 2, 128, 16, variant)
    mag = t.exp2(t.randint(-14, 13, (p.m, 2, 4, 1), generator=p.g, device="cuda").float())
    rows = [(t.randn(p.m, 2, 4, 32, generator=p.g, device="cuda") * mag).flatten(2).to(dtype_of(x)) for _ in range(2)]
    rows[0][3, 1, :32] = 0.0
    rows[0][4, 0, 7], rows[0][5, 1, 99], rows[1][6, 0, 3] = math.inf, math.nan, -math.inf
    rows[1][7, 0, :16] = -0.0
    assert rf4.rope_append(p.cache, None, rows[0], rows[1]) is None
    for which, r in zip(("K", "V"), rows):
        blocks, real = appended(p, which)
        want = rf4.quantize(r.reshape(p.m * 2, 128), variant).view(p.m, 2, 4, p.bb)
        assert t.equal(blocks, want[real])


def test_append_at_positions_of_its_own():
    t = torch()
    p = pu.Paged([4, 3], [10, 3], 1, 64, 16, rf4.DUAL)
    k, v, q = (t.randn(p.m, h, 64, generator=p.g, device="cuda") for h in (1, 1, 2))
    freq, _ = rf4.rotary_frequencies(64)
    pos = t.tensor([100, -3, 7, 7, 0, 65536, 5], dtype=t.int32, device="cuda")
    out = rf4.rope_append(p.cache, q, k, v, freq, positions=pos)
    check_rotary(out, q, pos, freq, False, 1.0)
    want, tol = pu.turned(k, pos, freq, False, 1.0)
    blocks, real = appended(p, "K")
    quantised_ok(blocks, want[real], tol[real], rf4.DUAL)


def test_many_sequences_find_their_rows():
    """Batches of every size near the search's powers of eight, sequences without rows among them."""
    t = torch()
    for B in (1, 2, 7, 8, 9, 63, 64, 65, 100, 513):
        r = t.Generator().manual_seed(B)
        ns = t.randint(0, 4, (B,), generator=r).tolist()
        ns[-1] = 1
        ts = [n + 5 for n in ns]
        p = pu.Paged(ns, ts, 1, 32, 16, rf4.DUAL, seed=B)
        k = t.randn(p.m, 1, 32, generator=p.g, device="cuda").half()
        rf4.rope_append(p.cache, None, k, k)
        ko, vo = rf4.cache_read(p.cache, p.m, dtype=t.float32)
        want = rf4.dequant(rf4.quantize(k.view(-1, 32)), p.m, 32).view(p.m, 1, 32)
        assert t.equal(ko, want) and t.equal(vo, want)


def test_whole_cache_read_and_large_offsets():
    """Pages behind the first 2^32 bytes: written and read at 64-bit offsets."""
    t = torch()
    page, hkv, d = 256, 8, 128
    size = page * hkv * 72
    pages = (1 << 32) // size + 40
    K = t.empty(pages * size, dtype=t.uint8, device="cuda")
    V = t.empty(pages * size, dtype=t.uint8, device="cuda")
    table = t.tensor([[pages - 1, 0], [3, pages - 2]], dtype=t.int32, device="cuda")
    lens = t.tensor([300, 512], dtype=t.int32, device="cuda")
    cu = t.tensor([0, 300, 812], dtype=t.int32, device="cuda")
    cache = rf4.PagedCache(K, V, table, lens, cu, kv_heads=hkv, head=d, page_size=page)
    k, v = (t.randn(812, hkv, d, device="cuda").half() for _ in range(2))
    rf4.rope_append(cache, None, k, v)
    ko, vo = rf4.cache_read(cache, 812, dtype=t.float32)
    for got, x in ((ko, k), (vo, v)):
        assert t.equal(got, rf4.dequant(rf4.quantize(x.reshape(-1, d)), 812 * hkv, d).view(812, hkv, d))
    q = t.randn(812, hkv, d, device="cuda").half()
    out = rf4.paged_attention(q, cache, d ** -0.5)
    s = t.einsum("nhd,thd->hnt", q[:300].double(), ko[:300].double()) * d ** -0.5
    s = t.where(t.arange(300, device="cuda") > t.arange(300, device="cuda")[:, None], -math.inf, s)
    want = t.einsum("hnt,thd->nhd", t.softmax(s, -1), vo[:300].double())
    assert float((out[:300].double() - want).norm() / want.norm()) < 2.0 ** -10


def test_bad_pages_are_reported_and_left_alone():
    t = torch()
    p = pu.Paged([20, 20], [40, 40], 2, 64, 16, rf4.DUAL)
    old = p.K.clone()
    table = p.table.clone()
    p.table[0, 1], p.table[1, 2] = p.pages, -2 ** 31
    k = t.randn(p.m, 2, 64, generator=p.g, device="cuda")
    rf4.rope_append(p.cache, None, k, k)
    assert rf4.device_error_bits() == 2
    ko, _ = rf4.cache_read(p.cache, p.m, dtype=t.float32)
    assert rf4.device_error_bits() == 2 and rf4.device_error_bits() == 0
    tok = [(0, i) for i in range(20, 40)] + [(1, i) for i in range(20, 40)]
    bad = t.tensor([(b, i // 16) in ((0, 1), (1, 2)) for b, i in tok], device="cuda")
    assert bool((ko[bad] == 0).all()) and bool((ko[~bad] != 0).any())
    for b, c in ((0, 1), (1, 2)):
        assert t.equal(p.K[int(table[b, c])], old[int(table[b, c])])
    # a sequence longer than its row of the table
    p.table.copy_(table)
    p.lens[1] = 49
    rf4.cache_read(p.cache, p.m)
    assert rf4.device_error_bits() == 2


def test_captured_and_replayed_at_other_lengths():
    t = torch()
    p = pu.Paged([1, 1, 1], [40, 40, 40], 2, 64, 16, rf4.FAST)
    k = t.randn(3, 2, 64, generator=p.g, device="cuda")
    ko, vo = rf4.cache_read(p.cache, 3)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        rf4.rope_append(p.cache, None, k, k)
        rf4.cache_read(p.cache, k_out=ko, v_out=vo)
    for lens in ([7, 40, 1], [33, 2, 16]):
        k.copy_(t.randn(3, 2, 64, generator=p.g, device="cuda"))
        p.lens.copy_(t.tensor(lens, dtype=t.int32))
        g.replay()
        p.ts = lens
        blocks, _ = appended(p, "K")
        assert t.equal(ko.double(), pu.decode(blocks, rf4.FAST)) and t.equal(ko, vo)
        quantised_ok(blocks, k.double(), t.zeros_like(k.double()), rf4.FAST)


def test_refusals():
    t = torch()
    p = pu.Paged([2], [5], 2, 64, 16, rf4.DUAL)
    k = t.randn(2, 2, 64, device="cuda")
    freq, _ = rf4.rotary_frequencies(64)
    f66 = t.ones(33, device="cuda")
    bad = [lambda: rf4.rope_append(p.cache, None, k[:, :1], k), lambda: rf4.rope_append(p.cache, None, k, k.half()), lambda: rf4.rope_append(p.cache, k.half(), k, k),
           lambda: rf4.rope_append(p.cache, None, k.cpu(), k.cpu()), lambda: rf4.rope_append(p.cache, None, k, k, freq.double()),
           lambda: rf4.rope_append(p.cache, None, k, k, freq, positions=t.zeros(2, dtype=t.int64, device="cuda")), lambda: rf4.rope_append(p.cache, None, k.transpose(1, 2), k),
           lambda: rf4.rope_append(p.cache, None, k, k, q_out=k), lambda: rf4.cache_read(p.cache), lambda: rf4.cache_read(p.cache, k_out=k[:, :1]),
           lambda: rf4.cache_read(p.cache, 3, k_out=k), lambda: rf4.rotary(k, freq, t.zeros(3, dtype=t.int32, device="cuda")),
           lambda: rf4.PagedCache(p.K.view(-1)[:-1], p.V.view(-1)[:-1], p.table, p.lens, p.cu, kv_heads=2, head=64, page_size=16),
           lambda: rf4.PagedCache(p.K.view(-1), p.V.view(-1), p.table, p.lens, p.cu[:1], kv_heads=2, head=64, page_size=16),
           lambda: rf4.PagedCache(p.K.view(-1), p.V.view(-1), p.table.long(), p.lens, p.cu, kv_heads=2, head=64, page_size=16),
           lambda: rf4.PagedCache(p.K.view(-1), p.V.view(-1).cpu(), p.table, p.lens, p.cu, kv_heads=2, head=64, page_size=16)]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    with pytest.raises(rf4.RocmFP4Error):
        rf4.rope_append(p.cache, None, k, k, f66)
    with pytest.raises(rf4.RocmFP4Error):
        rf4.cache_read(p.cache, k_out=k.double())
