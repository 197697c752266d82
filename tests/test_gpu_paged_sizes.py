"""GPU tests of the paged cache's operators where their ways of working change: rows around the choice between the two
attention kernels, tokens of few blocks read back four a warp, frequencies of any size."""
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


@pytest.mark.parametrize("variant", [rf4.DUAL, rf4.FAST])
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("ns,ts,H,hkv,D,page,causal,window", [
    ([16, 16], [300, 16], 2, 2, 64, 16, True, 0),                     # 16 rows each: tiles of eight
    ([16, 17], [300, 17], 2, 2, 64, 16, True, 0),                     # one more: tiles of 128
    ([4, 4, 4], [131, 4, 900], 8, 2, 128, 48, True, 0),               # 16 rows of four heads
    ([1], [1000], 16, 1, 128, 32, True, 0),                           # a token of 16 heads
    ([64, 0, 0, 0], [2000, 5, 0, 70], 3, 3, 128, 64, True, 0),        # one long chunk among waiting sequences
    ([3, 5, 1, 2], [50, 333, 97, 2], 6, 2, 64, 16, True, 33),         # windows that begin inside a page and a chunk
    ([9, 1], [40, 129], 1, 1, 128, 16, True, 1),                      # rows that see themselves alone
    ([7, 12], [65, 31], 4, 4, 64, 32, False, 0),                      # more queries than a tile, all tokens
])
def test_rows_around_the_choice_of_kernel(variant, name, ns, ts, H, hkv, D, page, causal, window):
    """The bound is that of the attention tests: paged_util.Paged.attention and half a step of the output's type."""
    t = torch()
    dtype = {"f16": t.float16, "bf16": t.bfloat16}[name]
    p = pu.Paged(ns, ts, hkv, D, page, variant, seed=7, extra=3)
    q = p.queries(H, dtype, pad=2)
    out = t.full((p.m + 2, H, D), 3.0, dtype=dtype, device="cuda")
    rf4.paged_attention(q, p.cache, D ** -0.5, causal=causal, window=window, out=out)
    want, tol = p.attention(q[:p.m], D ** -0.5, causal, window)
    assert bool(((out[:p.m].double() - want).abs() <= tol + pu.rounding(want, dtype) * (1 + 2.0 ** -6)).all())
    assert bool((out[p.m:] == 3.0).all())


@pytest.mark.parametrize("variant", [rf4.DUAL, rf4.FAST])
@pytest.mark.parametrize("D,hkv,page", [(32, 1, 16), (64, 1, 48), (96, 1, 64), (160, 1, 16), (128, 3, 32)])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_many_rows_of_few_blocks_read_back(variant, D, hkv, page, name):
    """Exact, at counts that leave the last warps and blocks of a token unfilled; rows that are no tokens of the call stay."""
    t = torch()
    dtype = {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[name]
    ts = [7001, 1, 6003, 0, 6999]
    p = pu.Paged(ts, ts, hkv, D, page, variant, seed=D)
    ahead, behind = 3, 2
    cache = rf4.PagedCache(p.K.view(-1), p.V.view(-1), p.table, p.lens, p.cu + ahead, kv_heads=hkv, head=D, page_size=page, variant=variant)
    k, v = (t.full((p.m + ahead + behind, hkv, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    rf4.cache_read(cache, k_out=k, v_out=v)
    alone = t.full_like(v, 3.0)
    rf4.cache_read(cache, v_out=alone)
    for got, which in ((k, "K"), (v, "V"), (alone, "V")):
        want = t.cat([p.tokens(which, b, 0, T)[0] for b, T in enumerate(ts) if T])
        assert t.equal(got[ahead:ahead + p.m].double(), want)
        assert bool((got[:ahead] == 3.0).all()) and bool((got[ahead + p.m:] == 3.0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 192])
def test_frequencies_of_any_size(D, interleaved):
    """Angles by integers of 300 bits.  Below 2 radians a token a fraction of a turn is off by 2^-62 at most, by 2^-31 at the
    farthest position; above, by fp64's 2^-52 of it.  Both are far below the sine's own 2^-23 (paged_util.turned)."""
    t = torch()
    one = 1 << 340

    def arctan(x):  # of 1 / x
        total = term = one // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total
    pi = 4 * (4 * arctan(5) - arctan(239))
    per_turn = one * one // (2 * pi)  # 1 / 2 pi, in units of 1 / one
    for sizes, places in (([1e-38, 1e-30, 1e-7, 0.0, 0.3, -0.7, 1.0, -1.0, 1.9999999, 2.0 ** -24], [0, 1, 2, 77777, 2 ** 31 - 1]),
                          ([2.0, -2.5, 3.1415927, 6.2831855, 100.0, -1e4, 0.5, 1.5], [0, 1, 3, 1000])):
        freq = t.tensor((sizes * D)[:D // 2], dtype=t.float32, device="cuda")
        pos = t.tensor(places, dtype=t.int32, device="cuda")
        g = t.Generator(device="cuda").manual_seed(D)
        x = t.randn(len(places), 3, D, generator=g, device="cuda")
        got = rf4.rotary(x, freq, pos, interleaved=interleaved, dtype=t.float16)
        angle = t.empty(len(places), D // 2, dtype=t.float64)
        for i, p in enumerate(places):
            for j, f in enumerate(freq.tolist()):
                m, e = math.frexp(f)
                m, e = int(m * 2 ** 24), e - 24
                turns = m * p * per_turn  # times 2^e / one
                unit = one << -e if e < 0 else one >> e
                angle[i, j] = 2 * math.pi * ((turns % unit) / unit)
        c, s = angle.cos()[:, None, :].cuda(), angle.sin()[:, None, :].cuda()
        xd = x.double()
        a, b = (xd[..., 0::2], xd[..., 1::2]) if interleaved else (xd[..., :D // 2], xd[..., D // 2:])
        want, size = t.empty_like(xd), t.empty_like(xd)
        for i, y in enumerate((a * c - b * s, b * c + a * s)):
            sl = slice(i, None, 2) if interleaved else slice(i * (D // 2), (i + 1) * (D // 2))
            want[..., sl], size[..., sl] = y, a.abs() + b.abs()
        assert bool(((got.double() - want).abs() <= size * 2.0 ** -21 + pu.rounding(want, t.float16) * (1 + 2.0 ** -6)).all())
