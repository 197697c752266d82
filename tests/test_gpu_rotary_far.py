"""GPU tests of rotary positions with frequencies of two radians a token and more at the farthest positions, and with frequencies
that are no numbers.

The reference angle comes from integers of 400 bits (1 / 2 pi from arctangents).  The kernel's fraction of a turn is off by 2^-62
at most, the angle by 2^-31 of a turn at the farthest position, far below the sine's own 2^-23 (paged_util.turned's bound)."""
import math

import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import torch

pytestmark = pytest.mark.gpu
if torch().cuda.is_available():
    import paged_util as pu

SIZES = [2.0, -2.0000002, 3.1415927, 6.2831855, 100.0, -12345.678, 1e7, 16777215.0, 1.6777216e7, -3e7, 1e10, 1.8e19, -4e19, 1e26, 2.5e38, 3.4028235e38, 0.75, 1.9999999]
PLACES = [0, 1, -1, 3, 70001, 2 ** 24 + 1, -2 ** 30 - 7, 2 ** 31 - 1, -2 ** 31]
ONE = 1 << 400


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    assert rf4.device_error_bits() == 0


def turns_a_radian():
    def arctan(x):  # of 1 / x
        total = term = ONE // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total
    return ONE * ONE // (2 * 4 * (4 * arctan(5) - arctan(239)))


def angles(freq, places):
    t, unit = torch(), turns_a_radian()
    out = t.empty(len(places), freq.numel(), dtype=t.float64)
    for j, f in enumerate(freq.tolist()):
        m, e = math.frexp(f)
        m, e = int(m * 2 ** 24), e - 24
        for i, p in enumerate(places):
            x = m * p * unit
            x = x << e if e >= 0 else x >> -e
            out[i, j] = 2 * math.pi * ((x % ONE >> 340) / (1 << 60))
    return out.cuda()


@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (96, 96, False), (64, 36, False), (64, 64, True), (64, 6, True)])
def test_fast_frequencies_at_far_positions(D, rot, interleaved):
    t = torch()
    for shift in (0, 9):
        freq = t.tensor(((SIZES[shift:] + SIZES[:shift]) * 6)[:rot // 2], dtype=t.float32, device="cuda")
        pos = t.tensor(PLACES, dtype=t.int32, device="cuda")
        x = t.randn(len(PLACES), 3, D, generator=t.Generator(device="cuda").manual_seed(D + rot), device="cuda")
        got = rf4.rotary(x, freq, pos, interleaved=interleaved, dtype=t.float16)
        th = angles(freq, PLACES)
        c, s = th.cos()[:, None, :], th.sin()[:, None, :]
        want, size = x.double(), t.zeros_like(x, dtype=t.float64)
        a, b = (want[..., 0:rot:2], want[..., 1:rot:2]) if interleaved else (want[..., :rot // 2], want[..., rot // 2:rot])
        turned, both = (a * c - b * s, b * c + a * s), a.abs() + b.abs()
        for i in (0, 1):
            sl = slice(i, rot, 2) if interleaved else slice(i * (rot // 2), (i + 1) * (rot // 2))
            want[..., sl], size[..., sl] = turned[i], both
        assert bool(((got.double() - want).abs() <= size * 2.0 ** -21 + pu.rounding(want, t.float16) * (1 + 2.0 ** -6)).all())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 40, False), (64, 64, True), (96, 30, True)])
def test_frequencies_that_are_no_numbers(D, rot, interleaved, bad):
    """Their pairs are no numbers, at position 0 too (infinity times 0 is none); all others are as before.  Packed, such values
    count as 0."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(1)
    freq, _ = rf4.rotary_frequencies(rot)
    pos = t.tensor([0, 5, 100000], dtype=t.int32, device="cuda")
    x = t.randn(3, 2, D, generator=g, device="cuda")
    clean = rf4.rotary(x, freq, pos, interleaved=interleaved, dtype=t.bfloat16)
    i = rot // 2 - 2
    freq[i] = bad
    got = rf4.rotary(x, freq, pos, interleaved=interleaved, dtype=t.bfloat16)
    hit = t.zeros(D, dtype=t.bool, device="cuda")
    hit[[2 * i, 2 * i + 1] if interleaved else [i, i + rot // 2]] = True
    assert bool(got[..., hit].isnan().all()) and t.equal(got[..., ~hit], clean[..., ~hit])
    p = pu.Paged([3], [3], 2, D, 16, rf4.DUAL)
    rf4.rope_append(p.cache, None, x, x, freq, positions=pos, interleaved=interleaved)
    k, _ = rf4.cache_read(p.cache, 3, dtype=t.float32)
    assert bool((k[..., hit] == 0).all()) and bool((k[..., ~hit] != 0).any()) and bool(k.isfinite().all())
