"""GPU tests of rocmfp4_logprobs on rows in which one token has nearly all of the probability, placed behind the first values
that a thread reads: a log probability is never above 0 and an entropy never below it.

Tolerances, from the arithmetic (u = 2^-24, half a unit of fp32 at 1): relative to the row's largest value the sum of the
exponentials is S = 1 + r, the 1 exact.  A term of r is off by at most 2^-21 of itself (two roundings of its exponent, the 2^x
instruction) and by what later sums add; S is rounded at most 10 times in a tile, once for each of at most 20 tiles, 10 times
where the threads join and 10 where the ranges do, by u S each, and ln S once more:
    |d logprob| <= 2^-17 r + 52 u,        below 2^-17 r + 2^-18;
the sum of e (z - m) has no term of the largest value, so
    |d entropy| <= 2^-16 H + 52 u,        below 2^-16 H + 2^-18."""
import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    assert rf4.device_error_bits() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,V", [(1, 131072), (3, 20000), (620, 20000), (620, 40001)])
@pytest.mark.parametrize("above", [4.0, 10.0, 15.0, 20.0, 23.14, 27.0, 27.7, 30.0, 40.0])
def test_signs_and_values(M, V, dtype, above):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(int(above * 100) + M)
    dt = getattr(t, dtype)
    z = t.randn(M, V, generator=g, device="cuda") * 0.25
    place = t.randint(0, V, (M,), generator=g, device="cuda")
    place[0] = V - 7
    if M > 1:
        place[1] = 0
    z.scatter_(1, place[:, None], above)
    z = z.to(dt)
    for n, scale in ((0, 1.0), (3, 1.0), (32, 0.85)):
        lp, ent, ids, top = rf4.logprobs(z, place.int(), top_n=n, scale=scale)
        assert bool((lp <= 0).all()) and bool((top <= 0).all()) and bool((ent >= 0).all())
        zs = z.double() * float(t.tensor(scale).float())
        zs = zs - zs.gather(1, place[:, None])
        rest = t.exp(zs).scatter(1, place[:, None], 0.0)
        r = rest.sum(1)
        ln = t.log1p(r)
        H = ln - (rest * zs).sum(1) / (1 + r)
        if above >= 10:
            assert float(zs.amax()) == 0.0
            assert bool(((lp.double() + ln).abs() <= 2.0 ** -17 * r + 2.0 ** -18).all())
            assert bool(((ent.double() - H).abs() <= 2.0 ** -16 * H + 2.0 ** -18).all())
            if n:
                assert t.equal(ids[:, 0].long(), place) and t.equal(top[:, 0], lp)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M", [2, 640])
def test_rising_rows(M, dtype):
    """Every tile has a larger value than those before it; the last is nearly certain."""
    t = torch()
    V = 24576
    z = (t.arange(V, device="cuda") // 2048).float()[None].repeat(M, 1) * 2.25
    z[:, V - 1] += 25.0
    z = z.to(getattr(t, dtype))
    target = t.full((M,), V - 1, dtype=t.int32, device="cuda")
    lp, ent, ids, top = rf4.logprobs(z, target, top_n=4)
    logp = t.log_softmax(z.double(), 1)
    H = -(logp.exp() * logp).sum(1)
    assert bool((lp <= 0).all()) and bool((top <= 0).all()) and bool((ent >= 0).all())
    r = -t.expm1(logp[:, -1])
    assert bool(((lp.double() - logp[:, -1]).abs() <= 2.0 ** -16 * r + 2.0 ** -18).all())
    assert bool(((ent.double() - H).abs() <= 2.0 ** -16 * H + 2.0 ** -18).all())


def test_certain_token():
    """Everything but one token masked, with -inf or with the least value: log probability 0, entropy 0, exactly."""
    t = torch()
    for low in (-float("inf"), t.finfo(t.float32).min):
        for M in (1, 620):
            z = t.full((M, 30000), low, device="cuda")
            z[:, 29000] = -3.5
            lp, ent, ids, top = rf4.logprobs(z, t.full((M,), 29000, dtype=t.int32, device="cuda"), top_n=1)
            assert bool((lp == 0).all()) and bool((ent == 0).all()) and bool((top == 0).all()) and bool((ids == 29000).all())
