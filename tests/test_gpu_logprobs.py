"""GPU tests of rocmfp4_logprobs against the definitions in 64 bits.

Tolerances, from the arithmetic (u = 2^-24): a term exp(z - m) carries the error of two roundings of its exponent and of
the 2^x instruction, at most 2^-21 (x exp(-x) is below 0.4); a sum of them has at most 16 additions in a tile, one per
tile (at most 60 here), 5 + 8 joins in the CTA and as many between ranges: below 2^-17 in all, and so is the error of
ln S.  So
    |d logprob| <= 2^-16 + 2^-22 (|logprob| + |z - m|),
    |d entropy| <= 2^-16 (1 + x) + 2^-22 entropy,  x = sum p (m - z).
Token indices and their order are exact.
"""
import numpy as np
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


def check(z, targets, n, scale, got):
    """z: [M, V] on the GPU, as given to the call."""
    t = torch()
    lp, ent, ids, top = (None if o is None else o.cpu().double() for o in got)
    raw = z.cpu().double()
    zs = raw * float(np.float32(scale))
    order = t.sort(raw, dim=1, descending=True, stable=True)[1][:, :n]
    assert t.equal(ids.long(), order)
    m = zs.amax(1, keepdim=True)
    none = m[:, 0] == -np.inf
    m = t.where(none[:, None], t.zeros_like(m), m)
    d = zs - m
    e = t.exp(d)
    ln = t.log(e.sum(1, keepdim=True))
    x = -t.where(e > 0, e * d, t.zeros_like(e)).sum(1) / e.sum(1)

    def close(a, b, lim):
        inf = t.isinf(b)
        assert t.equal(a[inf], b[inf])
        assert bool(((a - b).abs()[~inf] <= lim[~inf]).all()), float(((a - b).abs()[~inf] - lim[~inf]).max())

    ref = t.where(none[:, None], t.full_like(d, -np.inf), d - ln)
    big = t.where(t.isinf(ref.float()), t.full_like(ref, -np.inf), ref)  # what fp32 rounds to -inf
    if targets is not None:
        at = targets.cpu().long()[:, None]
        r, dd = big.gather(1, at)[:, 0], d.gather(1, at)[:, 0].abs()
        close(lp, r, 2.0 ** -16 + 2.0 ** -22 * (r.abs() + dd))
    r, dd = big.gather(1, order), d.gather(1, order).abs()
    close(top, r, 2.0 ** -16 + 2.0 ** -22 * (r.abs() + dd))
    h = t.where(none, t.zeros_like(x), ln[:, 0] + x)
    close(ent, h, 2.0 ** -16 * (1 + t.where(none, t.zeros_like(x), x)) + 2.0 ** -22 * h.abs())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (2, 5), (4, 33), (1, 257), (3, 1000), (2, 4097), (5, 16384), (1, 50257), (2, 152064), (650, 1031)])
def test_matches_definition(M, V, dtype):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(M * 1000003 + V)
    for off, pad in ((0, 0), (1, 3), (5, 8)):
        buf = t.empty(M * (V + pad) + off + 16, device="cuda", dtype=getattr(t, dtype))
        buf.normal_(0.0, 4.0, generator=g)
        z = buf[off:off + M * (V + pad)].view(M, V + pad)[:, :V]
        targets = t.randint(0, V, (M,), generator=g, device="cuda").int()
        for n in sorted({0, 1, min(V, 5), min(V, 32)}):
            for scale in (1.0, 0.7):
                check(z, targets, n, scale, rf4.logprobs(z, targets, top_n=n, scale=scale))


def special(t, V, dtype, kind, g):
    z = t.randn(1, V, generator=g, device="cuda") * 3
    if kind == "constant":
        z[:] = 1.25
    elif kind == "rising":
        z = t.linspace(-60, 60, V, device="cuda")[None]
    elif kind == "falling":
        z = t.linspace(60, -60, V, device="cuda")[None]
    elif kind == "two values":
        z = (z > 0).float()
    elif kind == "masked but three":
        keep = t.randint(0, V, (3,), generator=g, device="cuda")
        w = t.full_like(z, -np.inf)
        w[0, keep] = z[0, keep]
        z = w
    elif kind == "masked":
        z[:] = -np.inf
    elif kind == "lowest":
        z[:] = t.finfo(dtype).min
    elif kind == "lowest but one":
        z[:] = t.finfo(dtype).min
        z[0, V // 2] = 3.0
    elif kind == "zeros of both signs":
        z[:] = 0.0
        z[0, ::3] = -0.0
    elif kind == "spike":
        z[0, V - 1] = 80.0
    elif kind == "rising tiles":
        z = z + t.arange(V, device="cuda")[None] // 997 * 4.0
    return z.to(dtype)


KINDS = ["constant", "rising", "falling", "two values", "masked but three", "masked", "lowest", "lowest but one",
         "zeros of both signs", "spike", "rising tiles"]


@pytest.mark.parametrize("V", [40, 3001, 20000])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("copies", [1, 700])
def test_special_rows(V, dtype, copies):
    """Rows that fill the candidate list, tie or leave nothing: shared by several CTAs (few rows) and by one each (many)."""
    t = torch()
    if copies > 1 and V > 3001:
        copies = 620
    g = t.Generator(device="cuda")
    g.manual_seed(V)
    dt = getattr(t, dtype)
    z = t.cat([special(t, V, dt, k, g) for k in KINDS])
    z = z.repeat(-(-copies // len(KINDS)), 1).contiguous()
    targets = t.randint(0, V, (z.shape[0],), generator=g, device="cuda").int()
    for n in (0, 7, 32):
        got = rf4.logprobs(z, targets, top_n=n, scale=1.0)
        check(z, targets, n, 1.0, got)
        again = rf4.logprobs(z, targets, top_n=n, scale=1.0)
        assert all(t.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M", [1, 620])
@pytest.mark.parametrize("off", [0, 3])
def test_large_values_in_few_places(M, dtype, off):
    """Every large value of a row where a few threads read: more candidates than the list holds."""
    t = torch()
    V = 20000
    g = t.Generator(device="cuda")
    g.manual_seed(M + off)
    dt = getattr(t, dtype)
    per = 16 // dt.itemsize
    buf = t.rand(M * V + 16, generator=g, device="cuda").to(dt)
    z = buf[off:off + M * V].view(M, V)
    place = (t.arange(V, device="cuda") + off) // per % 256
    for n in (5, 20, 32):
        large = (place % 8 == 0) & (place < 8 * (n - 1))
        w = (z.float() + 20 * large).to(dt)
        buf2 = t.empty_like(buf)
        row = buf2[off:off + M * V].view(M, V)
        row.copy_(w)
        targets = t.randint(0, V, (M,), generator=g, device="cuda").int()
        check(row, targets, n, 1.0, rf4.logprobs(row, targets, top_n=n))


@pytest.mark.parametrize("M", [1, 620])
def test_rows_with_many_nan(M):
    """NaN ranks as the largest value, the lowest index first."""
    t = torch()
    z = t.randn(M, 9001, device="cuda")
    z[:, 5::3] = float("nan")
    z[M // 2:, :] = float("nan")
    z[M // 2:, 8] = 1.0
    _, _, ids, _ = rf4.logprobs(z, None, top_n=12)
    first = t.tensor([list(range(5, 41, 3))], device="cuda", dtype=t.int32)
    rest = t.tensor([[0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11, 12]], device="cuda", dtype=t.int32)
    assert t.equal(ids, t.cat([first.expand(M // 2, -1), rest.expand(M - M // 2, -1)]))


def test_nan_and_infinity():
    t = torch()
    z = t.randn(3, 5000, device="cuda")
    z[0, 77] = float("inf")
    z[0, 4000] = float("inf")
    z[1, 4321] = float("nan")
    targets = t.tensor([77, 3, 5], dtype=t.int32, device="cuda")
    lp, ent, ids, top = rf4.logprobs(z, targets, top_n=4)
    assert bool(lp[:2].isnan().all()) and bool(ent[:2].isnan().all()) and bool(top[:2].isnan().all())
    assert ids[0, :2].tolist() == [77, 4000] and int(ids[1, 0]) == 4321
    rest = t.sort(z[1].nan_to_num(-100.0), descending=True, stable=True)[1][:3]
    assert ids[1, 1:].tolist() == rest.tolist()
    check(z[2:], targets[2:], 4, 1.0, tuple(o[2:] for o in (lp, ent, ids, top)))


def test_targets_outside_and_absent():
    t = torch()
    z = t.randn(4, 300, device="cuda")
    lp, ent, ids, top = rf4.logprobs(z, t.tensor([-1, 300, 2 ** 31 - 1, 299], dtype=t.int32, device="cuda"), top_n=2)
    assert bool(lp[:3].isnan().all()) and bool(lp[3].isfinite())
    none, ent2, ids2, top2 = rf4.logprobs(z, top_n=2)
    assert none is None and t.equal(ent, ent2) and t.equal(ids, ids2) and t.equal(top, top2)


def test_offsets_past_32_bits():
    """The last row of a matrix of more than 2^32 values."""
    t = torch()
    M, V = 28300, 152064
    z = t.zeros(M, V, dtype=t.float16, device="cuda")
    z[-1, 9] = 4.0
    z[-1, 150000] = 5.0
    targets = t.full((M,), 9, dtype=t.int32, device="cuda")
    got = rf4.logprobs(z, targets, top_n=3)
    check(z[-1:], targets[-1:], 3, 1.0, tuple(o[-1:] for o in got))
    check(z[:1], targets[:1], 3, 1.0, tuple(o[:1] for o in got))


def test_graph_capture():
    t = torch()
    z = t.randn(2, 30000, device="cuda")
    targets = t.tensor([5, 6], dtype=t.int32, device="cuda")
    want = rf4.logprobs(z, targets, top_n=6)
    out = tuple(t.empty_like(o) for o in want)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        rf4.logprobs(z, targets, top_n=6, logprob=out[0], entropy=out[1], top_ids=out[2], top_logprobs=out[3])
    for _ in range(3):
        graph.replay()
    t.cuda.synchronize()
    assert all(t.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    t = torch()
    z = t.randn(2, 64, device="cuda")
    for kw in (dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(top_n=33), dict(top_n=65)):
        with pytest.raises(rf4.RocmFP4Error):
            rf4.logprobs(z, **kw)
    with pytest.raises(rf4.RocmFP4Error):
        rf4.logprobs(z.double())
    with pytest.raises(ValueError):
        rf4.logprobs(z, t.zeros(2, dtype=t.int64, device="cuda"))
    with pytest.raises(ValueError):
        rf4.logprobs(z.t())
    with pytest.raises(ValueError):
        rf4.logprobs(z, logprob=t.zeros(2, device="cuda"))
    assert rf4.logprobs(z[:0], top_n=3)[2].shape == (0, 3)
