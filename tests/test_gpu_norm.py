"""GPU tests of rocmfp4_add_rmsnorm against the formula in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, the rounding of fp32):
  * h = x + r is one fp32 addition: |dh| <= u |h|; stored in type t it is off by another eps(t) / 2 of itself;
  * the sum of squares has at most 32 additions in a thread and 37 across threads (5 in a warp, 32 warps), all of
    positive terms, so its relative error is below 72 u, half of which reaches 1 / sqrt(); rsqrtf, the division by D and
    the two products add less than 8 u.  Together, with room, 64 u = 2^-18 of |y|;
  * y in type t: eps(t) / 2 more (fp16 below 2^-14: half a subnormal step, 2^-25);
  * scales: 2^-18 and two roundings: below 2^-17 of themselves;
  * e4m3 codes: 2^-4 of the value (half of eps = 2^-3) or half a subnormal step (2^-10), and 2^-16 of the value for y and s.
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


def rows_of(t, M, D, dtype, pad, scale, g, offset=0):
    """[M, D] view with rows D + pad values apart, `offset` values into its buffer."""
    buf = t.zeros(M * (D + pad) + offset + 8, dtype=dtype, device="cuda")
    v = buf[offset:offset + M * (D + pad)].view(M, D + pad)[:, :D]
    v.copy_(t.randn(M, D, generator=g, device="cuda") * scale)
    return v


def check(out, x, r, w, eps, group):
    t = torch()
    h = x.double() + (r.double() if r is not None else 0.0)
    D = h.shape[1]
    ref = h / t.sqrt((h * h).sum(1, keepdim=True) / D + eps) * w.double()
    if r is not None:
        err = (out.residual.double() - h).abs()
        assert bool((err <= (t.finfo(out.residual.dtype).eps / 2 + 2.0 ** -23) * h.abs() + 2.0 ** -25).all())
    if out.y is not None:
        err = (out.y.double() - ref).abs()
        lim = (t.finfo(out.y.dtype).eps / 2 + 2.0 ** -18) * ref.abs() + 2.0 ** -25
        assert bool((err <= lim).all()), float((err - lim).max())
    if group:
        size = D if group < 0 else group
        parts = ref.split(size, dim=1)
        s = t.stack([p.abs().amax(1) for p in parts], 1) / 448.0
        assert out.scales.shape == s.shape
        assert bool(((out.scales.double() - s).abs() <= 2.0 ** -17 * s + 1e-45).all())
        each = t.cat([s[:, i:i + 1].expand(-1, p.shape[1]) for i, p in enumerate(parts)], 1)
        want = t.where(each > 0, ref / each.clamp(min=1e-300), t.zeros_like(ref))
        err = (out.q.float().double() - want).abs()
        assert bool((err <= (2.0 ** -4 + 2.0 ** -16) * want.abs() + 2.0 ** -10).all())


CASES = [(1, 1), (1, 8), (3, 31), (2, 64), (5, 100), (1, 1000), (4, 2049), (1, 5120), (9, 5120), (600, 40), (700, 257),
         (333, 5120), (2, 8192), (3, 8200), (1, 20000), (700, 8192), (1, 32768), (310, 32768)]


@pytest.mark.parametrize("M,D", CASES)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_matches_formula(M, D, pad):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(M * 100003 + D * 7 + pad)
    types = [t.float32, t.bfloat16, t.float16]
    w = None
    for k, xt in enumerate(types):
        rt = [t.bfloat16, None, t.float32, t.float16][(k + M + pad) % 4]
        x = rows_of(t, M, D, xt, pad, 2.0, g)
        r = rows_of(t, M, D, rt, pad, 30.0, g) if rt is not None else None
        w = (1 + 0.3 * t.randn(D, generator=g, device="cuda")).to(types[(k + 1) % 3])
        for group, yt in ((0, t.float16), (32, t.bfloat16), (64, None), (128, t.float16), (-1, None)):
            ro = t.empty(M, D, dtype=rt, device="cuda") if r is not None else None
            keep = r.clone() if r is not None else None
            out = rf4.add_rmsnorm(x, w, residual=r, eps=1e-6, dtype=yt, residual_out=ro, group=group)
            assert (out.y is None) == (yt is None) and (out.q is None) == (group == 0)
            check(out, x, r, w, 1e-6, group)
            if r is not None:
                assert t.equal(r, keep)  # the input residual is untouched
                first = out
                again = rf4.add_rmsnorm(x, w, residual=keep, eps=1e-6, dtype=yt, group=group)  # in place
                assert again.residual is keep and t.equal(keep, first.residual)
                assert (first.y is None or t.equal(first.y, again.y)) and (first.q is None or t.equal(first.scales, again.scales))


@pytest.mark.parametrize("M,D", [(1217, 1024), (1300, 2056), (1999, 5120), (2500, 8192), (1217, 12288), (1400, 16384)])
@pytest.mark.parametrize("pad", [0, 16])
def test_many_wide_rows(M, D, pad):
    """Rows enough for the persistent form (and too wide for it in some types), every pair of types, in place as well."""
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(M + D + pad)
    types = [t.float32, t.bfloat16, t.float16]
    w = (1 + 0.3 * t.randn(D, generator=g, device="cuda")).bfloat16()
    for k, xt in enumerate(types):
        x = rows_of(t, M, D, xt, pad, 2.0, g)
        for rt in [None] + types:
            r = rows_of(t, M, D, rt, pad, 30.0, g) if rt is not None else None
            group, yt = [(0, t.float16), (128, None), (-1, t.bfloat16), (32, t.float16)][(k + (types.index(rt) if rt else 3)) % 4]
            ro = t.empty(M, D, dtype=rt, device="cuda") if r is not None else None
            out = rf4.add_rmsnorm(x, w, residual=r, dtype=yt, residual_out=ro, group=group)
            check(out, x, r, w, 1e-6, group)
            if r is not None:
                again = rf4.add_rmsnorm(x, w, residual=r, dtype=yt, group=group)
                assert again.residual is r and t.equal(r, out.residual)
                assert (out.y is None or t.equal(out.y, again.y)) and (out.q is None or t.equal(out.q.view(t.uint8), again.q.view(t.uint8)))


@pytest.mark.parametrize("xoff,D", [(1, 512), (3, 514), (8, 512)])
def test_unaligned_pointers(xoff, D):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(xoff)
    x = rows_of(t, 7, D, t.bfloat16, 0, 1.0, g, offset=xoff)
    r = rows_of(t, 7, D, t.float32, 0, 3.0, g, offset=xoff)
    w = t.ones(D + 1, dtype=t.float16, device="cuda")[1:]
    out = rf4.add_rmsnorm(x, w, residual=r, residual_out=t.empty(7, D, device="cuda"), dtype=t.bfloat16, group=32)
    check(out, x, r, w, 1e-6, 32)


def test_writes_stay_inside():
    """Guard values around every output stay as they were, at a ragged width."""
    t = torch()
    M, D = 5, 203
    x = t.randn(M, D, device="cuda")
    w = t.ones(D, device="cuda", dtype=t.bfloat16)
    big_y = t.full((M * D + 64,), 7.0, dtype=t.float16, device="cuda")
    big_r = t.full((M, D + 5), 7.0, dtype=t.float32, device="cuda")
    big_q = t.full((M * D + 64,), 7.0, device="cuda").to(t.float8_e4m3fn)
    big_s = t.full((M * 7 + 32,), 7.0, device="cuda")
    rf4.add_rmsnorm(x, w, residual=t.zeros(M, D, device="cuda"), y=big_y[32:32 + M * D].view(M, D), residual_out=big_r[:, :D],
                    q=big_q[16:16 + M * D].view(M, D), scales=big_s[16:16 + M * 7].view(M, 7), group=32)
    assert bool((big_y[:32] == 7).all()) and bool((big_y[32 + M * D:] == 7).all()) and bool((big_r[:, D:] == 7).all())
    assert bool((big_q.float()[:16] == 7).all()) and bool((big_q.float()[16 + M * D:] == 7).all())
    assert bool((big_s[:16] == 7).all()) and bool((big_s[16 + M * 7:] == 7).all())


def test_zeros_infinities_and_nan():
    t = torch()
    D = 96
    x = t.randn(5, D, device="cuda")
    x[1] = 0.0
    x[2, 5] = float("inf")
    x[3, 40] = float("nan")
    x[4] *= 1e-30  # eps decides: values far below the least fp16
    w = t.ones(D, device="cuda", dtype=t.bfloat16)
    out = rf4.add_rmsnorm(x, w, dtype=t.bfloat16, group=32)
    assert bool((out.y[1] == 0).all()) and bool((out.scales[1] == 0).all()) and bool((out.q.float()[1] == 0).all())
    y2 = out.y[2].float()
    assert bool(y2[5].isnan()) and int(y2.isnan().sum()) == 1 and float(y2.nan_to_num().abs().max()) == 0.0
    assert bool(out.y[3].isnan().all()) and bool(out.scales[3].isnan().all()) and bool(out.q.float()[3].isnan().all())
    assert bool(out.scales[2, 0].isnan()) and bool((out.scales[2, 1:] == 0).all())
    check(rf4.AddRmsNorm(out.y[[0, 4]], None, out.q[[0, 4]], out.scales[[0, 4]]), x[[0, 4]], None, w, 1e-6, 32)


def test_graph_capture_and_other_stream():
    t = torch()
    x = t.randn(3, 640, device="cuda")
    r = t.randn(3, 640, device="cuda").to(t.bfloat16)
    w = t.ones(640, device="cuda", dtype=t.bfloat16)
    y, ro = t.empty(3, 640, dtype=t.float16, device="cuda"), t.empty_like(r)
    rf4.add_rmsnorm(x, w, residual=r, y=y, residual_out=ro)
    want = y.clone()
    t.cuda.synchronize()
    s = t.cuda.Stream()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=s):
        rf4.add_rmsnorm(x, w, residual=r, y=y, residual_out=ro)
    y.zero_()
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(y, want)
    y.zero_()
    t.cuda.synchronize()
    rf4.add_rmsnorm(x, w, residual=r, y=y, residual_out=ro, stream=s)
    s.synchronize()
    assert t.equal(y, want)


def test_refusals():
    t = torch()
    x = t.randn(2, 64, device="cuda")
    w = t.ones(64, device="cuda")
    for kw in (dict(group=48), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(rf4.RocmFP4Error):
            rf4.add_rmsnorm(x, w, **kw)
    with pytest.raises(rf4.RocmFP4Error):
        rf4.add_rmsnorm(x.double(), w)
    with pytest.raises(rf4.RocmFP4Error):
        rf4.add_rmsnorm(t.zeros(1, 32800, device="cuda"), t.ones(32800, device="cuda"))
    for kw in (dict(residual=t.zeros(2, 32, device="cuda")), dict(residual_out=x), dict(q=x), dict(y=t.zeros(1, 64, device="cuda"))):
        with pytest.raises(ValueError):
            rf4.add_rmsnorm(x, w, **kw)
    with pytest.raises(ValueError):
        rf4.add_rmsnorm(x.t(), w)
    empty = rf4.add_rmsnorm(x[:0], w)
    assert empty.y.shape == (0, 64)
    assert np.isfinite(rf4.add_rmsnorm(x[0], w).y.cpu().numpy().astype(np.float64)).all()
