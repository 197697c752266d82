"""GPU tests of calls on the first rows of a batch: a call of M rows below cu[B] gives what the whole batch's call gives its first
M rows, in each operator; the last sequence's rows keep the tokens that cu gives them."""
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


@pytest.mark.parametrize("ns,ts,rows", [([3, 6], [40, 300], 5), ([2, 5, 1], [9, 5, 70], 4), ([60, 200], [100, 700], 90), ([60, 200, 3], [100, 700, 5], 230), ([300], [300], 299)])
@pytest.mark.parametrize("window", [0, 20])
def test_the_first_rows_of_a_batch(ns, ts, rows, window):
    t = torch()
    p = pu.Paged(ns, ts, 2, 64, 16, rf4.DUAL, seed=rows)
    q = p.queries(4, t.float16)
    out = t.full((p.m, 4, 64), 3.0, dtype=t.float16, device="cuda")
    rf4.paged_attention(q[:rows], p.cache, 0.125, window=window, out=out[:rows])
    want, tol = p.attention(q, 0.125, True, window)
    off = (out[:rows].double() - want[:rows]).abs()
    assert bool((off <= tol[:rows] + pu.rounding(want[:rows], t.float16) * (1 + 2.0 ** -6)).all())
    assert bool((out[rows:] == 3.0).all())
    assert t.equal(rf4.cache_read(p.cache, rows)[0], rf4.cache_read(p.cache, p.m)[0][:rows])
    freq, _ = rf4.rotary_frequencies(64)
    kv = t.randn(p.m, 2, 64, generator=p.g, device="cuda").half()
    whole = rf4.rope_append(p.cache, q, kv, kv, freq)
    assert t.equal(rf4.rope_append(p.cache, q[:rows], kv[:rows], kv[:rows], freq), whole[:rows])
