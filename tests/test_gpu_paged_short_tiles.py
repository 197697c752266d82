"""GPU tests of attention over many short sequences: row tiles of one token tile one after the other in every block, alone and
between row tiles of two halves and of several token tiles.  The bound is that of the attention tests (paged_util.Paged.attention
and half a step of the output's type)."""
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


@pytest.mark.parametrize("D,variant,name", [(64, rf4.DUAL, "f16"), (128, rf4.FAST, "bf16"), (128, rf4.DUAL, "f16")])
@pytest.mark.parametrize("kind", ["one token tile", "one, two halves", "one, several"])
def test_short_row_tiles_one_after_the_other(D, variant, name, kind):
    t = torch()
    dtype = {"f16": t.float16, "bf16": t.bfloat16}[name]
    ns = [17 + i % 24 for i in range(500)]
    ts = [n + i % (129 - n) for i, n in enumerate(ns)]
    if kind == "one, two halves":
        for i in range(5, 500, 9):
            ns[i], ts[i] = 150 + i % 40, 300 + i
    elif kind == "one, several":
        for i in range(3, 500, 7):
            ts[i] = 129 + 3 * i
    p = pu.Paged(ns, ts, 4, D, 16, variant, seed=D)
    q = p.queries(4, dtype)
    out = rf4.paged_attention(q, p.cache, D ** -0.5)
    want, tol = p.attention(q, D ** -0.5)
    assert bool(((out.double() - want).abs() <= tol + pu.rounding(want, dtype) * (1 + 2.0 ** -6)).all())
    for _ in range(20):
        assert t.equal(rf4.paged_attention(q, p.cache, D ** -0.5), out)
