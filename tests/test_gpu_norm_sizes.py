"""GPU tests of rocmfp4_add_rmsnorm on matrices of more than 2^31 values: the last rows lie past 32-bit offsets in x, the
residual, y, the codes and the scales.  Rows are compared with the same rows in a matrix of their own (each row's result does
not depend on the others), and those with the formula; the tolerances are those of the norm's other tests."""
import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import torch
from test_gpu_norm import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    assert rf4.device_error_bits() == 0


@pytest.mark.parametrize("D,group", [(5120, 128), (5119, 32), (40, 32)])
def test_offsets_past_31_bits(D, group):
    """Persistent CTAs, a CTA a row, several rows a CTA."""
    t = torch()
    M = (1 << 31) // D + 700
    g = t.Generator(device="cuda")
    g.manual_seed(D)
    x = t.empty(M, D, dtype=t.bfloat16, device="cuda").normal_(0.0, 2.0, generator=g)
    r = t.empty(M, D, dtype=t.bfloat16, device="cuda").normal_(0.0, 30.0, generator=g)
    w = (1 + 0.3 * t.randn(D, generator=g, device="cuda")).bfloat16()
    keep = r[-5:].clone(), r[:5].clone()
    out = rf4.add_rmsnorm(x, w, residual=r, dtype=t.bfloat16, group=group)
    assert out.y.numel() > 1 << 31 and out.residual is r
    for rows, res in ((slice(-5, None), keep[0]), (slice(0, 5), keep[1])):
        part = rf4.AddRmsNorm(out.y[rows], out.residual[rows], out.q[rows], out.scales[rows])
        check(part, x[rows], res, w, 1e-6, group)
    m = M - 600
    assert bool((out.y[m:].float().abs().amax(1) > 0).all()) and bool((out.scales[m:] > 0).all())
