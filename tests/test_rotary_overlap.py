"""Outputs of rotary positions that share memory with the inputs are refused: the partners of a pair may be read after a value's
output was written.  On the CPU: every call below is refused before any pointer is used.  On the GPU: the calls next to them."""
import ctypes

import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gemm_rocmfp4_dequant_gb300 import build as lib_build

X = 1 << 20  # never dereferenced
M, H, D = 3, 4, 64


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return rf4.load()


def refused(L, status):
    return status == 1 and b"overlap" in L.rocmfp4_last_error()


@pytest.mark.parametrize("x_type,ld,offset", [(2, 256, 0), (1, 256, 0), (2, 400, 0), (2, 256, 8), (2, 256, -8), (2, 256, 3 * 256 * 2 - 8), (2, 256, -3 * 256 * 2 + 8),
                                              (0, 256, 0), (0, 256, 3 * 256 * 4 - 8), (0, 300, 2 * 300 * 4 + 1016), (2, (1 << 62) // 2, 1 << 40)])
def test_rotary(L, x_type, ld, offset):
    assert refused(L, L.rocmfp4_rotary(X, x_type, ld, 64, 64, D, 0, 1.0, X + offset, 0, M, H, D, None))


@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("rot", [64, 20, 0])
def test_append(L, which, rot):
    far = dict(q=2 * X, k=3 * X, v=4 * X)
    far[which] = X + 1528
    s = rf4._PagedCacheStruct(1 << 24, 1 << 24, 64, 64, 64, 2, 4, 4, 9, 16, 2, D, 0)
    assert refused(L, L.rocmfp4_rope_append(ctypes.addressof(s), far["q"], far["k"], far["v"], 2, 256, 128, 128, None, 64, rot, 0, 1.0, X, 0, M, H, None))


@pytest.mark.gpu
def test_neighbours_and_gaps_are_taken():
    """An output right before or behind the input's rows, and one token's, between the heads of its QKV row."""
    import __graft_entry__
    import torch as t
    __graft_entry__.build()
    rows = t.randn(3 * M, H, D, device="cuda").half()
    x = rows[M:2 * M]
    freq, _ = rf4.rotary_frequencies(24)
    pos = t.arange(M, dtype=t.int32, device="cuda")
    want = rf4.rotary(x, freq, pos)
    for out in (rows[:M], rows[2 * M:]):
        assert t.equal(rf4.rotary(x, freq, pos, out=out), want)
    for out in (x, rows[M - 1:2 * M - 1], rows[M + 1:2 * M + 1]):
        with pytest.raises(rf4.RocmFP4Error, match="overlap"):
            rf4.rotary(x, freq, pos, out=out)
    one = t.randn(1, 2 * H, D, device="cuda").half()
    want = rf4.rotary(one[:, :H], freq, pos[:1])
    assert t.equal(rf4.rotary(one[:, :H], freq, pos[:1], out=one[:, H:]), want)
    assert rf4.device_error_bits() == 0
