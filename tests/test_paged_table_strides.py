"""Page tables of any row stride: what PagedCache hands on (CPU, with stand-ins for CUDA tensors that have a shape, strides and an
address), what the C entry points take (CPU), and the operators over an expanded table against a written-out one (GPU)."""
import ctypes

import pytest
import torch

import gemm_rocmfp4_dequant_gb300 as rf4
from gemm_rocmfp4_dequant_gb300 import build as lib_build


class OnGpu:
    """A CPU tensor that says that it lies on a GPU."""

    def __init__(self, t):
        self._t, self.is_cuda, self.device = t, True, torch.device("cuda", 0)

    def __getattr__(self, name):
        return getattr(self._t, name)


def cache_of(table, B):
    lib_build.build()
    pages = OnGpu(torch.zeros(4 * 16 * 36, dtype=torch.uint8))
    ints = [OnGpu(torch.zeros(n, dtype=torch.int32)) for n in (B, B + 1)]
    return rf4.PagedCache(pages, pages, OnGpu(table), *ints, kv_heads=1, head=64, page_size=16)


@pytest.mark.parametrize("B,shape,make,stride", [
    (3, (3, 4), lambda: torch.zeros(3, 4, dtype=torch.int32), 4),
    (3, (3, 4), lambda: torch.zeros(3, 9, dtype=torch.int32)[:, :4], 9),
    (3, (3, 4), lambda: torch.zeros(1, 4, dtype=torch.int32).expand(3, -1), 0),
    (3, (3, 4), lambda: torch.zeros(4, dtype=torch.int32).as_strided((3, 4), (0, 1)), 0),
    (3, (3, 1), lambda: torch.zeros(1, 1, dtype=torch.int32).expand(3, -1), 0),
    (3, (3, 1), lambda: torch.zeros(3, 1, dtype=torch.int32), 1),
    (3, (3, 1), lambda: torch.zeros(3, 7, dtype=torch.int32)[:, 2:3], 7),
    (1, (1, 4), lambda: torch.zeros(4, dtype=torch.int32).as_strided((1, 4), (0, 1)), 4),
    (3, (3, 0), lambda: torch.zeros(3, 0, dtype=torch.int32), 0),
    (0, (0, 4), lambda: torch.zeros(0, 4, dtype=torch.int32), 4),
])
def test_the_table_s_own_stride(B, shape, make, stride):
    table = make()
    assert table.shape == shape
    s = cache_of(table, B)._struct
    assert (s.table_width, s.table_stride) == (shape[1], stride)
    # no row's last number lies behind the tensor's memory
    if B and shape[1]:
        assert (B - 1) * s.table_stride + s.table_width <= table.untyped_storage().nbytes() // 4 - table.storage_offset()


@pytest.mark.parametrize("step", [1, 2, 3])
def test_overlapping_rows_are_refused(step):
    with pytest.raises(ValueError, match="overlap"):
        cache_of(torch.zeros(12, dtype=torch.int32).as_strided((3, 4), (step, 1)), 3)


def test_strides_at_the_c_entry():
    lib_build.build()
    L = rf4.load()

    def call(stride, width):  # nothing to do: M = 0
        s = rf4._PagedCacheStruct(0x10000, 0x10000, 0x10000, 0x10000, 0x10000, 2, width, stride, 9, 16, 2, 64, 0)
        return L.rocmfp4_cache_read(ctypes.addressof(s), 0x10000, 0x10000, 0, 0, None)
    assert [call(s, 4) for s in (0, 4, 5)] == [0, 0, 0]
    assert [call(s, 4) for s in (1, 3, -1, -4)] == [1, 1, 1, 1]
    assert call(0, 0) == 0 and call(-1, 0) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("ns", [[1, 1, 1], [40, 3, 150]])
def test_one_row_of_pages_for_all_sequences(ns):
    """Beams over one encoder's states; every result is bitwise that of the table written out, row by row."""
    import __graft_entry__
    import paged_util as pu
    __graft_entry__.build()
    t = torch
    p = pu.Paged([0], [700], 2, 64, 16, rf4.DUAL, seed=3)
    lens = t.tensor([700, 333, 17], dtype=t.int32, device="cuda")
    cu = t.tensor([0, ns[0], ns[0] + ns[1], sum(ns)], dtype=t.int32, device="cuda")
    q = t.randn(sum(ns), 6, 64, device="cuda").half()
    got = []
    for table in (p.table.expand(3, -1), p.table.repeat(3, 1)):
        cache = rf4.PagedCache(p.K.view(-1), p.V.view(-1), table, lens, cu, kv_heads=2, head=64, page_size=16)
        got.append((rf4.paged_attention(q, cache, 0.125, causal=False), *rf4.cache_read(cache, sum(ns))))
    assert rf4.device_error_bits() == 0
    for a, b in zip(*got):
        assert t.equal(a, b) and bool(a.any())
