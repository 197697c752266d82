"""CPU tests of the argument checks of rocmfp4_rotary, rocmfp4_rope_append, rocmfp4_cache_read and rocmfp4_paged_attention
(every call below is refused on the host, or has nothing to do, before any pointer is used), and of rotary_frequencies."""
import ctypes
import math

import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gemm_rocmfp4_dequant_gb300 import build as lib_build

INVALID, UNSUPPORTED = 1, 2
PTR = 0x10000  # never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return rf4.load()


CACHE = dict(K=PTR, V=PTR, table=PTR, lens=PTR, cu=PTR, B=2, table_width=4, table_stride=4, num_pages=9, page_size=16, Hkv=2, D=64, variant=0)
BAD_CACHE = [(dict(variant=2), INVALID), (dict(B=-1), INVALID), (dict(table_width=-1), INVALID), (dict(num_pages=-1), INVALID), (dict(Hkv=0), INVALID),
             (dict(D=0), INVALID), (dict(D=48), INVALID), (dict(page_size=0), INVALID), (dict(table_stride=3), INVALID), (dict(cu=None), INVALID),
             (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(cu=PTR + 2), INVALID),
             (dict(lens=PTR + 1), INVALID), (dict(table=PTR + 3), INVALID), (dict(K=PTR + 8), UNSUPPORTED), (dict(V=PTR + 2), UNSUPPORTED),
             (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(D=288), UNSUPPORTED), (dict(num_pages=1 << 31), UNSUPPORTED),
             (dict(B=1 << 31), UNSUPPORTED), (dict(table_width=1 << 28, table_stride=1 << 28), UNSUPPORTED), (dict(Hkv=65537), UNSUPPORTED)]


def split(kw):
    c = dict(CACHE)
    c.update({k[2:]: v for k, v in kw.items() if k.startswith("c_")})
    s = rf4._PagedCacheStruct(*c.values())
    return s, {k: v for k, v in kw.items() if not k.startswith("c_")}


def append(L, **kw):
    s, kw = split(kw)
    a = dict(cache=ctypes.addressof(s), q=PTR, k=PTR, v=PTR, type=0, ldq=256, ldk=128, ldv=128, positions=None, freq=PTR, rot=64, interleaved=0, amplitude=1.0,
             q_out=PTR, q_type=0, M=3, H=4, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.rocmfp4_rope_append(*a.values())


def read(L, **kw):
    s, kw = split(kw)
    a = dict(cache=ctypes.addressof(s), k_out=PTR, v_out=PTR, type=0, M=3, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.rocmfp4_cache_read(*a.values())


def attend(L, **kw):
    s, kw = split(kw)
    a = dict(q=PTR, ldq=256, cache=ctypes.addressof(s), out=PTR, M=3, H=4, scale=0.1, causal=1, window=0, act=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.rocmfp4_paged_attention(*a.values())


def rotary(L, **kw):
    a = dict(x=PTR, x_type=0, ldx=256, positions=PTR, freq=PTR, rot=64, interleaved=0, amplitude=1.0, y=PTR, y_type=0, M=3, H=4, D=64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.rocmfp4_rotary(*a.values())


@pytest.mark.parametrize("call", [append, read, attend])
@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(L, call, kw, status):
    assert call(L, **{"c_" + k: v for k, v in kw.items()}) == status
    assert L.rocmfp4_last_error()


@pytest.mark.parametrize("call", [append, read, attend])
def test_no_cache_and_nothing_to_do(L, call):
    assert call(L, cache=None) == INVALID
    assert call(L, M=0) == 0
    assert call(L, c_B=0, c_lens=None) == 0
    assert call(L, M=-1) == INVALID


@pytest.mark.parametrize("kw", [dict(type=3), dict(q_type=2), dict(H=-1), dict(rot=-2), dict(rot=63), dict(rot=66), dict(amplitude=NAN), dict(amplitude=INF), dict(q=None),
                                dict(k=None), dict(v=None), dict(q_out=None), dict(freq=None), dict(ldq=255), dict(ldk=127), dict(ldv=64), dict(q=PTR + 2), dict(k=PTR + 1),
                                dict(freq=PTR + 2), dict(positions=PTR + 2), dict(q_out=PTR + 1)])
def test_append_invalid(L, kw):
    assert append(L, **kw) == INVALID
    assert L.rocmfp4_last_error()


@pytest.mark.parametrize("kw", [dict(q_out=PTR + 4), dict(M=1 << 31), dict(H=65537, ldq=1 << 30)])
def test_append_unsupported(L, kw):
    assert append(L, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(type=3), dict(k_out=None, v_out=None), dict(k_out=PTR + 2), dict(v_out=PTR + 1)])
def test_read_invalid(L, kw):
    assert read(L, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(k_out=PTR + 8), dict(v_out=PTR + 4), dict(M=1 << 31)])
def test_read_unsupported(L, kw):
    assert read(L, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(act=2), dict(H=-2), dict(H=3), dict(window=-1), dict(scale=0.0), dict(scale=-0.1), dict(scale=NAN), dict(scale=INF), dict(causal=2),
                                dict(causal=0, window=3), dict(q=None), dict(out=None), dict(q=PTR + 1), dict(out=PTR + 1), dict(ldq=255)])
def test_attention_invalid(L, kw):
    assert attend(L, **kw) == INVALID
    assert L.rocmfp4_last_error()


@pytest.mark.parametrize("kw", [dict(c_D=32), dict(c_D=256, ldq=1024), dict(q=PTR + 8), dict(ldq=260), dict(out=PTR + 2), dict(M=1 << 30)])
def test_attention_unsupported(L, kw):
    assert attend(L, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(x_type=3), dict(y_type=2), dict(M=-1), dict(H=-1), dict(D=0), dict(D=40), dict(rot=66), dict(rot=1), dict(amplitude=NAN), dict(x=None),
                                dict(y=None), dict(freq=None), dict(positions=None), dict(ldx=255), dict(x=PTR + 2), dict(positions=PTR + 1)])
def test_rotary_invalid(L, kw):
    assert rotary(L, **kw) == INVALID


def test_rotary_unsupported_and_empty(L):
    assert rotary(L, D=288, ldx=1152, rot=0) == UNSUPPORTED
    assert rotary(L, y=PTR + 4) == UNSUPPORTED
    assert rotary(L, M=0, x=None, y=None) == 0
    assert rotary(L, H=0, x=None, y=None) == 0


def test_frequencies():
    f, a = rf4.rotary_frequencies(8, 10000.0, device="cpu")
    assert a == 1.0 and [round(v, 6) for v in f.tolist()] == [1.0, 0.1, 0.01, 0.001]
    lin, _ = rf4.rotary_frequencies(8, method="linear", factor=4.0, device="cpu")
    assert (lin * 4 - f).abs().max() <= 2.0 ** -24
    ntk, _ = rf4.rotary_frequencies(8, method="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(ntk[-1]) * 4 / float(f[-1]) - 1) < 1e-6
    parts, a = rf4.rotary_frequencies(64, method="parts", factor=8.0, original=4096, device="cpu")
    full, _ = rf4.rotary_frequencies(64, device="cpu")
    turns = 4096 * full.double() / (2 * math.pi)
    for got, base, n in zip(parts.tolist(), full.tolist(), turns.tolist()):
        want = base if n >= 32 else base / 8 if n <= 1 else base * ((n - 1) / 31 + (32 - n) / 31 / 8)
        assert abs(got / want - 1) < 1e-6
    assert abs(a - (0.1 * math.log(8.0) + 1)) < 1e-12
    for kw in (dict(rot=3), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, factor=0.5), dict(rot=8, method="other"), dict(rot=2, method="ntk"),
               dict(rot=8, method="parts"), dict(rot=8, method="parts", original=9, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            rf4.rotary_frequencies(device="cpu", **kw)
