"""CPU tests of the argument checks of rocmfp4_add_rmsnorm, rocmfp4_moe and rocmfp4_logprobs: every call below is refused on the host
(or has nothing to do) before any pointer is used."""
import ctypes

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


def norm(L, **kw):
    a = dict(x=PTR, x_type=0, ldx=64, residual=PTR, residual_out=PTR, residual_type=0, ldr=64, ldro=64, weight=PTR, weight_type=0,
             eps=1e-6, y=PTR, y_type=0, q=PTR, scales=PTR, group=32, M=2, D=64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.rocmfp4_add_rmsnorm(*a.values())


@pytest.mark.parametrize("kw", [
    dict(x_type=3), dict(x_type=-1), dict(weight_type=5), dict(residual_type=3), dict(y_type=2), dict(M=-1), dict(D=-1), dict(D=0), dict(group=16),
    dict(group=-32), dict(group=(1 << 32) + 32), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(x=None), dict(weight=None),
    dict(residual_out=None), dict(y=None, q=None, scales=None), dict(scales=None), dict(q=None), dict(ldx=63), dict(ldr=63, ldro=63), dict(ldro=65),
    dict(x=PTR + 2), dict(residual=PTR + 1, residual_out=PTR + 1), dict(y=PTR + 1), dict(scales=PTR + 2), dict(weight=PTR + 1)])
def test_norm_invalid(L, kw):
    assert norm(L, **kw) == INVALID
    assert L.rocmfp4_last_error()


def test_norm_unsupported_and_empty(L):
    assert norm(L, D=32776, ldx=32776, ldr=32776, ldro=32776) == UNSUPPORTED
    assert norm(L, M=1 << 31) == UNSUPPORTED
    assert norm(L, M=0, x=None, weight=None, residual=None, y=None, q=None, scales=None) == 0


def logprobs(L, **kw):
    a = dict(logits=PTR, type=0, ld=100, targets=PTR, scale=1.0, logprob=PTR, entropy=PTR, top_ids=PTR, top_logprobs=PTR, top_n=5, M=2, V=100,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.rocmfp4_logprobs(*a.values())


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(M=-1), dict(V=-1), dict(V=0, top_n=0), dict(top_n=-1), dict(top_n=101), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
    dict(scale=INF), dict(scale=1e-31), dict(scale=1e31), dict(ld=99), dict(logits=None), dict(logprob=None), dict(top_ids=None), dict(top_logprobs=None), dict(logits=PTR + 2),
    dict(targets=PTR + 1), dict(top_ids=PTR + 2), dict(entropy=PTR + 2)])
def test_logprobs_invalid(L, kw):
    assert logprobs(L, **kw) == INVALID
    assert L.rocmfp4_last_error()


def test_logprobs_unsupported_and_empty(L):
    assert logprobs(L, top_n=33) == UNSUPPORTED
    assert logprobs(L, V=1 << 31, ld=1 << 31) == UNSUPPORTED
    assert logprobs(L, M=0, logits=None, targets=None) == 0


def moe(L, **kw):
    a = dict(X=PTR, router=PTR, router_type=1, Wgu=PTR, Wd=PTR, Y=PTR, ids=PTR, probs=PTR, M=2, E=8, top_k=2, K=64, I=96, route=1,
             route_scale=1.0, variant=0, act=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.rocmfp4_moe(*a.values())


@pytest.mark.parametrize("kw", [
    dict(variant=2), dict(act=2), dict(router_type=3), dict(route=3), dict(route=-1), dict(M=-1), dict(E=0), dict(top_k=0), dict(top_k=9),
    dict(K=0), dict(K=63), dict(I=0), dict(I=-32), dict(I=48), dict(route_scale=NAN), dict(route_scale=INF), dict(X=None), dict(router=None),
    dict(Wgu=None), dict(Wd=None), dict(Y=None), dict(Y=PTR + 2), dict(ids=PTR + 1), dict(probs=PTR + 2)])
def test_moe_invalid(L, kw):
    assert moe(L, **kw) == INVALID
    assert L.rocmfp4_last_error()


@pytest.mark.parametrize("kw", [
    dict(M=33), dict(E=513), dict(E=64, top_k=17), dict(K=32800), dict(I=32800), dict(M=32, E=16, top_k=16, I=32768), dict(X=PTR + 8),
    dict(router=PTR + 4), dict(Wgu=PTR + 2), dict(Wd=PTR + 8)])
def test_moe_unsupported(L, kw):
    assert moe(L, **kw) == UNSUPPORTED


def test_moe_empty(L):
    assert moe(L, M=0, X=None, router=None, Wgu=None, Wd=None, Y=None) == 0
