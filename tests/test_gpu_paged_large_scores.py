"""GPU tests of attention over a paged cache with scores so large that only the largest count, in both attention kernels.

Queries are +-2^15 or 0, keys whole multiples of 2^7 below 2^11, so that scores are multiples of 2^22 with few bits: exact in
fp32, whatever the order of the sum.  Two that differ are 2^22 * scale apart at least, so that a row's output is the mean of the
values of the tokens of its largest score.  P is exact then (a power of two, the same for all), the sum counts, and the mean is off
by fp32's accumulation of T values, (T / 16 + 16) * 2^-23 of their size, and half a step of the output's type."""
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


@pytest.mark.parametrize("scale", [2.0 ** -10, 0.125, 1.0, 37.7, 1e12, 1e30])
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("ns,ts", [([1, 4, 1], [9, 3000, 200]), ([40, 300, 7], [40, 2500, 1]), ([1], [20000]), ([70], [9000])])
def test_scores_of_which_the_largest_alone_counts(scale, name, ns, ts):
    t = torch()
    dtype = {"f16": t.float16, "bf16": t.bfloat16}[name]
    for D, variant in ((64, rf4.FAST), (128, rf4.DUAL)):
        p = pu.Paged(ns, ts, 2, D, 32, variant, seed=D)
        p.K[..., 16:] = 0x78  # half-scale 2^7
        for b in range(len(ts)):  # every third token's key stands twice
            for j in range(1, ts[b], 3):
                if j % 32 and j < 400:
                    p.K[int(p.table[b, j // 32]), :, j % 32] = p.K[int(p.table[b, j // 32]), :, j % 32 - 1]
        q = (2.0 ** 15 * t.randint(-1, 2, (p.m, 4, D), generator=p.g, device="cuda")).to(dtype)
        out = rf4.paged_attention(q, p.cache, scale)
        at = 0
        for b, (n, T) in enumerate(zip(ns, ts)):
            K, V = (p.tokens(which, b, 0, T)[0] for which in "KV")
            x = t.einsum("nkgd,tkd->nkgt", q[at:at + n].double().view(n, 2, 2, D), K)
            last = (T - n + t.arange(n, device="cuda"))[:, None]
            keep = (t.arange(T, device="cuda") <= last)[:, None, None, :]
            x = x.masked_fill(~keep, -float("inf"))
            top = (x == x.amax(-1, keepdim=True)) & keep
            share = top.double() / top.sum(-1, keepdim=True).clamp(min=1)
            want = t.einsum("nkgt,tkd->nkgd", share, V).reshape(n, 4, D)
            size = t.einsum("nkgt,tkd->nkgd", share, V.abs()).reshape(n, 4, D)
            off = (out[at:at + n].double() - want).abs()
            assert bool((off <= (T / 16 + 16) * 2.0 ** -23 * size + pu.rounding(want, dtype) * (1 + 2.0 ** -6)).all()), (D, b)
            at += n
