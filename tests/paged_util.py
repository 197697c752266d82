"""A paged ROCmFP4 cache for the tests, and the definitions of the operators over it in 64 bits (torch, any device)."""
from __future__ import annotations

import math

import torch as t

import gemm_rocmfp4_dequant_gb300 as rf4

MAGNITUDES = (0.0, 1.0, 2.0, 3.0, 4.0, 6.0, 8.0, 10.0)


def e4m3_values(device):
    e = t.arange(128, device=device)
    return t.where(e >= 8, (1 + (e % 8) / 8.0).double() * t.exp2((e // 8 - 7).double()), (e % 8).double() * 2.0 ** -9)


def decode(w, variant):
    """Blocks (..., blocks, 17 or 18 bytes), every scale byte below 0x80, to float64 values (..., blocks * 32)."""
    q = t.cat((w[..., :16] & 15, w[..., :16] >> 4), -1).long()
    v = t.tensor(MAGNITUDES, dtype=t.float64, device=w.device)[q % 8] * t.where(q >= 8, -1.0, 1.0)
    hs = 0.5 * e4m3_values(w.device)[(w[..., 16:] & 127).long()]
    return (v * hs.repeat_interleave(16 if variant == rf4.DUAL else 32, -1)).flatten(-2) + 0.0


class Paged:
    """ns new rows and ts tokens of each sequence, pages in no order, random valid blocks in every page; rows behind a
    sequence's last token hold scale bytes that are no numbers."""

    def __init__(self, ns, ts, hkv, d, page, variant, seed=0, spare=2, width=None, extra=0):
        g = t.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.ns, self.ts, self.hkv, self.d, self.page, self.variant = g, list(ns), list(ts), hkv, d, page, variant
        B = len(ns)
        counts = [-(-x // page) for x in ts]
        width = max(counts + [1]) if width is None else width
        self.pages = sum(counts) + spare
        order = t.randperm(self.pages, generator=g, device="cuda").int()
        self.table = t.full((B, width + extra), -7, dtype=t.int32, device="cuda")[:, :width]
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.lens = t.tensor(ts, dtype=t.int32, device="cuda")
        cu = [0]
        for n in ns:
            cu.append(cu[-1] + n)
        self.m = cu[-1]
        self.cu = t.tensor(cu, dtype=t.int32, device="cuda")
        self.bb = 18 if variant == rf4.DUAL else 17
        self.shape = (self.pages, hkv, page, d // 32, self.bb)
        self.K, self.V = self._blocks(), self._blocks()
        self.spoil()
        self.cache = rf4.PagedCache(self.K.view(-1), self.V.view(-1), self.table, self.lens, self.cu, kv_heads=hkv, head=d, page_size=page, variant=variant)

    def _blocks(self):
        w = t.randint(0, 256, self.shape, generator=self.g, device="cuda", dtype=t.uint8)
        w[..., 16:] = 24 + w[..., 16:] % 24
        return w

    def spoil(self):
        for b, n in enumerate(self.ts):
            used = -(-n // self.page)
            if n % self.page and used <= self.table.shape[1]:
                pg = int(self.table[b, used - 1])
                if 0 <= pg < self.pages:
                    self.K[pg, :, n % self.page:] = 255
                    self.V[pg, :, n % self.page:] = 255

    def tokens(self, which, b, lo, hi):
        """Values [hi - lo, hkv, d] of tokens lo .. hi - 1 of sequence b, and which of them exist."""
        i = t.arange(lo, hi, device="cuda")
        pg = i // self.page
        inside = pg < self.table.shape[1]
        page = self.table.long()[b, pg.clamp(max=max(0, self.table.shape[1] - 1))]
        real = inside & (page >= 0) & (page < self.pages)
        rows = (self.K if which == "K" else self.V)[page.clamp(0, self.pages - 1), :, i % self.page]
        return decode(rows, self.variant) * real[:, None, None], real

    def attention(self, q, scale, causal=True, window=0):
        """(out, bound) [m, H, D] in 64 bits: the definition, and how far the kernel's may be off (see test_gpu_paged_attention)."""
        H, D = q.shape[1], self.d
        G = H // self.hkv
        out = t.zeros(self.m, H, D, dtype=t.float64, device="cuda")
        tol = t.zeros_like(out)
        at = 0
        for b, (n, T) in enumerate(zip(self.ns, self.ts)):
            if n and T > 0:
                K, real = self.tokens("K", b, 0, T)
                V, _ = self.tokens("V", b, 0, T)
                tok = t.arange(T, device="cuda")
                keep = real[None, :].expand(n, T)
                if causal:
                    last = (T - n + t.arange(n, device="cuda"))[:, None]
                    keep = keep & (tok <= last)
                    if window:
                        keep = keep & (tok > last - window)
                qq = q[at:at + n].double().view(n, self.hkv, G, D)
                x = t.einsum("nkgd,tkd->nkgt", qq, K) * scale
                mag = t.einsum("nkgd,tkd->nkgt", qq.abs(), K.abs()) * scale
                x = t.where(keep[:, None, None, :], x, -math.inf)
                top = x.amax(-1, keepdim=True)
                p = t.exp(x - t.where(top.isinf(), t.zeros_like(top), top))
                s = p.sum(-1, keepdim=True)
                p = p / t.where(s > 0, s, t.ones_like(s))
                out[at:at + n] = t.einsum("nkgt,tkd->nkgd", p, V).reshape(n, H, D)
                dx = (t.where(keep[:, None, None, :], mag, t.zeros_like(mag)).amax(-1, keepdim=True) * (16 + D / 16) * 2.0 ** -23 + 2.0 ** -20)
                rel = 2.0 ** -11 + 2 * dx + (T / 16 + 16) * 2.0 ** -23
                tol[at:at + n] = (rel * t.einsum("nkgt,tkd->nkgd", p, V.abs())).reshape(n, H, D)
            at += n
        return out, tol

    def queries(self, H, dtype, scale=1.5, pad=0, stride=0):
        """[m + pad, H, D], rows `stride` values further apart than they are wide."""
        m = self.m + pad
        buf = t.zeros(m, H * self.d + stride, dtype=dtype, device="cuda")
        buf[:, :H * self.d] = (t.randn(m, H * self.d, generator=self.g, device="cuda") * scale).to(dtype)
        return buf[:, :H * self.d].unflatten(1, (H, self.d))


def turned(x, pos, freq, interleaved, amplitude):
    """(y, bound) in 64 bits of heads x [M, H, D] at positions pos [M]."""
    rot = 2 * freq.numel()
    th = pos.double()[:, None] * freq.double()[None, :]
    c, s = (amplitude * t.cos(th))[:, None, :], (amplitude * t.sin(th))[:, None, :]
    x = x.double()
    y, mag = x.clone(), t.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    parts = (a * c - b * s, b * c + a * s)
    size = abs(amplitude) * (a.abs() + b.abs())
    for i, p in enumerate(parts):
        sl = slice(i, rot, 2) if interleaved else slice(i * (rot // 2), (i + 1) * (rot // 2))
        y[..., sl], mag[..., sl] = p, size
    # sine and cosine to 2^-23 (an eighth of a turn in fp32, and 2^-32 of a turn), the amplitude's, a product's and a sum's rounding
    return y, mag * 2.0 ** -21


def rounding(y, dtype):
    """Half a step of `dtype` at y, normal or not."""
    least = 2.0 ** -25 if dtype is t.float16 else 2.0 ** -134
    return y.abs() * t.finfo(dtype).eps / 2 + least
