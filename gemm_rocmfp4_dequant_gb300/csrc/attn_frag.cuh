// Decode of ROCmFP4 cache rows in shared memory into mma.sync fragments, and the
// warp instructions around them; for the attention kernels of few query rows.
#pragma once
#include "common.cuh"

namespace rocmfp4 {

// Shared-memory loads are plain C++ loads, so the compiler may schedule them
// early (the mbarrier wait and the proxy fence carry "memory" clobbers, which
// keep them after the data lands and before the stage is refilled).
RF4_DEV uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }

// Four bytes at any shared-memory address (two aligned words and a funnel shift).
RF4_DEV uint32_t lds_bytes4(const uint8_t* p) {
  const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(p) & 3u;
  const uint8_t* a = p - mis;
  return __funnelshift_r(lds32(a), lds32(a + 4), mis * 8u);
}

// Four bytes at an address whose offset from a 4-byte boundary is al (0..3),
// or not known (al = -1).  Called with al a constant after unrolling, so the
// branches fold away.
RF4_DEV uint32_t lds_bytes4_al(const uint8_t* p, int al) {
  if (al == 0) return lds32(p);
  if (al > 0) return __funnelshift_r(lds32(p - al), lds32(p - al + 4), 8 * al);
  return lds_bytes4(p);
}

// Offset from a 4-byte boundary of byte `off` of a token row, when rows start
// on 4-byte boundaries (every row length here is a multiple of 4 except the
// single-scale rows of D = 64), else -1.
template <int V, int D>
RF4_HOSTDEV constexpr int row_align(int off) {
  return (Fmt<V>::BB * (D / 32)) % 4 == 0 ? off % 4 : -1;
}

// Scale pair of a block as f16x2 E4M3 values: (scale of weights 0-15, scale
// of weights 16-31); the single-scale variant repeats its one scale.
template <int V>
RF4_DEV uint32_t block_scales(const uint8_t* block, int al) {
  const uint8_t* a = block + 16;
  const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(a) & 3u;
  const uint32_t w = al >= 0 ? lds32(a - al) >> (8 * al) : lds32(a - mis) >> (mis * 8u);
  if constexpr (V == 0) {
    return e4m3x2<0>(w & 0xFFFFu);  // two bytes, never straddling a word (even address)
  } else {
    return e4m3x2<0>(__byte_perm(w, 0u, 0x0000u) & 0xFFFFu);  // the byte twice
  }
}

// The four decoded pairs of bytes 4c .. 4c+3 of a block, each
// (w_j, w_{j+16}) * (scale pair), exact in fp16.
RF4_DEV void decode4(uint32_t codes, uint32_t s2, uint32_t (&v)[4]) {
  v[0] = hmul2(clamp5(e2m1x2<0>(codes)), s2);
  v[1] = hmul2(clamp5(e2m1x2<1>(codes)), s2);
  v[2] = hmul2(clamp5(e2m1x2<2>(codes)), s2);
  v[3] = hmul2(clamp5(e2m1x2<3>(codes)), s2);
}

// The MMA and movmatrix wrappers below touch registers only, so they are not
// volatile: the compiler may schedule them among the softmax's dependent steps.
RF4_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

RF4_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit elements across the warp (fragment layout: lane
// (r, c) holds elements (r, 2c) and (r, 2c+1)).
RF4_DEV uint32_t movmatrix_t(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// 2^x by the hardware approximation (relative error about 2^-22; 2^-inf = +0,
// subnormal results flush to zero).
RF4_DEV float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

RF4_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// p = hi + lo in two fp16 pairs (p already scaled by 2^15).
// C = 0 form of mma_f16 / mma_bf16.
RF4_DEV void mma_z(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool bf16) {
  const float z = 0.f;
  if (bf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z));
}

RF4_DEV void split_half2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_half2(a - __low2float(h), b - __high2float(h));
}

}  // namespace rocmfp4
