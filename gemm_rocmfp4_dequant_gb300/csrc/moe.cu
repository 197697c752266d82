// A whole mixture-of-experts layer for a few tokens (M <= 32), in one kernel:
//   l = R x                         router logits of every expert, fp32
//   top_k experts by (l descending, index ascending), weights p by the route
//   h = SiLU(Wg x) * (Wu x)         per chosen expert, fp32
//   Y = sum over choices of p * (Wd h)
// with every expert's Wg, Wu (stacked) and Wd in packed ROCmFP4 blocks.  Only
// the blocks of chosen experts are read, each once.
//
// One persistent CTA per SM, launched cooperatively, in three phases with two
// grid barriers: router logits (and the activations in fragment order); gate
// and up products (h goes to the workspace); down products.  Every CTA repeats
// the small top-k selection for itself, which costs less than handing its
// result on.
//
// Products.  A tile is 16 rows: 8 gate and the 8 up rows of the same hidden
// values, or 16 output rows.  A span is 144 bytes (8 dual blocks) or 272 bytes
// (16 single-scale blocks) of each row.  A warp takes tiles on its own (or
// KP neighbouring warps share a tile's spans where tiles are few) and streams
// their spans through a private ring of shared-memory stages, by tensor copies
// of 16-row boxes.  The down tasks are known as soon as the routing is, so the
// ring runs on into them before the second barrier.
// The arithmetic is mma.sync m16n8k16 on fp16 with fp32 accumulators: A is
// the decoded weights, exact in fp16, decoded once for all the tokens of the
// expert; B's columns are tokens.  Lane (q, c) decodes blocks of rows q and
// q + 8; byte j of a block is the pair (j, j + 16), so activations are kept in
// that pair order, 16 bytes a lane and load.  Eight MMAs run in the tensor
// core's accumulator, then add to fp32 registers, round to nearest.
//
// Precision.  bf16 activations become fp16 after scaling a token by the power
// of two that brings its largest magnitude to [2^14, 2^15): values down to
// 2^-28 of the largest stay exact, smaller ones are off by at most 2^-39 of
// it.  h is fp32; the down product takes it as two fp16 columns, high and
// remainder, 22 bits together.  The pair is made where h is, times 16, if the
// choice's largest |h| proves to be in [2^-5, 2^11); a choice outside that
// range has its pairs made again from the fp32 h, scaled like a bf16 token,
// behind a third barrier that other calls do not meet.
//
// Bound: memory (3 I K / 32 blocks per chosen expert), with the decode's issue
// slots (about 3.7 instructions per pair of weights) close behind.
//
// Rows whose length is no multiple of 16 bytes (K / 32 not a multiple of 8,
// dual, or 16, single-scale) cannot be boxes of a tensor copy.  They come by a
// bulk copy per row from the 16-byte boundary before the span to the one
// after it (which stays inside the matrices, as their sizes are multiples of
// 16), and are shifted into place word by word.
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace rocmfp4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kTileRows = 16;
constexpr int kMaxStages = 8;
constexpr int kRouterTokens = 8;   // tokens a router pass holds
constexpr int kGuGroups = 4;       // groups of 8 tokens of an expert
constexpr int kDnGroups = 8;       // groups of 4 tokens: high and low columns
constexpr int kFastExp = 4;        // h times 2^4 in its fp16 pair

template <int V>
struct Unit {
  static constexpr int BLOCKS = Fmt<V>::BPL;       // blocks a lane has of a span: 2 / 4
  static constexpr int BYTES = Fmt<V>::LANE_BYTES; // 36 / 68
  static constexpr int SPAN = Fmt<V>::SPAN;        // 144 / 272
  static constexpr int SPAN_BLOCKS = 4 * BLOCKS;   // 8 / 16
  static constexpr int NS = V == 0 ? 2 : 1;        // spans a stage holds
  static constexpr int X_SPAN = SPAN_BLOCKS * 64;  // bytes of a span's fp16 activations
  static constexpr int PITCH = 304;                // row slots of unaligned rows: NS spans, 16-byte slack, no bank conflicts
  static constexpr int STAGE = (kTileRows * PITCH + 127) / 128 * 128;
  static_assert(NS * SPAN + 15 <= PITCH && NS * SPAN * kTileRows <= STAGE, "stage holds either form");
};

struct MoeParams {
  CUtensorMap map_gu;  // aligned rows: {words, I rows, 2 E halves}, box {span, 8, 2}
  CUtensorMap map_dn;  // {words, E K rows}, box {span, 16}
  const uint16_t* X;
  const void* router;
  const uint8_t* Wgu;
  const uint8_t* Wd;
  float* Y;
  int32_t* ids;
  float* probs;
  float* logits;       // workspace [M][E]
  float* x_unscale;    // workspace [M]
  uint32_t* amax;      // workspace [M * top_k]: bits of the largest |h|
  uint8_t* xf;         // workspace: activations in fragment order, fp16
  float* h;            // workspace [M * top_k][I]
  uint8_t* h_hi;       // workspace: h * 16 in fragment order, fp16 and its remainder
  uint8_t* h_lo;
  uint32_t* bars;      // workspace: three barrier counters and one of finished CTAs, zero between launches
  uint32_t* err;
  int M, E, top_k, K, I;
  int router_type, route;
  float route_scale;
  int parts;           // KP: warps that share a gate/up tile
  int stages;          // ring stages of a warp
  // offsets in shared memory
  int off_mask, off_list, off_slot, off_unscale, off_keys, off_x, off_acc, off_ring;
  int x_pitch;         // bytes between tokens of the activations in shared memory, 0: they stay in the workspace
  int acc_floats;      // per warp
};

template <int ACT>
RF4_DEV float act_f32(uint32_t bits16) {
  if constexpr (ACT == 1) return __uint_as_float(bits16 << 16);
  else return __half2float(__ushort_as_half((uint16_t)bits16));
}

// 2^k, k clamped to a range that its inverse shares.
RF4_DEV float exp2i(int k) { return __uint_as_float((uint32_t)(127 + max(-120, min(120, k))) << 23); }
// The power of two that brings a magnitude (its bits) to [2^14, 2^15); 0 for zero and non-finite ones.
RF4_DEV int scale_exp(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  if (e == 255 || amax_bits == 0) return 0;
  return max(-120, min(120, 141 - e));
}
// Whether the fp16 pair of h made with the fixed scale is good: 0, [2^-5, 2^11) or not finite (then so is the output).
RF4_DEV bool fast_range(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return amax_bits == 0 || e == 255 || (e >= 127 - 5 && e < 127 + 11);
}

RF4_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The five words that hold block PHI of a lane's unit (any byte address
// unless ALIGNED): code byte j at byte (PHI * block bytes) % 4 + j.
template <int V, bool ALIGNED, int PHI>
RF4_DEV void block_words(const uint8_t* unit, bool have, uint32_t (&w)[5]) {
  constexpr int FIRST = PHI * Fmt<V>::BB / 4;
  if constexpr (ALIGNED) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(unit) + FIRST;
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = p[i];
  } else {
    const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(unit) & 3u;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(unit - mis) + FIRST;
    uint32_t a[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) a[i] = have ? p[i] : 0u;  // past the row: zero codes under zero scales
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = __funnelshift_r(a[i], a[i + 1], 8 * mis);
  }
}

RF4_DEV uint32_t codes_at(const uint32_t (&w)[5], int pos) {
  const uint32_t word = w[pos >> 2];
  switch (pos & 3) {
    case 0: return e2m1x2<0>(word);
    case 1: return e2m1x2<1>(word);
    case 2: return e2m1x2<2>(word);
    default: return e2m1x2<3>(word);
  }
}

// A block's words and its scale pair (fp16).
template <int V, bool ALIGNED, int PHI>
struct Block {
  static constexpr int O = PHI * Fmt<V>::BB % 4;
  uint32_t w[5], s2;
  RF4_DEV Block(const uint8_t* unit, bool have) {
    block_words<V, ALIGNED, PHI>(unit, have, w);
    if constexpr (V == 0) s2 = O == 0 ? e4m3x2<0>(w[4]) : e4m3x2<1>(w[4]);
    else s2 = e4m3x2<0>(__byte_perm(w[4], 0u, O * 0x11));
  }
  // the pair (w_j, w_{j+16}), exact in fp16
  RF4_DEV uint32_t pair(int j) const { return hmul2(clamp5(codes_at(w, O + j)), s2); }
};

RF4_DEV void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
RF4_DEV void mma_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Byte offset of chunk kk (pairs 4 kk .. 4 kk + 3) of block PHI of lane group c
// in a span's activations: the four c lie side by side.
RF4_DEV int x_chunk(int phi, int kk, int c) { return ((phi * 4 + kk) * 4 + c) * 16; }

RF4_DEV void load_b(const uint8_t* p, uint4 (&b)[4]) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) b[kk] = *reinterpret_cast<const uint4*>(p + kk * 64);
}

// Activations of the lane's column, one pointer per group of tokens, moving on
// through the row 256 bytes a block.  One group (most experts of a few tokens):
// the next block's are loaded while this one's weights are decoded.  Columns
// beyond the expert's tokens repeat its first; their sums are not used.
template <int GROUPS>
struct Columns {
  const uint8_t* p[GROUPS];
  uint4 b[4];
  RF4_DEV void start() {
    if constexpr (GROUPS == 1) load_b(p[0], b);
  }
};

// One span of a tile: `ra`, `rb` are rows q and q + 8 at the lane's unit, blk
// the unit's first block.  A block is eight MMAs in two chains of four.
template <int V, bool ALIGNED, int PHI, int GROUPS>
RF4_DEV void span_products(const uint8_t* ra, const uint8_t* rb, int blk, int nb, int ng, Columns<GROUPS>& col, float (&acc)[GROUPS][4]) {
  const bool have = ALIGNED || blk + PHI < nb;
  const Block<V, ALIGNED, PHI> x(ra, have), y(rb, have);
  if constexpr (GROUPS == 1) {
    uint4 next[4];
    load_b(col.p[0] + 256, next);  // reads past the row's last block stay in the workspace
    float d[2][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint4 b = col.b[kk];
      if (kk < 2) mma_z(d[kk & 1], x.pair(4 * kk), y.pair(4 * kk), x.pair(4 * kk + 1), y.pair(4 * kk + 1), b.x, b.y);
      else mma(d[kk & 1], x.pair(4 * kk), y.pair(4 * kk), x.pair(4 * kk + 1), y.pair(4 * kk + 1), b.x, b.y);
      mma(d[kk & 1], x.pair(4 * kk + 2), y.pair(4 * kk + 2), x.pair(4 * kk + 3), y.pair(4 * kk + 3), b.z, b.w);
      col.b[kk] = next[kk];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[0][i] += d[0][i] + d[1][i];
    col.p[0] += 256;
  } else {
    uint32_t a0[16], a1[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) a0[j] = x.pair(j), a1[j] = y.pair(j);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      if (g < ng) {
        uint4 b[4];
        load_b(col.p[g], b);
        float d[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk == 0) mma_z(d, a0[0], a1[0], a0[1], a1[1], b[0].x, b[0].y);
          else mma(d, a0[4 * kk], a1[4 * kk], a0[4 * kk + 1], a1[4 * kk + 1], b[kk].x, b[kk].y);
          mma(d, a0[4 * kk + 2], a1[4 * kk + 2], a0[4 * kk + 3], a1[4 * kk + 3], b[kk].z, b[kk].w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][i] += d[i];
        col.p[g] += 256;
      }
    }
  }
  if constexpr (PHI + 1 < Unit<V>::BLOCKS) span_products<V, ALIGNED, PHI + 1, GROUPS>(ra, rb, blk, nb, ng, col, acc);
}

// The bytes [a, a + n) as a copy from 16-byte boundary to 16-byte boundary.
RF4_DEV uint32_t span_bytes(const uint8_t* a, int n) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(a) & ~uintptr_t(15), e = (reinterpret_cast<uintptr_t>(a) + n + 15) & ~uintptr_t(15);
  return (uint32_t)(e - b);
}
RF4_DEV void copy_span(uint8_t* dst, const uint8_t* a, int n, uint32_t bar) {
  bulk_g2s(smem_addr(dst), reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(a) & ~uintptr_t(15)), span_bytes(a, n), bar);
}
RF4_DEV int mis16(const uint8_t* a) { return (int)(reinterpret_cast<uintptr_t>(a) & 15u); }

// Barrier of some whole warps of the CTA (id 1 .. 15).
RF4_DEV void team_barrier(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

RF4_DEV uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Order-preserving bits of a router logit, above 0; NaN orders below every number.
RF4_DEV float logit_of(uint32_t key) {
  return key == 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
RF4_DEV uint32_t logit_key(float f) {
  if (f != f) return 1u;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

RF4_DEV void load8_router(int type, const void* base, int64_t off, float (&v)[8]) {
  if (type == 0) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = type == 1 ? act_f32<1>(w[i] & 0xFFFFu) : act_f32<0>(w[i] & 0xFFFFu);
      v[2 * i + 1] = type == 1 ? act_f32<1>(w[i] >> 16) : act_f32<0>(w[i] >> 16);
    }
  }
}

template <int V, int ACT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ MoeParams p) {
  using U = Unit<V>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_probs = reinterpret_cast<float*>(smem);                           // [M][top_k]
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + p.off_mask);         // [E]: tokens of an expert
  uint16_t* s_list = reinterpret_cast<uint16_t*>(smem + p.off_list);         // chosen experts, ascending
  uint8_t* s_slot = smem + p.off_slot;                                       // [M][E]: which choice of the token
  float* s_unscale = reinterpret_cast<float*>(smem + p.off_unscale);         // [M]: 1 / the activations' scale
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem + p.off_keys);         // [kWarps][E]: order of a token's logits
  float* s_acc = reinterpret_cast<float*>(smem + p.off_acc);                 // [kWarps][acc_floats]
  __shared__ uint64_t s_bars[kWarps * kMaxStages];
  __shared__ float s_red[kWarps][kRouterTokens];
  __shared__ int s_active, s_ok;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = gridDim.x;

  uint64_t* bars = s_bars + warp * kMaxStages;
  if (lane == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_addr(&bars[i]), 1);
    fence_mbar_init();
  }
  if (ALIGNED && tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_gu)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_dn)) : "memory");
  }
  if (tid == 0) s_ok = 1;
  for (int e = tid; e < p.E; e += kThreads) s_mask[e] = 0;
  __syncthreads();

  // Every CTA arrives and waits (bounded) for the others; false if one gave up.
  auto grid_barrier = [&](uint32_t* counter) {
    __syncthreads();
    if (tid == 0) {
      atomic_add_acq_rel_gpu(counter, 1u);
      const long long t0 = clock64();
      while (load_acquire(counter) < (uint32_t)G) {
        if (clock64() - t0 > (1ll << 32)) {
          atomicOr(p.err, kErrWaitTimeout);
          s_ok = 0;
          break;
        }
      }
    }
    __syncthreads();
    return s_ok != 0;
  };

  // ---- router logits: one expert per CTA and pass, eight tokens at a time ----
  for (int e = blockIdx.x; e < p.E; e += G) {
    for (int m0 = 0; m0 < p.M; m0 += kRouterTokens) {
      const int mc = min(kRouterTokens, p.M - m0);
      float acc[kRouterTokens];
#pragma unroll
      for (int m = 0; m < kRouterTokens; ++m) acc[m] = 0.f;
      for (int k = tid * 8; k < p.K; k += kThreads * 8) {
        float r[8];
        load8_router(p.router_type, p.router, (int64_t)e * p.K + k, r);
        uint4 a[kRouterTokens];
#pragma unroll
        for (int m = 0; m < kRouterTokens; ++m)
          if (m < mc) a[m] = __ldg(reinterpret_cast<const uint4*>(p.X + (int64_t)(m0 + m) * p.K + k));
#pragma unroll
        for (int m = 0; m < kRouterTokens; ++m) {
          if (m < mc) {
            const uint32_t w[4] = {a[m].x, a[m].y, a[m].z, a[m].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[m] = fmaf(r[2 * i], act_f32<ACT>(w[i] & 0xFFFFu), acc[m]);
              acc[m] = fmaf(r[2 * i + 1], act_f32<ACT>(w[i] >> 16), acc[m]);
            }
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kRouterTokens; ++m) {
        if (m >= mc) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
        if (lane == 0) s_red[warp][m] = acc[m];
      }
      __syncthreads();
      if (tid < kRouterTokens && m0 + tid < p.M) {
        float l = 0.f;
        for (int w = 0; w < kWarps; ++w) l += s_red[w][tid];
        p.logits[(int64_t)(m0 + tid) * p.E + e] = l;
      }
      __syncthreads();
    }
  }
  // ---- activations in fragment order, by the CTAs that have the fewest experts ----
  const int nb_k = p.K / 32, spans_k = (nb_k + U::SPAN_BLOCKS - 1) / U::SPAN_BLOCKS;
  for (int m = G - 1 - (int)blockIdx.x; m < p.M; m += G) {
    const uint16_t* x = p.X + (int64_t)m * p.K;
    float scale = 1.f;
    if constexpr (ACT == 1) {
      uint32_t mx = 0;  // bf16 magnitudes order as their bits
      for (int k = tid * 2; k < p.K; k += kThreads * 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(x + k) & 0x7FFF7FFFu;
        mx = max(mx, max(w & 0xFFFFu, w >> 16));
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) s_red[warp][0] = __uint_as_float(mx << 16);
      __syncthreads();
      mx = 0;
      for (int w = 0; w < kWarps; ++w) mx = max(mx, __float_as_uint(s_red[w][0]));
      const int k = scale_exp(mx);
      scale = exp2i(k);
      if (tid == 0) p.x_unscale[m] = exp2i(-k);
      __syncthreads();
    } else if (tid == 0) {
      p.x_unscale[m] = 1.f;
    }
    for (int i = tid; i < spans_k * U::SPAN_BLOCKS * 4; i += kThreads) {
      const int blk = i >> 2, kk = i & 3, in = blk % U::SPAN_BLOCKS;
      uint2 a = make_uint2(0, 0), b = a;  // zeros past the row
      if (blk < nb_k) {
        a = *reinterpret_cast<const uint2*>(x + blk * 32 + 4 * kk);
        b = *reinterpret_cast<const uint2*>(x + blk * 32 + 16 + 4 * kk);
      }
      uint4 v;
      if constexpr (ACT == 0) {
        v = make_uint4(__byte_perm(a.x, b.x, 0x5410), __byte_perm(a.x, b.x, 0x7632), __byte_perm(a.y, b.y, 0x5410), __byte_perm(a.y, b.y, 0x7632));
      } else {
        v.x = pack_half2(act_f32<1>(a.x & 0xFFFFu) * scale, act_f32<1>(b.x & 0xFFFFu) * scale);
        v.y = pack_half2(act_f32<1>(a.x >> 16) * scale, act_f32<1>(b.x >> 16) * scale);
        v.z = pack_half2(act_f32<1>(a.y & 0xFFFFu) * scale, act_f32<1>(b.y & 0xFFFFu) * scale);
        v.w = pack_half2(act_f32<1>(a.y >> 16) * scale, act_f32<1>(b.y >> 16) * scale);
      }
      uint8_t* dst = p.xf + ((int64_t)m * spans_k + blk / U::SPAN_BLOCKS) * U::X_SPAN + x_chunk(in % U::BLOCKS, kk, in / U::BLOCKS);
      *reinterpret_cast<uint4*>(dst) = v;
    }
  }
  const int choices = p.M * p.top_k;
  if (blockIdx.x == 0)
    for (int a = tid; a < choices; a += kThreads) p.amax[a] = 0u;
  const int nb_i = p.I / 32, spans_i = (nb_i + U::SPAN_BLOCKS - 1) / U::SPAN_BLOCKS;
  const int64_t h_row = (int64_t)spans_i * U::X_SPAN;  // bytes of a choice's h parts
  // Place of hidden value i in its row of h parts.
  auto h_place = [&](int i) {
    const int in = i / 32 % U::SPAN_BLOCKS, pj = i & 15;
    return (int64_t)(i / 32 / U::SPAN_BLOCKS) * U::X_SPAN + x_chunk(in % U::BLOCKS, pj >> 2, in / U::BLOCKS) + (pj & 3) * 4 + (i >> 4 & 1) * 2;
  };
  if constexpr (!ALIGNED) {  // zeros past the rows of h
    for (int a = blockIdx.x; a < choices; a += G)
      for (int i = p.I + tid; i < spans_i * U::SPAN_BLOCKS * 32; i += kThreads) {
        *reinterpret_cast<uint16_t*>(p.h_hi + a * h_row + h_place(i)) = 0;
        *reinterpret_cast<uint16_t*>(p.h_lo + a * h_row + h_place(i)) = 0;
      }
  }
  bool ok = grid_barrier(p.bars);

  // ---- top k of every token (one warp per token), repeated by every CTA ----
  if (ok) {
    uint32_t* keys = s_keys + warp * p.E;  // a lane reads only what it wrote: entries lane, lane + 32, ...
    for (int m = warp; m < p.M; m += kWarps) {
      const float* logits = p.logits + (int64_t)m * p.E;
      uint32_t best = 0, next = 0;  // the lane's largest remaining key and its expert
      for (int e = lane; e < p.E; e += 32) {
        const uint32_t k = logit_key(__ldcg(logits + e));
        keys[e] = k;
        if (k > best) best = k, next = e;
      }
      // the softmax over all experts needs its sum before choices leave the keys
      float denom = 0.f;
      const float top = logit_of(__reduce_max_sync(0xffffffffu, best));
      if (p.route == 0)
        for (int e = lane; e < p.E; e += 32) denom += expf(logit_of(keys[e]) - top);
      uint32_t my_key = 1;
      int my_id = 0;
      for (int j = 0; j < p.top_k; ++j) {
        const uint32_t mx = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == mx ? next : 0xFFFFu);
        if (lane == j) my_id = (int)e, my_key = mx;
        if ((int)(e & 31) == lane) {
          keys[e] = 0;
          best = 0;
          for (int i = lane; i < p.E; i += 32) {
            const uint32_t k = keys[i];
            if (k > best) best = k, next = i;
          }
        }
      }
      const float mine = logit_of(my_key);
      float num = 0.f;
      if (p.route == 2) {
        num = lane < p.top_k ? 1.f / (1.f + expf(-mine)) : 0.f;
        denom = num;
      } else {
        num = lane < p.top_k ? expf(mine - top) : 0.f;
        if (p.route == 1) denom = num;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) denom += __shfl_xor_sync(0xffffffffu, denom, o);
      if (lane < p.top_k) {
        const float pr = num / denom * p.route_scale;
        s_probs[m * p.top_k + lane] = pr;
        s_slot[m * p.E + my_id] = (uint8_t)lane;
        atomicOr(&s_mask[my_id], 1u << m);
        if (blockIdx.x == 0) {
          if (p.ids != nullptr) p.ids[m * p.top_k + lane] = my_id;
          if (p.probs != nullptr) p.probs[m * p.top_k + lane] = pr;
        }
      }
    }
  }
  if (ok && tid < p.M) s_unscale[tid] = __ldcg(p.x_unscale + tid);
  if (ok && p.x_pitch != 0) {
    const int per = spans_k * U::X_SPAN / 16;  // 16-byte chunks of a token
    for (int i = tid; i < p.M * per; i += kThreads)
      *reinterpret_cast<uint4*>(smem + p.off_x + i / per * p.x_pitch + i % per * 16) = __ldcg(reinterpret_cast<const uint4*>(p.xf) + i);
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const bool on = e0 + lane < p.E && s_mask[e0 + lane] != 0;
      const uint32_t b = __ballot_sync(0xffffffffu, on);
      if (on) s_list[n + __popc(b & ((1u << lane) - 1u))] = (uint16_t)(e0 + lane);
      n += __popc(b);
    }
    if (lane == 0) s_active = n;
  }
  __syncthreads();
  const int A = ok ? s_active : 0;

  // ---- this warp's stages: gate/up tiles, then down tiles --------------------------------
  const int rb_k = nb_k * Fmt<V>::BB, rb_i = nb_i * Fmt<V>::BB;
  const int KP = p.parts, team = warp / KP, part = warp % KP, teams = kWarps / KP;
  const int span0 = spans_k * part / KP, span1 = spans_k * (part + 1) / KP;  // this warp's spans of a gate/up tile
  const int per_expert = p.I / 8;                                          // gate/up tiles of an expert
  const int gu_tiles = A * per_expert;                                     // dealt round robin over CTAs, then teams
  const int first_gu = blockIdx.x + G * team;
  const int tiles = p.K / kTileRows;
  const int my_tiles = (int)blockIdx.x < tiles ? (tiles - (int)blockIdx.x + G - 1) / G : 0;
  const int sd = (spans_i + U::NS - 1) / U::NS;                            // stages of an expert's rows in a down tile
  const int u0 = warp * (A * sd) / kWarps, u1 = (warp + 1) * (A * sd) / kWarps;  // this warp's share of a down tile's stages
  uint8_t* ring = smem + p.off_ring + (size_t)warp * p.stages * U::STAGE;

  // Row r of a stage at the lane's unit of the stage's first span; further
  // spans lie SPAN_STEP on.  Unaligned rows start at their own place within 16 bytes.
  const int q = lane >> 2, c = lane & 3;
  constexpr int SPAN_STEP = ALIGNED ? kTileRows * U::SPAN : U::SPAN;
  auto unit_at = [&](const uint8_t* stage, int r, const uint8_t* src) {
    if constexpr (ALIGNED) return stage + r * U::SPAN + c * U::BYTES;
    else return stage + r * U::PITCH + mis16(src) + c * U::BYTES;
  };
  auto gu_row = [&](int e, int i0, int r) { return p.Wgu + ((int64_t)e * 2 * p.I + (r < 8 ? 0 : p.I) + i0 + (r & 7)) * rb_k; };
  auto dn_row = [&](int e, int n0, int r) { return p.Wd + ((int64_t)e * p.K + n0 + r) * rb_i; };

  // Copies of spans [span, span + n) of a tile's 16 rows into a stage.
  auto fill = [&](bool down, int e, int row0, int span, int n, int slot) {
    uint8_t* dst = ring + (size_t)slot * U::STAGE;
    const uint32_t bar = smem_addr(&bars[slot]);
    if constexpr (ALIGNED) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, (uint32_t)(n * kTileRows * U::SPAN));
        for (int k = 0; k < n; ++k) {
          const uint32_t to = smem_addr(dst + k * kTileRows * U::SPAN);
          if (down) tma_load_2d(to, &p.map_dn, (span + k) * (U::SPAN / 4), e * p.K + row0, bar);
          else tma_load_3d(to, &p.map_gu, (span + k) * (U::SPAN / 4), row0, 2 * e, bar);
        }
      }
    } else {
      const int rb = down ? rb_i : rb_k, lo = span * U::SPAN, len = min(rb - lo, n * U::SPAN);
      const uint8_t* src = (down ? dn_row(e, row0, lane & 15) : gu_row(e, row0, lane & 15)) + lo;
      const uint32_t bytes = __reduce_add_sync(0xffffffffu, lane < kTileRows ? span_bytes(src, len) : 0u);
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (lane < kTileRows) copy_span(dst + lane * U::PITCH, src, len, bar);
    }
  };
  // The next stage to fill.
  struct {
    bool gu, any;
    int id, e, row0, span;  // gate/up: tile number, expert, first row, next span
    int tile, u, a, s;      // down: tile of this CTA, unit, place in the list, stage of the row
  } nx;
  auto start_gu = [&](int id) {
    nx.id = id;
    nx.e = s_list[id / per_expert];
    nx.row0 = id % per_expert * 8;
    nx.span = span0;
  };
  auto start_dn = [&]() {
    nx.u = u0;
    nx.a = u0 / sd;
    nx.s = u0 - nx.a * sd;
  };
  nx.tile = 0;
  nx.gu = first_gu < gu_tiles;
  nx.any = nx.gu || (u0 < u1 && my_tiles > 0);
  if (nx.gu) start_gu(first_gu);
  if (u0 < u1) start_dn();
  int fill_slot = 0, filled = 0;
  auto fill_next = [&]() {
    if (!nx.any) return;
    if (nx.gu) {
      fill(false, nx.e, nx.row0, nx.span, min(U::NS, span1 - nx.span), fill_slot);
      nx.span += U::NS;
      if (nx.span >= span1) {
        if (nx.id + G * teams < gu_tiles) {
          start_gu(nx.id + G * teams);
        } else {
          nx.gu = false;
          nx.any = u0 < u1 && my_tiles > 0;
        }
      }
    } else {
      fill(true, s_list[nx.a], (blockIdx.x + nx.tile * G) * kTileRows, nx.s * U::NS, min(U::NS, spans_i - nx.s * U::NS), fill_slot);
      if (++nx.s == sd) nx.s = 0, ++nx.a;
      if (++nx.u == u1) {
        if (++nx.tile < my_tiles) start_dn();
        else nx.any = false;
      }
    }
    if (++fill_slot == p.stages) fill_slot = 0;
    ++filled;
  };
  int slot = 0, used = 0;
  uint32_t parity = 0;
  bool live = ok;
  if (ok)
    for (int i = 0; i < p.stages; ++i) fill_next();
  auto wait_stage = [&]() {  // warp-uniform: every lane waits on the same barrier
    const bool landed = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&bars[slot]), parity));
    if (!landed && lane == 0) atomicOr(p.err, kErrWaitTimeout);
    return landed;
  };
  auto next_slot = [&]() {
    ++used;
    if (++slot == p.stages) slot = 0, parity ^= 1u;
  };
  auto release_stage = [&]() {
    __syncwarp();
    fence_proxy_async();  // the stage's reads precede the next copy into it
    fill_next();
    next_slot();
  };
  // The token after `skip` others of a set, -1 for none.
  auto token_of = [&](uint32_t tokens, int skip) {
    for (int i = 0; i < skip; ++i) tokens &= tokens - 1;
    return tokens ? __ffs(tokens) - 1 : -1;
  };
  float* acc_w = s_acc + (size_t)warp * p.acc_floats;

  // ---- gate and up ----
  const uint8_t* x_base = p.x_pitch != 0 ? smem + p.off_x : p.xf;
  const int64_t x_row = p.x_pitch != 0 ? p.x_pitch : spans_k * U::X_SPAN;
  auto gu_tile = [&](auto groups, int e, int i0, uint32_t tokens) {
    constexpr int GROUPS = decltype(groups)::value;
    const int ng = GROUPS == 1 ? 1 : (__popc(tokens) + 7) / 8;
    int tok[GROUPS];
    float acc[GROUPS][4];
    Columns<GROUPS> col;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      tok[g] = g < ng ? token_of(tokens, 8 * g + q) : -1;
      col.p[g] = x_base + (tok[g] >= 0 ? tok[g] : __ffs(tokens) - 1) * x_row + span0 * U::X_SPAN + c * 16;
      acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
    }
    col.start();
    for (int span = span0; span < span1 && live; span += U::NS) {
      if (!wait_stage()) {
        live = false;
        break;
      }
      const uint8_t* st = ring + (size_t)slot * U::STAGE;
      const uint8_t* ra = unit_at(st, q, gu_row(e, i0, q) + span * U::SPAN);
      const uint8_t* rb = unit_at(st, q + 8, gu_row(e, i0, q + 8) + span * U::SPAN);
      const int n = min(U::NS, span1 - span);
      for (int k = 0; k < n; ++k)
        span_products<V, ALIGNED, 0, GROUPS>(ra + k * SPAN_STEP, rb + k * SPAN_STEP, (span + k) * U::SPAN_BLOCKS + c * U::BLOCKS, nb_k, ng, col, acc);
      release_stage();
    }
    if (KP > 1) {  // the parts' sums, in order
      if (part > 0) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
          if (g < ng) *reinterpret_cast<float4*>(acc_w + (g * 32 + lane) * 4) = make_float4(acc[g][0], acc[g][1], acc[g][2], acc[g][3]);
      }
      team_barrier(1 + team, KP * 32);
      if (part == 0) {
        for (int w = 1; w < KP; ++w) {
          const float* other = acc_w + (size_t)w * p.acc_floats;
#pragma unroll
          for (int g = 0; g < GROUPS; ++g)
            if (g < ng) {
              const float4 v = *reinterpret_cast<const float4*>(other + (g * 32 + lane) * 4);
              acc[g][0] += v.x, acc[g][1] += v.y, acc[g][2] += v.z, acc[g][3] += v.w;
            }
        }
      }
      team_barrier(1 + team, KP * 32);
      if (part > 0) return;
    }
    // Lane (q, c): gate and up of hidden value i0 + q for columns 2 c and 2 c + 1.
    const int i = i0 + q;
    const int64_t place = h_place(i);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      if (g >= ng) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = __shfl_sync(0xffffffffu, tok[g], (2 * c + j) * 4);
        float h = 0.f;
        int a = 0;
        if (m >= 0) {
          const float un = s_unscale[m], gate = acc[g][j] * un, up = acc[g][2 + j] * un;
          h = gate / (1.f + expf(-gate)) * up;
          a = m * p.top_k + s_slot[m * p.E + e];
          p.h[(int64_t)a * p.I + i] = h;
          const float hs = h * (float)(1 << kFastExp);
          const __half hi = __float2half_rn(hs);
          *reinterpret_cast<__half*>(p.h_hi + a * h_row + place) = hi;
          *reinterpret_cast<__half*>(p.h_lo + a * h_row + place) = __float2half_rn(hs - __half2float(hi));
        }
        uint32_t mx = __float_as_uint(h) & 0x7FFFFFFFu;
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        if (q == 0 && m >= 0) atomicMax(p.amax + a, mx);
      }
    }
  };
  for (int id = first_gu; id < gu_tiles; id += G * teams) {
    const int e = s_list[id / per_expert], i0 = id % per_expert * 8;
    const uint32_t tokens = s_mask[e];
    if (__popc(tokens) <= 8) gu_tile(std::integral_constant<int, 1>{}, e, i0, tokens);
    else gu_tile(std::integral_constant<int, kGuGroups>{}, e, i0, tokens);
  }
  ok = grid_barrier(p.bars + 1) && ok;  // every h is written

  // ---- h parts outside the fixed scale's range, made again; a choice's weight takes its scale ----
  {
    bool again = false;
    for (int a = tid; a < choices && ok; a += kThreads) {
      const uint32_t mx = __ldcg(p.amax + a);
      const bool out = !fast_range(mx);
      s_probs[a] *= exp2i(out ? -scale_exp(mx) : -kFastExp);
      again = again || out;
    }
    if (__syncthreads_or(again)) {  // the same answer in every CTA
      for (int a = blockIdx.x; a < choices; a += G) {
        const uint32_t mx = __ldcg(p.amax + a);
        if (fast_range(mx)) continue;
        const float scale = exp2i(scale_exp(mx));
        for (int i = tid; i < p.I; i += kThreads) {
          const float hs = __ldcg(p.h + (int64_t)a * p.I + i) * scale;
          const __half hi = __float2half_rn(hs);
          *reinterpret_cast<__half*>(p.h_hi + a * h_row + h_place(i)) = hi;
          *reinterpret_cast<__half*>(p.h_lo + a * h_row + h_place(i)) = __float2half_rn(hs - __half2float(hi));
        }
      }
      ok = grid_barrier(p.bars + 2) && ok;
    }
  }
  live = live && ok;

  // ---- down: a tile of output rows at a time, its experts' stages shared by the warps ----
  // column n < 4: the high part of the group's token n; n >= 4: the remainder of token n - 4
  const uint8_t* h_base = (q < 4 ? p.h_hi : p.h_lo) + c * 16;
  int u = 0;
  auto dn_run = [&](auto groups, int e, int n0, int at, int end, uint32_t tokens) {  // stages [u, end) of one expert
    constexpr int GROUPS = decltype(groups)::value;
    const int ng = GROUPS == 1 ? 1 : (__popc(tokens) + 3) / 4;
    int tok[GROUPS];
    float acc[GROUPS][4];
    Columns<GROUPS> col;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      tok[g] = g < ng ? token_of(tokens, 4 * g + (q & 3)) : -1;
      const int m = tok[g] >= 0 ? tok[g] : __ffs(tokens) - 1;
      col.p[g] = h_base + (m * p.top_k + s_slot[m * p.E + e]) * h_row + (u - at * sd) * (U::NS * U::X_SPAN);
      acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
    }
    col.start();
    for (; u < end; ++u) {
      if (!wait_stage()) {
        live = false;
        break;
      }
      const uint8_t* st = ring + (size_t)slot * U::STAGE;
      const int span = (u - at * sd) * U::NS, n = min(U::NS, spans_i - span);
      const uint8_t* ra = unit_at(st, q, dn_row(e, n0, q) + span * U::SPAN);
      const uint8_t* rb = unit_at(st, q + 8, dn_row(e, n0, q + 8) + span * U::SPAN);
      for (int k = 0; k < n; ++k)
        span_products<V, ALIGNED, 0, GROUPS>(ra + k * SPAN_STEP, rb + k * SPAN_STEP, (span + k) * U::SPAN_BLOCKS + c * U::BLOCKS, nb_i, ng, col, acc);
      release_stage();
    }
    // columns 2 c, 2 c + 1 (c < 2) with their remainders, of rows q and q + 8
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      if (g >= ng) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[g][i] += __shfl_xor_sync(0xffffffffu, acc[g][i], 2);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = __shfl_sync(0xffffffffu, tok[g], ((2 * c + j) & 3) * 4);
        if (c < 2 && m >= 0) {
          const float w = s_probs[m * p.top_k + s_slot[m * p.E + e]];
          acc_w[q * p.M + m] += w * acc[g][j];
          acc_w[(q + 8) * p.M + m] += w * acc[g][2 + j];
        }
      }
    }
  };
  for (int tile = 0; tile < my_tiles && ok; ++tile) {
    const int n0 = (blockIdx.x + tile * G) * kTileRows;
    for (int i = lane; i < kTileRows * p.M; i += 32) acc_w[i] = 0.f;
    __syncwarp();
    for (u = u0; u < u1 && live;) {
      const int at = u / sd, end = min(u1, (at + 1) * sd), e = s_list[at];
      const uint32_t tokens = s_mask[e];
      if (__popc(tokens) <= 4) dn_run(std::integral_constant<int, 1>{}, e, n0, at, end, tokens);
      else dn_run(std::integral_constant<int, kDnGroups>{}, e, n0, at, end, tokens);
    }
    __syncthreads();
    for (int i = tid; i < kTileRows * p.M; i += kThreads) {
      const int m = i / kTileRows, r = i % kTileRows;
      float y = 0.f;
      for (int w = 0; w < kWarps; ++w) y += s_acc[(size_t)w * p.acc_floats + r * p.M + m];
      p.Y[(int64_t)m * p.K + n0 + r] = y;
    }
    __syncthreads();
  }
  // copies that no one waited for (after a wait gave up) land before the CTA leaves
  for (; used < filled; next_slot()) (void)mbar_wait_bounded(smem_addr(&bars[slot]), parity);
  __syncthreads();
  if (tid == 0 && atomic_add_acq_rel_gpu(p.bars + 3, 1u) == (uint32_t)G - 1u)
    for (int i = 0; i < kMoeBarWords; ++i) store_relaxed_gpu(p.bars + i, 0u);
}

using MoeFn = void (*)(MoeParams);

template <int V>
MoeFn pick(int act, bool aligned) {
  if (act == 0) return aligned ? moe_kernel<V, 0, true> : moe_kernel<V, 0, false>;
  return aligned ? moe_kernel<V, 1, true> : moe_kernel<V, 1, false>;
}

constexpr int kSmemMax = 227 * 1024 - 2560;  // dynamic; the rest is the kernel's static shared memory
constexpr int kSlack = 32;                   // word reads past the last row slot

int up16(int v) { return (v + 15) / 16 * 16; }

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

template <int V>
cudaError_t set_up(const MoeArgs& a, int sms, MoeParams* p, int* smem) {
  using U = Unit<V>;
  int at = up16(p->M * p->top_k * 4);
  p->off_mask = at;
  at += up16(p->E * 4);
  p->off_list = at;
  at += up16(p->E * 2);
  p->off_slot = at;
  at += up16(p->M * p->E);
  p->off_unscale = at;
  at += up16(p->M * 4);
  p->off_keys = at;
  at += kWarps * up16(p->E * 4);
  p->off_acc = at;
  const int groups = (p->M + 7) / 8;
  p->acc_floats = kTileRows * p->M > groups * 128 ? kTileRows * p->M : groups * 128;
  at += kWarps * p->acc_floats * 4;
  const int64_t spans_k = (a.K / 32 + U::SPAN_BLOCKS - 1) / U::SPAN_BLOCKS, spans_i = (a.I / 32 + U::SPAN_BLOCKS - 1) / U::SPAN_BLOCKS;
  // The activations go to shared memory where the ring keeps two stages next
  // to them; rows 64 bytes off a multiple of 128, so that two tokens' loads
  // meet no bank twice.  Else they are read through L1.
  const int64_t x_bytes = a.M * (spans_k * U::X_SPAN + 64) + 256;
  p->off_x = at;
  if (x_bytes <= kSmemMax - kSlack - 128 - at - 2 * kWarps * U::STAGE) {
    p->x_pitch = (int)(spans_k * U::X_SPAN + 64);
    at += (int)x_bytes;
  }
  p->off_ring = (at + 127) / 128 * 128;
  const int room = (kSmemMax - p->off_ring - kSlack) / (kWarps * U::STAGE);
  p->stages = room < kMaxStages ? room : kMaxStages;
  if (p->stages < 1) return cudaErrorInvalidConfiguration;
  *smem = p->off_ring + kWarps * p->stages * U::STAGE + kSlack;
  // Warps to a gate/up tile: one where every SM has tiles for its warps, more
  // where the (at most min(E, M top_k)) chosen experts give it fewer.
  const int64_t experts = a.M * a.top_k < a.E ? a.M * a.top_k : a.E;
  p->parts = 1;
  while (kWarps % (2 * p->parts) == 0 && p->parts < 8 && 2 * p->parts <= spans_k && experts * (a.I / 8) * p->parts < 8 * (int64_t)sms) p->parts *= 2;
  // Workspace: logits, activation scales, largest |h|, then 16-byte aligned arrays.
  const int64_t choices = a.M * a.top_k;
  float* w = a.ws;
  p->logits = w;
  w += kMoeMaxTokens * kMoeMaxExperts;
  p->x_unscale = w;
  w += kMoeMaxTokens;
  p->amax = reinterpret_cast<uint32_t*>(w);
  w += kMoeMaxTokens * kMoeMaxTop;
  p->h = w;
  w += choices * a.I;
  p->xf = reinterpret_cast<uint8_t*>(w);
  p->h_hi = p->xf + a.M * spans_k * U::X_SPAN;
  p->h_lo = p->h_hi + choices * spans_i * U::X_SPAN;
  return cudaSuccess;
}

template <int V>
cudaError_t encode_maps(const MoeArgs& a, MoeParams* p) {
  using U = Unit<V>;
  const cuuint64_t rb_k = a.K / 32 * Fmt<V>::BB, rb_i = a.I / 32 * Fmt<V>::BB;
  const cuuint32_t one[3] = {1, 1, 1};
  {
    const cuuint64_t dims[3] = {rb_k / 4, (cuuint64_t)a.I, 2 * (cuuint64_t)a.E}, strides[2] = {rb_k, rb_k * a.I};
    const cuuint32_t box[3] = {U::SPAN / 4, 8, 2};
    if (g_encode(&p->map_gu, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(a.Wgu), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const cuuint64_t dims[2] = {rb_i / 4, (cuuint64_t)(a.E * a.K)}, strides[1] = {rb_i};
  const cuuint32_t box[2] = {U::SPAN / 4, kTileRows};
  if (g_encode(&p->map_dn, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(a.Wd), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

}  // namespace

cudaError_t moe_prepare() {
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorSymbolNotFound;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  for (int v = 0; v < 2; ++v)
    for (int act = 0; act < 2; ++act)
      for (int al = 0; al < 2; ++al) {
        const MoeFn fn = v == 0 ? pick<0>(act, al) : pick<1>(act, al);
        cudaError_t e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_moe(int variant, int act, const MoeArgs& a, int sms, cudaStream_t s) {
  MoeParams p{};
  p.X = a.X;
  p.router = a.router;
  p.Wgu = a.Wgu;
  p.Wd = a.Wd;
  p.Y = a.Y;
  p.ids = a.ids;
  p.probs = a.probs;
  p.bars = a.bars;
  p.err = a.err;
  p.M = (int)a.M;
  p.E = (int)a.E;
  p.top_k = (int)a.top_k;
  p.K = (int)a.K;
  p.I = (int)a.I;
  p.router_type = a.router_type;
  p.route = a.route;
  p.route_scale = a.route_scale;
  int smem = 0;
  cudaError_t e = variant == 0 ? set_up<0>(a, sms, &p, &smem) : set_up<1>(a, sms, &p, &smem);
  if (e != cudaSuccess) return e;
  const int ku = variant == 0 ? Fmt<0>::KU : Fmt<1>::KU;
  const bool aligned = a.K % ku == 0 && a.I % ku == 0 && a.E * a.K < (int64_t(1) << 31);
  if (aligned && (e = variant == 0 ? encode_maps<0>(a, &p) : encode_maps<1>(a, &p)) != cudaSuccess) return e;
  const MoeFn fn = variant == 0 ? pick<0>(act, aligned) : pick<1>(act, aligned);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // its CTAs wait on one another: all resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace rocmfp4
