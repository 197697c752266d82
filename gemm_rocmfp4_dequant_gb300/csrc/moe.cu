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
// (16 single-scale blocks) of each row.  A warp takes tiles on its own (the
// last of a CTA's gate/up tiles, too few for a tile a warp, go to teams of two
// or four warps that share a tile's spans) and streams their spans through a
// private ring of shared-memory stages, one tensor copy of a 16-row box a span.
// The down tasks are known as soon as the routing is, so the ring runs on into
// them before the second barrier.  The ring has two stages; one from 13 to 25
// tokens on (by experts, layout and alignment), where the tokens' outputs and
// sums take the room and a warp's next copy starts when it has done with the last.
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
// behind a third barrier that other calls do not meet.  There an infinite h
// (an overflow of its product) keeps a remainder of 0, so that its sign
// reaches the outputs.
//
// Bound: memory (3 I K / 32 blocks per chosen expert) and, as close, the
// decode: 387 cycles an SM quarter for 16 rows x 256 weights with everything in
// shared memory, 268 of them the conversion, clamp and scaling of the pairs.
// Short calls are bound by the chain of phases: 3 us to the first barrier, 2
// for the choices, 1.7 until the first copies are under way, 1.3 a barrier.
//
// Measured on one GB300, dual, 128 experts of [2 x 768, 2048] + [2048, 768], 8
// chosen: one token 20.5 us (21.8 MB; a cooperative launch starts every 2.048
// us at best), eight tokens 50 to 54 us (137.6 MB, 2.6 TB/s); 64 experts of
// [2 x 1536, 5120], single-scale, 6 chosen, four tokens: 85 to 94 us (2.9 TB/s).
// 16 warps: with 12 (and 168 registers) the last ran 104 us.  The first layer
// at 16, 24 and 32 tokens: 74, 96 and 113 us, 2.9, 2.8 and 2.5 TB/s of the
// blocks that they reach; the last two with one stage.
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

constexpr int kWarps = kMoeWarps;
constexpr int kThreads = kWarps * 32;
constexpr int kTileRows = kMoeTileRows;
constexpr int kMaxStages = kMoeMaxStages;
constexpr int kRouterTokens = 8;   // tokens a router pass holds
constexpr int kTouchBytes = 32768;  // activations asked for ahead of use
constexpr int kFastExp = 4;        // h times 2^4 in its fp16 pair

template <int V>
struct Unit {
  static constexpr int BLOCKS = Fmt<V>::BPL;       // blocks a lane has of a span: 2 / 4
  static constexpr int BYTES = Fmt<V>::LANE_BYTES; // 36 / 68
  static constexpr int SPAN = Fmt<V>::SPAN;        // 144 / 272
  static constexpr int SPAN_BLOCKS = 4 * BLOCKS;   // 8 / 16
  static constexpr int X_SPAN = SPAN_BLOCKS * 64;  // bytes of a span's fp16 activations
};

static_assert(Unit<0>::SPAN == moe_span_bytes(0) && Unit<1>::SPAN == moe_span_bytes(1), "the layout's spans");
static_assert(Unit<0>::SPAN_BLOCKS == moe_span_blocks(0) && Unit<1>::SPAN_BLOCKS == moe_span_blocks(1), "the layout's spans");

// Bytes from span to span of a stage.
template <int V, bool ALIGNED>
RF4_HOSTDEV constexpr int span_step() { return ALIGNED ? kTileRows * Unit<V>::SPAN : Unit<V>::SPAN; }

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
  MoeLayout l;
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
// Whether the fp16 pair of h made with the fixed scale is good: 0 or [2^-5, 2^11).
RF4_DEV bool fast_range(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return amax_bits == 0 || (e >= 127 - 5 && e < 127 + 11);
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

// One group of at most eight columns (most experts of a few tokens).  `p` moves
// through the lane's activations, 256 bytes a block; the next block's are
// loaded while this one's weights are decoded, in turn into a and b.  Columns
// beyond the expert's tokens repeat its first; their sums are not used.
struct Column {
  const uint8_t* p;
  uint4 a[4], b[4];
  float acc[4];
  RF4_DEV void start(const uint8_t* first) {
    p = first;
    load_b(p, a);
    acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
  }
  // Block PHI and those after it of a unit; ra, rb: rows q and q + 8 at the lane's unit; blk: its first block.
  template <int V, bool ALIGNED, int PHI>
  RF4_DEV void unit(const uint8_t* ra, const uint8_t* rb, int blk, int nb) {
    const bool have = ALIGNED || blk + PHI < nb;
    const Block<V, ALIGNED, PHI> x(ra, have), y(rb, have);
    uint4(&now)[4] = PHI % 2 ? b : a;
    load_b(p + 256 * (PHI + 1), PHI % 2 ? a : b);  // reads past the row's last block stay in the workspace
    float d[2][4];  // eight MMAs in two chains
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (kk < 2) mma_z(d[kk & 1], x.pair(4 * kk), y.pair(4 * kk), x.pair(4 * kk + 1), y.pair(4 * kk + 1), now[kk].x, now[kk].y);
      else mma(d[kk & 1], x.pair(4 * kk), y.pair(4 * kk), x.pair(4 * kk + 1), y.pair(4 * kk + 1), now[kk].x, now[kk].y);
      mma(d[kk & 1], x.pair(4 * kk + 2), y.pair(4 * kk + 2), x.pair(4 * kk + 3), y.pair(4 * kk + 3), now[kk].z, now[kk].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += d[0][i] + d[1][i];
    if constexpr (PHI + 1 < Unit<V>::BLOCKS) unit<V, ALIGNED, PHI + 1>(ra, rb, blk, nb);
    else p += 256 * Unit<V>::BLOCKS;
  }
};

// Several groups: the weights are decoded once, then meet each group's columns.
// The sums lie in shared memory (one float4 a lane and group): registers and
// code stay small, and the eight MMAs of a group cover the way there and back.
struct Columns {
  const uint8_t* p;
  const uint32_t* off;  // bytes from p to the activations of the lane's column, one in eight words a group
  float4* sums;
  int ng;
  template <int V, bool ALIGNED, int PHI>
  RF4_DEV void unit(const uint8_t* ra, const uint8_t* rb, int blk, int nb) {
    const bool have = ALIGNED || blk + PHI < nb;
    uint32_t a0[16], a1[16];
    {
      const Block<V, ALIGNED, PHI> x(ra, have), y(rb, have);
#pragma unroll
      for (int j = 0; j < 16; ++j) a0[j] = x.pair(j), a1[j] = y.pair(j);
    }
#pragma unroll 1
    for (int g = 0; g < ng; ++g) {
      uint4 b[4];
      load_b(p + off[8 * g] + 256 * PHI, b);
      float d[2][4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk < 2) mma_z(d[kk & 1], a0[4 * kk], a1[4 * kk], a0[4 * kk + 1], a1[4 * kk + 1], b[kk].x, b[kk].y);
        else mma(d[kk & 1], a0[4 * kk], a1[4 * kk], a0[4 * kk + 1], a1[4 * kk + 1], b[kk].x, b[kk].y);
        mma(d[kk & 1], a0[4 * kk + 2], a1[4 * kk + 2], a0[4 * kk + 3], a1[4 * kk + 3], b[kk].z, b[kk].w);
      }
      float4 s = sums[32 * g];
      s.x += d[0][0] + d[1][0], s.y += d[0][1] + d[1][1], s.z += d[0][2] + d[1][2], s.w += d[0][3] + d[1][3];
      sums[32 * g] = s;
    }
    if constexpr (PHI + 1 < Unit<V>::BLOCKS) unit<V, ALIGNED, PHI + 1>(ra, rb, blk, nb);
    else p += 256 * Unit<V>::BLOCKS;
  }
};

// The bytes [a, a + n) as a copy from 16-byte boundary to 16-byte boundary.
RF4_DEV uint32_t span_bytes(const uint8_t* a, int n) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(a) & ~uintptr_t(15), e = (reinterpret_cast<uintptr_t>(a) + n + 15) & ~uintptr_t(15);
  return (uint32_t)(e - b);
}
RF4_DEV void copy_span(uint8_t* dst, const uint8_t* a, int n, uint32_t bar) {
  bulk_g2s(smem_addr(dst), reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(a) & ~uintptr_t(15)), span_bytes(a, n), bar);
}
RF4_DEV int mis16(const uint8_t* a) { return (int)(reinterpret_cast<uintptr_t>(a) & 15u); }

// Asks for a line of global memory to be brought to L1; nothing waits for it.
RF4_DEV void touch(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.ca.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  (void)v;
}

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
  float* s_probs = reinterpret_cast<float*>(smem);                          // [M][top_k]
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + p.l.off_mask);      // [E]: tokens of an expert
  uint16_t* s_list = reinterpret_cast<uint16_t*>(smem + p.l.off_list);      // chosen experts, ascending
  uint8_t* s_slot = smem + p.l.off_slot;                                    // [M][E]: which choice of the token
  float* s_unscale = reinterpret_cast<float*>(smem + p.l.off_unscale);      // [M]: 1 / the activations' scale
  float* s_y = reinterpret_cast<float*>(smem + p.l.off_y);                  // [kWarps][M][16]: outputs of a down tile
  float* s_acc = reinterpret_cast<float*>(smem + p.l.off_acc);              // [kWarps][acc_floats]
  __shared__ uint64_t s_bars[kWarps * kMaxStages];
  __shared__ uint64_t s_pick[kWarps][kMoeMaxTop];
  __shared__ float s_red[kWarps][kRouterTokens];
  // Columns of the expert a warp is at: bytes to their activations, their
  // choice (gate/up) or token (down), -1 for none, and, of its activations, 1 / the scale (gate/up) or the choice's weight (down).
  __shared__ uint32_t s_off[kWarps * 64];
  __shared__ int16_t s_choice[kWarps * 64];
  __shared__ float s_un[kWarps * 64];
  __shared__ uint32_t s_amax[kMoeMaxTokens * kMoeMaxTop];  // bits of the choices' largest |h| in this CTA
  __shared__ int s_active, s_ok;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = gridDim.x;

  uint64_t* bars = s_bars + warp * kMaxStages;
  if (lane == 0) {
    for (int i = 0; i < p.l.stages; ++i) mbar_init(smem_addr(&bars[i]), 1);
    fence_mbar_init();
  }
  if (ALIGNED && tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_gu)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map_dn)) : "memory");
  }
  if (tid == 0) s_ok = 1;
  for (int e = tid; e < p.E; e += kThreads) s_mask[e] = 0;
  for (int a = tid; a < p.M * p.top_k; a += kThreads) s_amax[a] = 0;
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
#pragma unroll 1
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
#pragma unroll 2
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
#pragma unroll 1
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

  if (ok && tid < p.M) s_unscale[tid] = __ldcg(p.x_unscale + tid);
  // The activations on their way to L1 while the choices are made (the
  // products would meet each line's latency in turn); not more than it holds.
  for (int64_t i = (int64_t)tid * 128; ok && i < p.M * spans_k * U::X_SPAN && i < kTouchBytes; i += kThreads * 128) touch(p.xf + i);
  // ---- top k of every token (one warp per token), repeated by every CTA ----
  if (ok) {
    // Room in what is idle yet: the order of every expert's logit, then the
    // candidates: those that reach the top_k-th largest of the lanes' maxima.
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem + p.l.off_select + warp * p.l.select_bytes);
    uint64_t* cand = reinterpret_cast<uint64_t*>(keys + 2 * p.E);
    for (int m = warp; m < p.M; m += kWarps) {
      uint32_t best = 0;
      for (int e = lane; e < p.E; e += 32) {
        const uint32_t k = logit_key(__ldcg(p.logits + (int64_t)m * p.E + e));
        keys[e] = k;
        best = max(best, k);
      }
      __syncwarp();
      const float top = logit_of(__reduce_max_sync(0xffffffffu, best));
      int rank = 0;  // of the lane's maximum, equal ones in lane order
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const uint32_t o = __shfl_sync(0xffffffffu, best, i);
        rank += o > best || (o == best && i < lane) ? 1 : 0;
      }
      const uint32_t least = __shfl_sync(0xffffffffu, best, __ffs(__ballot_sync(0xffffffffu, rank == p.top_k - 1)) - 1);
      int n = 0;
#pragma unroll 1
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        const uint32_t k = e < p.E ? keys[e] : 0u;
        const bool in = e < p.E && k >= least;
        const uint32_t b = __ballot_sync(0xffffffffu, in);
        if (in) cand[n + __popc(b & ((1u << lane) - 1u))] = (uint64_t)k << 32 | (uint32_t)~e;  // equal logits: the lowest expert first
        n += __popc(b);
      }
      __syncwarp();
#pragma unroll 1
      for (int i = lane; i < n; i += 32) {
        const uint64_t k = cand[i];
        int r = 0;
#pragma unroll 2
        for (int o = 0; o < n; ++o) r += cand[o] > k ? 1 : 0;
        if (r < p.top_k) s_pick[warp][r] = k;
      }
      float denom = 0.f;
      if (p.route == 0)  // softmax over all experts
#pragma unroll 1
        for (int e = lane; e < p.E; e += 32) denom += expf(logit_of(keys[e]) - top);
      __syncwarp();
      const uint64_t pick = s_pick[warp][lane < p.top_k ? lane : 0];
      const uint32_t my_key = (uint32_t)(pick >> 32);
      const int my_id = (int)~(uint32_t)pick;
      __syncwarp();
      const float mine = logit_of(my_key);
      float num = 0.f;
      if (p.route == 2) {
        // Below 0 the sigmoids times exp(-top), which cancels: all of them may be too small for fp32.
        num = lane >= p.top_k ? 0.f : top < 0.f ? expf(mine - top) / (1.f + expf(mine)) : 1.f / (1.f + expf(-mine));
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
  fence_proxy_async();  // the ring's use above precedes the copies into it
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
  const int per_expert = p.I / 8;  // gate/up tiles of an expert
  // A CTA's gate/up tiles are neighbours, so that its warps share activations
  // in L1.  Rounds of a tile a warp; the tiles left over go to teams of KP
  // warps, each with its part of the spans (a round of few tiles would leave
  // most warps idle for as long as a whole tile takes.  Whole calls, a warp a
  // tile always: 22.6, 51.4, 90.0 and 28.7 us; teams: 20.5, 50.6, 88.0 and
  // 25.5, for the three sizes named on top and 13 tokens over 10 experts of
  // width 352).
  const int g0 = (int)((int64_t)A * per_expert * blockIdx.x / G), n_gu = (int)((int64_t)A * per_expert * (blockIdx.x + 1) / G) - g0;
  const int rounds_gu = n_gu / kWarps, left = n_gu - rounds_gu * kWarps;
  int KP = left > 8 ? 1 : left > 4 ? 2 : 4;
  while (KP > spans_k) KP /= 2;
  const int team = warp / KP, part = warp - team * KP;
  const int l0 = spans_k * part / KP, l1 = spans_k * (part + 1) / KP;  // spans of a tile left over
  const int jobs_gu = rounds_gu + (team < left ? 1 : 0);              // this warp's
  auto tile_of = [&](int j) { return g0 + rounds_gu * kWarps + (j < rounds_gu ? (j - rounds_gu) * kWarps + warp : team); };
  // Down: a CTA takes 16-row tiles, and its warps share the stages of a tile
  // (every chosen expert's rows) in equal runs.
  const int ns = p.l.ns, sd = (spans_i + ns - 1) / ns;
  const int tiles = p.K / kTileRows, my_tiles = (int)blockIdx.x < tiles ? (tiles - (int)blockIdx.x + G - 1) / G : 0;
  const int u0 = warp * (A * sd) / kWarps, u1 = (warp + 1) * (A * sd) / kWarps;
  uint8_t* ring = smem + p.l.off_ring + warp * p.l.stages * p.l.stage_bytes;

  // Lane (q, c) reads rows q and q + 8 of a stage at unit c of each span.
  // Unaligned rows start at their own place within 16 bytes.
  const int q = lane >> 2, c = lane & 3, pitch = moe_row_pitch(V, ALIGNED, ns);
  constexpr int STEP = span_step<V, ALIGNED>();
  const int unit_a = q * pitch + c * U::BYTES, unit_b = unit_a + 8 * pitch;
  auto gu_row = [&](int e, int i0, int r) { return p.Wgu + ((int64_t)e * 2 * p.I + (r < 8 ? 0 : p.I) + i0 + (r & 7)) * rb_k; };
  auto dn_row = [&](int e, int n0, int r) { return p.Wd + ((int64_t)e * p.K + n0 + r) * rb_i; };

  // Copies of ns spans from `span` on, up to `last`, of a tile's 16 rows into a stage.
  auto fill = [&](bool down, int e, int row0, int span, int last, int slot) {
    uint8_t* dst = ring + slot * p.l.stage_bytes;
    const uint32_t bar = smem_addr(&bars[slot]);
    if constexpr (ALIGNED) {
      if (lane == 0) {
        const int n = min(ns, last - span);
        mbar_arrive_expect_tx(bar, (uint32_t)(n * kTileRows * U::SPAN));
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
          const uint32_t to = smem_addr(dst) + k * (kTileRows * U::SPAN);
          if (down) tma_load_2d(to, &p.map_dn, (span + k) * (U::SPAN / 4), e * p.K + row0, bar);
          else tma_load_3d(to, &p.map_gu, (span + k) * (U::SPAN / 4), row0, 2 * e, bar);
        }
      }
    } else {
      const int rb = down ? rb_i : rb_k, lo = span * U::SPAN, len = min(rb - lo, min(ns, last - span) * U::SPAN);
      const uint8_t* src = (down ? dn_row(e, row0, lane & 15) : gu_row(e, row0, lane & 15)) + lo;
      const uint32_t bytes = __reduce_add_sync(0xffffffffu, lane < kTileRows ? span_bytes(src, len) : 0u);
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (lane < kTileRows) copy_span(dst + lane * pitch, src, len, bar);
    }
  };
  // The next stage to fill: of gate/up job `id` (expert, first row, next span and
  // the end), then of a down tile (stage u of tile `id` of this CTA's).
  struct {
    bool gu, any;
    int id, e, row0, span, last, u, at;  // at: place of e in the list
  } nx;
  auto start_gu = [&](int id) {
    const int tile = tile_of(id);
    while (tile >= (nx.at + 1) * per_expert) ++nx.at;
    nx.id = id;
    nx.e = s_list[nx.at];
    nx.row0 = (tile - nx.at * per_expert) * 8;
    nx.span = id < rounds_gu ? 0 : l0;
    nx.last = id < rounds_gu ? spans_k : l1;
  };
  auto start_dn = [&]() {
    nx.gu = false;
    nx.any = u0 < u1 && my_tiles > 0;
    nx.id = 0;
    nx.u = u0;
    nx.at = u0 / max(sd, 1);
    nx.last = spans_i;
  };
  nx.gu = nx.any = jobs_gu > 0;
  if (nx.gu) nx.at = tile_of(0) / per_expert, start_gu(0);
  else start_dn();
  int fill_slot = 0, filled = 0;
  auto fill_next = [&]() {
    if (!nx.any) return;
    if (!nx.gu) {
      if (nx.u == (nx.at + 1) * sd) ++nx.at;
      nx.e = s_list[nx.at];
      nx.row0 = (blockIdx.x + nx.id * G) * kTileRows;
      nx.span = (nx.u - nx.at * sd) * ns;
    }
    fill(!nx.gu, nx.e, nx.row0, nx.span, nx.last, fill_slot);
    if (nx.gu) {
      nx.span += ns;
      if (nx.span >= nx.last) {
        if (nx.id + 1 < jobs_gu) start_gu(nx.id + 1);
        else start_dn();
      }
    } else if (++nx.u == u1) {
      nx.u = u0;
      nx.at = u0 / sd;
      nx.any = ++nx.id < my_tiles;
    }
    if (++fill_slot == p.l.stages) fill_slot = 0;
    ++filled;
  };
  int slot = 0, used = 0;
  uint32_t parity = 0;
#pragma unroll 1
  for (int i = 0; i < p.l.stages; ++i) fill_next();
  auto next_slot = [&]() {
    ++used;
    if (++slot == p.l.stages) slot = 0, parity ^= 1u;
  };
  // The next stage, once its copies have landed.  If a wait gives up, nothing
  // more is copied or waited for: the outputs are invalid, and an error bit says so.
  auto wait_stage = [&]() {
    if (used < filled && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&bars[slot]), parity))) {
      if (lane == 0) atomicOr(p.err, kErrWaitTimeout);
      nx.any = false;
    }
    return ring + slot * p.l.stage_bytes;
  };
  auto release_stage = [&]() {
    __syncwarp();
    fence_proxy_async();  // the stage's reads precede the next copy into it
    fill_next();
    next_slot();
  };
  // The token after `skip` others of a set, -1 for none.
  auto token_of = [&](uint32_t tokens, int skip) {
#pragma unroll 1
    for (int i = 0; i < skip; ++i) tokens &= tokens - 1;
    return tokens ? __ffs(tokens) - 1 : -1;
  };
  float* acc_w = s_acc + (size_t)warp * p.l.acc_floats;
  uint32_t* off_w = s_off + warp * 64;
  int16_t* choice_w = s_choice + warp * 64;
  float* un_w = s_un + warp * 64;

  // The h parts of an expert's first token on their way to L1, one expert ahead of use.
  auto fetch_h = [&](int at) {
    const int e = s_list[at], m = __ffs(s_mask[e]) - 1;
    const int64_t row = (m * p.top_k + s_slot[m * p.E + e]) * h_row;
    for (int64_t i = lane * 128; i < h_row && i < 4096; i += 4096) touch(p.h_hi + row + i), touch(p.h_lo + row + i);
  };
  // ---- the two products: gate and up (phase 0), then down (phase 1) ----------------------
  // One loop for both, and one copy of its code: a launch meets most of it
  // once, and instruction fetches are a good part of a short call.
  float* y_w = s_y + warp * (kTileRows * p.M);  // down: the warp's part of a tile's outputs
  float4* sums = reinterpret_cast<float4*>(acc_w) + lane;
#pragma unroll 1
  for (int phase = 0; phase < 2; ++phase) {
    const bool down = phase == 1;
    const int nb = down ? nb_i : nb_k;
    // Columns: eight tokens; or the high parts of four tokens' h, then their remainders.
    const int width = down ? 4 : 8;
    const uint8_t* b0 = (down ? (q < 4 ? p.h_hi : p.h_lo) : p.xf) + c * 16;
    const uint32_t b_row = (uint32_t)(down ? h_row : (int64_t)spans_k * U::X_SPAN);
    const int rounds = !ok ? 0 : down ? my_tiles : 1;
    int noted = -1, ng = 0;  // the place in the list whose columns are noted
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
      if (down) {
        for (int i = lane; i < kTileRows * p.M; i += 32) y_w[i] = 0.f;
        __syncwarp();
      }
      // gate/up: job x; down: stages from x on of one expert
      const int per = down ? sd : per_expert;
      int at = (down ? u0 : tile_of(0)) / max(per, 1);
#pragma unroll 1
      for (int x = down ? u0 : 0; x < (down ? u1 : jobs_gu);) {
        const int place = down ? x : tile_of(x);
        while (place >= (at + 1) * per) ++at;
        const int e = s_list[at];
        int row0, s0, s1, parts = 1;
        if (down) {
          const int last = min(u1, (at + 1) * sd);
          row0 = (blockIdx.x + round * G) * kTileRows;
          s0 = (x - at * sd) * ns;
          s1 = min(spans_i, (last - at * sd) * ns);
          x = last;
        } else {
          row0 = (place - at * per_expert) * 8;
          s0 = x < rounds_gu ? 0 : l0, s1 = x < rounds_gu ? spans_k : l1;
          parts = x < rounds_gu ? 1 : KP;
          ++x;
        }
        if (at != noted) {
          if (down && x < u1) fetch_h(at + 1);
          noted = at;
          const uint32_t tokens = s_mask[e];
          ng = (__popc(tokens) + width - 1) / width;
          __syncwarp();
#pragma unroll 1
          for (int n = lane; n < 8 * ng; n += 32) {  // column n: token width * (n / 8) + n % width of the set
            const int t = token_of(tokens, width * (n >> 3) + (n & (width - 1))), m = t >= 0 ? t : __ffs(tokens) - 1;
            const int a = m * p.top_k + s_slot[m * p.E + e];
            off_w[n] = (uint32_t)(down ? a : m) * b_row;
            choice_w[n] = (int16_t)(t < 0 ? -1 : down ? m : a);
            un_w[n] = down ? s_probs[a] : s_unscale[m];
          }
          __syncwarp();
        }
        int ma = 0, mb = 0;
        if constexpr (!ALIGNED) {
          ma = mis16(down ? dn_row(e, row0, q) : gu_row(e, row0, q));
          mb = mis16(down ? dn_row(e, row0, q + 8) : gu_row(e, row0, q + 8));
        }
        auto stages = [&](auto& col) {
#pragma unroll 1
          for (int span = s0; span < s1; span += ns) {
            const uint8_t* st = wait_stage();
            const int n = min(ns, s1 - span);
#pragma unroll 1
            for (int k = 0; k < n; ++k)
              col.template unit<V, ALIGNED, 0>(st + unit_a + ma + k * STEP, st + unit_b + mb + k * STEP, (span + k) * U::SPAN_BLOCKS + c * U::BLOCKS, nb);
            release_stage();
          }
        };
        if (ng == 1) {
          Column col;
          col.start(b0 + off_w[q] + s0 * U::X_SPAN);
          stages(col);
          sums[0] = make_float4(col.acc[0], col.acc[1], col.acc[2], col.acc[3]);
        } else {
          Columns col{b0 + s0 * U::X_SPAN, off_w + q, sums, ng};
          for (int g = 0; g < ng; ++g) sums[32 * g] = make_float4(0.f, 0.f, 0.f, 0.f);
          stages(col);
        }
        // Lane (q, c): rows q and q + 8, columns 2 c and 2 c + 1 of every group.
        if (parts > 1) team_barrier(1 + team, KP * 32);
        if (down) {
#pragma unroll 1
          for (int g = 0; g < ng; ++g) {
            const float4 v = sums[32 * g];
            const float s[4] = {v.x + __shfl_xor_sync(0xffffffffu, v.x, 2), v.y + __shfl_xor_sync(0xffffffffu, v.y, 2),
                                v.z + __shfl_xor_sync(0xffffffffu, v.z, 2), v.w + __shfl_xor_sync(0xffffffffu, v.w, 2)};
            if (c < 2) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int n = 8 * g + 2 * c + j, m = choice_w[n];
                if (m >= 0) {
                  float* y = y_w + m * kTileRows + q;
                  y[0] += un_w[n] * s[j];
                  y[8] += un_w[n] * s[2 + j];
                }
              }
            }
          }
        } else if (parts == 1 || part == 0) {
          const int i = row0 + q;
          const int64_t place = h_place(i);
#pragma unroll 1
          for (int g = 0; g < ng; ++g) {
            float4 v = sums[32 * g];
#pragma unroll 1
            for (int w = 1; w < parts; ++w) {  // the parts' sums, in order
              const float4 o = *reinterpret_cast<const float4*>(acc_w + (size_t)w * p.l.acc_floats + (32 * g + lane) * 4);
              v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            const float gates[2] = {v.x, v.y}, ups[2] = {v.z, v.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int n = 8 * g + 2 * c + j, a = choice_w[n];
              if (a >= 0) {
                const float gate = gates[j] * un_w[n], up = ups[j] * un_w[n];
                const float h = gate / (1.f + expf(-gate)) * up, hs = h * (float)(1 << kFastExp);
                const __half hi = __float2half_rn(hs);
                p.h[(int64_t)a * p.I + i] = h;
                *reinterpret_cast<__half*>(p.h_hi + a * h_row + place) = hi;
                *reinterpret_cast<__half*>(p.h_lo + a * h_row + place) = __float2half_rn(hs - __half2float(hi));
                atomicMax(&s_amax[a], __float_as_uint(h) & 0x7FFFFFFFu);
              }
            }
          }
        }
        if (parts > 1) team_barrier(1 + team, KP * 32);
      }
      if (down) {  // the warps' parts, in order
        __syncthreads();
        const int n0 = (blockIdx.x + round * G) * kTileRows;
        for (int i = tid; i < kTileRows * p.M; i += kThreads) {
          float y = 0.f;
          for (int w = 0; w < kWarps; ++w) y += s_y[w * (kTileRows * p.M) + i];
          p.Y[(int64_t)(i / kTileRows) * p.K + n0 + i % kTileRows] = y;
        }
        __syncthreads();
      }
    }
    if (down) break;

    __syncthreads();
    for (int a = tid; a < choices; a += kThreads)
      if (s_amax[a] != 0) atomicMax(p.amax + a, s_amax[a]);
    ok = grid_barrier(p.bars + 1) && ok;  // every h is written
    // h parts outside the fixed scale's range are made again; a choice's weight takes its scale
    bool again = false;
    for (int a = tid; a < choices && ok; a += kThreads) {
      const uint32_t mx = __ldcg(p.amax + a);
      const bool out = !fast_range(mx);
      s_probs[a] *= exp2i(out ? -scale_exp(mx) : -kFastExp);
      again = again || out;
    }
    if (__syncthreads_or(again)) {  // the same answer in every CTA
#pragma unroll 1
      for (int a = blockIdx.x; a < choices; a += G) {
        const uint32_t mx = __ldcg(p.amax + a);
        if (fast_range(mx)) continue;
        const float scale = exp2i(scale_exp(mx));
#pragma unroll 1
        for (int i = tid; i < p.I; i += kThreads) {
          float hs = __ldcg(p.h + (int64_t)a * p.I + i) * scale;
          // Beside an infinite h (or a NaN) every output is infinite or NaN,
          // whatever the others are, as long as they stay finite.
          if (mx >= 0x7F800000u && fabsf(hs) < INFINITY) hs = fminf(fmaxf(hs, -65504.f), 65504.f);
          const __half hi = __float2half_rn(hs);
          *reinterpret_cast<__half*>(p.h_hi + a * h_row + h_place(i)) = hi;
          *reinterpret_cast<__half*>(p.h_lo + a * h_row + h_place(i)) = __float2half_rn(fabsf(hs) == INFINITY ? 0.f : hs - __half2float(hi));
        }
      }
      ok = grid_barrier(p.bars + 2) && ok;
    }
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

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

template <int V>
cudaError_t encode_maps(const MoeArgs& a, MoeParams* p) {
  const cuuint64_t rb_k = a.K / 32 * Fmt<V>::BB, rb_i = a.I / 32 * Fmt<V>::BB;
  const cuuint32_t one[3] = {1, 1, 1}, words = Unit<V>::SPAN / 4;
  {
    const cuuint64_t dims[3] = {rb_k / 4, (cuuint64_t)a.I, 2 * (cuuint64_t)a.E}, strides[2] = {rb_k, rb_k * a.I};
    const cuuint32_t box[3] = {words, 8, 2};
    if (g_encode(&p->map_gu, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(a.Wgu), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const cuuint64_t dims[2] = {rb_i / 4, (cuuint64_t)(a.E * a.K)}, strides[1] = {rb_i};
  const cuuint32_t box[2] = {words, kTileRows};
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
        cudaError_t e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeSmemMax);
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
  const int ku = variant == 0 ? Fmt<0>::KU : Fmt<1>::KU;
  const bool aligned = a.K % ku == 0 && a.I % ku == 0;
  if (!moe_layout(variant, aligned, a.M, a.E, a.top_k, a.K, a.I, &p.l)) return cudaErrorInvalidConfiguration;
  p.logits = a.ws + p.l.ws_logits;
  p.x_unscale = a.ws + p.l.ws_unscale;
  p.amax = reinterpret_cast<uint32_t*>(a.ws + p.l.ws_amax);
  p.h = a.ws + p.l.ws_h;
  p.xf = reinterpret_cast<uint8_t*>(a.ws + p.l.ws_x);
  p.h_hi = reinterpret_cast<uint8_t*>(a.ws + p.l.ws_hi);
  p.h_lo = reinterpret_cast<uint8_t*>(a.ws + p.l.ws_lo);
  cudaError_t e;
  if (aligned && (e = variant == 0 ? encode_maps<0>(a, &p) : encode_maps<1>(a, &p)) != cudaSuccess) return e;
  const MoeFn fn = variant == 0 ? pick<0>(act, aligned) : pick<1>(act, aligned);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.l.bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // its CTAs wait on one another: all resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace rocmfp4
