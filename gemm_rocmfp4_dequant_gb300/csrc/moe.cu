// A whole mixture-of-experts layer for a few tokens (M <= 32), in one kernel:
//   l = R x                         router logits of every expert, fp32
//   top_k experts by (l descending, index ascending), weights p by the route
//   h = SiLU(Wg x) * (Wu x)         per chosen expert, fp32
//   Y = sum over choices of p * (Wd h)
// with every expert's Wg, Wu (stacked) and Wd in packed ROCmFP4 blocks.  Only
// the blocks of chosen experts are read, each once.
//
// Bound: memory (3 I K / 32 blocks per chosen expert) at a token or two per
// expert; the decode's ALU work (about 5 instructions a byte) is close behind.
//
// One persistent CTA per SM, launched cooperatively, in three phases with two
// grid barriers: router logits; gate and up products (h goes to the
// workspace); down products.  Every CTA repeats the small top-k selection for
// itself, which costs less than handing its result on.  The products are
// cut into tasks of a few whole rows that warps take on their own: a warp
// streams its tasks' rows by bulk copies into a private ring of shared-memory
// stages, and because the down tasks are known as soon as the routing is, the
// ring runs on into them before the second barrier.
//
// Products.  A unit is a 4-byte multiple of whole blocks of a row: two dual
// blocks (36 bytes) or four single-scale blocks (68 bytes).  L lanes share a
// row, taking units c, c + L, ...; a warp holds 32 / L groups of R rows, and
// the activations of a block, loaded once, serve the R rows.  Unit strides
// of 9 or 17 words keep the shared-memory reads free of bank conflicts.  A
// block's codes become fp16 pairs (weights j, j + 16), widen to fp32 exactly,
// and accumulate by packed fp32 FMAs, one chain per half, so a half-scale is
// applied once per half.  Everything from the codes to the sums is fp32 round
// to nearest: h needs no second rounding to a 16-bit type.
//
// Rows whose length is no multiple of 4 bytes (K / 32 odd, dual; K / 32 not a
// multiple of 4, single-scale) are shifted into place word by word; copies
// start at the 16-byte boundary before a row and end at the one after it,
// which stays inside the matrices as their sizes are multiples of 16.
#include "common.cuh"
#include "kernels.h"

namespace rocmfp4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kTileRows = 16;    // output rows of a down tile
constexpr int kMaxStages = 4;
constexpr int kRouterTokens = 8;  // tokens a router pass holds

// Shape of one product: rows of nb blocks, cut among lanes and stages.
struct RowGeom {
  int nb;          // blocks per row
  int rb;          // bytes per row
  int lanes;       // L: lanes that share a row (4, 8, 16 or 32)
  int iters;       // units per lane
  int seg_iters;   // iterations held by one stage
  int segs;        // stages per task
  int rows;        // rows of a task: 32 / L * R
  int pitch;       // bytes between row slots of a stage (rb when a stage holds whole rows)
  int half;        // offset of the up rows' region (gate/up tasks)
};

struct MoeParams {
  const uint16_t* X;
  const void* router;
  const uint8_t* Wgu;
  const uint8_t* Wd;
  float* Y;
  int32_t* ids;
  float* probs;
  float* logits;   // workspace [M][E]
  float* h;        // workspace [M * top_k][I]
  uint32_t* bars;  // workspace: two barrier counters and one of finished CTAs, zero between launches
  uint32_t* err;
  int M, E, top_k, K, I;
  int router_type, route;
  float route_scale;
  RowGeom gu, dn;
  int stage_bytes, stages;
  // offsets in shared memory
  int off_mask, off_list, off_slot, off_acc, off_ring;
  int acc_floats;  // per warp
};

template <int V>
struct Unit {
  static constexpr int BLOCKS = V == 0 ? 2 : 4;
  static constexpr int BYTES = BLOCKS * Fmt<V>::BB;  // 36 / 68
  static constexpr int R_GU = V == 0 ? 4 : 2;        // rows a lane holds: gate and up rows in equal parts
  static constexpr int R_DN = V == 0 ? 2 : 1;
};

RF4_DEV uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
RF4_DEV float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
RF4_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
RF4_DEV uint64_t half2_to_f32x2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack2(f.x, f.y);
}

template <int ACT>
RF4_DEV float act_f32(uint32_t bits16) {
  if constexpr (ACT == 1) return __uint_as_float(bits16 << 16);
  else return __half2float(__ushort_as_half((uint16_t)bits16));
}

// A block's 32 activations as pairs (x_j, x_{j+16}).  SRC 0 / 1: fp16 / bf16 input; 2: fp32 workspace.
template <int SRC>
RF4_DEV void load_x(const void* base, int64_t off, uint64_t (&xp)[16]) {
  if constexpr (SRC == 2) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = p[i], b = p[4 + i];
      xp[4 * i] = pack2(a.x, b.x);
      xp[4 * i + 1] = pack2(a.y, b.y);
      xp[4 * i + 2] = pack2(a.z, b.z);
      xp[4 * i + 3] = pack2(a.w, b.w);
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 a = __ldg(p + i), b = __ldg(p + 2 + i);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (SRC == 1) {
          xp[8 * i + 2 * j] = pack2(__uint_as_float(u[j] << 16), __uint_as_float(v[j] << 16));
          xp[8 * i + 2 * j + 1] = pack2(__uint_as_float(u[j] & 0xFFFF0000u), __uint_as_float(v[j] & 0xFFFF0000u));
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
          const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
          xp[8 * i + 2 * j] = pack2(f.x, g.x);
          xp[8 * i + 2 * j + 1] = pack2(f.y, g.y);
        }
      }
    }
  }
}

// The five words that hold block PHI of a unit at `unit` (any byte address
// unless ALIGNED): code byte j at byte (PHI * block bytes) % 4 + j.
template <int V, bool ALIGNED, int PHI>
RF4_DEV void block_words(const uint8_t* unit, uint32_t (&w)[5]) {
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
    for (int i = 0; i < 6; ++i) a[i] = p[i];
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

// Adds block PHI of R rows (row r at unit + r * stride) times T tokens' activations.
template <int V, bool ALIGNED, int R, int T, int PHI>
RF4_DEV void block_rows(const uint8_t* const (&unit)[R], const uint64_t (&xp)[T][16], float (&tot)[R][T]) {
  constexpr int O = PHI * Fmt<V>::BB % 4;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint32_t w[5];
    block_words<V, ALIGNED, PHI>(unit[r], w);
    uint64_t acc[T][2];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t][0] = acc[t][1] = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint64_t wp = half2_to_f32x2(clamp5(codes_at(w, O + j)));
#pragma unroll
      for (int t = 0; t < T; ++t) acc[t][j & 1] = fma2(wp, xp[t][j], acc[t][j & 1]);
    }
    float2 s;
    if constexpr (V == 0) {
      const uint32_t h = O == 0 ? e4m3x2<0>(w[4]) : e4m3x2<1>(w[4]);
      s = __half22float2(*reinterpret_cast<const __half2*>(&h));
    } else {
      const uint32_t h = e4m3x2<0>(__byte_perm(w[4], 0u, O * 0x11));
      s = __half22float2(*reinterpret_cast<const __half2*>(&h));
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float2 a = unpack2(acc[t][0]), b = unpack2(acc[t][1]);
      tot[r][t] = fmaf(s.x, a.x + b.x, tot[r][t]);
      tot[r][t] = fmaf(s.y, a.y + b.y, tot[r][t]);
    }
  }
}

template <int V, bool ALIGNED, int R, int T, int SRC, int PHI>
RF4_DEV void unit_blocks(const uint8_t* const (&unit)[R], const void* xbase, const int64_t (&xoff)[T], int blk, int nb,
                         float (&tot)[R][T]) {
  if (blk + PHI < nb) {
    uint64_t xp[T][16];
#pragma unroll
    for (int t = 0; t < T; ++t) load_x<SRC>(xbase, xoff[t] + (int64_t)(blk + PHI) * 32, xp[t]);
    block_rows<V, ALIGNED, R, T, PHI>(unit, xp, tot);
  }
  if constexpr (PHI + 1 < Unit<V>::BLOCKS) unit_blocks<V, ALIGNED, R, T, SRC, PHI + 1>(unit, xbase, xoff, blk, nb, tot);
}

// One stage's products for T tokens: tot[r][t], summed over the lanes of a row
// (each of them gets the sum).  `row`: the row slots in shared memory; u0: the
// first unit held.
template <int V, bool ALIGNED, int R, int T, int SRC>
RF4_DEV void stage_products(const RowGeom& g, const uint8_t* const (&row)[R], int u0, int c, const void* xbase,
                            const int64_t (&xoff)[T], float (&tot)[R][T]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) tot[r][t] = 0.f;
  for (int i = 0; i < g.seg_iters; ++i) {
    const int ul = i * g.lanes + c;  // unit within the stage
    const int blk = (u0 + ul) * Unit<V>::BLOCKS;
    if (blk >= g.nb) break;
    const uint8_t* unit[R];
#pragma unroll
    for (int r = 0; r < R; ++r) unit[r] = row[r] + ul * Unit<V>::BYTES;
    unit_blocks<V, ALIGNED, R, T, SRC, 0>(unit, xbase, xoff, blk, g.nb, tot);
  }
  __syncwarp();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= g.lanes) continue;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t) tot[r][t] += __shfl_xor_sync(0xffffffffu, tot[r][t], o);
  }
}

// The bytes [a, a + n) as a copy from 16-byte boundary to 16-byte boundary.
RF4_DEV uint32_t span_bytes(const uint8_t* a, int64_t n) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(a) & ~uintptr_t(15), e = (reinterpret_cast<uintptr_t>(a) + n + 15) & ~uintptr_t(15);
  return (uint32_t)(e - b);
}
RF4_DEV void copy_span(uint8_t* dst, const uint8_t* a, int64_t n, uint32_t bar) {
  bulk_g2s(smem_addr(dst), reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(a) & ~uintptr_t(15)), span_bytes(a, n), bar);
}
RF4_DEV int mis16(const uint8_t* a) { return (int)(reinterpret_cast<uintptr_t>(a) & 15u); }

RF4_DEV uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Order-preserving bits of a router logit, above 0; NaN orders below every number.
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
  constexpr int RG = U::R_GU, RD = U::R_DN;
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_probs = reinterpret_cast<float*>(smem);                           // [M][top_k]
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + p.off_mask);         // [E]: tokens of an expert
  uint16_t* s_list = reinterpret_cast<uint16_t*>(smem + p.off_list);         // chosen experts, ascending
  uint8_t* s_slot = smem + p.off_slot;                                       // [M][E]: which choice of the token
  float* s_acc = reinterpret_cast<float*>(smem + p.off_acc);                 // [kWarps][acc_floats]
  __shared__ uint64_t s_bars[kWarps * kMaxStages];
  __shared__ float s_red[kWarps][kRouterTokens];
  __shared__ int s_active, s_ok;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = gridDim.x;

  uint64_t* bars = s_bars + warp * kMaxStages;
  if (lane == 0) {
    for (int i = 0; i < kMaxStages; ++i) mbar_init(smem_addr(&bars[i]), 1);
    fence_mbar_init();
  }
  if (tid == 0) s_ok = 1;
  for (int e = tid; e < p.E; e += kThreads) s_mask[e] = 0;
  __syncthreads();

  // Every CTA arrives and waits (bounded) for the others; false if one gave up.
  auto grid_barrier = [&](uint32_t* counter) {
    __threadfence();
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
      float acc[kRouterTokens];
#pragma unroll
      for (int m = 0; m < kRouterTokens; ++m) acc[m] = 0.f;
      for (int k = tid * 8; k < p.K; k += kThreads * 8) {
        float r[8];
        load8_router(p.router_type, p.router, (int64_t)e * p.K + k, r);
#pragma unroll
        for (int m = 0; m < kRouterTokens; ++m) {
          if (m0 + m >= p.M) break;
          const uint4 a = __ldg(reinterpret_cast<const uint4*>(p.X + (int64_t)(m0 + m) * p.K + k));
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[m] = fmaf(r[2 * i], act_f32<ACT>(w[i] & 0xFFFFu), acc[m]);
            acc[m] = fmaf(r[2 * i + 1], act_f32<ACT>(w[i] >> 16), acc[m]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kRouterTokens; ++m) {
        if (m0 + m >= p.M) break;
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
  bool ok = grid_barrier(p.bars);

  // ---- top k of every token (one warp per token), repeated by every CTA ----
  if (ok) {
    for (int m = warp; m < p.M; m += kWarps) {
      constexpr int PL = 16;  // experts per lane: E <= 512
      uint32_t key[PL];
      float val[PL];
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int e = i * 32 + lane;
        val[i] = e < p.E ? __ldcg(p.logits + (int64_t)m * p.E + e) : 0.f;
        key[i] = e < p.E ? logit_key(val[i]) : 0u;
      }
      float top = 0.f, mine = 0.f, denom = 0.f;
      int my_id = 0;
      for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = 0;
        int at = 0;
        float bv = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i)
          if (key[i] > best) best = key[i], at = i, bv = val[i];
        const uint32_t mx = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == mx ? (uint32_t)(at * 32 + lane) : 0xFFFFu);
        const float l = __shfl_sync(0xffffffffu, bv, e & 31);
        if ((int)(e & 31) == lane) {
#pragma unroll
          for (int i = 0; i < PL; ++i)
            if (i == (int)(e >> 5)) key[i] = 0u;
        }
        if (j == 0) top = l;
        if (lane == j) my_id = (int)e, mine = l;
      }
      float num = 0.f;
      if (p.route == 2) {
        num = lane < p.top_k ? 1.f / (1.f + expf(-mine)) : 0.f;
        denom = num;
      } else {
        num = lane < p.top_k ? expf(mine - top) : 0.f;
        if (p.route == 1) {
          denom = num;
        } else {
#pragma unroll
          for (int i = 0; i < PL; ++i)
            if (i * 32 + lane < p.E) denom += expf(val[i] - top);
        }
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

  // ---- this warp's stages: gate/up tasks, then down tasks -------------------------------
  const RowGeom gu = p.gu, dn = p.dn;
  const int pairs = gu.rows / 2;                          // gate/up row pairs of a task
  const int per_expert = (p.I + pairs - 1) / pairs;       // gate/up tasks of an expert
  const int gu_tasks = A * per_expert;                    // dealt round robin over all CTAs, then warps
  const int first_gu = blockIdx.x + G * warp;
  const int n_gu = first_gu < gu_tasks ? (gu_tasks - first_gu + G * kWarps - 1) / (G * kWarps) : 0;
  const int tiles = p.K / kTileRows;
  const int my_tiles = (int)blockIdx.x < tiles ? (tiles - (int)blockIdx.x + G - 1) / G : 0;
  const int subs = kTileRows / dn.rows;                   // down tasks of a tile and expert
  const int tile_tasks = A * subs;
  const int per_tile = warp < tile_tasks ? (tile_tasks - warp + kWarps - 1) / kWarps : 0;
  const int n_stages_gu = n_gu * gu.segs;
  const int n_stages = n_stages_gu + my_tiles * per_tile * dn.segs;
  uint8_t* ring = smem + p.off_ring + (size_t)warp * p.stages * p.stage_bytes;

  // na rows from `a` to slots from dst, nbr rows from `b` to slots from dst + half: part `seg` of each row
  auto arm_and_copy = [&](uint8_t* dst, const uint8_t* a, int na, const uint8_t* b, int nbr, int half, const RowGeom& g, int seg, int slot) {
    const uint32_t bar = smem_addr(&bars[slot]);
    if (g.segs == 1) {  // whole rows: one copy for each run of rows
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, span_bytes(a, (int64_t)na * g.rb) + (nbr ? span_bytes(b, (int64_t)nbr * g.rb) : 0u));
        copy_span(dst, a, (int64_t)na * g.rb, bar);
        if (nbr) copy_span(dst + half, b, (int64_t)nbr * g.rb, bar);
      }
    } else {  // part of every row: one copy per row, by lanes
      const int lo = seg * g.seg_iters * g.lanes * U::BYTES;
      const int len = min(g.rb - lo, g.seg_iters * g.lanes * U::BYTES);
      uint32_t bytes = 0;
      for (int r = lane; r < na + nbr; r += 32) bytes += span_bytes((r < na ? a + (int64_t)r * g.rb : b + (int64_t)(r - na) * g.rb) + lo, len);
      bytes = __reduce_add_sync(0xffffffffu, bytes);
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      for (int r = lane; r < na + nbr; r += 32) {
        const uint8_t* src = (r < na ? a + (int64_t)r * g.rb : b + (int64_t)(r - na) * g.rb) + lo;
        copy_span(dst + (r < na ? r * g.pitch : half + (r - na) * g.pitch), src, len, bar);
      }
    }
  };
  struct Task {
    int expert, row0, rows, seg, tile;
  };
  auto task_of = [&](int s) {
    Task t;
    if (s < n_stages_gu) {
      const int id = first_gu + s / gu.segs * (G * kWarps);
      t.seg = s % gu.segs;
      t.expert = s_list[id / per_expert];
      t.row0 = id % per_expert * pairs;
      t.rows = min(pairs, p.I - t.row0);
      t.tile = -1;
    } else {
      const int q = s - n_stages_gu, task = q / dn.segs;
      t.seg = q % dn.segs;
      t.tile = task / per_tile;
      const int idx = warp + kWarps * (task % per_tile);
      t.expert = s_list[idx / subs];
      t.row0 = (blockIdx.x + t.tile * G) * kTileRows + idx % subs * dn.rows;
      t.rows = dn.rows;  // rows divide a tile, and tiles divide K
    }
    return t;
  };
  auto issue = [&](int s) {
    const Task t = task_of(s);
    const int slot = s % p.stages;
    uint8_t* dst = ring + (size_t)slot * p.stage_bytes;
    if (t.tile < 0) {
      const uint8_t* a = p.Wgu + ((int64_t)t.expert * 2 * p.I + t.row0) * gu.rb;
      arm_and_copy(dst, a, t.rows, a + (int64_t)p.I * gu.rb, t.rows, gu.half, gu, t.seg, slot);
    } else {
      const uint8_t* a = p.Wd + ((int64_t)t.expert * p.K + t.row0) * dn.rb;
      arm_and_copy(dst, a, t.rows, nullptr, 0, 0, dn, t.seg, slot);
    }
  };
  int issued = 0, s = 0;
  for (; issued < p.stages && issued < n_stages; ++issued) issue(issued);
  auto wait_stage = [&](int i) {  // warp-uniform: every lane waits on the same barrier
    const bool landed = mbar_wait_bounded(smem_addr(&bars[i % p.stages]), (uint32_t)((i / p.stages) & 1));
    if (__all_sync(0xffffffffu, landed)) return true;
    if (lane == 0) atomicOr(p.err, kErrWaitTimeout);
    return false;
  };
  auto release_stage = [&]() {
    __syncwarp();
    fence_proxy_async();  // the stage's reads precede the next copy into it
    if (issued < n_stages) issue(issued), ++issued;
  };

  float* acc = s_acc + (size_t)warp * p.acc_floats;
  bool live = ok;

  // ---- gate and up ----
  {
    const int c = lane % gu.lanes, g = lane / gu.lanes, groups = 32 / gu.lanes;
    for (; s < n_stages_gu && live; ++s) {
      if (!wait_stage(s)) {
        live = false;
        break;
      }
      const Task t = task_of(s);
      const uint8_t* st = ring + (size_t)(s % p.stages) * p.stage_bytes;
      const uint8_t* ga = p.Wgu + ((int64_t)t.expert * 2 * p.I + t.row0) * gu.rb;
      const uint8_t* ua = ga + (int64_t)p.I * gu.rb;
      const bool whole = gu.segs == 1;
      const uint8_t* row[RG];
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const int i = r % (RG / 2) * groups + g;  // pair of the task
        const uint8_t* a = r < RG / 2 ? ga : ua;
        row[r] = st + (r < RG / 2 ? 0 : gu.half) + i * gu.pitch + mis16(whole ? a : a + (int64_t)i * gu.rb);
      }
      const int u0 = t.seg * gu.seg_iters * gu.lanes;
      // products of one or two tokens at a time
      auto finish = [&](float gate, float up, int i, int pos, int m) {
        if (gu.segs > 1) {
          float* q = acc + 2 * (pos * pairs + i);
          if (t.seg > 0) gate += q[0], up += q[1];
          if (t.seg < gu.segs - 1) {
            q[0] = gate, q[1] = up;
            return;
          }
        }
        const int j = s_slot[m * p.E + t.expert];
        p.h[(int64_t)(m * p.top_k + j) * p.I + t.row0 + i] = gate / (1.f + expf(-gate)) * up;
      };
      uint32_t tokens = s_mask[t.expert];
      for (int pos = 0; tokens != 0; pos += 2) {
        const int m0 = __ffs(tokens) - 1;
        tokens &= tokens - 1;
        if (tokens == 0) {
          const int64_t off[1] = {(int64_t)m0 * p.K};
          float tot[RG][1];
          stage_products<V, ALIGNED, RG, 1, ACT>(gu, row, u0, c, p.X, off, tot);
#pragma unroll
          for (int r = 0; r < RG / 2; ++r) {
            const int i = r * groups + g;
            if (c == 0 && i < t.rows) finish(tot[r][0], tot[r + RG / 2][0], i, pos, m0);
          }
        } else {
          const int m1 = __ffs(tokens) - 1;
          tokens &= tokens - 1;
          const int64_t off[2] = {(int64_t)m0 * p.K, (int64_t)m1 * p.K};
          float tot[RG][2];
          stage_products<V, ALIGNED, RG, 2, ACT>(gu, row, u0, c, p.X, off, tot);
#pragma unroll
          for (int r = 0; r < RG / 2; ++r) {
            const int i = r * groups + g;
            if (c == 0 && i < t.rows) {
              finish(tot[r][0], tot[r + RG / 2][0], i, pos, m0);
              finish(tot[r][1], tot[r + RG / 2][1], i, pos + 1, m1);
            }
          }
        }
      }
      release_stage();
    }
  }
  ok = grid_barrier(p.bars + 1) && ok;  // every h is written
  live = live && ok;

  // ---- down: a tile of output rows at a time, the warps over its experts ----
  if (ok) {
    const int c = lane % dn.lanes, g = lane / dn.lanes, groups = 32 / dn.lanes;
    for (int tile = 0; tile < my_tiles; ++tile) {
      for (int i = lane; i < kTileRows * p.M; i += 32) acc[i] = 0.f;
      __syncwarp();
      for (int q = 0; q < per_tile * dn.segs && live; ++q, ++s) {
        if (!wait_stage(s)) {
          live = false;
          break;
        }
        const Task t = task_of(s);
        const uint8_t* st = ring + (size_t)(s % p.stages) * p.stage_bytes;
        const uint8_t* da = p.Wd + ((int64_t)t.expert * p.K + t.row0) * dn.rb;
        const int in_tile = t.row0 - (blockIdx.x + tile * G) * kTileRows;
        const uint8_t* row[RD];
#pragma unroll
        for (int r = 0; r < RD; ++r) {
          const int i = r * groups + g;
          row[r] = st + i * dn.pitch + mis16(dn.segs == 1 ? da : da + (int64_t)i * dn.rb);
        }
        const int u0 = t.seg * dn.seg_iters * dn.lanes;
        uint32_t tokens = s_mask[t.expert];
        while (tokens != 0) {
          const int m0 = __ffs(tokens) - 1;
          tokens &= tokens - 1;
          const int a0 = m0 * p.top_k + s_slot[m0 * p.E + t.expert];
          if (tokens == 0) {
            const int64_t off[1] = {(int64_t)a0 * p.I};
            float tot[RD][1];
            stage_products<V, ALIGNED, RD, 1, 2>(dn, row, u0, c, p.h, off, tot);
#pragma unroll
            for (int r = 0; r < RD; ++r) {
              const int i = r * groups + g;
              if (c == 0 && i < t.rows) acc[(in_tile + i) * p.M + m0] += s_probs[a0] * tot[r][0];
            }
          } else {
            const int m1 = __ffs(tokens) - 1;
            tokens &= tokens - 1;
            const int a1 = m1 * p.top_k + s_slot[m1 * p.E + t.expert];
            const int64_t off[2] = {(int64_t)a0 * p.I, (int64_t)a1 * p.I};
            float tot[RD][2];
            stage_products<V, ALIGNED, RD, 2, 2>(dn, row, u0, c, p.h, off, tot);
#pragma unroll
            for (int r = 0; r < RD; ++r) {
              const int i = r * groups + g;
              if (c == 0 && i < t.rows) {
                acc[(in_tile + i) * p.M + m0] += s_probs[a0] * tot[r][0];
                acc[(in_tile + i) * p.M + m1] += s_probs[a1] * tot[r][1];
              }
            }
          }
        }
        release_stage();
      }
      __syncthreads();
      const int n0 = (blockIdx.x + tile * G) * kTileRows;
      for (int i = tid; i < kTileRows * p.M; i += kThreads) {
        const int m = i / kTileRows, r = i % kTileRows;
        float y = 0.f;
        for (int w = 0; w < kWarps; ++w) y += s_acc[(size_t)w * p.acc_floats + r * p.M + m];
        p.Y[(int64_t)m * p.K + n0 + r] = y;
      }
      __syncthreads();
    }
  }
  // copies that no one waited for (after a wait gave up) land before the CTA leaves
  for (; s < issued; ++s) (void)mbar_wait_bounded(smem_addr(&bars[s % p.stages]), (uint32_t)((s / p.stages) & 1));
  __syncthreads();
  if (tid == 0 && atomic_add_acq_rel_gpu(p.bars + 2, 1u) == (uint32_t)G - 1u) {
    store_relaxed_gpu(p.bars, 0u);
    store_relaxed_gpu(p.bars + 1, 0u);
    store_relaxed_gpu(p.bars + 2, 0u);
  }
}

using MoeFn = void (*)(MoeParams);

template <int V>
MoeFn pick(int act, bool aligned) {
  if (act == 0) return aligned ? moe_kernel<V, 0, true> : moe_kernel<V, 0, false>;
  return aligned ? moe_kernel<V, 1, true> : moe_kernel<V, 1, false>;
}

constexpr int kSmemMax = 227 * 1024 - 2048;  // dynamic; the rest is the kernel's static shared memory
constexpr int kStageTarget = 6144;           // a stage holds whole rows where they fit into this
constexpr int kStageSlack = 32;              // word reads past a row's end

int up16(int v) { return (v + 15) / 16 * 16; }

// Rows of K weights over R rows a lane; `both`: gate and up rows in two regions.
RowGeom geometry(int variant, int64_t K, int R, bool both, int* stage_bytes) {
  RowGeom g{};
  const int ub = variant == 0 ? Unit<0>::BYTES : Unit<1>::BYTES, per = variant == 0 ? Unit<0>::BLOCKS : Unit<1>::BLOCKS;
  g.nb = (int)(K / 32);
  g.rb = g.nb * (variant == 0 ? 18 : 17);
  const int units = (g.nb + per - 1) / per;
  // Lanes to a row: as few idle as possible, the most lanes among equals
  // (rows then lie in fewer places of the shared-memory banks).
  int best = 1 << 30;
  for (int L = 32; L >= 4; L /= 2) {
    const int padded = (units + L - 1) / L * L;
    if (padded < best) best = padded, g.lanes = L;
  }
  g.iters = (units + g.lanes - 1) / g.lanes;
  g.rows = 32 / g.lanes * R;
  const int parts = both ? 2 : 1, n = g.rows / parts;
  g.pitch = g.rb;
  g.half = up16(n * g.rb) + 16 + kStageSlack;
  g.seg_iters = g.iters;
  g.segs = 1;
  if (parts * g.half > kStageTarget && g.iters > 1) {  // not whole rows: slots of up to seg_iters units a lane
    const int fit = (kStageTarget / g.rows - 16 - kStageSlack) / (g.lanes * ub);
    g.segs = (g.iters + (fit > 1 ? fit : 1) - 1) / (fit > 1 ? fit : 1);
    g.seg_iters = (g.iters + g.segs - 1) / g.segs;
    g.segs = (g.iters + g.seg_iters - 1) / g.seg_iters;
    g.pitch = up16(g.seg_iters * g.lanes * ub) + 16 + kStageSlack;
    g.half = n * g.pitch;
  }
  if (g.segs == 1) g.pitch = g.rb, g.half = up16(n * g.rb) + 16 + kStageSlack;
  *stage_bytes = parts * g.half;
  return g;
}

}  // namespace

cudaError_t moe_prepare() {
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
  p.logits = a.ws;
  p.h = a.ws + kMoeMaxTokens * kMoeMaxExperts;
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
  int gu_bytes = 0, dn_bytes = 0;
  p.gu = geometry(variant, a.K, variant == 0 ? Unit<0>::R_GU : Unit<1>::R_GU, true, &gu_bytes);
  p.dn = geometry(variant, a.I, variant == 0 ? Unit<0>::R_DN : Unit<1>::R_DN, false, &dn_bytes);
  p.stage_bytes = (gu_bytes > dn_bytes ? gu_bytes : dn_bytes) / 128 * 128 + 128;
  int at = up16(p.M * p.top_k * 4);
  p.off_mask = at;
  at += up16(p.E * 4);
  p.off_list = at;
  at += up16(p.E * 2);
  p.off_slot = at;
  at += up16(p.M * p.E);
  p.off_acc = at;
  p.acc_floats = kTileRows * p.M;
  if (p.gu.segs > 1 && p.gu.rows * p.M > p.acc_floats) p.acc_floats = p.gu.rows * p.M;
  at += kWarps * p.acc_floats * 4;
  p.off_ring = (at + 127) / 128 * 128;
  const int room = (kSmemMax - p.off_ring - kStageSlack) / (kWarps * p.stage_bytes);
  p.stages = room < kMaxStages ? room : kMaxStages;
  if (p.stages < 1) return cudaErrorInvalidConfiguration;
  const int smem = p.off_ring + kWarps * p.stages * p.stage_bytes + kStageSlack;
  const bool aligned = p.gu.rb % 4 == 0 && p.dn.rb % 4 == 0;
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
