// Attention of few rows over a paged ROCmFP4 cache: single tokens, mostly.  The
// same operator as paged_attention.cu, for row tiles of at most eight (row,
// head) pairs, which a 128-row tensor-core tile would leave empty.
//
// A row tile's rows are the eight columns of mma.sync m16n8k16:
//   scores: A = 16 tokens x 16 of D of K, decoded in registers (exact), B = q;
//   P V:    A = 16 of D x 16 tokens of V^T (decoded rows, transposed by
//           movmatrix), B = P^T, rounded to fp16 after a factor of 2^15.
// Scores, maxima, sums and the weighted sum are fp32; a score is subtracted from its maximum before
// the scaling, so that large ones differ as they do.  P's half step of 2^-11 is
// the output type's own (fp16) or an eighth of it (bf16).
//
// A CTA's four warps take a row tile's 32-token chunks in turn, each with a ring
// of bulk copies of its own (a chunk is two groups of 16 tokens, each within a
// page), and keep a running maximum and sum each; no warp waits for another
// until the CTA's part of the row tile is done.  The work is cut as in
// paged_work.cuh, over two CTAs an SM; the CTA that arrives last at a shared row
// tile adds the parts, its warps a quarter of them each.
//
// Measured (40 query heads over 8 of D = 128, in a graph): one token over 32768
// 24.7 us (38 MB, 1.5 TB/s), 16 over 4096 40.4 us (71 MB, 1.8 TB/s), 64 over 2000
// 64.6 us (147 MB, 2.3 TB/s), one over 100 7.1 us.  What bounds it is the decode and its
// latencies (about 1400 warp instructions a chunk, half of the issue slots used);
// of the 40.4 us, copies and the joining of parts alone take 20.  Tried
// and not better: three CTAs an SM (40.9 / 66.9 us), V transposed by byte permutes instead of movmatrix
// with rows in conflict-free order (41.7 / 71.0), one CTA of twelve warps an SM (22.6 / 40.5
// but 8.1 for 100 tokens and 74 for 64 x 2000), the same with copies that run on into the next row tile
// (24.1 / 43.7).
#include "attn_frag.cuh"
#include "kernels.h"
#include "paged_work.cuh"

namespace rocmfp4 {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kChunk = 32;   // tokens a warp takes at a time
constexpr int kStages = 3;   // chunks under way per warp
constexpr int kCtasPerSm = kPagedCtas;
constexpr int kCols = 8;     // rows of a row tile
constexpr float kPScale = 32768.0f, kPUnscale = 1.0f / 32768.0f;
constexpr float kLog2e = 1.4426950408889634f;

struct Shape {
  static constexpr int kRows = kCols, kNarrow = kCols, kTok = kWarps * kChunk, kMinShare = 2;
  static RF4_DEV int fixed(int) { return 1; }
};

struct Params : Batch {
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq;
  int H;
  float scale_log2;
  float* ws;      // [ctas][2] parts of kCols rows of D, then as many pairs (m, l)
  uint32_t* cnt;  // [ctas], zero between launches
};

template <int V, int D>
struct Fmt2 {
  static constexpr int BB = Fmt<V>::BB, NB = D / 32, RB = NB * BB;
  static constexpr int CB = kChunk * RB, STAGE = 2 * CB, RING = kStages * STAGE;
  static constexpr int KS = D / 16;
  static constexpr int STATE = 2 * kCols + kCols * D;  // floats of a warp's state
  static constexpr int MAX_PARTS = 512;                // CTAs of a launch, at most
  // shared memory: the rings; between row tiles, the warps' states; while parts are added, their weights behind the sums
  static constexpr int SUMS = kWarps * kCols * D * 4, ADD = SUMS + kCols * MAX_PARTS * 4;
  static constexpr int AREA = kWarps * RING > ADD ? kWarps * RING : ADD;
  static constexpr int OFF_CTL = (AREA + 15) / 16 * 16;
  static_assert(kWarps * STATE * 4 <= AREA && CB % 16 == 0, "shared memory");
};

struct Control {
  uint64_t full[kWarps][kStages];
  uint32_t have[kWarps][kStages];  // of a chunk's two groups: those that were copied
  Stretch work;
  int last;
};

RF4_DEV uint32_t pack_act(float lo, float hi, int act) {
  if (act == 0) return pack_half2(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Adds a shared row tile's parts and writes its rows; all threads.
template <int D, int ACT>
RF4_DEV void add_parts(const Params& p, const Item& it, const float2* ml, float* area) {
  constexpr int Q4 = D / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = it.last - it.first + 1;
  float* sums = area;
  float* weight = area + kWarps * kCols * D;  // [rows][parts]
  // part n: the first CTA's in its slot 1, the others' in slot 0
  auto record = [&](int n) { return (size_t)((it.first + n) * 2 + (n == 0)) * kCols; };
  for (int row = warp; row < it.rows; row += kWarps) {
    float M = -INFINITY, L = 0.f;
    for (int n = lane; n < parts; n += 32) M = fmaxf(M, __ldcg(&ml[record(n) + row]).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;
    for (int n = lane; n < parts; n += 32) {
      const float2 v = __ldcg(&ml[record(n) + row]);
      const float e = v.y == 0.f ? 0.f : ex2_approx((v.x - M) * p.scale_log2);
      weight[row * parts + n] = e;
      L += e * v.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    __syncwarp();
    for (int n = lane; n < parts; n += 32) weight[row * parts + n] *= inv;
  }
  __syncthreads();
  // warp w: parts w, w + kWarps, ...; a lane's places are four values each
  constexpr int K = kCols * Q4 / 32;
  const int places = it.rows * Q4;
  float4 a[K];
#pragma unroll
  for (int k = 0; k < K; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int n = warp; n < parts; n += kWarps) {
    const float4* base = reinterpret_cast<const float4*>(p.ws + record(n) * D);
    float4 x[K];
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = lane + 32 * k < places ? __ldcg(base + lane + 32 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float u = weight[min((lane + 32 * k) / Q4, it.rows - 1) * parts + n];
      a[k].x += u * x[k].x, a[k].y += u * x[k].y, a[k].z += u * x[k].z, a[k].w += u * x[k].w;
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (lane + 32 * k < places) reinterpret_cast<float4*>(sums + warp * kCols * D)[lane + 32 * k] = a[k];
  __syncthreads();
  for (int i = threadIdx.x; i < it.rows * D / 2; i += kThreads) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      x += sums[w * kCols * D + 2 * i];
      y += sums[w * kCols * D + 2 * i + 1];
    }
    const int rr = 2 * i / D, row = it.r0 + rr, token = row / p.G, g = row - token * p.G;
    *reinterpret_cast<uint32_t*>(p.out + ((int64_t)(it.s.row0 + token) * p.H + (int64_t)it.hk * p.G + g) * D + 2 * i % D) = pack_act(x, y, ACT);
  }
}

template <int V, int D, int ACT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_few_kernel(const __grid_constant__ Params p) {
  using F = Fmt2<V, D>;
  extern __shared__ __align__(128) uint8_t smem[];
  Control& ctl = *reinterpret_cast<Control*>(smem + F::OFF_CTL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;  // fragment row (token; column of B) and column group
  uint8_t* ring = smem + warp * F::RING;
  if (lane < kStages) {
    mbar_init(smem_addr(&ctl.full[warp][lane]), 1);
    fence_mbar_init();
  }
  grid_dependency_wait();  // lengths, tables and everything else may be the preceding kernel's output
  bool any_wide;
  if (!find_work<Shape, kThreads>(p, ctl.work, any_wide)) return;
  Walk<Shape> walk(p, ctl.work);
  Item it;
  const int ps = p.c.page_size;
  const int64_t page_bytes = (int64_t)p.c.Hkv * ps * F::RB;
  uint32_t stage = 0, phase = 0, put = 0;  // of the chunk to be taken next; stage of the one to be brought next
  bool ok = true;
  while (walk.next(p, it)) {
    int lo, hi, lo1, hi0;
    seen(p, it.s, it.r0 / p.G, lo, hi0);
    seen(p, it.s, (it.r0 + it.rows - 1) / p.G, lo1, hi);
    if (threadIdx.x == 0 && it.s.over) atomicOr(p.c.err, kErrBadPage);
    const int first = max(4 * it.c0, lo / kChunk), end = min(4 * (it.c0 + it.tiles), (hi + kChunk - 1) / kChunk);
    const int32_t* pages = p.c.table + (int64_t)it.b * p.c.ldt;
    const int64_t head = (int64_t)it.hk * ps * F::RB;

    // this warp's chunks: first + warp, + 4, ...
    auto bring = [&](int ch) {
      if (lane == 0) {
        const int t0 = ch * kChunk, at = t0 / ps, off = t0 - at * ps;
        const bool same = off + 16 < ps;  // both groups in one page
        const bool want0 = t0 + 16 > lo, want1 = t0 + 16 < hi;  // (the chunk itself is wanted)
        const int p0 = want0 ? pages[at] : -1, p1 = want1 ? (same && want0 ? p0 : pages[same ? at : at + 1]) : -1;
        const bool have0 = p0 >= 0 && p0 < p.c.num_pages, have1 = p1 >= 0 && p1 < p.c.num_pages;
        if ((want0 && !have0) || (want1 && !have1)) atomicOr(p.c.err, kErrBadPage);
        const uint32_t bar = smem_addr(&ctl.full[warp][put]);
        ctl.have[warp][put] = (have0 ? 1u : 0u) | (have1 ? 2u : 0u);
        mbar_arrive_expect_tx(bar, (have0 ? F::CB : 0) + (have1 ? F::CB : 0));
        const int64_t s0 = head + p0 * page_bytes + (int64_t)off * F::RB;
        const int64_t s1 = head + p1 * page_bytes + (int64_t)(same ? off + 16 : 0) * F::RB;
        const uint32_t dst = smem_addr(ring + put * F::STAGE);
        if (have0 && have1 && same) {
          bulk_g2s(dst, p.c.K + s0, F::CB, bar);
          bulk_g2s(dst + F::CB, p.c.V + s0, F::CB, bar);
        } else {
          if (have0) {
            bulk_g2s(dst, p.c.K + s0, F::CB / 2, bar);
            bulk_g2s(dst + F::CB, p.c.V + s0, F::CB / 2, bar);
          }
          if (have1) {
            bulk_g2s(dst + F::CB / 2, p.c.K + s1, F::CB / 2, bar);
            bulk_g2s(dst + F::CB + F::CB / 2, p.c.V + s1, F::CB / 2, bar);
          }
        }
      }
      put = put + 1 == kStages ? 0 : put + 1;
    };
    int next = first + warp;  // the chunk to be brought next
    int under_way = 0;
    for (; under_way < kStages && next < end && ok; ++under_way, next += kWarps) bring(next);

    // B fragments of q: k step (block kb, half h) pairs byte j = 4c + 2h of every block with columns (2c, 2c + 1) and byte
    // j + 1 with (2c + 8, 2c + 9)
    uint32_t qb0[F::KS], qb1[F::KS];
    {
      const int row = it.r0 + min(r, it.rows - 1), token = row / p.G, g = row - token * p.G;
      const uint16_t* qr = p.q + (int64_t)(it.s.row0 + token) * p.ldq + ((int64_t)it.hk * p.G + g) * D;
#pragma unroll
      for (int kb = 0; kb < F::NB; ++kb) {
        const uint2 x = *reinterpret_cast<const uint2*>(qr + 32 * kb + 4 * c), y = *reinterpret_cast<const uint2*>(qr + 32 * kb + 16 + 4 * c);
        qb0[2 * kb] = r < it.rows ? __byte_perm(x.x, y.x, 0x5410) : 0u;
        qb1[2 * kb] = r < it.rows ? __byte_perm(x.x, y.x, 0x7632) : 0u;
        qb0[2 * kb + 1] = r < it.rows ? __byte_perm(x.y, y.y, 0x5410) : 0u;
        qb1[2 * kb + 1] = r < it.rows ? __byte_perm(x.y, y.y, 0x7632) : 0u;
      }
    }
    // what columns 2c and 2c + 1 see (columns behind the rows: anything)
    int clo[2], chi[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      clo[j] = 0;
      chi[j] = 0x7fffffff;
      if (2 * c + j < it.rows) seen(p, it.s, (it.r0 + 2 * c + j) / p.G, clo[j], chi[j]);
    }

    float mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.f, 0.f};
    float oacc[2 * F::NB][4];
#pragma unroll
    for (int m = 0; m < 2 * F::NB; ++m) oacc[m][0] = oacc[m][1] = oacc[m][2] = oacc[m][3] = 0.f;

    for (int ch = first + warp; ch < end && ok; ch += kWarps) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&ctl.full[warp][stage]), phase))) {
        ok = false;
        break;
      }
      const uint8_t* ks_base = ring + stage * F::STAGE;
      const uint8_t* vs_base = ks_base + F::CB;
      const uint32_t have = ctl.have[warp][stage];
      const int t0 = ch * kChunk;
      // some column does not see some token of the chunk, or a token is not there
      const bool part = t0 < lo1 || t0 + kChunk > hi0 || have != 3u;

      // ---- scores: token rows 16mt + r and 16mt + r + 8 ----
      float x[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint8_t* ra = ks_base + (16 * mt + r) * F::RB;
        const uint8_t* rb = ra + 8 * F::RB;
#pragma unroll
        for (int kb = 0; kb < F::NB; ++kb) {
          uint32_t va[4], vb[4];
          const int alc = row_align<V, D>(kb * F::BB), als = row_align<V, D>(kb * F::BB + 16);
          decode4(lds_bytes4_al(ra + kb * F::BB + 4 * c, alc), block_scales<V>(ra + kb * F::BB, als), va);
          decode4(lds_bytes4_al(rb + kb * F::BB + 4 * c, alc), block_scales<V>(rb + kb * F::BB, als), vb);
          if constexpr (ACT == 1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              va[k] = f16x2_to_bf16x2(va[k]);
              vb[k] = f16x2_to_bf16x2(vb[k]);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {va[2 * h], vb[2 * h], va[2 * h + 1], vb[2 * h + 1]};
            if (kb == 0 && h == 0)
              mma_z(x[mt], a, qb0[0], qb1[0], ACT == 1);
            else if constexpr (ACT == 1)
              mma_bf16(x[mt], a, qb0[2 * kb + h], qb1[2 * kb + h]);
            else
              mma_f16(x[mt], a, qb0[2 * kb + h], qb1[2 * kb + h]);
          }
        }
      }

      // ---- softmax over the chunk (columns 2c, 2c + 1 in this lane) ----
      float cmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (part) {
            const int t = t0 + 16 * mt + r + (e >= 2 ? 8 : 0);
            if (t < clo[e & 1] || t >= chi[e & 1] || !(have >> mt & 1u)) x[mt][e] = -INFINITY;
          }
          cmax[e & 1] = fmaxf(cmax[e & 1], x[mt][e]);
        }
      float alpha[2], pv[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        cmax[j] = fmaxf(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 4));
        cmax[j] = fmaxf(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 8));
        cmax[j] = fmaxf(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 16));
        const float m = fmaxf(mrun[j], cmax[j]), ref = m == -INFINITY ? 0.f : m;
        alpha[j] = ex2_approx((mrun[j] - ref) * p.scale_log2);
        mrun[j] = m;
        float sum = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = j; e < 4; e += 2) {
            pv[mt][e] = ex2_approx((x[mt][e] - ref) * p.scale_log2);
            sum += pv[mt][e];
          }
        lrun[j] = lrun[j] * alpha[j] + sum;
      }

      // ---- P V ----
      float cacc[2 * F::NB][4];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        // lane (r, c) holds P of token 16kk + r (+ 8) for columns 2c, 2c + 1; transposed, column r at tokens 2c, 2c + 1 (+ 8)
        const uint32_t b0 = movmatrix_t(pack_half2(pv[kk][0] * kPScale, pv[kk][1] * kPScale));
        const uint32_t b1 = movmatrix_t(pack_half2(pv[kk][2] * kPScale, pv[kk][3] * kPScale));
        const int ta = t0 + 16 * kk + r, tb = ta + 8;
        const bool there = have >> kk & 1u;
        const uint8_t* ra = vs_base + (16 * kk + r) * F::RB;
        const uint8_t* rb = ra + 8 * F::RB;
#pragma unroll
        for (int kb = 0; kb < F::NB; ++kb) {
          uint32_t va[4], vb[4];
          const int alc = row_align<V, D>(kb * F::BB), als = row_align<V, D>(kb * F::BB + 16);
          decode4(lds_bytes4_al(ra + kb * F::BB + 4 * c, alc), block_scales<V>(ra + kb * F::BB, als), va);
          decode4(lds_bytes4_al(rb + kb * F::BB + 4 * c, alc), block_scales<V>(rb + kb * F::BB, als), vb);
          if (part) {  // rows that are no tokens may hold anything
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              va[k] = there && ta < hi ? va[k] : 0u;
              vb[k] = there && tb < hi ? vb[k] : 0u;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {movmatrix_t(va[2 * h]), movmatrix_t(va[2 * h + 1]), movmatrix_t(vb[2 * h]), movmatrix_t(vb[2 * h + 1])};
            if (kk == 0)
              mma_z(cacc[2 * kb + h], a, b0, b1, false);
            else
              mma_f16(cacc[2 * kb + h], a, b0, b1);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2 * F::NB; ++m) {
        oacc[m][0] = fmaf(oacc[m][0], alpha[0], cacc[m][0]);
        oacc[m][1] = fmaf(oacc[m][1], alpha[1], cacc[m][1]);
        oacc[m][2] = fmaf(oacc[m][2], alpha[0], cacc[m][2]);
        oacc[m][3] = fmaf(oacc[m][3], alpha[1], cacc[m][3]);
      }
      if (++stage == kStages) stage = 0, phase ^= 1u;
      --under_way;
      __syncwarp();
      fence_proxy_async();  // the ring's reads precede the next bulk copy into it
      if (next < end) {
        bring(next);
        next += kWarps;
        ++under_way;
      }
    }
    if (!ok) {  // copies under way land before the block goes on
      if (lane == 0) atomicOr(p.c.err, kErrWaitTimeout);
      for (; under_way > 0; --under_way) {
        (void)mbar_wait_bounded(smem_addr(&ctl.full[warp][stage]), phase);
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      lrun[j] += __shfl_xor_sync(0xffffffffu, lrun[j], 4);
      lrun[j] += __shfl_xor_sync(0xffffffffu, lrun[j], 8);
      lrun[j] += __shfl_xor_sync(0xffffffffu, lrun[j], 16);
    }

    // ---- the warps' states, in warp order ----
    __syncthreads();  // every ring is idle
    float* area = reinterpret_cast<float*>(smem);
    float* mine = area + warp * F::STATE;
    if (r == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mine[2 * c + j] = mrun[j];
        mine[kCols + 2 * c + j] = lrun[j];
      }
    }
#pragma unroll
    for (int m = 0; m < 2 * F::NB; ++m) {
      const int kb = m / 2, h = m % 2;
      const int d = 32 * kb + 4 * (r / 2) + 2 * h + 16 * (r % 2);
      float* o = mine + 2 * kCols;
      *reinterpret_cast<float2*>(o + (2 * c) * D + d) = make_float2(oacc[m][0] * kPUnscale, oacc[m][2] * kPUnscale);
      *reinterpret_cast<float2*>(o + (2 * c + 1) * D + d) = make_float2(oacc[m][1] * kPUnscale, oacc[m][3] * kPUnscale);
    }
    __syncthreads();
    const bool whole = it.first == it.last;
    float2* ml = reinterpret_cast<float2*>(p.ws + (size_t)gridDim.x * 2 * kCols * D);
    const size_t record = ((size_t)blockIdx.x * 2 + (it.slot & 1)) * kCols;
    for (int i = threadIdx.x; i < it.rows * D / 2; i += kThreads) {
      const int rr = 2 * i / D, d = 2 * i % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, area[w * F::STATE + rr]);
      const float ref = M == -INFINITY ? 0.f : M;
      float x = 0.f, y = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* s = area + w * F::STATE;
        const float e = ex2_approx((s[rr] - ref) * p.scale_log2);
        L += e * s[kCols + rr];
        x += e * s[2 * kCols + rr * D + d];
        y += e * s[2 * kCols + rr * D + d + 1];
      }
      if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int row = it.r0 + rr, token = row / p.G, g = row - token * p.G;
        *reinterpret_cast<uint32_t*>(p.out + ((int64_t)(it.s.row0 + token) * p.H + (int64_t)it.hk * p.G + g) * D + d) = pack_act(x * inv, y * inv, ACT);
      } else {
        __stcg(reinterpret_cast<float2*>(p.ws + (record + rr) * D + d), make_float2(x, y));
        if (d == 0) __stcg(&ml[record + rr], make_float2(M, L));
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const uint32_t n = atomic_add_acq_rel_gpu(&p.cnt[it.first], 1u);
        ctl.last = n == (uint32_t)(it.last - it.first);
        if (ctl.last) store_relaxed_gpu(&p.cnt[it.first], 0u);
      }
      __syncthreads();
      if (ctl.last) {
        __threadfence();
        add_parts<D, ACT>(p, it, ml, area);
      }
    }
    fence_proxy_async();
    __syncthreads();  // the rings may be filled again
  }
}

using Fn = void (*)(Params);
template <int V, int D>
Fn kernel_for(int act) {
  return act == 0 ? paged_few_kernel<V, D, 0> : paged_few_kernel<V, D, 1>;
}
Fn kernel_for(int variant, int D, int act) {
  if (variant == 0) return D == 64 ? kernel_for<0, 64>(act) : kernel_for<0, 128>(act);
  return D == 64 ? kernel_for<1, 64>(act) : kernel_for<1, 128>(act);
}
template <int V, int D>
constexpr int smem_of() {
  return Fmt2<V, D>::OFF_CTL + (int)sizeof(Control);
}
int smem_for(int variant, int D) {
  if (variant == 0) return D == 64 ? smem_of<0, 64>() : smem_of<0, 128>();
  return D == 64 ? smem_of<1, 64>() : smem_of<1, 128>();
}

}  // namespace

cudaError_t paged_few_prepare() {
  for (int v = 0; v < 2; ++v)
    for (int D : {64, 128})
      for (int act = 0; act < 2; ++act) {
        cudaError_t e = cudaFuncSetAttribute((const void*)kernel_for(v, D, act), cudaFuncAttributeMaxDynamicSharedMemorySize, smem_for(v, D));
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_paged_few(int variant, int act, const PagedAttnArgs& a, int sms, cudaStream_t s) {
  Params p{};
  p.q = a.q;
  p.out = a.out;
  p.ldq = a.ldq;
  p.M = (int)a.M;
  p.H = a.H;
  p.G = a.H / a.cache.Hkv;
  p.causal = a.causal;
  p.window = a.window;
  p.scale_log2 = a.scale * kLog2e;
  p.c = a.cache;
  p.ws = a.ws;
  p.cnt = a.cnt;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kCtasPerSm * sms < 512 ? kCtasPerSm * sms : 512));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_for(variant, a.cache.D);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel_for(variant, a.cache.D, act), p);
}

}  // namespace rocmfp4
