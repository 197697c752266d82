// Rows of a paged ROCmFP4 K/V cache: rotary positions, packing into pages,
// reading back.
//
// rope_kernel.  Row m of a call is a token with position p.  In the first
// `rot` values of a head the pairs (i, i + rot/2) or (2i, 2i + 1), i < rot/2,
// are turned by the angle p * freq[i] and scaled by `amplitude`:
//   y_a = A (x_a cos - x_b sin),  y_b = A (x_b cos + x_a sin).
// Heads of q are rounded once to fp16 / bf16.  Heads of k (turned) and of v
// (as they are) become ROCmFP4 rows by the quantiser's rule, from the fp32
// values: the smallest scale byte e with 5 * E4M3(e) >= the group's largest
// magnitude, and the nearest Codebook10 magnitudes, ties to the smaller; every
// comparison is exact in fp32, non-finite values count as 0.
//
// Angles.  freq / 2 pi mod 1 is held as a 64-bit fixed-point fraction of a
// turn, so that position * fraction mod 2^64 is the turned angle mod 2 pi by
// one integer product, as exact at position 2^31 as at 1 (a product in fp32
// would be off by 2^-24 of the whole angle).  The top 32 bits, reduced to an
// eighth of a turn either side, are what the fp32 sine and cosine see.
//
// Split: eight threads own one 32-value block place of a token (4 values a
// thread: a group of 16 is four lanes) and walk over heads, so that sines and
// cosines are computed once for all heads of a walk.  Few rows: one head a
// walk, for latency; many rows: as few walks as fill the GPU.
//
// cache_read_kernel.  The rows' blocks back as dense values, exact in every
// output type; four threads a block.
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace rocmfp4 {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  const void* x[3];  // q, k, v
  int64_t ld[3];
  const int32_t* positions;  // nullptr: the token's place in its sequence
  const float* freq;
  uint16_t* q_out;
  int64_t M;
  int H, heads;  // heads of q; of q, k and v together
  int rot, nb, slices, act;
  float amplitude;
  int paged;
  PagedArgs c;
};

// The sequence of a row, found by eight lanes that probe eight places at a
// time: the last b with cu[b] <= row.
RF4_DEV int sequence_of(const int32_t* cu, int B, int64_t row, uint32_t mask, int l) {
  int lo = 0, n = B;  // the answer lies in lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 7) / 8;
    const int at = lo + l * step;
    const bool le = l * step < n && (l == 0 || cu[at] <= row);
    const uint32_t hits = __ballot_sync(mask, le) & mask;
    const int k = __popc(hits) - 1;  // lane 0 always hits, and cu does not decrease
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// cos and sin of 2 pi * turns / 2^64.
RF4_DEV void turn(uint64_t turns, float& c, float& s) {
  const uint32_t t = (uint32_t)(turns >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(t - (quarter << 30)) * 0x1p-31f;  // half turns, at most a quarter
  float s0, c0;
  sincospif(x, &s0, &c0);
  c = quarter == 0 ? c0 : quarter == 1 ? -s0 : quarter == 2 ? -c0 : s0;
  s = quarter == 0 ? s0 : quarter == 1 ? c0 : quarter == 2 ? -s0 : -c0;
}

template <int T>
struct Raw4 {
  uint2 v;
};
template <>
struct Raw4<0> {
  float4 v;
};

template <int T>
RF4_DEV float one_f32(const void* p, int64_t i) {
  if constexpr (T == 0) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  if constexpr (T == 1) return __uint_as_float((uint32_t)h << 16);
  return __half2float(__ushort_as_half(h));
}

// Four consecutive values from element i on.
template <int T, bool VEC>
RF4_DEV void load4(const void* p, int64_t i, float (&x)[4]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = one_f32<T>(p, i + k);
  } else if constexpr (T == 0) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (T == 1) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      } else {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[k]);
        x[2 * k] = __low2float(h);
        x[2 * k + 1] = __high2float(h);
      }
    }
  }
}

// Code of |x| = a for half-scale hs: the number of midpoints below a.
RF4_DEV uint32_t code_of(float x, float a, float hs) {
  uint32_t k = (a > 0.5f * hs) + (a > 1.5f * hs) + (a > 2.5f * hs) + (a > 3.5f * hs) + (a > 5.f * hs) + (a > 7.f * hs) +
               (a > 9.f * hs);
  return k && x < 0.f ? k | 8u : k;
}

// T: type of q, k and v (0 fp32, 1 bf16, 2 fp16).  V: block layout.
// INTER: pairs (2i, 2i + 1).  VEC: every four values are one aligned vector,
// and so are their partners.
template <int T, int V, bool INTER, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  const int lane = threadIdx.x & 31, l = lane & 7;
  const uint32_t mask = 0xFFu << (lane & 24);
  const int64_t group = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 3;
  const int block = (int)(group % p.nb);
  const int64_t rest = group / p.nb;
  const int slice = (int)(rest % p.slices);
  const int64_t row = rest / p.slices;
  grid_launch_dependents();
  if (row >= p.M) return;
  const int D = p.nb * 32, d0 = block * 32 + 4 * l;
  const int rot = p.rot, half = rot / 2;

  grid_dependency_wait();  // everything read below may be the preceding kernel's output
  uint64_t turns[4];
  uint32_t turned = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    turns[i] = 0;
    const int d = d0 + i;
    if (d < rot) {
      turned |= 1u << i;
      const double f = (double)p.freq[INTER ? d / 2 : d < half ? d : d - half] * 0.15915494309189533577;
      turns[i] = (uint64_t)((f - floor(f)) * 18446744073709551616.0);
    }
  }

  int64_t pos = 0;
  int64_t slot = -1;  // row of the pages for head 0 of the token
  if (p.paged) {
    if (row >= p.c.cu[p.c.B] || row < p.c.cu[0]) return;  // padding
    const int b = sequence_of(p.c.cu, p.c.B, row, mask, l);
    const int64_t len = p.c.lens[b];
    pos = len - ((int64_t)p.c.cu[b + 1] - row);
    if (pos >= 0 && pos < len) {
      const int64_t pg = pos / p.c.page_size;
      const int page = pg < p.c.width ? p.c.table[b * p.c.ldt + pg] : -1;
      if (page >= 0 && page < p.c.num_pages)
        slot = (int64_t)page * p.c.Hkv * p.c.page_size + pos % p.c.page_size;
      else if (l == 0)
        atomicOr(p.c.err, kErrBadPage);
    }
  }
  if (p.positions != nullptr) pos = p.positions[row];
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER && (i & 1)) {
      cs[i] = cs[i - 1];
      sn[i] = -sn[i - 1];
      continue;
    }
    turn(turns[i] * (uint64_t)pos, cs[i], sn[i]);
    cs[i] *= p.amplitude;
    sn[i] *= INTER || d0 + i < half ? -p.amplitude : p.amplitude;
  }

#pragma unroll 2
  for (int h = slice; h < p.heads; h += p.slices) {
    const int kind = h < p.H ? 0 : h < p.H + p.c.Hkv ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.H : h - p.H - p.c.Hkv;
    if (kind != 0 && slot < 0) break;
    const int64_t at = row * p.ld[kind] + (int64_t)hh * D + d0;
    float x[4];
    load4<T, VEC>(p.x[kind], at, x);
    if (kind != 2 && turned) {
      float o[4];
      if constexpr (INTER) {
        o[0] = x[1], o[1] = x[0], o[2] = x[3], o[3] = x[2];
      } else if constexpr (VEC) {
        load4<T, true>(p.x[kind], at + (d0 < half ? half : -half), o);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = turned >> i & 1u ? one_f32<T>(p.x[kind], at + i + (d0 + i < half ? half : -half)) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (turned >> i & 1u) x[i] = fmaf(x[i], cs[i], o[i] * sn[i]);
    }
    if (kind == 0) {
      uint16_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = p.act == 0 ? __half_as_ushort(__float2half_rn(x[i])) : __bfloat16_as_ushort(__float2bfloat16_rn(x[i]));
      // q_out is contiguous and 8-byte aligned, D a multiple of 32
      *reinterpret_cast<uint2*>(p.q_out + (row * p.H + hh) * D + d0) =
          make_uint2(r[0] | (uint32_t)r[1] << 16, r[2] | (uint32_t)r[3] << 16);
      continue;
    }
    float amax = 0.f, a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = fabsf(x[i]);
      if (!(a[i] <= 3.402823466e38f)) a[i] = 0.f;
      amax = fmaxf(amax, a[i]);
    }
    amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 2));
    if constexpr (V == 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 4));
    const uint32_t e = quant_scale(amax);
    const float hs = 0.5f * ue4m3_f32(e);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c |= code_of(x[i], a[i], hs) << (8 * i);
    // byte j: value j below, value j + 16 above
    const uint32_t other = __shfl_xor_sync(mask, c, 4), e_other = __shfl_xor_sync(mask, e, 4);
    uint8_t* blk = (kind == 1 ? p.c.K : p.c.V) + ((slot + (int64_t)hh * p.c.page_size) * p.nb + block) * Fmt<V>::BB;
    if (l < 4) {
      const uint32_t w = c | other << 4;
      if constexpr (V == 0) {
        uint16_t* o = reinterpret_cast<uint16_t*>(blk) + 2 * l;
        o[0] = (uint16_t)w;
        o[1] = (uint16_t)(w >> 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) blk[4 * l + i] = (uint8_t)(w >> (8 * i));
      }
    } else if (l == 4) {
      if constexpr (V == 0)
        *reinterpret_cast<uint16_t*>(blk + 16) = (uint16_t)(e_other | e << 8);
      else
        blk[16] = (uint8_t)e;
    }
  }
}

constexpr int kReadThreads = 256;

struct ReadParams {
  void* out[2];  // K's and V's values, nullptr: not wanted
  int64_t M;
  int nb, type;
  PagedArgs c;
};

// OUT: 0 fp32, 1 bf16, 2 fp16.
template <int V, int OUT>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
  using F = Fmt<V>;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, l = lane & 7, q = lane & 3;
  const uint32_t mask = 0xFFu << (lane & 24);
  const int per_row = p.c.Hkv * p.nb;  // blocks of K (or V) a token has
  // eight lanes take K's and V's block of the same place
  const int64_t groups = p.M * per_row;
  for (int64_t g = ((int64_t)blockIdx.x * kReadThreads + threadIdx.x) >> 3; g < groups;
       g += (int64_t)gridDim.x * (kReadThreads / 8)) {
    const int64_t row = g / per_row;
    const int r = (int)(g - row * per_row), hh = r / p.nb, block = r - hh * p.nb;
    if (row >= p.c.cu[p.c.B] || row < p.c.cu[0]) continue;  // padding
    const int b = sequence_of(p.c.cu, p.c.B, row, mask, l);
    const int64_t len = p.c.lens[b];
    const int64_t pos = len - ((int64_t)p.c.cu[b + 1] - row);
    int page = -1;
    if (pos >= 0 && pos < len) {
      const int64_t pg = pos / p.c.page_size;
      page = pg < p.c.width ? p.c.table[b * p.c.ldt + pg] : -1;
      if (page < 0 || page >= p.c.num_pages) {
        page = -1;
        if (l == 0) atomicOr(p.c.err, kErrBadPage);
      }
    }
    const int which = l >> 2;
    void* out = p.out[which];
    if (out == nullptr) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (page >= 0) {
      const uint8_t* blk = (which ? p.c.V : p.c.K) +
                           ((((int64_t)page * p.c.Hkv + hh) * p.c.page_size + pos % p.c.page_size) * p.nb + block) * F::BB;
      uint32_t w, s;
      if constexpr (V == 0) {
        const uint16_t* b16 = reinterpret_cast<const uint16_t*>(blk);
        w = b16[2 * q] | (uint32_t)b16[2 * q + 1] << 16;
        s = b16[8];
      } else {
        w = blk[4 * q] | (uint32_t)blk[4 * q + 1] << 8 | (uint32_t)blk[4 * q + 2] << 16 | (uint32_t)blk[4 * q + 3] << 24;
        s = blk[16];
        s |= s << 8;
      }
      const uint32_t s2 = e4m3x2<0>(s);
      const uint32_t h[4] = {hmul2(clamp5(e2m1x2<0>(w)), s2), hmul2(clamp5(e2m1x2<1>(w)), s2),
                             hmul2(clamp5(e2m1x2<2>(w)), s2), hmul2(clamp5(e2m1x2<3>(w)), s2)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 t = *reinterpret_cast<const __half2*>(&h[i]);
        v[i] = __fadd_rn(__low2float(t), 0.f);  // -0 to +0
        v[4 + i] = __fadd_rn(__high2float(t), 0.f);
      }
    }
    const int64_t o = (row * per_row + r) * 32 + 4 * q;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (OUT == 0) {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + o + 16 * k) =
            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      } else {
        uint16_t t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[i] = OUT == 1 ? __bfloat16_as_ushort(__float2bfloat16_rn(v[4 * k + i]))
                          : __half_as_ushort(__float2half_rn(v[4 * k + i]));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o + 16 * k) =
            make_uint2(t[0] | (uint32_t)t[1] << 16, t[2] | (uint32_t)t[3] << 16);
      }
    }
  }
}

template <class P>
cudaError_t launch_dependent(void (*fn)(P), int64_t grid, int threads, cudaStream_t s, const P& params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, params);
}

using RopeFn = void (*)(RopeParams);
template <int T, int V>
RopeFn rope_for(bool inter, bool vec) {
  if (inter) return vec ? rope_kernel<T, V, true, true> : rope_kernel<T, V, true, false>;
  return vec ? rope_kernel<T, V, false, true> : rope_kernel<T, V, false, false>;
}
template <int T>
RopeFn rope_for(int variant, bool inter, bool vec) {
  return variant == 0 ? rope_for<T, 0>(inter, vec) : rope_for<T, 1>(inter, vec);
}

}  // namespace

cudaError_t launch_rope(int variant, const RopeArgs& a, int sms, cudaStream_t s) {
  RopeParams p{};
  p.positions = a.positions;
  p.freq = a.freq;
  p.q_out = a.q_out;
  p.M = a.M;
  p.H = (int)a.H;
  p.rot = (int)a.rot;
  p.act = a.act;
  p.amplitude = a.amplitude;
  p.paged = a.paged;
  p.c = a.cache;
  if (!a.paged) p.c.Hkv = 0;
  p.heads = p.H + 2 * p.c.Hkv;
  p.nb = (int)(a.D / 32);
  const int64_t need = a.type == 0 ? 16 : 8;  // bytes of four values
  bool vec = a.interleaved || (a.rot / 2) % 4 == 0;
  for (int i = 0; i < 3; ++i) {
    p.x[i] = a.x[i];
    p.ld[i] = a.ld[i];
    if (a.x[i] != nullptr && (reinterpret_cast<uintptr_t>(a.x[i]) % need != 0 || a.ld[i] % 4 != 0)) vec = false;
  }
  // Walks: as many as give every SM 2048 threads, at most one per head.
  const int64_t want = (int64_t)sms * 256;
  int64_t slices = (want + a.M * p.nb - 1) / (a.M * p.nb);
  p.slices = (int)(slices < 1 ? 1 : slices > p.heads ? p.heads : slices);
  const RopeFn fn = a.type == 0 ? rope_for<0>(variant, a.interleaved, vec)
                    : a.type == 1 ? rope_for<1>(variant, a.interleaved, vec)
                                  : rope_for<2>(variant, a.interleaved, vec);
  const int64_t groups = a.M * p.nb * p.slices;
  return launch_dependent(fn, (groups * 8 + kRopeThreads - 1) / kRopeThreads, kRopeThreads, s, p);
}

cudaError_t launch_cache_read(int variant, int type, const CacheReadArgs& a, int sms, cudaStream_t s) {
  ReadParams p{};
  p.out[0] = a.k_out;
  p.out[1] = a.v_out;
  p.M = a.M;
  p.nb = a.cache.D / 32;
  p.type = type;
  p.c = a.cache;
  const int64_t groups = a.M * p.c.Hkv * p.nb;
  int64_t grid = (groups * 8 + kReadThreads - 1) / kReadThreads;
  const int64_t most = (int64_t)sms * 64;
  grid = grid > most ? most : grid;
  using Fn = void (*)(ReadParams);
  const Fn fn = variant == 0 ? (type == 0 ? (Fn)cache_read_kernel<0, 0> : type == 1 ? (Fn)cache_read_kernel<0, 1> : (Fn)cache_read_kernel<0, 2>)
                             : (type == 0 ? (Fn)cache_read_kernel<1, 0> : type == 1 ? (Fn)cache_read_kernel<1, 1> : (Fn)cache_read_kernel<1, 2>);
  return launch_dependent(fn, grid, kReadThreads, s, p);
}

}  // namespace rocmfp4
