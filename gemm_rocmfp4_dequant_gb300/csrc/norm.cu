// Residual addition and RMS norm, the step between two products of a decode
// step or a prefill:
//   h = x + r,  y = h / sqrt(mean(h^2) + eps) * w,
// with h stored in the residual's type, y as fp16 / bf16 activations and, where
// asked for, y in 8 bits: q = e4m3(y / s), s = max|y| / 448 over each group of
// a row.  The norm is taken of the unrounded fp32 sum; the sum of squares, the
// norm and the group maxima are fp32, and each output is rounded once.
//
// Bound: memory (x and r read once, h, y and q written once; about 6 flops a
// value).  A row is held in registers between its two uses (sum of squares,
// scaling), so nothing is read twice: a group of threads owns a row, every
// thread 1 to kMaxVec vectors of 8 consecutive values.  Rows of up to 256
// values share a CTA (one warp or part of one per row).
//
// Many wide rows: a CTA per row leaves the memory idle while it sums and
// scales (8.5 to 9 ns a row whatever its bytes).  There, persistent CTAs bring
// whole rows to shared memory by bulk copies two rows ahead of use.
//
// Measured on one GB300: 23552 rows of 5120, fp32 into a bf16 stream, bf16 out:
// 193.5 us, 6.23 TB/s, 92 % of the copy bandwidth (198.9 us with a CTA per
// row); 4096 rows of 5120 with an 8-bit output: 30.6 us, 4.8 TB/s (37.4 us);
// one row of 5120: 2.6 us in a graph, 7.3 us called alone (the host's time).
#include "common.cuh"
#include "kernels.h"

namespace rocmfp4 {
namespace {

constexpr float kFp8Max = 448.0f;
constexpr int kMaxVec = 4;

enum : int { kTypeF32 = 0, kTypeBF16 = 1, kTypeF16 = 2, kTypeNone = 3 };

template <int T>
struct Elem {
  using type = uint16_t;
};
template <>
struct Elem<kTypeF32> {
  using type = float;
};

template <int T>
RF4_DEV float to_f32(typename Elem<T>::type v) {
  if constexpr (T == kTypeF32) return v;
  else if constexpr (T == kTypeBF16) return __uint_as_float((uint32_t)v << 16);
  else return __half2float(__ushort_as_half(v));
}

template <int T>
RF4_DEV typename Elem<T>::type from_f32(float f) {
  if constexpr (T == kTypeF32) return f;
  else if constexpr (T == kTypeBF16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  else return __half_as_ushort(__float2half_rn(f));
}

// Eight consecutive values starting at p; n of them exist (the rest read as 0).
template <int T, bool VEC>
RF4_DEV void load8(const void* base, int off, int n, float (&v)[8]) {
  using E = typename Elem<T>::type;
  const E* p = static_cast<const E*>(base) + off;
  if constexpr (VEC) {
    if constexpr (T == kTypeF32) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = to_f32<T>((uint16_t)w[i]);
        v[2 * i + 1] = to_f32<T>((uint16_t)(w[i] >> 16));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.f;
  }
}

template <int T, bool VEC>
RF4_DEV void store8(void* base, int off, int n, const float (&v)[8]) {
  using E = typename Elem<T>::type;
  E* p = static_cast<E*>(base) + off;
  if constexpr (VEC) {
    if constexpr (T == kTypeF32) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = from_f32<T>(v[2 * i]) | ((uint32_t)from_f32<T>(v[2 * i + 1]) << 16);
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// The types that are not template parameters (weight, y) are the same for the
// whole launch: a uniform branch per vector.
template <bool VEC>
RF4_DEV void load8_any(int type, const void* base, int off, int n, float (&v)[8]) {
  if (type == kTypeF32) load8<kTypeF32, VEC>(base, off, n, v);
  else if (type == kTypeBF16) load8<kTypeBF16, VEC>(base, off, n, v);
  else load8<kTypeF16, VEC>(base, off, n, v);
}

// Larger of two values; NaN if either is NaN (a row that holds one shows it in its scales).
RF4_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two e4m3 codes of (lo, hi), round to nearest even, saturating at 448; NaN stays NaN.
RF4_DEV uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The 8-bit codes of eight values whose group's largest magnitude is amax.
// The quotient y / s is y * (448 / amax), off by a few ulp of fp32: far below
// the 2^-4 steps of e4m3, and one product instead of a division a value.  A
// group below 1e-30 divides, as 448 / amax would leave fp32's range.
template <bool VEC>
RF4_DEV void quantise8(uint8_t* q, int n, const float (&v)[8], float amax) {
  float z[8];
  if (amax < 1e-30f) {
    const float s = amax / kFp8Max;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = s > 0.f ? v[j] / s : 0.f;
  } else {
    float inv;
    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(amax));
    inv *= kFp8Max;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = v[j] * inv;
  }
  const uint32_t c0 = e4m3_pair(z[0], z[1]) | (e4m3_pair(z[2], z[3]) << 16);
  const uint32_t c1 = e4m3_pair(z[4], z[5]) | (e4m3_pair(z[6], z[7]) << 16);
  if constexpr (VEC) {
    *reinterpret_cast<uint2*>(q) = make_uint2(c0, c1);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) q[j] = (uint8_t)((j < 4 ? c0 : c1) >> (8 * (j & 3)));
  }
}

// Sum (or largest) over the threads of a row: `lanes` of a warp (a power of two), or the whole CTA.
template <bool MAX>
RF4_DEV float row_reduce(float v, int lanes, int nwarps, float* red) {
  for (int o = (lanes < 32 ? lanes : 32) >> 1; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  if (lanes <= 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < nwarps; ++i) v = MAX ? max_nan(v, red[i]) : v + red[i];
  __syncthreads();
  return v;
}

// The rest of a row once its threads hold h: residual, sum of squares, norm and
// outputs.  `taken()` runs behind the first barrier of the row's sum, when
// every thread has h.  values(e): how many values a vector from e on has.
template <int RT, int NV, bool VEC, class Values, class Taken>
RF4_DEV void finish_row(const NormArgs& a, int64_t row, bool live, int t, int lanes, int nwarps, float* red, float (&h)[NV][8], Values&& values,
                        Taken&& taken) {
  const int D = (int)a.D;
  float ss = 0.f;
  uint8_t* res_out = RT == kTypeNone ? nullptr : static_cast<uint8_t*>(a.residual_out) + row * a.ldro * (RT == kTypeF32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (RT != kTypeNone) {
      const int e = 8 * (i * lanes + t), n = values(e);
      if (n > 0) store8<RT, VEC>(res_out, e, n, h[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
  }
  ss = row_reduce<false>(ss, lanes, nwarps, red);
  taken();
  const float rstd = rsqrtf(ss / (float)D + a.eps);
  const int group = a.group, shift = 31 - __clz(group | 1), groups = group ? (D + group - 1) >> shift : 1;
  void* y = a.y == nullptr ? nullptr : static_cast<uint16_t*>(a.y) + row * D;
  uint8_t* q = a.q == nullptr ? nullptr : a.q + row * D;
  float* scales = a.scales + row * groups;
  float rowmax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 8 * (i * lanes + t), n = values(e);
    if (n > 0) {
      float w[8];
      load8_any<VEC>(a.weight_type, a.weight, e, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] *= rstd * w[j];
      if (y != nullptr) {
        if (a.y_act == 1) store8<kTypeBF16, VEC>(y, e, n, h[i]);
        else store8<kTypeF16, VEC>(y, e, n, h[i]);
      }
    }
    if (q == nullptr) continue;
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (VEC || j < n) m = max_nan(m, fabsf(h[i][j]));
    rowmax = max_nan(rowmax, m);
    if (group == 0) continue;
    // a group is group / 8 consecutive lanes (4, 8 or 16, aligned in the warp)
    for (int o = group >> 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (n > 0) {
      if ((e & (group - 1)) == 0) scales[e >> shift] = m * (1.f / kFp8Max);
      quantise8<VEC>(q + e, n, h[i], m);
    }
  }
  if (q == nullptr || group != 0) return;
  rowmax = row_reduce<true>(rowmax, lanes, nwarps, red);
  if (live && t == 0) scales[0] = rowmax * (1.f / kFp8Max);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 8 * (i * lanes + t), n = values(e);
    if (n > 0) quantise8<VEC>(q + e, n, h[i], rowmax);
  }
}

// XT, RT: types of x and of the residual (kTypeNone: no residual).  NV:
// vectors a thread holds.  VEC: every row of every operand starts on a 16-byte
// boundary and D is a multiple of 8.
template <int XT, int RT, int NV, bool VEC>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a, int lanes) {
  __shared__ float red[32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const int rows_per_cta = blockDim.x / lanes;
  const int t = tid % lanes;
  const int64_t row = (int64_t)blockIdx.x * rows_per_cta + tid / lanes;
  const bool live = row < a.M;
  const int D = (int)a.D;
  // the row of every operand (a row past the last one reads and writes nothing)
  const int64_t r = live ? row : 0;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + r * a.ldx * (XT == kTypeF32 ? 4 : 2);
  const uint8_t* res = static_cast<const uint8_t*>(a.residual) + r * a.ldr * (RT == kTypeF32 ? 4 : 2);
  auto values = [&](int e) { return !live || e >= D ? 0 : VEC || D - e >= 8 ? 8 : D - e; };
  float h[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 8 * (i * lanes + t), n = values(e);
    if (n > 0) {
      load8<XT, VEC>(x, e, n, h[i]);
      if constexpr (RT != kTypeNone) {
        float v[8];
        load8<RT, VEC>(res, e, n, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += v[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
    }
  }
  finish_row<RT, NV, VEC>(a, r, live, t, lanes, blockDim.x >> 5, red, h, values, [] {});
}

constexpr int kStages = 2;

// Bytes of a stage: a row of x, then a row of the residual.
RF4_HOSTDEV constexpr int stage_bytes(int xt, int rt, int D) {
  return D * (xt == kTypeF32 ? 4 : 2) + (rt == kTypeNone ? 0 : D * (rt == kTypeF32 ? 4 : 2));
}

// The persistent form: a CTA takes rows blockIdx.x, + gridDim.x, ...; thread t
// its vectors t, t + blockDim.x, ... of each.
template <int XT, int RT, int NV>
__global__ void __launch_bounds__(512) norm_stream_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[32];
  __shared__ uint64_t bars[kStages];
  __shared__ int gave_up;
  const int t = threadIdx.x, lanes = blockDim.x, D = (int)a.D;
  const int xb = stage_bytes(XT, kTypeNone, D), bytes = stage_bytes(XT, RT, D);
  if (t == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_addr(&bars[i]), 1);
    fence_mbar_init();
    gave_up = 0;
  }
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
  auto issue = [&](int64_t row, int s) {  // thread 0
    const uint32_t bar = smem_addr(&bars[s]);
    uint8_t* dst = ring + s * bytes;
    mbar_arrive_expect_tx(bar, (uint32_t)bytes);
    bulk_g2s(smem_addr(dst), static_cast<const uint8_t*>(a.x) + row * a.ldx * (XT == kTypeF32 ? 4 : 2), (uint32_t)xb, bar);
    if constexpr (RT != kTypeNone)
      bulk_g2s(smem_addr(dst + xb), static_cast<const uint8_t*>(a.residual) + row * a.ldr * (RT == kTypeF32 ? 4 : 2), (uint32_t)(bytes - xb), bar);
  };
  if (t == 0)
    for (int s = 0; s < kStages; ++s)
      if (blockIdx.x + (int64_t)s * gridDim.x < a.M) issue(blockIdx.x + (int64_t)s * gridDim.x, s);
  auto values = [&](int e) { return e < D ? 8 : 0; };
  int s = 0;
  uint32_t parity = 0;
  int64_t row = blockIdx.x;
  bool stopped = false;
  for (; row < a.M && !stopped; row += gridDim.x) {
    if (!mbar_wait_bounded(smem_addr(&bars[s]), parity)) gave_up = 1;
    const uint8_t* st = ring + s * bytes;
    float h[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 8 * (i * lanes + t);
      if (e < D) {
        load8<XT, true>(st, e, 8, h[i]);
        if constexpr (RT != kTypeNone) {
          float v[8];
          load8<RT, true>(st + xb, e, 8, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += v[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      }
    }
    // Behind the barrier every thread has read the stage: the row two ahead may
    // come in.  A wait that gave up ends the loop, the same for all threads.
    auto taken = [&] {
      stopped = gave_up != 0;
      if (t == 0 && !stopped && row + (int64_t)kStages * gridDim.x < a.M) {
        fence_proxy_async();
        issue(row + (int64_t)kStages * gridDim.x, s);
      }
    };
    finish_row<RT, NV, true>(a, row, true, t, lanes, lanes >> 5, red, h, values, taken);
    if (++s == kStages) s = 0, parity ^= 1u;
  }
  if (stopped && t == 0) {  // the copies under way land before the CTA leaves
    atomicOr(a.err, kErrWaitTimeout);
    for (int i = 0; i < kStages; ++i) (void)mbar_wait_bounded(smem_addr(&bars[i]), i < s ? parity ^ 1u : parity);
  }
}

using NormFn = void (*)(NormArgs, int);

using StreamFn = void (*)(NormArgs);

template <int XT, int RT, bool VEC>
NormFn pick_nv(int nv) {
  switch (nv) {
    case 1: return norm_kernel<XT, RT, 1, VEC>;
    case 2: return norm_kernel<XT, RT, 2, VEC>;
    default: return norm_kernel<XT, RT, kMaxVec, VEC>;
  }
}

template <int XT, bool VEC>
NormFn pick_rt(int rt, int nv) {
  switch (rt) {
    case kTypeF32: return pick_nv<XT, kTypeF32, VEC>(nv);
    case kTypeBF16: return pick_nv<XT, kTypeBF16, VEC>(nv);
    case kTypeF16: return pick_nv<XT, kTypeF16, VEC>(nv);
    default: return pick_nv<XT, kTypeNone, VEC>(nv);
  }
}

template <bool VEC>
NormFn pick(int xt, int rt, int nv) {
  switch (xt) {
    case kTypeF32: return pick_rt<kTypeF32, VEC>(rt, nv);
    case kTypeBF16: return pick_rt<kTypeBF16, VEC>(rt, nv);
    default: return pick_rt<kTypeF16, VEC>(rt, nv);
  }
}

template <int XT, int NV>
StreamFn pick_stream_rt(int rt) {
  switch (rt) {
    case kTypeF32: return norm_stream_kernel<XT, kTypeF32, NV>;
    case kTypeBF16: return norm_stream_kernel<XT, kTypeBF16, NV>;
    case kTypeF16: return norm_stream_kernel<XT, kTypeF16, NV>;
    default: return norm_stream_kernel<XT, kTypeNone, NV>;
  }
}

template <int NV>
StreamFn pick_stream(int xt, int rt) {
  switch (xt) {
    case kTypeF32: return pick_stream_rt<kTypeF32, NV>(rt);
    case kTypeBF16: return pick_stream_rt<kTypeBF16, NV>(rt);
    default: return pick_stream_rt<kTypeF16, NV>(rt);
  }
}

constexpr int kStreamSmem = 96 * 1024;  // most a CTA of the persistent form takes

template <class... Args>
cudaError_t launch_dependent(void (*fn)(Args...), int64_t grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

int64_t norm_max_width() { return (int64_t)1024 * 8 * kMaxVec; }

cudaError_t norm_prepare() {
  for (int xt = 0; xt < 3; ++xt)
    for (int rt = 0; rt < 4; ++rt) {
      for (const StreamFn fn : {pick_stream<2>(xt, rt), pick_stream<4>(xt, rt)}) {
        cudaError_t e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
        if (e != cudaSuccess) return e;
      }
    }
  return cudaSuccess;
}

cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t s) {
  const int rt = a.residual != nullptr ? a.residual_type : (int)kTypeNone;
  const bool vec = a.D % 8 == 0 && a.ldx % 8 == 0 && al16(a.x) && al16(a.weight) && al16(a.y) && al16(a.q) &&
                   (rt == kTypeNone || (a.ldr % 8 == 0 && a.ldro % 8 == 0 && al16(a.residual) && al16(a.residual_out)));
  const int64_t vecs = (a.D + 7) / 8;
  // Persistent CTAs for rows of 1024 values and more, from eight rows an SM on
  // (fewer do not repay their start), where two rows fit a CTA's share.  Two
  // vectors a thread for the 8-bit output, whose extra work wants more threads
  // (4096 rows of 5120: 30.6 us against 35.7 with four), and for rows of up to
  // 24 KB (8192 rows of 2048, fp32 into bf16: 28.6 us against 33.8); else four
  // (23552 rows of 5120, fp32 into bf16: 193.5 us against 204.5 with two).
  const int64_t smem = kStages * (int64_t)stage_bytes(a.x_type, rt, (int)a.D);
  const int per = (a.q != nullptr || smem <= kStages * 24 * 1024) && vecs <= 1024 ? 2 : 4;
  if (vec && vecs >= 128 && vecs <= 512 * per && a.M >= 8 * (int64_t)sms && smem <= kStreamSmem) {
    const int threads = (int)(((vecs + per - 1) / per + 31) / 32 * 32);
    const StreamFn fn = per == 2 ? pick_stream<2>(a.x_type, rt) : pick_stream<4>(a.x_type, rt);
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads, (size_t)smem);
    if (e != cudaSuccess) return e;
    if (per_sm > 0) return launch_dependent(fn, (int64_t)per_sm * sms, threads, (int)smem, s, a);
  }
  // Vectors a thread holds: one where the rows are too few to fill the GPU (a
  // row's latency counts), four where they are many (fewer threads wait at
  // the row's reduction).
  int nv = a.M <= 2 * (int64_t)sms ? 1 : vecs >= 512 ? 4 : vecs >= 128 ? 2 : 1;
  while (nv < kMaxVec && (vecs + nv - 1) / nv > 1024) nv *= 2;
  int64_t lanes = (vecs + nv - 1) / nv;
  if (lanes <= 32) {
    int p = a.q != nullptr && a.group != 0 ? 16 : 4;  // a group's lanes share a warp and a row
    while (p < lanes) p *= 2;
    lanes = p;
  } else {
    lanes = (lanes + 31) / 32 * 32;
  }
  const int threads = lanes <= 32 ? 128 : (int)lanes;
  const int64_t rows_per_cta = threads / lanes;
  return launch_dependent(vec ? pick<true>(a.x_type, rt, nv) : pick<false>(a.x_type, rt, nv), (a.M + rows_per_cta - 1) / rows_per_cta, threads, 0, s,
                          a, (int)lanes);
}

}  // namespace rocmfp4
