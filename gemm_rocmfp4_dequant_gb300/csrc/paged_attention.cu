// Attention of a chunk of rows of every sequence over a paged ROCmFP4 cache:
//   out[r][h] = softmax_t(scale * q[r][h] . K[t]) . V[t]
// over the tokens t that row r sees.  A CTA takes one (row, head); its warps
// take alternate tokens and keep a running maximum and sum each.
#include "common.cuh"
#include "kernels.h"

namespace rocmfp4 {
namespace {

constexpr int kWarps = 4;

struct Params {
  PagedAttnArgs a;
};

RF4_DEV float act_f32(uint16_t bits, int act) {
  return act == 0 ? __half2float(__ushort_as_half(bits)) : __uint_as_float((uint32_t)bits << 16);
}

template <int V, int D>
RF4_DEV void row_values(const uint8_t* row, int lane, float (&v)[D / 32]) {
  constexpr int N = D / 32;
  const int d0 = lane * N, i = d0 & 31;
  const uint8_t* blk = row + d0 / 32 * Fmt<V>::BB;
  const float hs = halfscale_f32(blk[16 + (V == 0 ? i >> 4 : 0)]);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t byte = blk[(i + k) & 15], q = i >= 16 ? byte >> 4 : byte & 15u;
    const int m = (int)(q & 7u), c = m <= 4 ? m : 2 * m - 4;
    v[k] = (float)(q & 8u ? -c : c) * hs;
  }
}

template <int V, int D>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const __grid_constant__ Params p, int act) {
  constexpr int N = D / 32;
  constexpr int RB = D / 32 * Fmt<V>::BB;
  __shared__ float sm[kWarps][D + 2];
  const PagedAttnArgs& a = p.a;
  const PagedArgs& c = a.cache;
  grid_dependency_wait();
  const int64_t row = blockIdx.x / a.H;
  const int h = (int)(blockIdx.x % a.H), hk = h / (a.H / c.Hkv), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (row >= c.cu[c.B] || row < c.cu[0]) return;
  int b = 0;
  for (int n = c.B; n > 1;) {
    const int step = n / 2;
    if (c.cu[b + step] <= row) b += step, n -= step;
    else n = step;
  }
  int64_t len = c.lens[b];
  len = len < 0 ? 0 : len > (int64_t)c.width * c.page_size ? (int64_t)c.width * c.page_size : len;
  int64_t hi = len, lo = 0;
  if (a.causal) {
    hi = (int64_t)c.lens[b] - (c.cu[b + 1] - row) + 1;
    if (a.window > 0) lo = hi - a.window > 0 ? hi - a.window : 0;
    if (hi > len) hi = len;
  }
  float q[N], o[N], m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    q[k] = act_f32(a.q[row * a.ldq + (int64_t)h * D + lane * N + k], act);
    o[k] = 0.f;
  }
  for (int64_t t = lo + warp; t < hi; t += kWarps) {
    const int page = c.table[b * c.ldt + t / c.page_size];
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) atomicOr(c.err, kErrBadPage);
      continue;
    }
    const int64_t at = (((int64_t)page * c.Hkv + hk) * c.page_size + t % c.page_size) * RB;
    float kv[N], s = 0.f;
    row_values<V, D>(c.K + at, lane, kv);
#pragma unroll
    for (int k = 0; k < N; ++k) s = fmaf(q[k], kv[k], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale;
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn, al = expf(m - ref), e = expf(s - ref);
    row_values<V, D>(c.V + at, lane, kv);
    sum = sum * al + e;
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = o[k] * al + e * kv[k];
    m = mn;
  }
  if (lane == 0) sm[warp][D] = m, sm[warp][D + 1] = sum;
#pragma unroll
  for (int k = 0; k < N; ++k) sm[warp][lane * N + k] = o[k];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float M = -INFINITY, O = 0.f, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][D]);
    if (M == -INFINITY) M = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float e = sm[w][D] == -INFINITY ? 1.f : expf(sm[w][D] - M);
      O += e * sm[w][d];
      L += e * sm[w][D + 1];
    }
    const float y = L > 0.f || L != L ? O / L : 0.f;
    a.out[(row * a.H + h) * D + d] = act == 0 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
}

}  // namespace

cudaError_t launch_paged_attention(int variant, int act, const PagedAttnArgs& a, int sms, cudaStream_t s) {
  Params p{a};
  using Fn = void (*)(Params, int);
  const Fn fn = variant == 0 ? (a.cache.D == 64 ? (Fn)attend_kernel<0, 64> : (Fn)attend_kernel<0, 128>)
                             : (a.cache.D == 64 ? (Fn)attend_kernel<1, 64> : (Fn)attend_kernel<1, 128>);
  fn<<<(unsigned)(a.M * a.H), kWarps * 32, 0, s>>>(p, act);
  return cudaGetLastError();
}

}  // namespace rocmfp4
