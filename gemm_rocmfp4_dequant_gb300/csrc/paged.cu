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
// cosines are computed once for all heads of a walk.  Where the pairs are
// halves of whole blocks (rot = D, a multiple of 64) they own the partners' block
// too.  Few rows: one head a walk, for latency; many rows: one wave of walks.
// Measured, 4096 tokens of 40 + 8 + 8 heads of 128 in fp32, in a graph with their
// reading back: 52 us, 41 of them here (163 MB in and out, 4.0 TB/s).  82 with a
// block a thread, angles in fp64 and five walks; 64 with angles in integers and four
// heads' loads in flight; 56 with pairs of blocks; 55 with one wave of walks, in CTAs
// of 256 threads, four an SM, which leave some SMs three; 53 with fp64 for frequencies
// of 2 and more.  Six CTAs an SM: 60.  512 x 40 x 128 alone: 4.5 us, 8192 rows 40 us (6.2
// TB/s).  Bound by issue and latency together: 28 warps an SM, 23 on the average, 43 % of
// the issue slots.
//
// cache_read_kernel.  The rows' blocks back as dense values, exact in every
// output type; four threads a block, one or four tokens a warp.  Measured,
// 16 x 4096 tokens of 8 heads of 128 in bf16: 75 us (344 MB, 4.6 TB/s).  198 with
// every block's place looked up by itself; 98 with a token a warp; 77 with one
// block's loads in flight a thread, 89 with three.  Bound by the ALU (58 %) and the
// latency of the places.
#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace rocmfp4 {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 7;  // CTAs an SM, at least: bounds the registers
constexpr int kBatch = 4;     // heads whose loads a thread has in flight

struct RopeParams {
  const void* x[3];  // q, k, v
  int64_t ld[3];
  const int32_t* positions;  // nullptr: the token's place in its sequence
  const float* freq;
  uint16_t* q_out;
  int64_t M;
  int H;  // heads of q
  int rot, nb, act;
  int places, slices;  // threads' blocks of a head; walks over the heads
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

// freq / 2 pi mod 1 in units of 2^-64: freq = m 2^-sh with a 24-bit m, so it is m times the bits of 1 / 2 pi, shifted, of which
// the turns above 1 fall away.  In integers, as this GPU has few fp64 units (the product and floor in fp64 took a third of a
// long append's time).  Below 2 radians a token the first 64 bits do; above, 128 of the first 256 (the digits come from
// arctangents of 1/5 and 1/239 in long integers).  Less than 2^-62 off, then, whatever the frequency.
RF4_DEV uint64_t turn_fraction(float freq) {
  constexpr uint64_t k0 = 0x28BE60DB9391054Aull, k1 = 0x7F09D5F47D4D3770ull, k2 = 0x36D8A5664F10E410ull, k3 = 0x7F9458EAF7AEF158ull;
  const uint32_t u = __float_as_uint(freq), E = u >> 23 & 255u;
  const uint64_t m = E ? (u & 0x7FFFFFu) | 0x800000u : 0u;
  uint64_t r;
  if (E > 127u) {
    // from bit `skip` on: before it stand whole turns for any m
    const uint32_t skip = E > 150u ? E - 150u : 0u, sh = E < 150u ? 150u - E : 0u, part = skip & 63u;
    const uint64_t a = skip < 64u ? k0 : k1, b = skip < 64u ? k1 : k2, c = skip < 64u ? k2 : k3;
    const uint64_t w0 = part ? a << part | b >> (64u - part) : a, w1 = part ? b << part | c >> (64u - part) : b;
    const uint64_t lo = m * w0, mid = lo + __umul64hi(m, w1), hi = __umul64hi(m, w0) + (mid < lo);
    r = sh ? hi << (64u - sh) | mid >> sh : mid;
  } else {
    const uint32_t sh = 150u - E;  // at least 23
    const uint64_t lo = m * k0, hi = __umul64hi(m, k0);
    r = sh < 64u ? hi << (64u - sh) | lo >> sh : sh < 128u ? hi >> (sh - 64u) : 0u;
  }
  return u >> 31 ? 0ull - r : r;
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

// All ones if a > t.
RF4_DEV int above(float a, float t) {
  int r;
  asm("set.gt.s32.f32 %0, %1, %2;" : "=r"(r) : "f"(a), "f"(t));
  return r;
}

// The codes of four values, a byte each: the number of midpoints that |x| lies
// above, and the sign of what is not zero.  a: |x|, 0 for what is not finite.
RF4_DEV uint32_t codes_of(const float (&x)[4], const float (&a)[4], float hs) {
  const float t[7] = {0.5f * hs, 1.5f * hs, 2.5f * hs, 3.5f * hs, 5.f * hs, 7.f * hs, 9.f * hs};
  int n = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    int k = 0;
#pragma unroll
    for (int j = 0; j < 7; ++j) k += above(a[i], t[j]);
    n = n * 256 + k;
  }
  const uint32_t c = (uint32_t)-n;
  const uint32_t top = __byte_perm(__byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0073),
                                   __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0073), 0x5410);
  return c | (top >> 4 & (c + 0x07070707u) & 0x08080808u);
}

RF4_DEV void store_q(const RopeParams& p, int64_t at, const float (&x)[4]) {
  uint2 r;
  if (p.act == 0) {
    const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
    r = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    r = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  *reinterpret_cast<uint2*>(p.q_out + at) = r;  // q_out is contiguous and 8-byte aligned, D a multiple of 32
}

// Quantises a block that eight threads hold, four values each, and writes it.
template <int V>
RF4_DEV void store_block_of(uint8_t* pages, int64_t at, const float (&x)[4], uint32_t mask, int l) {
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
  const uint32_t c = codes_of(x, a, hs);
  // byte j: value j below, value j + 16 above
  const uint32_t other = __shfl_xor_sync(mask, c, 4), e_other = __shfl_xor_sync(mask, e, 4);
  uint8_t* blk = pages + at * Fmt<V>::BB;
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

template <int N>
struct Kind {  // 0 q, 1 k, 2 v
  static constexpr int value = N;
};

// How a thread's values are paired.
enum Pairs {
  kInterleaved,  // (2i, 2i + 1): four values hold their own partners
  kHalves,       // (i, i + rot / 2): the partners are read a second time
  kWhole         // the same with rot = D, a multiple of 64: the thread takes the block of the partners too
};

// T: type of q, k and v (0 fp32, 1 bf16, 2 fp16).  V: block layout.  VEC: every
// four values are one aligned vector, and so are their partners.
template <int T, int V, int PAIRS, bool VEC>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int N = PAIRS == kWhole ? 2 : 1;  // blocks of a thread
  constexpr int BATCH = kBatch / N;
  const int lane = threadIdx.x & 31, l = lane & 7;
  const uint32_t mask = 0xFFu << (lane & 24);
  const uint32_t group = (uint32_t)(((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 3);
  const uint32_t rest = group / (uint32_t)p.places;
  const int block = (int)(group - rest * p.places);
  const int64_t row = rest / (uint32_t)p.slices;
  const int slice = (int)(rest - (uint32_t)row * p.slices);
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
    if (PAIRS == kWhole || d < rot) {
      turned |= 1u << i;
      if (PAIRS != kInterleaved || i % 2 == 0) {
        const float f = p.freq[PAIRS == kInterleaved ? d / 2 : PAIRS == kWhole || d < half ? d : d - half];
        turns[i] = turn_fraction(f);
        if (!(fabsf(f) <= 3.402823466e38f)) turned |= 16u << i;  // no angle: NaN
      }
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
      const uint32_t pg = (uint32_t)pos / (uint32_t)p.c.page_size;
      const int page = pg < (uint32_t)p.c.width ? p.c.table[b * p.c.ldt + pg] : -1;
      if (page >= 0 && page < p.c.num_pages)
        slot = (int64_t)page * p.c.Hkv * p.c.page_size + ((uint32_t)pos - pg * (uint32_t)p.c.page_size);
      else if (l == 0)
        atomicOr(p.c.err, kErrBadPage);
    }
  }
  if (p.positions != nullptr) pos = p.positions[row];
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (PAIRS == kInterleaved && (i & 1)) {
      cs[i] = cs[i - 1];
      sn[i] = -sn[i - 1];
      continue;
    }
    turn(turns[i] * (uint64_t)pos, cs[i], sn[i]);
    if (turned >> (4 + i) & 1u) cs[i] = sn[i] = __uint_as_float(0x7FC00000u);
    cs[i] *= p.amplitude;
    sn[i] *= PAIRS != kHalves || d0 + i < half ? -p.amplitude : p.amplitude;
  }

  // A batch of heads of one kind: all loads, then the arithmetic.
  auto batch = [&](auto kind_, int h0, int n) {
    constexpr int kind = decltype(kind_)::value;
    const int64_t at0 = row * p.ld[kind] + d0;
    float x[BATCH][4], o[BATCH][4];  // o: the partners
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int h = h0 + u * p.slices;
      if (h >= n) break;
      const int64_t at = at0 + (int64_t)h * D;
      load4<T, VEC>(p.x[kind], at, x[u]);
      if constexpr (PAIRS == kWhole) {
        load4<T, VEC>(p.x[kind], at + half, o[u]);
      } else if constexpr (PAIRS == kHalves && kind != 2) {
        if (!turned) continue;
        if constexpr (VEC) {
          load4<T, true>(p.x[kind], at + (d0 < half ? half : -half), o[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[u][i] = turned >> i & 1u ? one_f32<T>(p.x[kind], at + i + (d0 + i < half ? half : -half)) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int h = h0 + u * p.slices;
      if (h >= n) break;
      if constexpr (PAIRS == kWhole && kind != 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[u][i], b = o[u][i];
          x[u][i] = fmaf(a, cs[i], b * sn[i]);
          o[u][i] = fmaf(b, cs[i], a * -sn[i]);
        }
      } else if constexpr (kind != 2) {
        if (turned) {
          if constexpr (PAIRS == kInterleaved) o[u][0] = x[u][1], o[u][1] = x[u][0], o[u][2] = x[u][3], o[u][3] = x[u][2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((VEC && PAIRS == kHalves) || (turned >> i & 1u)) x[u][i] = fmaf(x[u][i], cs[i], o[u][i] * sn[i]);
        }
      }
      if constexpr (kind == 0) {
        store_q(p, (row * p.H + h) * D + d0, x[u]);
        if constexpr (PAIRS == kWhole) store_q(p, (row * p.H + h) * D + d0 + half, o[u]);
      } else {
        uint8_t* pages = kind == 1 ? p.c.K : p.c.V;
        const int64_t at = (slot + (int64_t)h * p.c.page_size) * p.nb + block;
        store_block_of<V>(pages, at, x[u], mask, l);
        if constexpr (PAIRS == kWhole) store_block_of<V>(pages, at + p.places, o[u], mask, l);
      }
    }
  };
  for (int h = slice; h < p.H; h += BATCH * p.slices) batch(Kind<0>(), h, p.H);
  if (slot < 0) return;
  // the walks go on where q's heads ended
  const int first = (slice + p.slices - p.H % p.slices) % p.slices;
  for (int h = first; h < p.c.Hkv; h += BATCH * p.slices) batch(Kind<1>(), h, p.c.Hkv);
  const int second = (first + p.slices - p.c.Hkv % p.slices) % p.slices;
  for (int h = second; h < p.c.Hkv; h += BATCH * p.slices) batch(Kind<2>(), h, p.c.Hkv);
}

constexpr int kReadThreads = 128;
constexpr int kReadUnroll = 2;  // blocks of K and of V whose loads a thread has in flight

struct ReadParams {
  void* out[2];  // K's and V's values, nullptr: not wanted
  int64_t M;
  int nb, rows;     // blocks of a head; tokens of a warp, 1 or 4
  uint32_t inv_nb;  // 2^32 / nb rounded up, 0 for nb = 1
  PagedArgs c;
};

// A block's word 4q .. 4q + 3 of codes and its scales, by words on 4-byte
// boundaries: each holds a byte of the block, so none lies outside of the pages
// (whose size is a multiple of 16).
template <int V>
RF4_DEV void load_block(const uint8_t* blk, int q, uint32_t (&w)[3]) {
  const uint8_t* a = blk + 4 * q;
  const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(a) & 3u, mis_s = (uint32_t)reinterpret_cast<uintptr_t>(blk + 16) & 3u;
  w[0] = *reinterpret_cast<const uint32_t*>(a - mis);
  w[1] = mis ? *reinterpret_cast<const uint32_t*>(a - mis + 4) : 0u;
  w[2] = *reinterpret_cast<const uint32_t*>(blk + 16 - mis_s);
  w[0] = __funnelshift_r(w[0], w[1], 8 * mis);
  w[2] >>= 8 * mis_s;
}

// The four pairs (value j, value j + 16) of a word, exact; a zero has no sign.
template <int V>
RF4_DEV void decode_word(uint32_t w, uint32_t scales, uint32_t (&h)[4]) {
  const uint32_t s2 = e4m3x2<0>(V == 0 ? scales & 0xFFFFu : __byte_perm(scales, 0u, 0x4400u));
  const __half2 s = *reinterpret_cast<const __half2*>(&s2), zero = __half2half2(__ushort_as_half(0));
  const uint32_t m[4] = {clamp5(e2m1x2<0>(w)), clamp5(e2m1x2<1>(w)), clamp5(e2m1x2<2>(w)), clamp5(e2m1x2<3>(w))};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 z = __hfma2(*reinterpret_cast<const __half2*>(&m[i]), s, zero);
    h[i] = *reinterpret_cast<const uint32_t*>(&z);
  }
}

// Writes a thread's eight values of block r.  Two bytes a value: neighbours swap, so that the even thread has eight of the
// first half and the odd one eight of the second, 16 bytes each.
template <int OUT>
RF4_DEV void store_block(void* out, int64_t at, int q, const uint32_t (&h)[4], bool want) {
  if constexpr (OUT == 0) {
    if (!want) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 t = *reinterpret_cast<const __half2*>(&h[i]);
      v[i] = __low2float(t);
      v[4 + i] = __high2float(t);
    }
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at + 4 * q);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[4] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = OUT == 1 ? f16x2_to_bf16x2(h[i]) : h[i];
    const bool odd = q & 1;
    const uint32_t mine = odd ? 0x7632 : 0x5410, other = odd ? 0x5410 : 0x7632;
    const uint32_t k0 = __byte_perm(x[0], x[1], mine), k1 = __byte_perm(x[2], x[3], mine);
    const uint32_t a = __shfl_xor_sync(0xffffffffu, __byte_perm(x[0], x[1], other), 1);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, __byte_perm(x[2], x[3], other), 1);
    if (!want) return;
    // even: 4q .. 4q + 7; odd: 16 + 4 (q - 1) .. + 7
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at + (odd ? 12 + 4 * q : 4 * q));
    *o = odd ? make_uint4(a, b, k0, k1) : make_uint4(k0, k1, a, b);
  }
}

// OUT: 0 fp32, 1 bf16, 2 fp16.
template <int V, int OUT>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
  using F = Fmt<V>;
  constexpr uint32_t kAll = 0xffffffffu;
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, q = lane & 3;
  const uint32_t mask = 0xFFu << (lane & 24);
  const int64_t row0 = ((int64_t)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5)) * p.rows;
  if (row0 >= p.M) return;
  grid_dependency_wait();
  // where the tokens lie, eight lanes a token: the byte of head 0; -1: nowhere, -2: padding
  int64_t place = -2;
  const int64_t row = row0 + (p.rows == 1 ? 0 : lane >> 3);
  if (row < p.M && row < p.c.cu[p.c.B] && row >= p.c.cu[0]) {
    const int b = sequence_of(p.c.cu, p.c.B, row, mask, lane & 7);
    const int64_t len = p.c.lens[b];
    const int64_t pos = len - ((int64_t)p.c.cu[b + 1] - row);
    place = -1;
    if (pos >= 0 && pos < len) {
      const uint32_t pg = (uint32_t)pos / (uint32_t)p.c.page_size;
      const int page = pg < (uint32_t)p.c.width ? p.c.table[b * p.c.ldt + pg] : -1;
      if (page >= 0 && page < p.c.num_pages)
        place = ((int64_t)page * p.c.Hkv * p.c.page_size + ((uint32_t)pos - pg * (uint32_t)p.c.page_size)) * p.nb * F::BB;
      else if ((lane & 7) == 0)
        atomicOr(p.c.err, kErrBadPage);
    }
  }
  __syncwarp();
  // The warp's tokens are p.rows * per_row blocks in a row of the output: eight at a time, four lanes each.
  const int per_row = p.c.Hkv * p.nb, total = p.rows * per_row;
  const int row_step = 8 / per_row, block_step = 8 - row_step * per_row;
  const int64_t skip = (int64_t)(p.c.page_size - 1) * p.nb;  // blocks from a head's row to the next head's, less a row's own
  int t = (lane >> 2) / per_row, r = (lane >> 2) - t * per_row;  // token, block of the token
  for (int f = lane >> 2; f - (lane >> 2) < total; f += 8 * kReadUnroll) {
    uint32_t w[kReadUnroll][2][3];
    bool want[kReadUnroll];
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int64_t at = __shfl_sync(kAll, place, p.rows == 1 ? 0 : min(t, 3) * 8);
      want[u] = f + 8 * u < total && at != -2;
      const uint32_t head = p.inv_nb ? __umulhi((uint32_t)r, p.inv_nb) : (uint32_t)r;
      const int64_t byte = at + (r + head * skip) * F::BB;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        w[u][k][0] = w[u][k][1] = w[u][k][2] = 0u;
        if (want[u] && at >= 0 && p.out[k] != nullptr) load_block<V>((k ? p.c.V : p.c.K) + byte, q, w[u][k]);
      }
      t += row_step;
      r += block_step;
      if (r >= per_row) {
        r -= per_row;
        ++t;
      }
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (p.out[k] == nullptr) continue;
        uint32_t h[4];
        decode_word<V>(w[u][k][0], w[u][k][2], h);  // nothing loaded: zeros
        store_block<OUT>(p.out[k], (row0 * per_row + f + 8 * u) * 32, q, h, want[u]);
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
RopeFn rope_for(int pairs, bool vec) {
  if (pairs == kWhole) return rope_kernel<T, V, kWhole, true>;
  if (pairs == kHalves) return vec ? rope_kernel<T, V, kHalves, true> : rope_kernel<T, V, kHalves, false>;
  return vec ? rope_kernel<T, V, kInterleaved, true> : rope_kernel<T, V, kInterleaved, false>;
}
template <int T>
RopeFn rope_for(int variant, int pairs, bool vec) {
  return variant == 0 ? rope_for<T, 0>(pairs, vec) : rope_for<T, 1>(pairs, vec);
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
  p.nb = (int)(a.D / 32);
  const int64_t need = a.type == 0 ? 16 : 8;  // bytes of four values
  bool vec = a.interleaved || (a.rot / 2) % 4 == 0;
  for (int i = 0; i < 3; ++i) {
    p.x[i] = a.x[i];
    p.ld[i] = a.ld[i];
    if (a.x[i] != nullptr && (reinterpret_cast<uintptr_t>(a.x[i]) % need != 0 || a.ld[i] % 4 != 0)) vec = false;
  }
  const int pairs = a.interleaved ? kInterleaved : vec && a.rot == a.D && a.D % 64 == 0 ? kWhole : kHalves;
  p.places = pairs == kWhole ? p.nb / 2 : p.nb;
  // Walks: as many as all SMs hold at a time (more would compute the angles again), at most one per head.
  const int64_t heads = p.H + 2 * (int64_t)p.c.Hkv;
  const int64_t slices = (int64_t)sms * kRopeCtas * (kRopeThreads / 8) / (a.M * p.places);
  p.slices = (int)(slices < 1 ? 1 : slices > heads ? heads : slices);
  const RopeFn fn = a.type == 0 ? rope_for<0>(variant, pairs, vec) : a.type == 1 ? rope_for<1>(variant, pairs, vec) : rope_for<2>(variant, pairs, vec);
  const int64_t groups = a.M * p.places * p.slices;
  return launch_dependent(fn, (groups * 8 + kRopeThreads - 1) / kRopeThreads, kRopeThreads, s, p);
}

cudaError_t launch_cache_read(int variant, int type, const CacheReadArgs& a, int sms, cudaStream_t s) {
  ReadParams p{};
  p.out[0] = a.k_out;
  p.out[1] = a.v_out;
  p.M = a.M;
  p.nb = a.cache.D / 32;
  p.inv_nb = p.nb == 1 ? 0u : (uint32_t)(((1ull << 32) + p.nb - 1) / p.nb);
  p.c = a.cache;
  // Four tokens a warp look their places up at the same time; one where there are not warps enough for all SMs.
  p.rows = a.M >= (int64_t)sms * 4 * 32 ? 4 : 1;
  const int64_t warps = (a.M + p.rows - 1) / p.rows;
  const int64_t grid = (warps + kReadThreads / 32 - 1) / (kReadThreads / 32);
  using Fn = void (*)(ReadParams);
  const Fn fn = variant == 0 ? (type == 0 ? (Fn)cache_read_kernel<0, 0> : type == 1 ? (Fn)cache_read_kernel<0, 1> : (Fn)cache_read_kernel<0, 2>)
                             : (type == 0 ? (Fn)cache_read_kernel<1, 0> : type == 1 ? (Fn)cache_read_kernel<1, 1> : (Fn)cache_read_kernel<1, 2>);
  return launch_dependent(fn, grid, kReadThreads, s, p);
}

}  // namespace rocmfp4
