// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits, in one pass over the logits:
//   z_v = scale * logit_v,  m = max z,  S = sum exp(z_v - m),
//   logprob(t) = z_t - m - ln S,   entropy = ln S - (sum exp(z_v - m) (z_v - m)) / S,
//   top n by (logit descending, index ascending) with their log probabilities.
// Every thread keeps its largest value m and the sums S and
// A = sum exp(z - m) (z - m) relative to it; sums are fp32.
//
// Bound: memory for many rows (each logit is read once; without
// alternatives 5.1 TB/s at 1024 rows of 152064 bf16, 5.3 at 608, one for each
// CTA that is resident at once), latency for few.  A row is cut into contiguous ranges, one per CTA, when
// there are too few rows to fill the GPU; the last CTA of a row to finish
// joins the ranges' records in range order, so the result does not depend on
// which that was.
//
// Measured on one GB300: 1024 rows of 152064 bf16 logits, 8 alternatives:
// 69.7 us, 4.47 TB/s, 66 % of the copy bandwidth; 333 rows of 32001 fp16, none:
// 9.6 us (9.1 in a graph); one row of 152064 fp32, 5: 8.6 us.
//
// Top n.  Values are compared as 64-bit keys (order-preserving bits of the
// logit, complement of the index), so ties go to the lowest index and keys are
// distinct.  In the pass a thread keeps the largest value of each of at most 8
// runs of tiles, its chunks.  The n-th largest of 64 groups' largest values, as
// a key with the last index that it can have, is a threshold that at least n
// values reach; only chunks whose largest value reaches it can hold the top n,
// little more than n as a rule, and their vectors alone are read again.  The
// pass has no barrier and costs the same in whatever order the values come.
// A candidate list filled during the pass, behind a threshold that was raised
// after 2, 4, 8, ... tiles, took 80.8 against 69.5 us on the first case above
// and 8.3 against 8.7 on the third.  One chunk a thread, and so all vectors of
// the few threads read again, took 85.8.
#include "common.cuh"
#include "kernels.h"

namespace rocmfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 2;        // 16-byte vectors a thread takes of a tile
constexpr int kGroups = 64;     // groups of 4 neighbouring threads
constexpr int kChunks = 8;      // runs of tiles whose largest values a thread keeps
constexpr int kCap = 1024;      // room of the candidate list
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving bits: a < b as floats iff key(a) < key(b); -0 counts as +0
// and every NaN as the largest.
RF4_DEV uint32_t ordered(float f) {
  if (f != f) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
RF4_DEV float unordered(uint32_t k) {
  if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
RF4_DEV uint64_t key_of(float f, uint32_t index) { return ((uint64_t)ordered(f) << 32) | (uint32_t)~index; }

// A distance at which exp(scale * distance) is 0 for every accepted scale;
// takes the place of -inf, so that 0 * distance stays 0.
constexpr float kFarBelow = -3.0e38f;

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
RF4_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
RF4_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
RF4_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

RF4_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
RF4_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Running softmax of some of a row's logits: S and A are the sums of e and
// e * (logit - m) with e = exp(scale * (logit - m)), m the largest of them.  Its
// own term is exactly 1 and no d is above 0, so S >= 1 and A <= 0 whatever
// rounds: log probabilities are at most 0 and entropies at least 0.  (An m that
// lags behind the largest value spares most tiles the rescaling, 69.1 against
// 69.7 us for 1024 rows of 152064 bf16, but leaves differences of numbers near
// 28, off by 2e-6 with either sign, where one token is nearly certain.)
struct Stats {
  float m = -INFINITY, S = 0.f, A = 0.f;
};

// Moves (S, A) from the reference `from` to `to` >= from; no values yet (m = -inf) stay nothing.
RF4_DEV void rescale(float& S, float& A, float from, float to, float c) {
  if (from == to || (S == 0.f && A == 0.f)) return;
  const float d = from - to, e = ex2(d * c);
  // e = 0 (a maximum far above): both sums vanish, and d may be infinite
  A = e > 0.f ? e * (A + d * S) : 0.f;
  S = e * S;
}
// The statistics of the lanes together, in every lane; the sums in a fixed order.
RF4_DEV Stats join(Stats s, float c) {
  float m = s.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  rescale(s.S, s.A, s.m, m, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
    s.A += __shfl_xor_sync(0xffffffffu, s.A, o);
  }
  s.m = m;
  return s;
}
// The statistics of the CTA's threads together, in every thread of warp 0 and
// in all[0] behind the next barrier.  `all`: room for a warp's each.
RF4_DEV void join_cta(Stats s, float c, Stats* all) {
  s = join(s, c);
  if ((threadIdx.x & 31) == 0) all[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = join(threadIdx.x < kThreads / 32 ? all[threadIdx.x] : Stats{}, c);
    __syncwarp();
    if (threadIdx.x == 0) all[0] = s;
  }
}

template <int TYPE>
struct Logit;
template <>
struct Logit<0> {
  using type = float;
  static constexpr int PER = 4;
  static RF4_DEV float one(float v) { return v; }
  // the largest value of some words (NaN only where there is nothing else)
  template <int W>
  static RF4_DEV float largest(const uint4 (&w)[W]) {
    float m = __uint_as_float(w[0].x);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      m = fmaxf(fmaxf(m, __uint_as_float(w[i].x)), __uint_as_float(w[i].y));
      m = fmaxf(fmaxf(m, __uint_as_float(w[i].z)), __uint_as_float(w[i].w));
    }
    return m;
  }
  static RF4_DEV void unpack(const uint4& w, float* v) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  }
};
template <>
struct Logit<1> {
  using type = uint16_t;
  static constexpr int PER = 8;
  static RF4_DEV float one(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static RF4_DEV uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  template <int W>
  static RF4_DEV float largest(const uint4 (&w)[W]) {
    uint32_t m = w[0].x;
#pragma unroll
    for (int i = 0; i < W; ++i) m = max2(max2(max2(max2(m, w[i].x), w[i].y), w[i].z), w[i].w);
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  static RF4_DEV void unpack(const uint4& w, float* v) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
};
template <>
struct Logit<2> {
  using type = uint16_t;
  static constexpr int PER = 8;
  static RF4_DEV float one(uint16_t v) { return __half2float(__ushort_as_half(v)); }
  static RF4_DEV uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  template <int W>
  static RF4_DEV float largest(const uint4 (&w)[W]) {
    uint32_t m = w[0].x;
#pragma unroll
    for (int i = 0; i < W; ++i) m = max2(max2(max2(max2(m, w[i].x), w[i].y), w[i].z), w[i].w);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return fmaxf(f.x, f.y);
  }
  static RF4_DEV void unpack(const uint4& w, float* v) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
};

struct TopState {  // in shared memory
  int count;       // candidates pushed (may pass the capacity)
  int chunks;      // that may have some
  int kept;        // scratch of cut()
  uint64_t floor;  // values must have a larger key to become candidates
  uint64_t group[kGroups];
  uint64_t best[kMaxTop];
};

// The n-th largest of the groups' largest keys (0 where fewer than n groups
// have one): at least n keys reach it.  `mine` is the thread's largest key, 0
// for none.  Every thread of the CTA calls it.
RF4_DEV uint64_t group_threshold(TopState& st, uint64_t mine, int n) {
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const uint64_t u = __shfl_xor_sync(0xffffffffu, mine, o);
    mine = u > mine ? u : mine;
  }
  __shared__ uint64_t threshold;
  if ((threadIdx.x & 3) == 0) st.group[threadIdx.x >> 2] = mine;
  if (threadIdx.x == 0) threshold = 0;
  __syncthreads();
  // a group's four lanes compare with a quarter of the groups each
  const int part = threadIdx.x & 3;
  int rank = 0;
#pragma unroll
  for (int i = 0; i < kGroups; i += 4) rank += st.group[i + part] > mine ? 1 : 0;
  rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  rank += __shfl_xor_sync(0xffffffffu, rank, 2);
  if (part == 0 && rank == n - 1 && mine != 0) threshold = mine;  // distinct keys: one group
  __syncthreads();
  return threshold;
}

// The n-th largest of `count` (n < count <= kThreads) distinct keys, of which
// zeros are none (then there may be fewer: 0).  Every thread of the CTA calls it.
RF4_DEV uint64_t nth_of(const uint64_t* keys, int count, int n) {
  __shared__ uint64_t threshold;
  if (threadIdx.x == 0) threshold = 0;
  __syncthreads();
  const int lanes = count <= kThreads / 4 ? 4 : count <= kThreads / 2 ? 2 : 1;  // a key's
  const int at = threadIdx.x / lanes, part = threadIdx.x % lanes;
  const uint64_t mine = at < count ? keys[at] : 0;
  int rank = 0;
#pragma unroll 8
  for (int i = part; i < count; i += lanes) rank += keys[i] > mine ? 1 : 0;
  if (lanes > 1) rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  if (lanes > 2) rank += __shfl_xor_sync(0xffffffffu, rank, 2);
  if (part == 0 && mine != 0 && rank == n - 1) threshold = mine;
  __syncthreads();
  return threshold;
}

// The n largest of the candidate list's `count` keys to the list's front, in
// order; floor becomes the n-th (if there are n).  Every thread calls it.
RF4_DEV void cut(TopState& st, uint64_t* list, uint64_t* spare, int count, int n) {
  int c = count;
  uint64_t* from = list;
  if (count > 2 * kGroups) {  // few enough to rank: those that reach the groups' threshold
    uint64_t mine = 0;
    for (int i = threadIdx.x; i < count; i += kThreads) mine = list[i] > mine ? list[i] : mine;
    const uint64_t t = group_threshold(st, mine, n);
    if (threadIdx.x == 0) st.kept = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads)
      if (list[i] >= t) spare[atomicAdd(&st.kept, 1)] = list[i];
    __syncthreads();
    c = st.kept;
    from = spare;
  }
  for (int i = threadIdx.x; i < c; i += kThreads) {
    const uint64_t k = from[i];
    int rank = 0;
    for (int j = 0; j < c; ++j) rank += from[j] > k ? 1 : 0;
    if (rank < n) st.best[rank] = k;
  }
  __syncthreads();
  c = c < n ? c : n;
  if (threadIdx.x < c) list[threadIdx.x] = st.best[threadIdx.x];
  if (threadIdx.x == 0) {
    st.count = c;
    st.kept = c;
    if (c == n) st.floor = st.best[n - 1];
  }
  __syncthreads();
}

// One record per range of a split row: m, S, A, the number of keys, then kMaxTop keys.
constexpr int kRecordBytes = 16 + 8 * kMaxTop;
constexpr int kMaxSplits = kThreads;  // one record a thread at the join

template <int TYPE, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const __grid_constant__ LogprobsArgs a) {
  using L = Logit<TYPE>;
  using E = typename L::type;
  constexpr int PER = L::PER, N = kVecs * PER, TILE = kThreads * kVecs;  // vectors of a tile
  constexpr int kPicked = 4 * kMaxTop;  // threads that may have some of the top n
  static_assert(kThreads * kChunks * sizeof(float) <= kCap * sizeof(uint64_t), "the chunks' largest values fit the spare list");
  static_assert(kThreads + kMaxTop <= kCap && kMaxTop * kMaxTop <= kCap, "what is pushed without a check has room");
  __shared__ TopState st;
  __shared__ uint64_t lists[TOP ? 2 * kCap : 1];
  __shared__ Stats warp_stats[kThreads / 32];
  __shared__ int picked[kMaxTop];
  __shared__ uint16_t chunks[TOP ? kPicked * kChunks : 1];  // thread and chunk
  __shared__ int last;
  uint64_t* list = lists;
  uint64_t* spare = lists + (TOP ? kCap : 0);
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, n = a.top_n, P = a.splits;
  const int64_t row = blockIdx.x / P;
  const int part = blockIdx.x % P;
  const E* z = static_cast<const E*>(a.logits) + row * a.ld;
  const float c = a.scale * kLog2e;
  if (TOP && tid == 0) {
    st.count = 0;
    st.chunks = 0;
    st.floor = 0;
  }
  __syncthreads();

  // The row as vectors of PER values from the 16-byte boundary at or before
  // its start: places before value 0 and past value V - 1 count as absent.
  const int lead = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(E));
  const uint4* vz = reinterpret_cast<const uint4*>(z - lead);
  const int vecs = (int)((a.V + lead + PER - 1) / PER);
  const int v0 = (int)((int64_t)vecs * part / P), v1 = (int)((int64_t)vecs * (part + 1) / P);
  // A tile from `base` on whose every vector is this range's and wholly inside the row.
  const int whole_from = v0 + (v0 * PER < lead ? 1 : 0);
  const int whole_to = min(v1, (int)((a.V + lead) / PER)) - TILE;
  auto whole = [&](int base) { return base >= whole_from && base <= whole_to; };
  auto fetch = [&](int base, uint4 (&w)[kVecs]) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) w[k] = __ldcs(vz + (base + tid) + k * kThreads);
  };
  // index of value i of this thread's in a tile, and whether there is such a value
  auto index = [&](int base, int i) { return (int64_t)(base + (i / PER) * kThreads + tid) * PER - lead + i % PER; };
  auto present = [&](int base, int i) {
    const int64_t e = index(base, i);
    return base + (i / PER) * kThreads + tid < v1 && e >= 0 && e < a.V;
  };

  auto values = [&](int base, float (&v)[N]) {  // of a tile at an end, absent ones -inf
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      // a vector inside the row in one load, one at an end of it value by value
      if (present(base, k * PER) && present(base, k * PER + PER - 1)) {
        L::unpack(__ldg(vz + base + k * kThreads + tid), v + k * PER);
      } else {
#pragma unroll
        for (int i = k * PER; i < k * PER + PER; ++i) v[i] = present(base, i) ? L::one(z[index(base, i)]) : -INFINITY;
      }
    }
  };

  float given = __uint_as_float(0x7FC00000u);  // the target's logit, asked for ahead of use
  if (tid == 0 && a.targets != nullptr) {
    const int64_t t = a.targets[row];
    if (t >= 0 && t < a.V) given = L::one(z[t]);
  }

  Stats s;
  uint4 w[kVecs];
  if (v0 < v1 && whole(v0)) fetch(v0, w);
  // This thread's chunks' largest values; `spare` is not needed until they are done with.
  float* top = reinterpret_cast<float*>(spare) + tid;
  const int per_chunk = TOP ? ((v1 - v0 + TILE - 1) / TILE + kChunks - 1) / kChunks : 1;  // tiles
  float chunk_top = -INFINITY;
  int chunk = 0, in_chunk = 0;
#pragma unroll 1
  for (int base = v0; base < v1; base += TILE) {
    float v[N], tm;
    const bool full = whole(base);
    if (full) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) L::unpack(w[k], v + k * PER);
      tm = L::largest(w);
    } else {
      values(base, v);
      tm = v[0];
#pragma unroll
      for (int i = 1; i < N; ++i) tm = fmaxf(tm, v[i]);
    }
    if (whole(base + TILE)) fetch(base + TILE, w);  // the next tile is on its way while this one is summed
    if (tm > s.m) {
      rescale(s.S, s.A, s.m, tm, c);
      s.m = tm;
    }
    const float mm = s.m == -INFINITY ? 0.f : s.m;  // nothing but -inf yet: e = 0
    // the tile's sums on their own: short chains
    uint64_t S[2] = {0, 0}, A[2] = {0, 0};
    const uint64_t minus = pack2(-mm, -mm), cc = pack2(c, c);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint64_t d = add2(pack2(v[2 * i], v[2 * i + 1]), minus);
      const float2 t = unpack2(mul2(d, cc));
      const uint64_t e = pack2(ex2(t.x), ex2(t.y));
      S[i & 1] = add2(S[i & 1], e);
      A[i & 1] = fma2(e, d, A[i & 1]);
    }
    const float2 sum = unpack2(add2(S[0], S[1])), part_a = unpack2(add2(A[0], A[1]));
    float tile_a = part_a.x + part_a.y;
    if (tile_a != tile_a) {  // a value of -inf (0 * -inf) or a NaN: again, with a finite factor for e = 0
      tile_a = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = v[i] - mm;
        tile_a = fmaf(ex2(d * c), max_nan(d, kFarBelow), tile_a);
      }
    }
    s.S += sum.x + sum.y;
    s.A += tile_a;
    if constexpr (TOP) {
      chunk_top = fmaxf(chunk_top, tm);
      if (++in_chunk == per_chunk) {
        top[chunk++ * kThreads] = chunk_top;
        chunk_top = -INFINITY;
        in_chunk = 0;
      }
    }
  }
  if constexpr (TOP) {
    if (in_chunk > 0) top[chunk++ * kThreads] = chunk_top;
    const int count = chunk, vecs_chunk = per_chunk * kVecs;  // of a thread and chunk
    auto vec_of = [&](int thread, int at, int r) { return v0 + (at * vecs_chunk + r) * kThreads + thread; };
    // indices that values of a chunk lie between
    auto from_index = [&](int thread, int at) { return (uint32_t)max((int64_t)vec_of(thread, at, 0) * PER - lead, (int64_t)0); };
    auto to_index = [&](int thread, int at) { return (uint32_t)((int64_t)vec_of(thread, at, vecs_chunk - 1) * PER - lead + PER - 1); };

    // Bounds of the thread's largest key, 0 for none.
    uint64_t low = 0, high = 0;
    int look_from = v0, look_to = v1;
    const bool nan = s.S != s.S;  // perhaps: fmaxf() has passed over it, and it is the largest of values
    if (nan) {
      for (int k = 0; k < count; ++k) top[k * kThreads] = __uint_as_float(0x7FC00000u);
    } else if (v0 + tid < v1) {
      int at = 0;
      float best = top[0];
      for (int k = 1; k < count; ++k)
        if (top[k * kThreads] > best) best = top[k * kThreads], at = k;
      low = key_of(best, to_index(tid, at));
      high = key_of(best, from_index(tid, at));
      look_from = v0 + at * per_chunk * TILE;
      look_to = min(v1, look_from + per_chunk * TILE);
    }
    uint64_t least = 0;
    bool mine = false, look = nan;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      if (look) {
        low = 0;
#pragma unroll 1
        for (int base = look_from; base < look_to; base += TILE) {
          float v[N];
          values(base, v);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint64_t k = key_of(v[i], (uint32_t)index(base, i));
            if (k > low && present(base, i)) low = k;
          }
        }
        high = low;
      }
      least = group_threshold(st, low, n);
      mine = high != 0 && high >= least;
      if (__syncthreads_count(mine) <= kPicked) break;
      // Many threads tie at the threshold: their keys themselves, of which at
      // most 4 n reach their threshold.
      look = mine && !nan;
      if (!mine) low = high = 0;
    }
    if (mine)
      for (int k = 0; k < count; ++k)
        if (key_of(top[k * kThreads], from_index(tid, k)) >= least) chunks[atomicAdd(&st.chunks, 1)] = (uint16_t)(k * kThreads + tid);
    __syncthreads();
    const int items = st.chunks * vecs_chunk;
    auto item_vec = [&](int item) {
      const int k = item < items ? chunks[item / vecs_chunk] : 0;
      return item < items ? vec_of(k % kThreads, k / kThreads, item % vecs_chunk) : v1;
    };
    auto push = [&](uint64_t k) {
      const int at = atomicAdd(&st.count, 1);
      if (at < kCap) list[at] = k;
    };
    const float lv = unordered((uint32_t)(least >> 32));  // a NaN if there is no threshold
#pragma unroll 1
    for (int item = tid; item < items; item += kThreads) {
      const int x = item_vec(item);
      if (x >= v1) continue;
      const int64_t e = (int64_t)x * PER - lead;  // index of its first value
      if (e >= 0 && e + PER <= a.V) {
        float v[PER];
        L::unpack(__ldg(vz + x), v);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (!(v[i] < lv)) {
            const uint64_t k = key_of(v[i], (uint32_t)(e + i));
            if (k >= least) push(k);
          }
      } else {  // at an end of the row
#pragma unroll 1
        for (int i = 0; i < PER; ++i)
          if (e + i >= 0 && e + i < a.V) {
            const uint64_t k = key_of(L::one(z[e + i]), (uint32_t)(e + i));
            if (k >= least) push(k);
          }
      }
    }
    __syncthreads();
    const int pushed = st.count;
    __syncthreads();
    if (pushed > kCap) {
      // Few chunks with a thousand of the range's largest values.  Again, a
      // value a thread at a time, cut to n each time.
      if (tid == 0) st.count = 0, st.floor = least > 0 ? least - 1 : 0;
      __syncthreads();
#pragma unroll 1
      for (int from = 0; from < items; from += kThreads) {
        const int x = item_vec(from + tid);
#pragma unroll 1
        for (int i = 0; i < PER; ++i) {
          const int64_t e = x < v1 ? (int64_t)x * PER - lead + i : -1;
          if (e >= 0 && e < a.V) {
            const uint64_t k = key_of(L::one(z[e]), (uint32_t)e);
            if (k > st.floor) push(k);
          }
          __syncthreads();
          const int have = st.count;
          __syncthreads();
          cut(st, list, spare, have, n);
        }
      }
    }
  }
  join_cta(s, c, warp_stats);
  if (TOP) cut(st, list, spare, st.count, n);
  __syncthreads();

  if (P > 1) {
    uint8_t* records = reinterpret_cast<uint8_t*>(a.ws) + (size_t)row * P * kRecordBytes;
    uint8_t* mine = records + (size_t)part * kRecordBytes;
    if (tid == 0) *reinterpret_cast<float4*>(mine) = make_float4(warp_stats[0].m, warp_stats[0].S, warp_stats[0].A, 0.f);
    if (TOP && tid < n) reinterpret_cast<uint64_t*>(mine + 16)[tid] = tid < st.count ? list[tid] : 0;  // 0: none
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const bool l = atomic_add_acq_rel_gpu(a.cnt + row, 1u) == (uint32_t)P - 1u;
      if (l) store_relaxed_gpu(a.cnt + row, 0u);
      last = l;
    }
    __syncthreads();
    if (!last) return;
    // Thread p has record p (P is at most the CTA's threads).
    const uint8_t* own = records + (size_t)(tid < P ? tid : 0) * kRecordBytes;
    s = Stats{};
    uint64_t first = 0;  // the record's largest key
    if (tid < P) {
      const float4 r = __ldcg(reinterpret_cast<const float4*>(own));
      s = Stats{r.x, r.y, r.z};
      if (TOP) first = __ldcg(reinterpret_cast<const unsigned long long*>(own + 16));
    }
    if constexpr (TOP) {
      // The n-th largest of the records' largest keys is reached by at most n
      // records; the top n are among the keys of these.
      if (tid == 0) st.count = 0, st.floor = 0;
      if (tid < P) spare[tid] = first;
      __syncthreads();
      const uint64_t t = P > n ? nth_of(spare, P, n) : 0;
      if (first != 0 && first >= t) picked[atomicAdd(&st.count, 1)] = tid;
      __syncthreads();
      const int records_in = st.count;
      __syncthreads();
      if (tid == 0) st.count = 0;
      __syncthreads();
      for (int i = tid; i < records_in * n; i += kThreads) {
        const uint64_t k = __ldcg(reinterpret_cast<const unsigned long long*>(records + (size_t)picked[i / n] * kRecordBytes + 16) + i % n);
        if (k != 0 && k >= t) list[atomicAdd(&st.count, 1)] = k;
      }
    }
    join_cta(s, c, warp_stats);
    __syncthreads();
    if (TOP) cut(st, list, spare, st.count, n);
  }

  s = warp_stats[0];
  const bool empty = s.m == -INFINITY && s.S == 0.f;  // every logit is -inf: no token is possible
  const float ln = logf(s.S);
  if (tid == 0) {
    if (a.targets != nullptr) {
      const int64_t t = a.targets[row];
      a.logprob[row] = t >= 0 && t < a.V ? (empty ? -INFINITY : a.scale * (given - s.m) - ln) : given;
    }
    if (a.entropy != nullptr) a.entropy[row] = empty ? 0.f : ln - a.scale * s.A / s.S;
  }
  if (TOP && tid < n) {
    const uint64_t k = list[tid];
    a.top_ids[row * n + tid] = (int32_t)~(uint32_t)k;
    a.top_logprobs[row * n + tid] = empty ? -INFINITY : a.scale * (unordered((uint32_t)(k >> 32)) - s.m) - ln;
  }
}

using LogprobsFn = void (*)(LogprobsArgs);

}  // namespace

// Split rows have at most 4 * sms parts together.
size_t logprobs_ws_bytes(int sms) { return (size_t)4 * sms * kRecordBytes; }
size_t logprobs_cnt_words(int sms) { return (size_t)4 * sms; }

cudaError_t launch_logprobs(const LogprobsArgs& args, int sms, cudaStream_t s) {
  LogprobsArgs a = args;
  const int per = a.type == 0 ? 4 : 8;
  const int64_t tiles = (a.V / per + 1 + kThreads * kVecs - 1) / (kThreads * kVecs);
  // As many CTAs as are resident at once, four per SM, and no more: a second
  // wave of a few costs as much as the first (rounded up instead of down, 333
  // rows of 32001 fp16 14.5 against 10.0 us in a graph; with 8 alternatives 23.0
  // against 15.1; 24 of 152064 fp32 18.2 against 12.2).  Each has at least one
  // whole tile of its row.
  int64_t P = a.M >= 4 * (int64_t)sms ? 1 : 4 * (int64_t)sms / a.M;
  P = P < tiles ? P : tiles;
  P = P < kMaxSplits ? P : kMaxSplits;
  a.splits = (int)P;
  LogprobsFn fn;
  if (a.top_n > 0) fn = a.type == 0 ? logprobs_kernel<0, true> : a.type == 1 ? logprobs_kernel<1, true> : logprobs_kernel<2, true>;
  else fn = a.type == 0 ? logprobs_kernel<0, false> : a.type == 1 ? logprobs_kernel<1, false> : logprobs_kernel<2, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M * P));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace rocmfp4
