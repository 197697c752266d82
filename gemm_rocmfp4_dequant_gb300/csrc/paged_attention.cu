// Attention of a chunk of rows of every sequence over a paged ROCmFP4 cache:
//   out[r][h] = softmax_t(scale * q[r][h] . K[t]) . V[t]
// over the tokens t that row r sees (causal, causal with a window, or all).
//
// Tiles.  The G query heads of a KV head share its tokens, so the (row, head)
// pairs of a sequence and a KV head are the rows of one matrix, token-major:
// row r is row r / G of the chunk, head r % G.  They are cut into tiles of up to
// 256; a tile walks over the tokens it sees, 128 at a time:
//   S = Q K^T    tcgen05.mma, 128 rows x 128 tokens, Q and K in shared memory
//   P = 2^((S - m) scale log2 e + 7), m a running maximum, into tensor memory
//   O += P V     tcgen05.mma, P from tensor memory, V from shared memory
// K and V are decoded from their blocks into shared memory, exact in fp16 (K in
// q's type), once for all rows of the tile.
//
// Two chains.  A "wide" tile (more than 128 rows) is two halves of 128 rows
// over the same tokens; a "narrow" one is one half whose even and odd token
// tiles go to the two chains, merged at the end.  While one chain's softmax
// runs, the tensor core works for the other.
//
// Softmax.  A thread owns a row (a lane of tensor memory), so maxima and sums
// need no exchange; both are fp32.  The reference m follows the maximum only
// when that has grown by more than 2^8 (the sum and O are scaled then), so
// P <= 2^15 fits fp16; P is rounded to fp16, whose half step of 2^-11 is the
// output type's own (fp16) or an eighth of it (bf16), and the sum keeps the
// unrounded values.  The factor 2^7 keeps weights down to 2^-21 normal in fp16; it
// cancels in O / l.
//
// Order of D.  Byte j of a block decodes to the pair (j, j + 16).  The
// contraction of S does not care for the order of D, so Q is stored in that
// order and K as it falls out; V's columns, and so O's, are in it too, and the
// output puts them back.
//
// Work: see paged_work.cuh; a wide tile's token tile counts twice.
//
// Warps (512 threads), registers moved from the others to the softmax:
//   0-3, 4-7   Q rows, softmax and output of chain 0 and 1
//   8-11       decode of K and V, one token row a thread
//   12, 13     MMA issue of chain 0 (and tensor-memory allocation) and 1
//   14         the stretch's row tiles; bulk copies of raw rows, one for each run
//              within a page
// (Measured when 512 rows over 33280 tokens took 286 us: two sets of decode
// warps, which leave the softmax 144 registers, 322; decode warps that fetch
// their own rows 376.)
//
// Measured (40 query heads over 8 of D = 128, in a graph): a prompt of 4096 246 us
// in bf16 (700 TFLOP/s of the products a causal mask asks for), 229 in fp16; 512 rows
// over 33280 tokens 283 us (1225 TFLOP/s, fp16).  Bound by shared memory: a wide token tile stores
// 64 KB of decoded K and V, reads their raw rows, and the four products read Q, K
// and V again, 2336 cycles at 128 bytes a cycle, and the 512 rows take about 4000 a
// wide token tile.  In bf16 K needs a second conversion.
// Every wait is bounded: a warp that gives up goes on without waiting, so that
// all meet at the end.  Where the chains meet, a warp that has no more row tiles,
// or gave up, stands in until all are as far.  At the end kErrWaitTimeout is
// recorded, and products and copies that nobody waited for are waited for.
#include <cstddef>
#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "paged_work.cuh"

namespace rocmfp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kTok = 128;     // tokens per tile
constexpr int kHalf = 128;    // rows per chain
constexpr int kMaxRaw = 8;    // stages of the raw ring
constexpr int kTiles = 16;    // token tiles described at a time
constexpr int kItems = 4;     // row tiles described at a time
constexpr int kSlots = 3;     // parts a CTA may hold: of its first, its last, and its current row tile
constexpr uint32_t kSuspendNs = 1000000;
constexpr float kGrow = 8.f;  // log2 of how far a maximum may lead its reference
constexpr float kLift = 7.f;  // log2 of P's factor
constexpr float kLarge = 4096.f;  // references (times scale log2 e) from which on scores are subtracted before they are scaled
constexpr float kLog2e = 1.4426950408889634f;

struct Params : Batch {
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq;
  int H;
  float scale_log2;
  float* ws;      // [ctas][kSlots][2][kHalf] rows of D, then as many pairs (m, l)
  uint32_t* cnt;  // [ctas], zero between launches
};

template <int V, int D>
struct Plan {
  static constexpr int RB = D / 32 * Fmt<V>::BB;  // raw bytes per token row
  static constexpr int RAW = kTok * RB;           // raw bytes per tile of K or V
  static constexpr int TILE = kTok * D * 2;       // decoded tile
  static constexpr int PANEL = kTok * 128;        // 64 columns of a tile
  static constexpr int STAGES = 2;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + STAGES * TILE;
  static constexpr int OFF_Q0 = OFF_V + STAGES * TILE;
  static constexpr int OFF_Q1 = OFF_Q0 + TILE;  // raw stages where no row tile is wide
  static constexpr int OFF_RAW = OFF_Q1 + TILE;
  static constexpr int ROOM = 227 * 1024 - 1024 - 2048;  // less alignment and barriers
  static constexpr int most(int n) { return n > kMaxRaw ? kMaxRaw : n; }
  static constexpr int RSTAGES = most((ROOM - OFF_RAW) / RAW), RSTAGES_NARROW = most((ROOM - OFF_Q1) / RAW);
  static constexpr int END = OFF_RAW + RSTAGES * RAW, END_NARROW = OFF_Q1 + RSTAGES_NARROW * RAW;
  static constexpr int OFF_BAR = END > END_NARROW ? END : END_NARROW;
  static constexpr int SMEM = OFF_BAR + 2048 + 1024;
  static_assert(RSTAGES >= 3 && OFF_BAR <= ROOM && SMEM <= 227 * 1024, "shared memory");
  static_assert(RAW % 16 == 0, "bulk copies");
};

// A token tile: rows from .. to - 1 of it were copied, but for `bad` groups of 16.
struct Tile {
  int from, to;
  uint32_t bad;
  int stop;  // no more tiles
};

struct Control {  // at OFF_BAR
  // barriers, each with the number of its arrivals
  uint64_t k_full[2], v_full[2];    // 4: decode warps
  uint64_t k_empty[2], v_empty[2];  // 2: chains
  uint64_t s_full[2], o_full[2], turn[2], drained[2];  // 1
  uint64_t p_full[2], q_full[2];                       // 4: softmax warps
  uint64_t raw_full[kMaxRaw];                          // 1, and the copies' bytes
  uint64_t raw_empty[kMaxRaw];                         // 4: decode warps
  uint64_t item_full[kItems];                          // 1
  uint64_t item_empty[kItems];                         // 8 + 2: softmax and MMA warps
  Stretch work;
  int last;
  uint32_t tmem;
  uint32_t first, copies;  // uses of raw stages: the first that the loader has not seen emptied, and how many there were
  Item items[kItems];
  Tile tiles[kTiles];
};
constexpr int kBars = 20 + 2 * kMaxRaw + 2 * kItems;
static_assert(offsetof(Control, work) == 8 * kBars && sizeof(Control) <= 2048, "control block");

struct Shape {
  static constexpr int kRows = 2 * kHalf, kNarrow = kHalf, kTok = 128, kMinShare = 4;
  static RF4_DEV int fixed(int weight) { return weight == 2 ? 3 : 1; }
};

// ---- tensor-core instructions -------------------------------------------------
RF4_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
RF4_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
RF4_DEV void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
RF4_DEV void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Shared-memory operands are in the 128-byte swizzle: rows of 128 bytes,
// groups of eight rows 1024 bytes apart (stride, in the descriptor's high word),
// 64-column panels the low word's upper half apart (used where the columns are
// the operand's outer dimension), address / 16 in its lower half.
//
// kind::f16, fp32 accumulator, A and B both fp16 (type 0) or bf16 (type 1), M =
// 128; `b_outer`: B's rows in memory are its contraction index.
RF4_HOSTDEV constexpr uint32_t instr_desc(int type, int n, int b_outer) {
  return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | ((uint32_t)b_outer << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
}
RF4_DEV bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
RF4_DEV void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
RF4_DEV void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
RF4_DEV void tmem_ld32(uint32_t addr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr));
}
RF4_DEV void tmem_st32(uint32_t addr, const float (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]),
      "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]),
      "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
      : "memory");
}
RF4_DEV void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// Waits for the loads; the registers pass through, so that no use of theirs comes before.
RF4_DEV void tmem_wait_ld(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
               :
               : "memory");
}
RF4_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

RF4_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
RF4_DEV uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
RF4_DEV uint32_t pack_act(float lo, float hi, int act) {
  if (act == 0) return pack_h2(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Registers between warpgroups: the block was launched with 512 x 128; two
// warpgroups take 176 a thread, two are left with 80.
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= kThreads * 128, "register split");
template <int N>
RF4_DEV void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
RF4_DEV void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Both chains' softmax warps meet; true if all of them were leaving.
RF4_DEV bool chains_meet(bool leaving) {
  uint32_t all;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, 1, 256, q;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(all) : "r"((uint32_t)leaving) : "memory");
  return all != 0;
}

// A wait for a phase that the hardware may suspend the warp in (plain polls
// measured the same).  Gives up after about 2^32 cycles.
RF4_DEV bool wait_suspended(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (ok) return true;
    if (clock64() - t0 > (1ll << 32)) return false;
  }
}

// Waits that go on without waiting once one has given up.
struct Waits {
  bool ok = true;
  RF4_DEV void warp(const uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_addr(bar), parity))) return;
    if (ok) ok = __all_sync(0xffffffffu, wait_suspended(smem_addr(bar), parity));
  }
};

// A place in a ring of stages and the parity of its use.  One set of warps waits
// for each of a ring's barriers, use by use: a set that left uses out could take an
// earlier phase's parity for the one it waits for.
struct Ring {
  uint32_t stage = 0, phase = 0;
  RF4_DEV void next(uint32_t n) {
    if (++stage == n) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// ---- decode ---------------------------------------------------------------------
template <int N>
RF4_DEV uint32_t pair_at(const uint32_t (&w)[N], int pos) {
  const uint32_t word = w[pos >> 2];
  switch (pos & 3) {
    case 0: return e2m1x2<0>(word);
    case 1: return e2m1x2<1>(word);
    case 2: return e2m1x2<2>(word);
    default: return e2m1x2<3>(word);
  }
}
template <int V, int N>
RF4_DEV uint32_t scales_at(const uint32_t (&w)[N], int pos) {
  if constexpr (V == 0) return (pos & 2) ? e4m3x2<1>(w[pos >> 2]) : e4m3x2<0>(w[pos >> 2]);
  return e4m3x2<0>(__byte_perm(w[pos >> 2], 0u, (uint32_t)(pos & 3) * 0x11u));
}

// A token's raw row as words.
template <int V, int D>
RF4_DEV void load_row(const uint8_t* raw, int row, uint32_t (&w)[(D / 32 * Fmt<V>::BB + 3) / 4]) {
  constexpr int RB = D / 32 * Fmt<V>::BB, N = (RB + 3) / 4;
  if constexpr (RB % 8 == 0) {
    const uint2* s = reinterpret_cast<const uint2*>(raw + row * RB);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 v = s[i];
      w[2 * i] = v.x;
      w[2 * i + 1] = v.y;
    }
  } else if constexpr (RB % 4 == 0) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(raw + row * RB);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = s[i];
  } else {  // 34 bytes: odd rows begin in the middle of a word
    static_assert(RB == 34, "row bytes");
    const uint32_t* s = reinterpret_cast<const uint32_t*>(raw + (row >> 1) * 68 + (row & 1) * 32);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = s[i];
    if (row & 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], i + 1 < N ? w[i + 1] : 0u, 16);
    }
  }
}

// The row's values into the swizzled tile: 64-column panels of 128-byte rows,
// 16-byte chunk c of row r at c ^ (r % 8).
template <int V, int D, bool BF16>
RF4_DEV void decode_row(const uint8_t* raw, uint8_t* tile, int row, bool real) {
  constexpr int BB = Fmt<V>::BB;
  uint8_t* dst = tile + row * 128;
  if (!real) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      *reinterpret_cast<uint4*>(dst + c / 8 * (kTok * 128) + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
    return;
  }
  uint32_t w[(D / 32 * BB + 3) / 4];
  load_row<V, D>(raw, row, w);
#pragma unroll
  for (int kb = 0; kb < D / 32; ++kb) {
    const uint32_t s2 = scales_at<V>(w, kb * BB + 16);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = hmul2(clamp5(pair_at(w, kb * BB + 4 * c + i)), s2);
        if constexpr (BF16) v[i] = f16x2_to_bf16x2(v[i]);
      }
      const int chunk = (kb & 1) * 4 + c;
      *reinterpret_cast<uint4*>(dst + kb / 2 * (kTok * 128) + ((chunk ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// ---- softmax of one tile's row -----------------------------------------------------
struct Row {
  float m = -INFINITY, l = 0.f;
};

// Column i of a group of 32, or -inf where bit i of `keep` is clear.
template <bool MASK>
RF4_DEV float masked(float x, int i, uint32_t keep) {
  if constexpr (MASK) return keep & (1u << i) ? x : -INFINITY;
  return x;
}

// Which of the 32 tokens from column c on a row sees: a .. e - 1 of the tile, but for `bad` groups of 16.
RF4_DEV uint32_t kept(int c, int a, int e, uint32_t bad) {
  const int lo = min(max(a - c, 0), 32), hi = min(max(e - c, 0), 32);
  const uint32_t from = lo < 32 ? 0xffffffffu << lo : 0u, to = hi < 32 ? ~(0xffffffffu << hi) : 0xffffffffu;
  const uint32_t two = bad >> (c >> 4);
  return from & to & ~((two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u));
}

RF4_DEV uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
RF4_DEV void un2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
RF4_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
RF4_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
RF4_DEV float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

template <bool MASK>
RF4_DEV float top_of(const float (&x)[32], uint32_t keep) {
  float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    t0 = max3(t0, masked<MASK>(x[i], i, keep), masked<MASK>(x[i + 1], i + 1, keep));
    t1 = max3(t1, masked<MASK>(x[i + 2], i + 2, keep), masked<MASK>(x[i + 3], i + 3, keep));
  }
  return fmaxf(t0, t1);
}

// 32 columns of S to P, packed; their sum is added to `sum`.
template <bool MASK>
RF4_DEV void weights(const float (&x)[32], uint32_t (&h)[16], uint64_t scale2, uint64_t lift2, uint64_t (&sum)[2], uint32_t keep) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float y0, y1;
    un2(fma2(f2(masked<MASK>(x[2 * i], 2 * i, keep), masked<MASK>(x[2 * i + 1], 2 * i + 1, keep)), scale2, lift2), y0, y1);
    y0 = ex2(y0);
    y1 = ex2(y1);
    sum[i & 1] = add2(sum[i & 1], f2(y0, y1));
    h[i] = pack_h2(y0, y1);
  }
}

// S of a tile's row in tensor memory less its reference where that is kLarge or more.  Below, (S - m) scale
// is S scale - m scale, fused, with the second product rounded: off by 2^-24 of it, 2^-12 at most, the same for a whole
// row; where scores are in the millions it would be powers of two, and P outside of fp16.  (The difference first for all:
// a prompt of 4096 255 us, not 246.)
__device__ __noinline__ void subtract(uint32_t s, float ref) {
#pragma unroll 1
  for (int c = 0; c < kTok; c += 32) {
    float x[32];
    tmem_ld32(s + c, x);
    tmem_wait_ld(x);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] -= ref;
    tmem_st32(s + c, x);
  }
  tmem_wait_st();
}

// S of this lane's row in tensor memory at `s` -> P at the same columns, O
// (at `o`, D columns) scaled where the reference moves.  Tokens a .. e - 1 of
// the tile are seen, but for `bad` groups of 16.  S is read twice, in loops that
// are kept short: this serves a row tile's first and last token tiles, and code
// that runs seldom had better not push the rest out of the instruction cache.
// Returns whether the warp has a large reference.
template <int D>
RF4_DEV bool softmax_tile(uint32_t s, uint32_t o, Row& st, float scale_log2, bool first, bool used, int a, int e, uint32_t bad) {
  float x[32], top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kTok; c += 32) {
    tmem_ld32(s + c, x);
    const uint32_t keep = kept(c, a, e, bad);
    tmem_wait_ld(x);
    top = fmaxf(top, top_of<true>(x, keep));
  }
  if (first) {
    st.m = top;
  } else {
    const bool grow = used && (top - st.m) * scale_log2 > kGrow;
    if (__any_sync(0xffffffffu, grow)) {
      const float alpha = grow ? ex2((st.m - top) * scale_log2) : 1.f;
      if (grow) st.m = top;
      st.l *= alpha;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        tmem_ld32(o + c, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= alpha;
        tmem_st32(o + c, x);
      }
    }
  }
  float ref = st.m == -INFINITY ? 0.f : st.m;
  const bool mine = used && fabsf(ref) * scale_log2 >= kLarge, large = __any_sync(0xffffffffu, mine);
  if (large) {
    subtract(s, mine ? ref : 0.f);  // a row's results do not depend on its neighbours'
    if (mine) ref = 0.f;
  }
  const float lift = fmaf(-ref, scale_log2, kLift);
  const uint64_t scale2 = f2(scale_log2, scale_log2), lift2 = f2(lift, lift);
  uint64_t sum[2] = {0, 0};
#pragma unroll 1
  for (int c = 0; c < kTok; c += 32) {
    uint32_t h[16];
    tmem_ld32(s + c, x);
    const uint32_t keep = kept(c, a, e, bad);
    tmem_wait_ld(x);
    weights<true>(x, h, scale2, lift2, sum, keep);
    tmem_st16(s + c / 2, h);
  }
  float s0, s1;
  un2(add2(sum[0], sum[1]), s0, s1);
  st.l += s0 + s1;
  tmem_wait_st();
  return large;
}

// The same for a tile that is seen whole and is not the row's first, of a warp without large
// references: P by the
// reference as it stands, in one pass, with the maximum beside it; P waits in
// registers until that shows whether the reference holds, and where it does
// not (a maximum that has grown by more than 2^8, seldom) the tile is done again.
template <int D>
RF4_DEV bool softmax_next(uint32_t s, Row& st, float scale_log2, bool used) {
  const float ref = st.m == -INFINITY ? 0.f : st.m, lift = fmaf(-ref, scale_log2, kLift);
  const uint64_t scale2 = f2(scale_log2, scale_log2), lift2 = f2(lift, lift);
  uint64_t sum[2] = {0, 0};
  uint32_t h[4][16];
  float x[32], y[32];
  tmem_ld32(s, x);
  tmem_wait_ld(x);
  tmem_ld32(s + 32, y);
  float top = top_of<false>(x, 0);
  weights<false>(x, h[0], scale2, lift2, sum, 0);
  tmem_wait_ld(y);
  tmem_ld32(s + 64, x);
  top = fmaxf(top, top_of<false>(y, 0));
  weights<false>(y, h[1], scale2, lift2, sum, 0);
  tmem_wait_ld(x);
  tmem_ld32(s + 96, y);
  top = fmaxf(top, top_of<false>(x, 0));
  weights<false>(x, h[2], scale2, lift2, sum, 0);
  tmem_wait_ld(y);
  top = fmaxf(top, top_of<false>(y, 0));
  weights<false>(y, h[3], scale2, lift2, sum, 0);
  if (__any_sync(0xffffffffu, used && (top - st.m) * scale_log2 > kGrow)) {
    return false;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_st16(s + 16 * c, h[c]);
  float s0, s1;
  un2(add2(sum[0], sum[1]), s0, s1);
  st.l += s0 + s1;
  tmem_wait_st();
  return true;
}

// Position p of O's columns is value d_of(p) of the head.
RF4_DEV int d_of(int p) { return (p & ~31) + ((p & 31) >> 1) + ((p & 1) << 4); }

// Adds the parts of a row tile in order and writes its rows; 256 threads.  A
// thread deals with several places of O at a time, so that loads of many
// parts are on their way together.
template <int D, int ACT>
RF4_DEV void merge_parts(const Params& p, const Item& it, const float2* ml) {
  constexpr int U = 4, Q4 = D / 4;
  const int parts = (it.last - it.first + 1) << (it.wide ? 0 : 1), work = it.rows * Q4;
  const bool whole = it.first == it.last;
  // part n of row rr: of CTA first + n / chains; the first CTA's in its slot 1, the others' in slot 0, a whole row tile's in slot 2
  auto record = [&](int n, int rr) __attribute__((always_inline)) {
    const int c = it.wide ? n : n >> 1, ch = it.wide ? rr / kHalf : n & 1;
    const int slot = whole ? 2 : c == 0 ? 1 : 0;
    return (((it.first + c) * kSlots + slot) * 2 + ch) * kHalf + rr % kHalf;
  };
  for (int i0 = threadIdx.x; i0 < work; i0 += U * 256) {
    int rr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) rr[u] = min(i0 + u * 256, work - 1) / Q4;
    float M[U];
#pragma unroll
    for (int u = 0; u < U; ++u) M[u] = -INFINITY;
#pragma unroll 2
    for (int n = 0; n < parts; ++n) {
#pragma unroll
      for (int u = 0; u < U; ++u) M[u] = fmaxf(M[u], __ldcg(&ml[record(n, rr[u])]).x);
    }
    float L[U];
    float4 O[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (M[u] == -INFINITY) M[u] = 0.f;
      L[u] = 0.f;
      O[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int n = 0; n < parts; ++n) {
      float2 v[U];
      float4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = record(n, rr[u]);
        v[u] = __ldcg(&ml[at]);
        x[u] = __ldcg(reinterpret_cast<const float4*>(p.ws + (size_t)at * D) + (i0 + u * 256) % Q4);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // a sum of zero: nothing seen, O may never have been written
        const float e = v[u].y == 0.f ? 0.f : ex2((v[u].x - M[u]) * p.scale_log2);
        L[u] += e * v[u].y;
        O[u].x += v[u].y == 0.f ? 0.f : e * x[u].x;
        O[u].y += v[u].y == 0.f ? 0.f : e * x[u].y;
        O[u].z += v[u].y == 0.f ? 0.f : e * x[u].z;
        O[u].w += v[u].y == 0.f ? 0.f : e * x[u].w;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * 256 >= work) break;
      const float inv = L[u] == 0.f ? 0.f : 1.f / L[u];
      const int row = it.r0 + rr[u], token = row / p.G, g = row - token * p.G;
      uint16_t* out = p.out + ((int64_t)(it.s.row0 + token) * p.H + (int64_t)it.hk * p.G + g) * D + d_of(4 * ((i0 + u * 256) % Q4));
      *reinterpret_cast<uint32_t*>(out) = pack_act(O[u].x * inv, O[u].z * inv, ACT);
      *reinterpret_cast<uint32_t*>(out + 16) = pack_act(O[u].y * inv, O[u].w * inv, ACT);
    }
  }
}

// Items in the order in which the scheduling warp wrote them; all lanes of a
// warp.  An item is read where it lies, until the warp is done with it.
struct Items {
  uint32_t n = 0;
  // The item `ahead` of the next one to be done with, or nullptr behind the last.
  RF4_DEV const Item* get(const Control& ctl, Waits& wait, uint32_t ahead = 0) {
    const uint32_t i = n + ahead;
    wait.warp(&ctl.item_full[i % kItems], (i / kItems) & 1u);
    const Item* it = &ctl.items[i % kItems];
    return wait.ok && it->rows > 0 ? it : nullptr;
  }
  RF4_DEV void done(Control& ctl) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&ctl.item_empty[n % kItems]));
    ++n;
  }
};

// Bulk copies of raw rows, K's and V's tiles in turn; one warp.  Lanes 0-7
// follow a group of 16 tokens each through the pages; the first of a run of
// groups that lie in one page copies the run.
template <int V, int D>
struct Loader {
  using F = Plan<V, D>;
  int stages;
  uint8_t* raw;
  Ring ring;
  int tile = 0;
  uint32_t issued = 0, stopped = 0;
  RF4_DEV Loader(int stages, uint8_t* raw) : stages(stages), raw(raw) {}

  RF4_DEV void item(const Params& p, Control& ctl, Waits& wait, const Item& it) {
    const int lane = threadIdx.x & 31, group = lane & 7, ps = p.c.page_size;
    int lo, hi, x;
    seen(p, it.s, it.r0 / p.G, lo, x);
    seen(p, it.s, (it.r0 + it.rows - 1) / p.G, x, hi);
    const int32_t* row = p.c.table + (int64_t)it.b * p.c.ldt;
    const int64_t head = (int64_t)it.hk * ps * F::RB, page_bytes = (int64_t)p.c.Hkv * ps * F::RB;
    int t0 = it.c0 * kTok, g0 = t0 + 16 * group, at = g0 / ps, off = g0 - at * ps;
    const int step = kTok / ps, rest = kTok - step * ps;
    auto look_up = [&](int g) __attribute__((always_inline)) { return lane < 8 && g < hi && g + 16 > lo ? row[at] : -1; };
    int page = look_up(g0);
    for (int j = 0; j < it.tiles; ++j, ++tile, t0 += kTok) {
      const bool want = lane < 8 && g0 < hi && g0 + 16 > lo, have = want && page >= 0 && page < p.c.num_pages;
      const int64_t src = head + page * page_bytes + (int64_t)off * F::RB;
      const uint32_t bad = __ballot_sync(0xffffffffu, want && !have), there = __ballot_sync(0xffffffffu, have);
      const bool lead = have && (lane == 0 || off == 0 || !(there >> (lane - 1) & 1u));
      const uint32_t leads = __ballot_sync(0xffffffffu, lead);
      const uint32_t run = __ffs((leads | ~there) >> (lane + 1 & 31)) * 16 * F::RB;
      // the next tile's page, on its way meanwhile
      g0 += kTok;
      at += step;
      off += rest;
      if (off >= ps) off -= ps, ++at;
      page = j + 1 < it.tiles ? look_up(g0) : -1;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        wait.warp(&ctl.raw_empty[ring.stage], ring.phase ^ 1u);
        if (!wait.ok) return;
        const uint32_t bar = smem_addr(&ctl.raw_full[ring.stage]);
        if (lane == 0) {
          if (which == 0) {
            ctl.tiles[tile % kTiles] = Tile{max((lo & ~15) - t0, 0), hi - t0, bad, 0};
            if (bad) atomicOr(p.c.err, kErrBadPage);
          }
          mbar_arrive_expect_tx(bar, (uint32_t)__popc(there) * 16u * F::RB);
        }
        __syncwarp();
        if (lead) bulk_g2s(smem_addr(raw + ring.stage * F::RAW + group * 16 * F::RB), (which ? p.c.V : p.c.K) + src, run, bar);
        ring.next(stages);
        ++issued;
      }
    }
  }

  // No more tiles.  (The stage that this takes is empty, and its barrier goes on by a phase.)
  RF4_DEV void stop(Control& ctl, Waits& wait) {
    wait.warp(&ctl.raw_empty[ring.stage], ring.phase ^ 1u);
    if (!wait.ok) return;
    if ((threadIdx.x & 31) == 0) {
      ctl.tiles[tile % kTiles] = Tile{0, 0, 0, 1};
      mbar_arrive(smem_addr(&ctl.raw_full[ring.stage]));
    }
    stopped = 1;
  }

  // What a block that gave up waits for at its end.
  RF4_DEV void leave(Control& ctl) const {
    if ((threadIdx.x & 31) != 0) return;
    ctl.copies = issued;
    ctl.first = issued + stopped > (uint32_t)stages ? issued + stopped - stages : 0;
  }
};

// Up to 128 rows of q into a swizzled tile, each 32-value block in the order (j, j + 16); 128 threads.
template <int D>
__device__ __noinline__ void load_q(const Params& p, const Item& it, int half, uint8_t* tile, int tid) {
  constexpr int NB = D / 32, PANEL = kTok * 128, PASS = 128 / NB;  // rows a pass
  const int rows = min(it.rows - half * kHalf, kHalf), kb = tid % NB;
  int rr = tid / NB;
#pragma unroll 1
  for (int pass = 0; pass < kHalf / PASS; pass += 2) {
    uint4 x[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = rr + u * PASS;
      if (r < rows) {
        const int row = it.r0 + half * kHalf + r, token = row / p.G, g = row - token * p.G;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(it.s.row0 + token) * p.ldq + ((int64_t)it.hk * p.G + g) * D + kb * 32);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[u][c] = src[c];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = rr + u * PASS;
      if (r < rows) {
        uint8_t* dst = tile + kb / 2 * PANEL + r * 128;
        // values 0-7 with 16-23, and 8-15 with 24-31
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 a = x[u][h], b = x[u][h + 2];
          const int chunk = (kb & 1) * 4 + 2 * h;
          *reinterpret_cast<uint4*>(dst + ((chunk ^ (r & 7)) << 4)) =
              make_uint4(__byte_perm(a.x, b.x, 0x5410), __byte_perm(a.x, b.x, 0x7632), __byte_perm(a.y, b.y, 0x5410), __byte_perm(a.y, b.y, 0x7632));
          *reinterpret_cast<uint4*>(dst + (((chunk + 1) ^ (r & 7)) << 4)) =
              make_uint4(__byte_perm(a.z, b.z, 0x5410), __byte_perm(a.z, b.z, 0x7632), __byte_perm(a.w, b.w, 0x5410), __byte_perm(a.w, b.w, 0x7632));
        }
      }
    }
    rr += 2 * PASS;
    if (rr >= rows) break;
  }
}

template <int V, int D, int ACT>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_kernel(const __grid_constant__ Params p) {
  using F = Plan<V, D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Control& ctl = *reinterpret_cast<Control*>(smem + F::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x < kBars) {
    const int i = threadIdx.x;
    const uint32_t arrivals = i < 4 ? 4 : i < 8 ? 2 : i < 16 ? 1 : i < 20 ? 4 : i < 20 + kMaxRaw ? 1 : i < 20 + 2 * kMaxRaw ? 4 : i < 20 + 2 * kMaxRaw + kItems ? 1 : 8 + 2;
    mbar_init(smem_addr(reinterpret_cast<uint64_t*>(&ctl) + i), arrivals);
    fence_mbar_init();
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&ctl.tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  grid_dependency_wait();  // lengths, tables and everything else may be the preceding kernel's output
  bool any_wide;
  const bool busy = find_work<Shape, kThreads>(p, ctl.work, any_wide);
  __syncthreads();
  tc_fence_after();
  if (!busy) {
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(ctl.tmem), "r"(512));
    return;
  }
  const uint32_t tmem = ctl.tmem;
  // columns: S (and P) of chain t at 128 t, O at 256 + D t
  const int raw_stages = any_wide ? F::RSTAGES : F::RSTAGES_NARROW;
  uint8_t* raw = smem + (any_wide ? F::OFF_RAW : F::OFF_Q1);
  Waits wait;

  if (warp < 8) {
    // ---- softmax and output ----
    take_registers<kSoftmaxRegs>();
    const int t = warp >> 2, r = threadIdx.x & (kHalf - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + 128u * t, o_at = tmem + lanes + 256u + (uint32_t)D * t;
    uint32_t n_s = 0, n_o = 0;  // uses of s_full and o_full
    Items items;
    // Chain t's half of a row tile's queries; a narrow tile's one half is chain 0's to bring.
    auto bring_q = [&](const Item& of) __attribute__((always_inline)) {
      if (t == 1 && !of.wide) return;
      load_q<D>(p, of, t, smem + (t ? F::OFF_Q1 : F::OFF_Q0), r);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.q_full[t]));
    };
    const Item* at = items.get(ctl, wait);
    if (at) bring_q(*at);
    for (const Item* nx; at; at = nx, items.done(ctl)) {
      const Item& it = *at;
      const int wide = it.wide, tiles = it.tiles, tile0 = it.tile, c0 = it.c0;
      const bool whole = it.first == it.last;
      const int row = it.r0 + (wide ? t * kHalf : 0) + r;
      const bool used = row < it.r0 + it.rows, idle = row - lane >= it.r0 + it.rows;  // idle: none of the warp's rows is used
      int lo = 0, hi = 0;
      if (used) seen(p, it.s, row / p.G, lo, hi);
      Row st;
      bool first = true, large = false;
      for (int j = wide ? 0 : t; j < tiles; j += wide ? 1 : 2) {
        const int t0 = (c0 + j) * kTok;
        const int a = max(lo - t0, 0), e = min(max(hi - t0, 0), kTok);
        wait.warp(&ctl.s_full[t], n_s++ & 1u);
        tc_fence_after();
        const uint32_t bad = ctl.tiles[(tile0 + j) % kTiles].bad;
        const bool part = __any_sync(0xffffffffu, used && (a > 0 || e < kTok)) || bad;
        // (P of rows that nobody reads may be anything)
        if (!idle && (part || first || large || !softmax_next<D>(s_at, st, p.scale_log2, used)))
          large = softmax_tile<D>(s_at, o_at, st, p.scale_log2, first, used, a, e, bad);
        first = false;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ctl.p_full[t]));
      }
      // The last scores are there, so this chain's products are done with its
      // queries: the next row tile's take their place while the output of this
      // one is dealt with.  A narrow tile's queries are the other chain's as
      // well, whose end the synchronisation below tells.
      nx = items.get(ctl, wait, 1);
      if (nx && wide) bring_q(*nx);
      if (!first) {
        wait.warp(&ctl.o_full[t], n_o++ & 1u);
        tc_fence_after();
      }
      if (wide && whole) {
        // the whole of this row is here
        const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
        const int token = row / p.G, g = row - token * p.G;
        uint16_t* out = p.out + ((int64_t)(it.s.row0 + token) * p.H + (int64_t)it.hk * p.G + g) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float x[32];
          tmem_ld32(o_at + c, x);
          tmem_wait_ld(x);
          if (used) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = pack_act(x[4 * i + h] * inv, x[4 * i + 2 + h] * inv, ACT);
              uint4* o4 = reinterpret_cast<uint4*>(out + c + 16 * h);
              o4[0] = make_uint4(w[0], w[1], w[2], w[3]);
              o4[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
        tc_fence_before();
        continue;
      }
      // a part: into the workspace
      float2* ml = reinterpret_cast<float2*>(p.ws + (size_t)gridDim.x * kSlots * 2 * kHalf * D);
      const size_t mine = (((size_t)blockIdx.x * kSlots + it.slot) * 2 + t) * kHalf + r;
      if (used) __stcg(&ml[mine], make_float2(st.m, st.l));
      if (!first) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float x[32];
          tmem_ld32(o_at + c, x);
          tmem_wait_ld(x);
          if (used) {
            float4* w = reinterpret_cast<float4*>(p.ws + mine * D + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) __stcg(w + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
          }
        }
        tc_fence_before();
      }
      __threadfence();
      chains_meet(false);
      bool merge = true;
      if (!whole) {
        if (threadIdx.x == 0) {
          const uint32_t n = atomic_add_acq_rel_gpu(&p.cnt[it.first], 1u);
          ctl.last = n == (uint32_t)(it.last - it.first);
          if (ctl.last) store_relaxed_gpu(&p.cnt[it.first], 0u);
        }
        chains_meet(false);
        merge = ctl.last;
        if (merge) __threadfence();
      }
      if (merge) {
        merge_parts<D, ACT>(p, it, ml);
      }
      chains_meet(false);  // the records and ctl.last may be written again
      if (nx && !wide) bring_q(*nx);
    }
    while (!chains_meet(true)) {
    }
  } else if (warp < 12) {
    // ---- decode ----
    give_registers<kOtherRegs>();
    const int row = threadIdx.x & (kTok - 1);
    Ring ring, kv;
    for (uint32_t n = 0;; ++n, kv.next(F::STAGES)) {
      bool real = false;
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        wait.warp(&ctl.raw_full[ring.stage], ring.phase);
        if (!wait.ok) break;
        if (which == 0) {
          const Tile tile = ctl.tiles[n % kTiles];
          if (tile.stop) break;
          real = row >= tile.from && row < tile.to && !(tile.bad >> (row >> 4) & 1u);
        }
        wait.warp(which ? &ctl.v_empty[kv.stage] : &ctl.k_empty[kv.stage], kv.phase ^ 1u);
        if (!wait.ok) break;
        const uint8_t* src = raw + ring.stage * F::RAW;
        uint8_t* dst = smem + (which ? F::OFF_V : F::OFF_K) + kv.stage * F::TILE;
        if (ACT == 1 && which == 0)
          decode_row<V, D, true>(src, dst, row, real);
        else
          decode_row<V, D, false>(src, dst, row, real);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&ctl.raw_empty[ring.stage]));
          mbar_arrive(smem_addr(which ? &ctl.v_full[kv.stage] : &ctl.k_full[kv.stage]));
        }
        ring.next(raw_stages);
      }
      if (!wait.ok || ctl.tiles[n % kTiles].stop) break;
    }
  } else {
    give_registers<kOtherRegs>();
    if (warp < 14) {
      // ---- MMA issue ----
      // The whole warp walks along, one elected lane issues: what the
      // instructions take is then uniform and stays in uniform registers.  A
      // chain's products are issued by one warp, so that they run in order: S of
      // its next token tile comes after the product that reads P in its place.
      constexpr uint32_t id_s = instr_desc(ACT, kTok, 0), id_o = instr_desc(0, D, 1);
      constexpr uint32_t desc_hi = (1024u >> 4) | 1u << 14 | 2u << 29;
      const uint32_t t = warp == 13;
      const uint32_t q_lo = (smem_addr(smem + F::OFF_Q0) >> 4) | 1u << 16, k_lo = (smem_addr(smem + F::OFF_K) >> 4) | 1u << 16;
      const uint32_t v_lo = (smem_addr(smem + F::OFF_V) >> 4) | (uint32_t)(F::PANEL >> 4) << 16;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t s_at = tm + 128u * t, o_at = tm + 256u + (uint32_t)D * t;
      Ring kr, vr;
      uint32_t n_q0 = 0, n_q1 = 0, n_p = 0, n_turn = 0;
      Items items;
      while (const Item* it = items.get(ctl, wait)) {
        const uint32_t wide = __shfl_sync(0xffffffffu, it->wide, 0);
        const int tiles = __shfl_sync(0xffffffffu, it->tiles, 0);
        items.done(ctl);
        int kj = 0, vj = 0;
        // Goes on to this chain's next tile of K (or V) and waits for it; the other chain's tiles are let go.
        auto next_own = [&](Ring& r, int& j, uint64_t* full, uint64_t* empty) __attribute__((always_inline)) {
          for (; j < tiles; ++j) {
            wait.warp(&full[r.stage], r.phase);
            if (wide || (j & 1) == (int)t) return true;
            if (lane == 0) mbar_arrive(smem_addr(&empty[r.stage]));
            r.next(F::STAGES);
          }
          return false;
        };
        auto scores = [&]() __attribute__((always_inline)) {
          tc_fence_after();
          const uint32_t a = q_lo + (wide & t) * (F::TILE >> 4), b = k_lo + kr.stage * (F::TILE >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k / 4) * (F::PANEL >> 4) + (k % 4) * 2;
              mma_ss(s_at, a + off, b + off, desc_hi, id_s, k != 0);
            }
            mma_commit(smem_addr(&ctl.s_full[t]));
            mma_commit(smem_addr(&ctl.k_empty[kr.stage]));
          }
          __syncwarp();
          ++kj;
          kr.next(F::STAGES);
        };
        // The chains take turns at the tensor core, product and next scores in
        // one go: left to themselves they fall into step, both at their softmax
        // and then both at half the core's rate (4.8k cycles a token tile).
        bool have = false;  // scores of a tile are on their way, or P of it
        uint32_t again = 0;  // O holds something already
#pragma unroll 1
        for (;;) {
          // K's and V's next tiles are there before P, mostly: only that wait counts
          // (V's first, for a tile of the other chain's to be let go that K's may wait for)
          if (have) next_own(vr, vj, ctl.v_full, ctl.v_empty);
          const bool more = next_own(kr, kj, ctl.k_full, ctl.k_empty);
          if (!have) {
            // A chain waits for the queries that it reads, and for no others, whose barrier may be two phases ahead: the
            // other half's, or those of a narrow row tile's only token tile.  Phases left out here are over before this
            // chain's next look at the barrier: its turn comes only after the other chain has waited for them.
            const uint32_t half = wide & t;
            if (more) wait.warp(&ctl.q_full[half], (half ? n_q1 : n_q0) & 1u);
            ++n_q0;
            n_q1 += wide;
          } else {
            wait.warp(&ctl.turn[t], (n_turn++ & 1u) ^ (t ^ 1u));
            wait.warp(&ctl.p_full[t], n_p++ & 1u);
            tc_fence_after();
            const uint32_t b = v_lo + vr.stage * (F::TILE >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kTok / 16; ++k) mma_ts(o_at, s_at + 8u * k, b + k * (2048 >> 4), desc_hi, id_o, again | (k != 0));
              mma_commit(smem_addr(&ctl.v_empty[vr.stage]));
              if (!more) mma_commit(smem_addr(&ctl.o_full[t]));
            }
            __syncwarp();
            again = 1;
            ++vj;
            vr.next(F::STAGES);
          }
          if (more) scores();
          if (have && lane == 0) mbar_arrive(smem_addr(&ctl.turn[t ^ 1]));
          if (!more) break;
          have = true;
        }
        if (t == 1 && !wide && (tiles & 1)) {  // an odd tile, the other chain's
          wait.warp(&ctl.turn[1], n_turn++ & 1u);
          if (lane == 0) mbar_arrive(smem_addr(&ctl.turn[0]));
        }
        next_own(vr, vj, ctl.v_full, ctl.v_empty);  // the other chain's last tile, perhaps
      }
    } else if (warp == 14) {
      // ---- row tiles, raw rows ----
      Walk<Shape> walk(p, ctl.work);
      Loader<V, D> load(raw_stages, raw);
      uint32_t n = 0;
      Item it;
      for (bool more = true; more && wait.ok; ++n) {
        more = walk.next(p, it);
        wait.warp(&ctl.item_empty[n % kItems], ((n / kItems) & 1u) ^ 1u);
        if (!wait.ok) break;
        if (!more) it.rows = 0;
        it.tile = load.tile;
        if (lane == 0) {
          ctl.items[n % kItems] = it;
          mbar_arrive(smem_addr(&ctl.item_full[n % kItems]));
          if (more && it.s.over) atomicOr(p.c.err, kErrBadPage);
        }
        if (more) load.item(p, ctl, wait, it);
        else load.stop(ctl, wait);
      }
      load.leave(ctl);
    }
  }
  tc_fence_before();
  if (__syncthreads_or(!wait.ok)) {
    // Some warp gave up.  Copies land and products end before the block does, by waits of their own.
    if (threadIdx.x == 0) atomicOr(p.c.err, kErrWaitTimeout);
    if (warp == 12 || warp == 13) {
      const uint32_t bar = smem_addr(&ctl.drained[warp - 12]);
      if (elect_one()) {
        mma_commit(bar);
        (void)mbar_wait_bounded(bar, 0);
      }
    } else if (warp == 14) {
      for (uint32_t i = ctl.first; i < ctl.copies; ++i) (void)mbar_wait_bounded(smem_addr(&ctl.raw_full[i % raw_stages]), i / raw_stages & 1u);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

using Fn = void (*)(Params);
template <int V, int D>
Fn kernel_for(int act) {
  return act == 0 ? paged_attention_kernel<V, D, 0> : paged_attention_kernel<V, D, 1>;
}
Fn kernel_for(int variant, int D, int act) {
  if (variant == 0) return D == 64 ? kernel_for<0, 64>(act) : kernel_for<0, 128>(act);
  return D == 64 ? kernel_for<1, 64>(act) : kernel_for<1, 128>(act);
}
int smem_for(int variant, int D) {
  if (variant == 0) return D == 64 ? Plan<0, 64>::SMEM : Plan<0, 128>::SMEM;
  return D == 64 ? Plan<1, 64>::SMEM : Plan<1, 128>::SMEM;
}

}  // namespace

size_t paged_attn_ws_floats(int sms) { return (size_t)sms * kSlots * 2 * kHalf * (128 + 2); }

cudaError_t paged_attn_prepare() {
  for (int v = 0; v < 2; ++v)
    for (int D : {64, 128})
      for (int act = 0; act < 2; ++act) {
        cudaError_t e = cudaFuncSetAttribute((const void*)kernel_for(v, D, act), cudaFuncAttributeMaxDynamicSharedMemorySize, smem_for(v, D));
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_paged_attention(int variant, int act, const PagedAttnArgs& a, int sms, cudaStream_t s) {
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
  cfg.gridDim = dim3((unsigned)sms);
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
