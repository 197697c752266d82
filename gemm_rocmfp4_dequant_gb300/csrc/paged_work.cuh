// How the attention over a paged cache is cut into work for CTAs, by the
// lengths on the device.
//
// The G query heads of a KV head share its tokens, so the (row, head) pairs of
// a sequence and a KV head are the rows of one matrix, token-major: row r is row
// r / G of the sequence's chunk, head r % G.  They are cut into row tiles, a row
// tile's tokens into token tiles.  All token tiles are numbered in one row
// (sequence, KV head, row tile, token tile) and every CTA takes an equal stretch
// of it.  A row tile that falls to several CTAs leaves parts in a workspace; the
// CTA that arrives last adds them in order.  Nothing waits for another CTA.
#pragma once
#include "common.cuh"
#include "paged.h"

namespace rocmfp4 {

// What the work's shape depends on.
struct Batch {
  PagedArgs c;
  int M, G, causal, window;  // rows of the call; query heads of a KV head
};

struct Seq {
  int row0, n;  // rows of the call
  int at;       // token that the first of them is, counted from the sequence's last row, which may lie behind the call's
  int lim;      // tokens that the table has room for
  bool over;    // whether the sequence has more
};

// A row tile's share of this CTA.
struct Item {
  int b, hk, r0, rows, wide;  // wide: a token tile of it counts twice
  int c0, tiles;              // this CTA's token tiles
  Seq s;
  int first, last;  // CTAs that share the row tile
  int slot;         // of this CTA's part
  int tile;         // number of the first token tile among this CTA's
};

// Where a CTA's stretch of the work lies; in shared memory.
struct Stretch {
  long long start, end, total;  // of the CTA's stretch; of all work
  long long base;               // where its first row tile begins
  long long scan[32];
  int scan_items[32];
  int b, hk, k, ctas;  // that row tile; CTAs that have work
};

RF4_DEV Seq sequence(const Batch& p, int b) {
  Seq s;
  const int r0 = min(max(p.c.cu[b], 0), p.M), r1 = min(max(p.c.cu[b + 1], 0), p.M);
  s.row0 = r0;
  s.n = max(r1 - r0, 0);
  const int len = max(p.c.lens[b], 0);
  s.at = len - max(max(p.c.cu[b + 1], 0) - r0, 0);
  const long long room = (long long)p.c.width * p.c.page_size;
  s.lim = (int)(len < room ? len : room);
  s.over = len > s.lim;
  return s;
}

// Tokens lo .. hi - 1 that row i of a sequence's chunk sees.
RF4_DEV void seen(const Batch& p, const Seq& s, int i, int& lo, int& hi) {
  lo = 0;
  hi = s.lim;
  if (p.causal) {
    const long long end = (long long)s.at + i + 1;
    hi = (int)(end < 0 ? 0 : end < s.lim ? end : s.lim);
    if (p.window > 0 && end > p.window) lo = (int)(end - p.window < hi ? end - p.window : hi);
  }
}

struct RowTile {
  int rows, weight;  // rows; work of one token tile
  int c0, tiles;     // first token tile, and how many (at least one)
  int fixed;         // work of a row tile whatever its length (queries, output), before that of its token tiles
  RF4_DEV long long all() const { return fixed + (long long)tiles * weight; }
};

// S: how a kernel cuts the work.  kRows and kTok: rows and tokens of a tile;
// kNarrow: rows up to which a token tile counts once, not twice; fixed(weight);
// kMinShare: token tiles that are worth a CTA.
template <class S>
RF4_DEV RowTile row_tile(const Batch& p, const Seq& s, int k) {
  RowTile t;
  const int r0 = k * S::kRows;
  t.rows = min(S::kRows, s.n * p.G - r0);
  t.weight = t.rows > S::kNarrow ? 2 : 1;
  t.fixed = S::fixed(t.weight);
  int lo, hi, x;
  seen(p, s, r0 / p.G, lo, x);
  seen(p, s, (r0 + t.rows - 1) / p.G, x, hi);
  t.c0 = lo / S::kTok;
  t.tiles = max(1, (hi + S::kTok - 1) / S::kTok - t.c0);
  return t;
}

// The row tiles of a CTA's stretch.
template <class S>
struct Walk {
  int b, hk, k, ctas;
  long long base, start, end, total;
  Seq s;  // of sequence b
  RF4_DEV Walk(const Batch& p, const Stretch& ctl)
      : b(ctl.b), hk(ctl.hk), k(ctl.k), ctas(ctl.ctas), base(ctl.base), start(ctl.start), end(ctl.end), total(ctl.total) {
    s = sequence(p, b);
  }
  RF4_DEV int owner(long long u) const {
    if (total < 1 << 22) return (int)(((uint32_t)(u + 1) * ctas - 1) / (uint32_t)total);
    return (int)(((u + 1) * ctas - 1) / total);
  }
  RF4_DEV bool next(const Batch& p, Item& it) {
    while (base < end) {
      const RowTile t = row_tile<S>(p, s, k);
      // token tiles whose places lie in start .. end - 1
      const long long at = base + t.fixed;
      const long long from = start - at + t.weight - 1, to = end - at + t.weight - 1;
      const int j0 = from <= 0 ? 0 : from >> (t.weight - 1) < t.tiles ? (int)(from >> (t.weight - 1)) : t.tiles;
      const int j1 = to <= 0 ? 0 : to >> (t.weight - 1) < t.tiles ? (int)(to >> (t.weight - 1)) : t.tiles;
      it.b = b;
      it.hk = hk;
      it.r0 = k * S::kRows;
      it.rows = t.rows;
      it.wide = t.weight - 1;
      it.c0 = t.c0 + j0;
      it.tiles = j1 - j0;
      it.s = s;
      it.first = it.last = blockIdx.x;
      it.slot = 2;
      if (j0 > 0 || j1 < t.tiles) {
        it.first = owner(at);
        it.last = owner(at + (long long)(t.tiles - 1) * t.weight);
        it.slot = j0 > 0 ? 0 : 1;
      }
      base += t.all();
      if ((long long)(++k) * S::kRows >= (long long)s.n * p.G) {
        k = 0;
        if (++hk == p.c.Hkv) {
          hk = 0;
          do {
            if (++b >= p.c.B) {
              base = total;
              break;
            }
            s = sequence(p, b);
          } while (s.n == 0);
        }
      }
      if (j0 < j1) return true;
    }
    return false;
  }
};

struct Work {
  long long cost;
  int tiles;  // row tiles; negative: some is wide
};

// Work of sequence b for one KV head: row tiles lane, lane + step, ...
template <class S>
RF4_DEV Work work_of(const Batch& p, int b, int lane, int step) {
  const Seq s = sequence(p, b);
  const int tiles = (s.n * p.G + S::kRows - 1) / (S::kRows);
  Work w{0, 0};
  bool wide = false;
  for (int k = lane; k < tiles; k += step) {
    const RowTile t = row_tile<S>(p, s, k);
    w.cost += t.all();
    ++w.tiles;
    wide |= t.weight > 1;
  }
  if (wide) w.tiles = -w.tiles;
  return w;
}

RF4_DEV long long divide(long long a, long long b) {
  if ((a | b) >> 31 == 0) return (uint32_t)a / (uint32_t)b;  // the short division
  return a / b;
}

// This CTA's stretch and where it begins; false if it has none.  `any`: whether
// some row tile of the call is wide.  All threads.
template <class S, int THREADS>
RF4_DEV bool find_work(const Batch& p, Stretch& ctl, bool& any) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.c.B;
  // few sequences: a warp each, its lanes over row tiles; many: a thread each, or several in a row
  const bool by_warp = B <= THREADS / 32;
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = by_warp ? min(warp, B) : min(tid * per, B), b1 = by_warp ? min(warp + 1, B) : min(b0 + per, B);
  long long mine = 0;
  int items = 0;
  bool wide = false;
  for (int b = b0; b < b1; ++b) {
    const Work w = work_of<S>(p, b, by_warp ? lane : 0, by_warp ? 32 : 1);
    mine += w.cost * p.c.Hkv;
    items += abs(w.tiles) * p.c.Hkv;
    wide |= w.tiles < 0;
  }
  if (by_warp) {
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane != 0) mine = 0;
  }
  long long before = mine;  // inclusive within the warp
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  items = __reduce_add_sync(0xffffffffu, items);
  if (lane == 31) {
    ctl.scan[warp] = before;
    ctl.scan_items[warp] = items;
  }
  const int any_wide = __syncthreads_or(wide);
  any = any_wide;
  long long total = 0, lower = 0;
  items = 0;
#pragma unroll 4
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) lower = total;
    total += ctl.scan[w];
    items += ctl.scan_items[w];
  }
  before += lower - mine;
  // A CTA for every row tile, or for every kMinShare token tiles where that
  // is more.  A wide token tile counts 2, and a CTA's stretch is never
  // shorter than one, so that every CTA between the first and the last of a
  // shared row tile has a part of it.
  long long most = total / S::kMinShare;
  most = most > items ? most : items;
  if (any_wide) most = most < total / 2 ? most : total / 2;
  if (most < 1) most = 1;
  const int ctas = (int)(most < (long long)gridDim.x ? most : (long long)gridDim.x);
  if (total == 0 || (int)blockIdx.x >= ctas) return false;
  const long long start = divide(total * blockIdx.x, ctas), end = divide(total * (blockIdx.x + 1), ctas);
  const uint32_t hit = __ballot_sync(0xffffffffu, start >= before && start < before + mine);
  if (hit) {  // one warp: the sequence of one of its lanes, then the row tile, 32 at a time
    int b = b0;
    long long base = before, w = mine;
    if (!by_warp)
      for (; b < b1; ++b) {
        w = work_of<S>(p, b, 0, 1).cost * p.c.Hkv;
        if (start < base + w) break;
        base += w;
      }
    const int from = __ffs(hit) - 1;
    b = __shfl_sync(0xffffffffu, b, from);
    base = __shfl_sync(0xffffffffu, base, from);
    w = __shfl_sync(0xffffffffu, w, from);
    const long long head = divide(w, p.c.Hkv);
    const int hk = (int)divide(start - base, head);
    base += hk * head;
    const Seq s = sequence(p, b);
    for (int k0 = 0;; k0 += 32) {
      const int k = k0 + lane;
      long long all = 0;
      if ((long long)k * S::kRows < (long long)s.n * p.G) {
        const RowTile t = row_tile<S>(p, s, k);
        all = t.all();
      }
      long long upto = all;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, start < base + upto);
      if (in) {
        if (lane == __ffs(in) - 1) {
          ctl.b = b;
          ctl.hk = hk;
          ctl.k = k;
          ctl.base = base + upto - all;
          ctl.start = start;
          ctl.end = end;
          ctl.total = total;
          ctl.ctas = ctas;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  __syncthreads();
  return true;
}

}  // namespace rocmfp4
