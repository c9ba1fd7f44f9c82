// Integer rules of the 8-bit paged cache, for the kernels and for host code alike (no CUDA needed).
#pragma once

#include <limits.h>

#include "lowram.h"

#ifdef __CUDACC__
#define LR_HD __host__ __device__ __forceinline__
#else
#define LR_HD inline
#endif

namespace lr {
namespace kv8 {

constexpr int kPage = LR_BLOCK_TOKENS;  // tokens of a page

// A number of the caller's, constant during the kernel.
LR_HD int input(const int* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}
template <class T>
LR_HD T least(T x, T y) { return y < x ? y : x; }
template <class T>
LR_HD T most(T x, T y) { return x < y ? y : x; }

// ------------------------------------------------------------------ append

// Sequence b's pages are the units from cu[b] / 64 + 2 b on: always enough of them (n tokens touch
// at most n / 64 + 2 pages), without a scan over the batch.
template <class Args>
LR_HD int unit_of(const Args& a, int b) { return input(a.cu + b) / kPage + 2 * b; }
template <class Args>
LR_HD int n_units(const Args& a) { return a.n_tokens / kPage + 2 * a.B; }
// The sequence that unit u is of: the largest b with unit_of(b) <= u.
template <class Args>
LR_HD int sequence_of_unit(const Args& a, int u) {
  int b = 0, len = a.B;
  while (len > 1) {
    const int half = len / 2;
    if (unit_of(a, b + half) <= u) {
      b += half;
      len -= half;
    } else {
      len = half;
    }
  }
  return b;
}

// CTAs that share a page's heads, each of `threads`. Up to 8 fill the machine evenly to the end, but each finds the
// page's angles again. With more pages than SMs a share therefore has eight query heads at least. Of 32 + 8 heads of
// 128 bf16 numbers, 8 shares and 4: 32K tokens 122 and 127 us by themselves, 132 and 133 in a long run; 24 ragged
// sequences 76 and 74; 200 tokens each of 128 sequences 112 and 108. Of 8 + 8 heads, 8, 2 and one: 88, 70 and 68.
// With under half a page of tokens for a sequence a share's beginning weighs more, and there are no more CTAs with
// something to do than run at once and a third: 64 registers leave an SM 1024 threads, and a sequence touches one page
// or two. The third was fitted; of 8, 4, 2 shares and one the best or within 4 % of it for 16 to 512 sequences of 2 to
// 31 tokens and 2, 4, 6 or 8 KV heads, in bf16 with head_dim 64, 128 and 256 and in fp32 with 64 and 128; with 5
// or 7 heads up to 1.3 times the best. 4 tokens each of 64 sequences 12.8, 9.9,
// 11.6 and 17.7 us (it takes 4), 31 tokens 18.0, 15.6, 20.6 and 28.6 (4), fp32 32.7, 30.5, 50.9 and 56.4 (4), 4
// tokens each of 256 sequences 40.6, 30.4, 25.6 and 23.1 (one).
template <class Args>
LR_HD int append_shares(const Args& a, int threads, int sm_count) {
  int ny = least(a.Hkv, 8);
  if (a.n_tokens < (long long)kPage / 2 * a.B) {
    const long long pages = a.B + a.n_tokens / kPage, at_once = (long long)sm_count * (1024 / threads);
    while (ny > 1 && 3 * pages * ny > 4 * at_once) ny = ny > 4 ? 4 : ny > 2 ? 2 : 1;
  } else if (n_units(a) > sm_count) {
    ny = most(1, least(ny, a.Hq / 8));
  }
  return ny;
}

// The positions [first, end) of a page of a sequence that receive new tokens.
struct PageRows {
  int page;  // index in the sequence
  int first, end;
};
// Page i, counted from 0, of those that n new tokens from position p0 on go to; false behind the last one. A
// sequence may end at the last page boundary that an int holds: page indices are compared, and no position behind
// the sequence is formed.
LR_HD bool page_rows(int p0, int n, int i, PageRows& r) {
  if (n < 1 || i < 0) return false;
  const int page0 = p0 / kPage, last = (p0 + n - 1) / kPage;
  if (i > last - page0) return false;
  r.page = page0 + i;
  r.first = i == 0 ? p0 : r.page * kPage;
  r.end = r.page == last ? p0 + n : (r.page + 1) * kPage;
  return true;
}

// ------------------------------------------------------------------ attention: the division of work
//
// A segment is one (sequence, KV head); its tokens are cut into tiles of two pages. The segments, in
// the order of (sequence, head), are laid out on a line of units, one for each tile and kSegmentUnits at
// the end for what a segment costs by itself, and the line is divided evenly among the CTAs: CTA c
// takes units [c W / C, (c + 1) W / C), so ragged lengths cost nothing and one long sequence
// fills the machine. A CTA's range touches at most two segments that others share: its first
// and its last one. What it has of those are pieces (unnormalised sums with their maximum) in the
// slots 2c and 2c + 1; a second kernel joins a segment's pieces in the order of the CTAs, which it finds
// written down: CTA c does so for the segment that its range is the first to start inside of. (Joined by
// the last CTA to finish instead, one of them was busy for 5 us with 8 pieces and 20 us with 37, its
// own tiles waiting; with the division worked out again in the second kernel, that one took 6 us.)

constexpr int kTilePages = 2;
constexpr int kTileTokens = kTilePages * kPage;
constexpr int kSegmentUnits = 2;

struct Span {
  int lo, n;        // tokens [lo, n) are attended
  int page0;        // page (index in the sequence) of the first tile
  int tiles;        // tiles of one head
  int units;        // its stretch of the line
};

template <class Args>
LR_HD Span span_of(const Args& a, int len) {
  Span s;
  s.n = least(most(len, 0), a.max_pages * kPage);
  s.lo = a.window > 0 ? most(0, s.n - a.window) : 0;
  s.page0 = s.lo / kPage;
  s.tiles = s.n == 0 ? 0 : ((s.n + kPage - 1) / kPage - s.page0 + kTilePages - 1) / kTilePages;
  s.units = s.n == 0 ? 0 : s.tiles + kSegmentUnits;
  return s;
}
template <class Args>
LR_HD Span seq_span(const Args& a, int b) { return span_of(a, input(a.lens + b)); }

// First unit of CTA c's range.
LR_HD long long range_begin(long long total, int c, int active) {
  if (total <= INT_MAX / 2048) return (unsigned)total * (unsigned)c / (unsigned)active;  // active <= 1024: no 64-bit division
  return total * c / active;
}

// A CTA's range of units and where it starts.
struct Work {
  long long begin, end;
  long long total;       // of the whole batch
  int active;            // CTAs that have a range
  int b;                 // sequence of the first unit
  long long b_first;     // first unit of that sequence
  bool bad_len;          // this thread has seen a length out of bounds
  int pieces;            // small calls: CTAs of the cluster that have tiles
};

// Small calls are one launch: a cluster for every segment, which joins it itself, if that gives no CTA more than
// four tiles (two with mma.sync). CTAs of a segment's cluster, 0 for a call that is not small. The rule goes by the page
// table's width: the lengths are on the device. 8 KV heads, bf16: 1000 tokens 7.4 us and 7.9 from Python, with the second
// kernel 9.0 and 9.7; 4000 tokens 9.8 and 9.9. fp32: 2000 tokens 10.3 and 10.2, 4000 tokens 13.4 and 11.4.
constexpr int kSmallCtas = 256;  // clusters of 8 find room for all of them at once
LR_HD int small_cluster(int batch, int n_kv_heads, int max_pages, bool tensor) {
  const long long segments = (long long)batch * n_kv_heads, tiles = (max_pages + 1) / kTilePages;
  if (segments < 1 || segments > kSmallCtas) return 0;
  int c = 8;
  while (c > 1 && (segments * c > kSmallCtas || c / 2 >= tiles)) c /= 2;
  return tiles <= (tensor ? 4 : 2) * c ? c : 0;
}

// Small calls: a cluster has a segment to itself, its CTAs the tiles in order, as many each as they take. The line
// is that of the segment's sequence.
template <class Args>
LR_HD Work small_work(const Args& a, int cta) {
  const int seg = cta / a.cluster, rank = cta % a.cluster;
  Work wk{};
  wk.b = seg / a.Hkv;
  const Span sp = seq_span(a, wk.b);
  if (sp.tiles == 0) return wk;
  const int per = (sp.tiles + a.cluster - 1) / a.cluster, first = seg % a.Hkv * sp.units;
  wk.pieces = (sp.tiles + per - 1) / per;
  wk.begin = first + least(rank * per, sp.tiles);
  wk.end = first + least((rank + 1) * per, sp.tiles);
  return wk;
}

// The CTA whose range holds unit t, for total units over `active` CTAs: largest c with
// c * total / active <= t.
LR_HD int cta_of_unit(long long t, long long total, int active) {
  if (total <= INT_MAX / 2048) return (int)(((unsigned)(t + 1) * (unsigned)active - 1) / (unsigned)total);
  return (int)(((t + 1) * active - 1) / total);
}

// A place on the line that moves forward. It stays inside the batch even if somebody changes the lengths under the
// kernel (a caller's mistake: then the result is garbage, and nothing else).
struct Place {
  int b, h;
  Span sp;
  long long b_first, seg_first;  // first unit of the sequence, of the segment
  int tile;                      // >= sp.tiles in a segment's last units

  template <class Args>
  LR_HD void start(const Args& a, const Work& wk) {
    b = wk.b;
    b_first = wk.b_first;
    sp = seq_span(a, b);
  }
  template <class Args>
  LR_HD void seek(const Args& a, long long unit) {
    while (unit >= b_first + (long long)sp.units * a.Hkv && b + 1 < a.B) {
      b_first += (long long)sp.units * a.Hkv;
      sp = seq_span(a, ++b);
    }
    const long long in = unit - b_first;
    const int units = most(1, sp.units);
    h = least(in <= INT_MAX ? (int)in / units : (int)least(in / units, (long long)INT_MAX), a.Hkv - 1);
    seg_first = b_first + (long long)h * sp.units;
    tile = (int)(unit - seg_first);
  }
};

// Walks the segments of a CTA's range in order.
template <class Args>
struct Walk : Place {
  const Args& a;
  Work wk;
  long long at;       // next unit
  int tile0, tile1;   // the range's tiles of the current segment

  LR_HD Walk(const Args& a_, const Work& w) : a(a_), wk(w), at(w.begin) {
    if (at < wk.end) start(a, wk);
  }
  // Moves to the next segment with tiles in the range; false at its end.
  LR_HD bool next() {
    while (at < wk.end) {
      seek(a, at);
      at = most(at + 1, seg_first + sp.units);
      tile0 = tile;
      tile1 = (int)least((long long)sp.tiles, wk.end - seg_first);
      if (tile0 < tile1) return true;
    }
    return false;
  }
  LR_HD bool whole() const { return tile0 == 0 && tile1 == sp.tiles; }
};

// The slot of CTA c's piece of a segment.
LR_HD int piece_slot(const Work& wk, int c, long long seg_first) {
  return 2 * c + (wk.begin < seg_first ? 1 : 0);
}

// A split segment: b * Hkv + h, the CTAs that share it, and whether the first one's range starts before it (its
// piece is its second one then).
struct alignas(16) Pieces {
  int head, n, c0, mid;
  LR_HD int slot(int i) const { return 2 * (c0 + i) + (i == 0 && mid ? 1 : 0); }
};

// The segment that CTA c's range is the first to start inside of, or none (n = 0).
template <class Args>
LR_HD Pieces pieces_of(const Args& a, const Work& wk, int c) {
  Pieces p{0, 0, 0, 0};
  if (wk.begin < wk.end && c > 0) {
    Place at;
    at.start(a, wk);
    at.seek(a, wk.begin);
    if (at.tile > 0 && at.tile < at.sp.tiles && range_begin(wk.total, c - 1, wk.active) <= at.seg_first) {
      p.head = at.b * a.Hkv + at.h;
      p.c0 = cta_of_unit(at.seg_first, wk.total, wk.active);
      p.n = cta_of_unit(at.seg_first + at.sp.tiles - 1, wk.total, wk.active) - p.c0 + 1;
      p.mid = range_begin(wk.total, p.c0, wk.active) < at.seg_first;
    }
  }
  return p;
}

}  // namespace kv8
}  // namespace lr
