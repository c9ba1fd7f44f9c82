// Device helpers of the 8-bit paged cache: e4m3 conversions, and for the attention the division
// of the batch's tiles among CTAs and the joining of the pieces of a split segment.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "lr_common.cuh"
#include "lr_kv8.h"

namespace lr {
namespace kv8 {

// Two fp32 values to e4m3 codes (nearest even, saturating, NaN kept); lo in bits 0-7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The values of two e4m3 codes (exact in fp16).
__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ------------------------------------------------------------------ attention: the division of work
//
// A segment is one (sequence, KV head); its tokens are cut into tiles of two pages. The tiles
// of all segments, in the order of (sequence, head, page), are divided evenly among the CTAs: CTA c
// takes tiles [c W / C, (c + 1) W / C), so ragged lengths cost nothing and one long sequence
// fills the machine. A CTA's range touches at most two segments that others share: its first
// and its last one. What it has of those are pieces (unnormalised sums with their maximum) in the
// slots 2c and 2c + 1; the last CTA to finish a piece of a segment joins all of them in the
// order of the CTAs, so the result does not depend on which CTA that is.

constexpr int kTilePages = 2;
constexpr int kTileTokens = kTilePages * kBlock;

struct Span {
  int lo, n;        // tokens [lo, n) are attended
  int page0;        // page (index in the sequence) of the first tile
  int tiles;        // tiles of one head
};

__device__ __forceinline__ Span seq_span(const Kv8AttnArgs& a, int b) {
  Span s;
  s.n = min(max(__ldg(a.lens + b), 0), a.max_pages * kBlock);
  s.lo = a.window > 0 ? max(0, s.n - a.window) : 0;
  s.page0 = s.lo / kBlock;
  s.tiles = ((s.n + kBlock - 1) / kBlock - s.page0 + kTilePages - 1) / kTilePages;
  if (s.n == 0) s.tiles = 0;
  return s;
}

// A CTA's range of tiles and where it starts.
struct Work {
  long long begin, end;  // tiles of the whole batch
  long long total;
  int active;            // CTAs that have work
  int b;                 // sequence of the first tile
  long long b_first;     // first tile of that sequence
};

// Called by all NT threads of the CTA; `scratch` holds NT + 4 long longs of shared memory.
template <int NT>
__device__ __forceinline__ Work find_work(const Kv8AttnArgs& a, long long* scratch) {
  const int tid = threadIdx.x;
  const int per = (a.B + NT - 1) / NT, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += (long long)seq_span(a, b).tiles * a.Hkv;
  // inclusive scan over the warp, then over the warps
  long long run = mine;
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  if (lane == 31) scratch[warp] = run;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const long long first = before + run - mine;
  Work wk;
  wk.total = total;
  wk.active = (int)min((long long)a.n_cta, total);
  const int c = blockIdx.x;
  const bool has = c < wk.active;
  wk.begin = has ? total * c / wk.active : 0;
  wk.end = has ? total * (c + 1) / wk.active : 0;
  if (has && wk.begin >= first && wk.begin < first + mine) {
    long long at = first;
    for (int b = b0; b < b1; ++b) {
      const long long n = (long long)seq_span(a, b).tiles * a.Hkv;
      if (wk.begin < at + n) {
        scratch[NT] = b;
        scratch[NT + 1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  wk.b = has ? (int)scratch[NT] : 0;
  wk.b_first = has ? scratch[NT + 1] : 0;
  return wk;
}

// The CTA whose range holds tile t, for total tiles over `active` CTAs: largest c with
// c * total / active <= t.
__device__ __forceinline__ int cta_of_tile(long long t, long long total, int active) {
  return (int)(((t + 1) * active - 1) / total);
}

// Walks the segments of a CTA's range in order.
struct Walk {
  const Kv8AttnArgs& a;
  Work wk;
  long long at;       // next tile of the batch
  int b, h;
  Span sp;
  long long b_first;
  // the current segment's part in this range
  int tile0, tile1;   // tiles of the segment, relative to its start
  long long seg_first;

  __device__ Walk(const Kv8AttnArgs& a_, const Work& w) : a(a_), wk(w), at(w.begin), b(w.b), b_first(w.b_first) {
    if (at < wk.end) sp = seq_span(a, b);
  }
  // Moves to the next segment with tiles in the range; false at its end.
  __device__ bool next() {
    if (at >= wk.end) return false;
    while (at >= b_first + (long long)sp.tiles * a.Hkv) {
      b_first += (long long)sp.tiles * a.Hkv;
      sp = seq_span(a, ++b);
    }
    h = (int)((at - b_first) / sp.tiles);
    seg_first = b_first + (long long)h * sp.tiles;
    tile0 = (int)(at - seg_first);
    tile1 = (int)min((long long)sp.tiles, wk.end - seg_first);
    at = seg_first + tile1;
    return true;
  }
  __device__ bool whole() const { return tile0 == 0 && tile1 == sp.tiles; }
};

// Output of one (sequence, query head): acc / l with the scores' reference m (2^x units), joined with
// the earlier partial result where there is one.
struct Joined {
  float inv, w_prev;  // o = acc * inv + o_prev * w_prev
  float lse;
};
__device__ __forceinline__ Joined join_prev(const Kv8AttnArgs& a, size_t row, float m, float l) {
  Joined j;
  const float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  const float lp = a.lse_prev ? a.lse_prev[row] * kLog2e : -CUDART_INF_F;
  const float own = l > 0.f || l != l ? m : -CUDART_INF_F;
  const float top = fmaxf(own, lp);
  if (top == -CUDART_INF_F && l == l && lp == lp) {
    j.inv = j.w_prev = 0.f;
    j.lse = -CUDART_INF_F;
    return j;
  }
  const float w = own == -CUDART_INF_F ? 0.f : exp2f(m - top);
  const float wp = lp == -CUDART_INF_F ? 0.f : exp2f(lp - top);
  const float sum = fmaf(l, w, wp);
  j.inv = w / sum;
  j.w_prev = wp / sum;  // NaN where the sum is: o_prev may be null all the same
  j.lse = kLn2 * (top + log2f(sum));
  return j;
}
template <typename T>
__device__ __forceinline__ T joined_value(const Kv8AttnArgs& a, size_t row, int d, const Joined& j, float acc) {
  float y = j.inv != 0.f ? acc * j.inv : 0.f;
  if (a.o_prev && j.w_prev != 0.f) y = fmaf(to_f32(((const T*)a.o_prev)[row * a.hd + d]), j.w_prev, y);
  return from_f32<T>(y);
}

// ---- pieces of a split segment

// The CTAs that share a segment, and the slot of each one's piece.
struct Pieces {
  int c0, n;
  long long seg_first, total;
  int active;
  __device__ int slot(int i) const {
    const int c = c0 + i;
    return 2 * c + (total * c / active < seg_first ? 1 : 0);
  }
};
__device__ __forceinline__ Pieces pieces_of(const Walk& k) {
  Pieces p;
  p.seg_first = k.seg_first;
  p.total = k.wk.total;
  p.active = k.wk.active;
  p.c0 = cta_of_tile(k.seg_first, p.total, p.active);
  p.n = cta_of_tile(k.seg_first + k.sp.tiles - 1, p.total, p.active) - p.c0 + 1;
  return p;
}

__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums the pieces in the order of the CTAs, 32 at a time: lane i of every warp weighs piece i, the
// thread adds up column d of the accumulators. All lanes of a warp call it together.
template <int MG>
__device__ __forceinline__ void join_pieces(const Kv8AttnArgs& a, const Pieces& pc, int d, bool has_d, float (&acc)[MG],
                                            float (&m)[MG], float (&l)[MG]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int g = 0; g < MG; ++g) {
    acc[g] = l[g] = 0.f;
    m[g] = -CUDART_INF_F;
  }
  for (int i0 = 0; i0 < pc.n; i0 += 32) {
    const int n = min(32, pc.n - i0);
    const float* mine = a.part + (size_t)pc.slot(i0 + min(lane, n - 1)) * a.part_stride;
    float w[MG];
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      if (g >= a.G) break;
      const float mi = lane < n ? __ldcg(mine + a.G * a.hd + g) : -CUDART_INF_F;
      const float li = lane < n ? __ldcg(mine + a.G * a.hd + 8 + g) : 0.f;
      const float top = fmaxf(m[g], warp_max(mi));
      const float ref = top == -CUDART_INF_F ? 0.f : top;
      const float old = exp2f(m[g] - ref);
      w[g] = exp2f(mi - ref);
      l[g] = fmaf(l[g], old, warp_sum(li * w[g]));
      acc[g] *= old;
      m[g] = top;
    }
    for (int i = 0; i < n; ++i) {
      const float* from = a.part + (size_t)pc.slot(i0 + i) * a.part_stride + d;
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        if (g >= a.G) break;
        const float wi = __shfl_sync(0xffffffffu, w[g], i);
        if (has_d) acc[g] = fmaf(wi, __ldcg(from + g * a.hd), acc[g]);
      }
    }
  }
}

// o = 0, lse = -inf (or the earlier partial result) for the sequences without tokens, shared out
// among the CTAs, and the device checks of the lengths. Called by `threads` threads (whole warps) of
// the CTA, `tid` counted among them.
template <typename T>
__device__ __forceinline__ void empty_sequences(const Kv8AttnArgs& a, int tid, int threads) {
  for (int b = blockIdx.x; b < a.B; b += a.n_cta) {
    const int len = __ldg(a.lens + b);
    if (tid == 0 && (len < 0 || len > a.max_pages * kBlock)) flag_error(a.err, LR_DEVERR_LEN);
    if (len > 0) continue;
    const int Hq = a.Hkv * a.G;
    for (int r = tid / 32; r < Hq; r += threads / 32) {
      const size_t row = (size_t)b * Hq + r;
      const Joined j = join_prev(a, row, -CUDART_INF_F, 0.f);
      for (int d = tid & 31; d < a.hd; d += 32) ((T*)a.o)[row * a.hd + d] = joined_value<T>(a, row, d, j, 0.f);
      __syncwarp();
      if (a.lse && (tid & 31) == 0) a.lse[row] = j.lse;
    }
  }
}

}  // namespace kv8
}  // namespace lr
