// Device helpers of the 8-bit paged cache: e4m3 conversions, and for the attention what a CTA does to find its
// share of the batch's tiles and to join the pieces of a split segment.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math_constants.h>

#include "lr_common.cuh"
#include "kv8_rules.h"
#include "lr_kv8.h"
#include "sm100.cuh"

namespace lr {
namespace kv8 {

// Two fp32 values to e4m3 codes (nearest even, saturating, NaN kept); lo in bits 0-7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return r;
}

// The values of two e4m3 codes (exact in fp16).
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) { return __half22float2(e4m3x2_half2(codes)); }

// Two fp32 operations in one instruction.
struct Two {
  uint64_t v;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Waits for the grid before in the stream, then lets the next one be launched: what that one reads before
// its own wait was complete before this grid went on.
__device__ __forceinline__ void grid_dependency() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// Launches a kernel that may start while the grid before drains: it waits for that grid (grid_dependency)
// before it reads what the grid writes.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int cluster, int threads, size_t smem, cudaStream_t st,
                              A&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// 2^x; -inf gives 0, results under 2^-126 too.
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ attention: the division of work (kv8_rules.h)

// The lengths and the page table on their way to L2 while the grid before may still run: they are read one after the
// other at the start, and after a step over many bytes they are in HBM again. Nothing is read
// here, so it does not matter who is still writing them.
__device__ __forceinline__ void prefetch_inputs(const Kv8AttnArgs& a) {
  const long long line = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long ids = (long long)a.B * a.max_pages;
  if (line * 32 < ids) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + line * 32));
  if (line * 32 < a.B) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.lens + line * 32));
}

// Called by all NT threads of the CTA; `scratch` holds NT + 4 long longs of shared memory. Up to 32 sequences
// are a warp's own business, a lane for each, without a barrier.
template <int NT>
__device__ __forceinline__ Work find_work(const Kv8AttnArgs& a, long long* scratch) {
  const int tid = threadIdx.x;
  if (a.B <= 32) {
    const int lane = tid & 31, len = lane < a.B ? __ldg(a.lens + lane) : 0;
    Work wk;
    wk.bad_len = len < 0 || len > a.max_pages * kBlock;
    const long long mine = lane < a.B ? (long long)span_of(a, len).units * a.Hkv : 0;
    long long run = mine;
    for (int o = 1; o < a.B; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    wk.total = __shfl_sync(0xffffffffu, run, a.B - 1);
    wk.active = (int)min((long long)a.n_cta, wk.total);
    const int c = blockIdx.x;
    const bool has = c < wk.active;
    wk.begin = has ? range_begin(wk.total, c, wk.active) : 0;
    wk.end = has ? range_begin(wk.total, c + 1, wk.active) : 0;
    const uint32_t hit = __ballot_sync(0xffffffffu, has && wk.begin >= run - mine && wk.begin < run);
    wk.b = max(0, __ffs(hit) - 1);
    wk.b_first = __shfl_sync(0xffffffffu, run - mine, wk.b);
    return wk;
  }
  const int per = (a.B + NT - 1) / NT, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  Work wk;
  wk.bad_len = false;
  for (int b = b0; b < b1; ++b) {
    mine += (long long)seq_span(a, b).units * a.Hkv;
    const int len = __ldg(a.lens + b);
    wk.bad_len |= len < 0 || len > a.max_pages * kBlock;
  }
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
  wk.total = total;
  wk.active = (int)min((long long)a.n_cta, total);
  const int c = blockIdx.x;
  const bool has = c < wk.active;
  wk.begin = has ? range_begin(total, c, wk.active) : 0;
  wk.end = has ? range_begin(total, c + 1, wk.active) : 0;
  if (has && wk.begin >= first && wk.begin < first + mine) {
    long long at = first;
    for (int b = b0; b < b1; ++b) {
      const long long n = (long long)seq_span(a, b).units * a.Hkv;
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

// Small calls: the device checks of every length and attended page, by the threads [0, step) of one CTA. They go through the
// whole table (2048 ids at most), an id with its sequence's length: loads that depend on one another, sequence by
// sequence, made this CTA 49 us late with 256 sequences.
__device__ __forceinline__ int check_all(const Kv8AttnArgs& a, int first, int step) {
  int bits = 0;
  const int ids = a.B * a.max_pages;
#pragma unroll 8
  for (int i = first; i < ids; i += step) {
    const int b = (unsigned)i / (unsigned)a.max_pages, p = i - b * a.max_pages;
    const int id = __ldg(a.table + i), len = __ldg(a.lens + b);
    if (len < 0 || len > a.max_pages * kBlock) bits |= LR_DEVERR_LEN;
    const Span sp = span_of(a, len);
    if (p >= sp.page0 && p * kBlock < sp.n && (unsigned)id >= (unsigned)a.n_pages) bits |= LR_DEVERR_PAGE;
  }
  return bits;
}

// Sums of weights times values are kept in units of 2^32: a weight is 1 at most, so no number of tokens that an int
// holds takes them out of fp32's range, whatever finite values the codes and scales stand for.
constexpr float kSumUnit = 4294967296.f;

// Output of one (sequence, query head): acc / l with the scores' reference m (2^x units), joined with
// the earlier partial result where there is one.
struct Joined {
  float inv, w_prev;  // o = acc * inv + o_prev * w_prev, acc in units of kSumUnit
  float top, sum;     // lse = ln 2 (top + log2 sum)
  __device__ __forceinline__ float lse() const {
    return sum == 0.f ? -CUDART_INF_F : 0.6931471805599453f * (top + log2f(sum));
  }
};
// `prev`: the earlier part's lse, -inf for none.
__device__ __forceinline__ Joined join_with(float m, float l, float prev) {
  Joined j;
  const float lp = prev * 1.4426950408889634f;
  const float own = l > 0.f || l != l ? m : -CUDART_INF_F;
  j.top = fmaxf(own, lp);
  if (j.top == -CUDART_INF_F && l == l && lp == lp) {
    j.inv = j.w_prev = j.sum = 0.f;
    return j;
  }
  const float w = own == -CUDART_INF_F ? 0.f : exp2f(m - j.top);
  const float wp = lp == -CUDART_INF_F ? 0.f : exp2f(lp - j.top);
  j.sum = fmaf(l, w, wp);
  const float r = __frcp_rn(j.sum);
  j.inv = w * r * kSumUnit;
  j.w_prev = wp * r;  // NaN where the sum is, with or without an earlier part
  return j;
}
__device__ __forceinline__ float prev_lse(const Kv8AttnArgs& a, size_t row) { return a.lse_prev ? a.lse_prev[row] : -CUDART_INF_F; }
__device__ __forceinline__ Joined join_prev(const Kv8AttnArgs& a, size_t row, float m, float l) {
  return join_with(m, l, prev_lse(a, row));
}
// acc * inv + prev * w; what a weight of 0 goes with is left out, whatever it is.
__device__ __forceinline__ float join_value(float acc, float inv, float prev, float w) {
  const float y = inv != 0.f ? acc * inv : 0.f;
  return w != 0.f ? fmaf(prev, w, y) : y;
}
template <typename T>
__device__ __forceinline__ T joined_value(const Kv8AttnArgs& a, size_t row, int d, const Joined& j, float acc) {
  const float prev = a.o_prev ? to_f32(((const T*)a.o_prev)[row * a.hd + d]) : 0.f;
  return from_f32<T>(join_value(acc, j.inv, prev, j.w_prev));
}

// o = 0 and lse = -inf, or the earlier partial result, for the sequences without tokens. One warp, `first` of `step`
// that share the rows: neighbouring ones go to different warps.
template <typename T>
__device__ __forceinline__ void empty_rows(const Kv8AttnArgs& a, int first, int step) {
  const int lane = threadIdx.x & 31, Hq = a.Hkv * a.G;
  const long long rows = (long long)a.B * Hq;
  for (long long at = first; at < rows; at += 32LL * step) {
    const long long mine = at + (long long)lane * step;
    uint32_t todo = __ballot_sync(0xffffffffu, mine < rows && __ldg(a.lens + mine / Hq) <= 0);
    for (; todo; todo &= todo - 1) {
      const size_t row = at + (long long)(__ffs(todo) - 1) * step;
      const Joined j = join_prev(a, row, -CUDART_INF_F, 0.f);
      for (int d = lane; d < a.hd; d += 32) ((T*)a.o)[row * a.hd + d] = joined_value<T>(a, row, d, j, 0.f);
      __syncwarp();  // lse may be lse_prev: every lane has read it
      if (a.lse && lane == 0) a.lse[row] = j.lse();
    }
  }
}

// Maximum over the warp; a NaN counts only where every lane has one.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Small calls: one warp joins the pieces of query head g of the cluster's segment, at most 8 of them.
template <typename T>
__device__ __forceinline__ void warp_join(const Kv8AttnArgs& a, int n, int g) {
  const int lane = threadIdx.x & 31, seg = blockIdx.x / a.cluster, cols = a.hd / 4;
  const size_t row = (size_t)seg * a.G + g, stride = 2 * (size_t)a.part_stride;
  const float* part = a.part + (size_t)seg * a.cluster * stride;
  const float* ml = part + (size_t)min(lane, n - 1) * stride + a.G * a.hd + g;
  const float mi = lane < n ? __ldcg(ml) : -CUDART_INF_F, li = lane < n ? __ldcg(ml + 8) : 0.f;
  const float prev = prev_lse(a, row);
  Joined j;
  float w = 0.f;
  for (int c0 = 0; c0 < cols; c0 += 32) {
    const int col = c0 + lane;
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = i < n && col < cols ? __ldcg(reinterpret_cast<const float4*>(part + i * stride + g * a.hd) + col)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    if (c0 == 0) {
      const float m = warp_max(mi);
      w = exp2_ftz(mi - (m == -CUDART_INF_F ? 0.f : m));
      j = join_with(m, warp_sum(w * li), prev);
    }
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      s.x = fmaf(wi, v[i].x, s.x);
      s.y = fmaf(wi, v[i].y, s.y);
      s.z = fmaf(wi, v[i].z, s.z);
      s.w = fmaf(wi, v[i].w, s.w);
    }
    if (col < cols) {
      T* o = (T*)a.o + row * a.hd + 4 * col;
      o[0] = joined_value<T>(a, row, 4 * col, j, s.x);
      o[1] = joined_value<T>(a, row, 4 * col + 1, j, s.y);
      o[2] = joined_value<T>(a, row, 4 * col + 2, j, s.z);
      o[3] = joined_value<T>(a, row, 4 * col + 3, j, s.w);
    }
  }
  __syncwarp();  // lse may be lse_prev: every lane has read it
  if (a.lse && lane == 0) a.lse[row] = j.lse();
}

// Small calls: the end of a CTA, all of its threads. The pieces are in place when the cluster has met. `bits`: its
// device error bits, of CTA 0 those of check_all too: that CTA writes the word, which nobody has to clear; a
// wait of another that ran out, seconds later, is added to it.
template <typename T>
__device__ __forceinline__ void finish_small(const Kv8AttnArgs& a, int pieces, int bits) {
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) *a.err = bits;
    else if (bits & LR_DEVERR_TIMEOUT) atomicOr(a.err, LR_DEVERR_TIMEOUT);
  }
  __syncwarp();  // the cluster barrier is warp-aligned
  if (a.cluster > 1) sm100::cluster_sync();
  if (pieces < 2) return;
  const int warps = blockDim.x / 32;
  for (int g = blockIdx.x % a.cluster * warps + (int)threadIdx.x / 32; g < a.G; g += a.cluster * warps) warp_join<T>(a, pieces, g);
}

}  // namespace kv8
}  // namespace lr
