// Decode attention over the 8-bit paged cache: the choice of the kernel, the kernel for every storage type,
// head_dim and group size that the tcgen05 kernel does not take, and the joining of pieces.
//
// Products by mma.sync (m16n8k16, fp16 in, fp32 sums): codes are exact in fp16, one conversion for two of them,
// and what multiplies them is a sum of two fp16 numbers, the second one 2^11 times as fine:
//   q = 2^e (q0 + q1 / 2048),   p = (p0 + p1 / 2048) / 2^15,
// each right to 2^-24, as good as fp32. The 16 rows of an operand are 8 query heads times two terms: row h
// and row h + 8, which the same lanes hold, so
//   S = Q K^T   (16 x 8 tokens): lane 4h + c has both terms of head h for tokens 2c and 2c + 1, and so
//   O = P V     (16 x 8 dims) takes the weights from the registers that the scores were in.
// The order of the dims is free: in S, lane 4t + c reads a quarter of token t's row, in O, lane 4d + c an eighth
// of the rows of its four tokens. Everything else is fp32.
//
// One CTA of 128 threads walks its share of the batch's tiles (kv8_common.cuh). Warp w takes the 32 tokens from
// 32 w on of every tile, by itself: its own maximum, sum and accumulators, joined with the other warps' at the
// segment's end. The values of a tile and the keys of the next are on their way while the scores are
// worked out. Bound by HBM latency and by the conversions; on the CUDA cores, with two
// multiply-adds to an instruction, it was bound by instructions at a third of HBM's rate.
#include <algorithm>

#include "kv8_common.cuh"

namespace lr {
namespace kv8 {
namespace {

constexpr int NT = 128, kWarps = NT / 32;
static_assert(kTileTokens == NT, "32 tokens of a tile to a warp");

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bits(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ uint32_t code_pair(uint32_t codes) { return bits(e4m3x2_half2(codes & 0xffffu)); }

// Two terms of two numbers.
__device__ __forceinline__ void split(float x, float y, uint32_t& t0, uint32_t& t1) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  t0 = bits(h);
  t1 = bits(__floats2half2_rn((x - f.x) * 2048.f, (y - f.y) * 2048.f));
}

// This lane's part of a row: `n` bytes of it (a multiple of 8) are there, the rest is 0.
template <int kWords>
__device__ __forceinline__ void load_row(const uint8_t* at, int n, bool wide, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < kWords; i += 4) {
    if (kWords >= 4 && wide && n >= 4 * i + 16) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(at + 4 * i));
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
      continue;
    }
#pragma unroll
    for (int x = i; x < i + 4 && x < kWords; x += 2) {
      uint2 v = make_uint2(0u, 0u);
      if (n > 4 * x) v = __ldg(reinterpret_cast<const uint2*>(at + 4 * x));
      w[x] = v.x;
      w[x + 1] = v.y;
    }
  }
}

// CTAs on an SM: what the registers allow.
constexpr int resident(int hd) { return hd <= 64 ? 4 : 2; }

template <int HD>  // head_dim <= HD
__global__ void __launch_bounds__(NT, resident(HD)) kv8_attn_kernel(Kv8AttnArgs a, bool bf16) {
  constexpr int kBatch = HD <= 128 ? 32 : 16, kBatches = 32 / kBatch;  // tokens under way at once
  constexpr int kKeyWords = HD / 16, kValueWords = HD / 32;            // of a lane's part of a row
  __shared__ long long scratch[NT + 4];
  __shared__ float ml[kWarps][2][8];
  __shared__ float sums[kWarps][8][HD];
  __shared__ uint4 queries[HD / 16][32];  // the same for every warp
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hi = lane >> 2, c = lane & 3;
  const int hd = a.hd, G = a.G;
  const int key_dim = c * (HD / 4), key_bytes = max(0, min(HD / 4, hd - key_dim));
  const int value_dim = hi * (HD / 8), value_bytes = max(0, min(HD / 8, hd - value_dim));
  const bool wide = hd % 16 == 0;
  if (tid == 0) err = 0;
  grid_dependency();
  Walk k(a, find_work<NT>(a, scratch));
  while (k.next()) {
    const int* table = a.table + (size_t)k.b * a.max_pages;
    const size_t row0 = ((size_t)k.b * a.Hkv + k.h) * G;

    // head `hi` of the queries, the dims of this lane's keys: scaled to [2^14, 2^15) and split
    __syncthreads();
    float factor;
    {
      float x[HD / 4], top = 0.f;
#pragma unroll
      for (int d = 0; d < HD / 4; d += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const size_t at = (row0 + hi) * hd + key_dim + d;
        if (hi < G && d < key_bytes) {
          if (bf16) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>((const __nv_bfloat16*)a.q + at));
            v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                            __uint_as_float(u.y & 0xffff0000u));
          } else {
            v = __ldg(reinterpret_cast<const float4*>((const float*)a.q + at));
          }
        }
        x[d] = v.x;
        x[d + 1] = v.y;
        x[d + 2] = v.z;
        x[d + 3] = v.w;
        top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max((int)(__float_as_uint(top) >> 23) - 127 - 14, -112);
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      factor = top < CUDART_INF_F ? __uint_as_float((uint32_t)(127 + e) << 23) * a.scale : CUDART_NAN_F;
#pragma unroll
      for (int j = 0; j < HD / 16; ++j) {
        uint4 q;
        split(x[4 * j] * inv, x[4 * j + 1] * inv, q.x, q.y);
        split(x[4 * j + 2] * inv, x[4 * j + 3] * inv, q.z, q.w);
        if (j % kWarps == warp) queries[j][lane] = q;
      }
    }
    __syncthreads();
    // acc[j]: head `hi`, dims 2c HD / 8 + j and (2c + 1) HD / 8 + j of both terms, in units of `unit`
    float acc[HD / 8][4];
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    float m = -CUDART_INF_F, l = 0.f;  // of head `hi`; the sum is this lane's share
    float unit = 0.f, largest = 0.f;   // of the value scales so far

    // batch i of the range is batch i % kBatches of the warp's tokens of tile tile0 + i / kBatches
    const int n_batches = (k.tile1 - k.tile0) * kBatches;
    struct Part {  // a batch's page (-1: none) and the tokens that are attended, counted from its first: [from, to)
      int id, from, to;
      unsigned row;  // of its first token in the page
      float ks, vs;
    };
    // the page id is on its way a batch before it is looked at, the scales a batch before they are used
    auto part_of = [&](int i) {
      Part b{-1, 0, 0, 0, 0.f, 0.f};
      if (i >= n_batches) return b;
      const int t = (k.sp.page0 + (k.tile0 + i / kBatches) * kTilePages) * kBlock + warp * 32 + i % kBatches * kBatch;
      if (t / kBlock * kBlock >= k.sp.n) return b;
      b.id = __ldg(table + t / kBlock);
      b.from = max(0, k.sp.lo - t);
      b.to = min(kBatch, k.sp.n - t);
      b.row = t % kBlock;
      return b;
    };
    auto resolve = [&](Part& b) {
      if ((unsigned)b.id < (unsigned)a.n_pages) {
        b.ks = __ldg(a.ks + (size_t)b.id * a.Hkv + k.h);
        b.vs = __ldg(a.vs + (size_t)b.id * a.Hkv + k.h);
      } else {
        if (lane == 0 && (b.to || b.from)) atomicOr(&err, LR_DEVERR_PAGE);
        b.from = b.to = 0;
      }
    };
    auto page_head = [&](const uint8_t* codes, const Part& b) {
      return codes + (size_t)b.id * a.page_stride + ((size_t)k.h * kBlock + b.row) * hd;
    };
    // rows of the keys: token 8 n + hi
    auto load_keys = [&](const Part& b, uint32_t (&w)[kBatch / 8][kKeyWords]) {
      const bool any = b.to > b.from;
      const uint8_t* at = any ? page_head(a.kc, b) + (unsigned)(hi * hd + key_dim) : nullptr;
#pragma unroll
      for (int n = 0; n < kBatch / 8; ++n) {
        const int t = 8 * n + hi;
        load_row<kKeyWords>(at + (unsigned)(8 * n * hd), any && t >= b.from && t < b.to ? key_bytes : 0, wide, w[n]);
      }
    };
    // rows of the values: tokens 16 n + {2c, 2c + 1, 2c + 8, 2c + 9}
    auto load_values = [&](const Part& b, uint32_t (&w)[kBatch / 16][4][kValueWords]) {
      const bool any = b.to > b.from;
      const uint8_t* at = any ? page_head(a.vc, b) + (unsigned)(2 * c * hd + value_dim) : nullptr;
#pragma unroll
      for (int n = 0; n < kBatch / 16; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 16 * n + (x & 1) + (x >> 1) * 8, t = 2 * c + row;
          load_row<kValueWords>(at + (unsigned)(row * hd), any && t >= b.from && t < b.to ? value_bytes : 0, wide, w[n][x]);
        }
    };
    Part now = part_of(0), next = part_of(1);
    uint32_t kw[kBatch / 8][kKeyWords], vw[kBatch / 16][4][kValueWords];
    resolve(now);
    load_keys(now, kw);
    for (int i = 0; i < n_batches; ++i) {
      load_values(now, vw);
      resolve(next);
      float x[kBatch / 8][2];  // scores of tokens 8 n + 2c and 8 n + 2c + 1
      {
        float s[kBatch / 8][4] = {};
#pragma unroll
        for (int j = 0; j < HD / 16; ++j) {
          const uint4 q = queries[j][lane];
#pragma unroll
          for (int n = 0; n < kBatch / 8; ++n) mma_f16(s[n], q.x, q.y, q.z, q.w, code_pair(kw[n][j]), code_pair(kw[n][j] >> 16));
        }
#pragma unroll
        for (int n = 0; n < kBatch / 8; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) x[n][y] = fmaf(s[n][2 + y], 1.f / 2048.f, s[n][y]) * (factor * now.ks);
      }
      load_keys(next, kw);
      const Part after = part_of(i + 2);
      if (now.from > 0 || now.to < kBatch) {
#pragma unroll
        for (int n = 0; n < kBatch / 8; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int t = 8 * n + 2 * c + y;
            if (t < now.from || t >= now.to) x[n][y] = -CUDART_INF_F;
          }
      }
      float top = m;
#pragma unroll
      for (int n = 0; n < kBatch / 8; ++n) top = fmaxf(top, fmaxf(x[n][0], x[n][1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float ref = top == -CUDART_INF_F ? 0.f : top;
      float old = exp2f(m - ref);
      m = top;
      l *= old;
      // sums are kept in units of the page's value scale, or of 2^-64 of the largest so far, so that
      // neither they nor the weights leave their type's range
      float share = 0.f;
      if (now.to > now.from) {
        largest = fmaxf(largest, now.vs);
        const float u = fmaxf(now.vs, largest * 5.421010862427522e-20f);
        if (unit != u) old *= unit / u;
        unit = u;
        share = now.vs == u ? 1.f : now.vs / u;
      }
      if (__any_sync(0xffffffffu, old != 1.f)) {
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[j][y] *= old;
      }
#pragma unroll
      for (int n = 0; n < kBatch / 16; ++n) {
        uint32_t p[4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float p0 = exp2f(x[2 * n + y][0] - ref), p1 = exp2f(x[2 * n + y][1] - ref);
          l += p0 + p1;
          split(p0 * share * 32768.f, p1 * share * 32768.f, p[2 * y], p[2 * y + 1]);
        }
#pragma unroll
        for (int j = 0; j < HD / 8; j += 4) {
          uint32_t b[2][4];  // of the rows 2c, 2c + 1 and of the rows 2c + 8, 2c + 9: pairs of dims j .. j + 3
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t r0 = vw[n][2 * y][j / 4], r1 = vw[n][2 * y + 1][j / 4];
            const uint32_t lo = __byte_perm(r0, r1, 0x5140), up = __byte_perm(r0, r1, 0x7362);
            b[y][0] = code_pair(lo);
            b[y][1] = code_pair(lo >> 16);
            b[y][2] = code_pair(up);
            b[y][3] = code_pair(up >> 16);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) mma_f16(acc[j + y], p[0], p[1], p[2], p[3], b[0][y], b[1][y]);
        }
      }
      now = next;
      next = after;
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    __syncthreads();  // the last segment's sums have been read
    if (c == 0) {
      ml[warp][0][hi] = m;
      ml[warp][1][hi] = l;
    }
    const float scale = unit * (1.f / 32768.f);
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      sums[warp][hi][2 * c * (HD / 8) + j] = fmaf(acc[j][2], 1.f / 2048.f, acc[j][0]) * scale;
      sums[warp][hi][(2 * c + 1) * (HD / 8) + j] = fmaf(acc[j][3], 1.f / 2048.f, acc[j][1]) * scale;
    }
    __syncthreads();
    const bool whole = k.whole();
    float* slot = whole ? nullptr : a.part + (size_t)piece_slot(k.wk, k.seg_first) * a.part_stride;
    for (int g = 0; g < G; ++g) {
      float top = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][0][g]);
      const float ref = top == -CUDART_INF_F ? 0.f : top;
      float f[kWarps], sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[w] = exp2f(ml[w][0][g] - ref);
        sum = fmaf(ml[w][1][g], f[w], sum);
      }
      Joined j;
      if (whole) {
        j = join_prev(a, row0 + g, top, sum);
        __syncthreads();  // lse may be lse_prev: every thread has read it
        if (a.lse && tid == 0) a.lse[row0 + g] = j.lse;
      } else if (tid == 0) {
        slot[G * hd + g] = top;
        slot[G * hd + 8 + g] = sum;
      }
      for (int d = tid; d < hd; d += NT) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v = fmaf(sums[w][g][d], f[w], v);
        if (!whole) slot[g * hd + d] = v;
        else if (bf16) ((__nv_bfloat16*)a.o)[(row0 + g) * hd + d] = joined_value<__nv_bfloat16>(a, row0 + g, d, j, v);
        else ((float*)a.o)[(row0 + g) * hd + d] = joined_value<float>(a, row0 + g, d, j, v);
      }
    }
  }
  __syncthreads();
  if (tid == 0) a.cta_err[blockIdx.x] = err;
}

void (*attn_kernel(int hd))(Kv8AttnArgs, bool) {
  return hd <= 64 ? kv8_attn_kernel<64> : hd <= 128 ? kv8_attn_kernel<128> : kv8_attn_kernel<256>;
}

// ------------------------------------------------------------------ joining the pieces
//
// CTA (c, g): query head g of the segment that the range of CTA c of the attention kernel is the first to start inside
// of (none, most of the time). Four numbers to a thread, the pieces spread over the rest of the threads,
// so that all of them are under way at once; the order of the sums is fixed by the threads. The same
// grid answers the empty sequences, a row to a warp, and collects the device errors. It may be launched
// while the attention kernel still runs: only lens is read before it has ended.

constexpr int JT = 128;
constexpr int kMaxCtas = 1024;

template <typename T>
__global__ void __launch_bounds__(JT) kv8_join_kernel(Kv8AttnArgs a) {
  __shared__ long long scratch[JT + 4];
  __shared__ float weight[kMaxCtas], sum_of[kMaxCtas];
  __shared__ float red[2][JT / 32];
  __shared__ __align__(16) float sums[JT * 4];
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x, g = blockIdx.y, Hq = a.Hkv * a.G, hd = a.hd;
  const Work wk = find_work<JT>(a, scratch);
  Walk k(a, wk);
  // the first of the CTAs whose range starts inside the segment
  const bool mine = c > 0 && k.next() && k.tile0 > 0 && range_begin(wk.total, c - 1, wk.active) <= k.seg_first;
  const bool errors = c == 0 && g == 0;
  if (errors) {
    if (tid == 0) err = 0;
    __syncthreads();
    bool bad = false;
    for (int b = tid; b < a.B; b += JT) {
      const int len = __ldg(a.lens + b);
      bad |= len < 0 || len > a.max_pages * kBlock;
    }
    if (bad) atomicOr(&err, LR_DEVERR_LEN);
  }
  const long long n_warps = (long long)gridDim.x * gridDim.y * (JT / 32), rows = (long long)a.B * Hq;
  for (long long row = ((long long)g * gridDim.x + c) * (JT / 32) + warp; row < rows; row += n_warps) {
    if (__ldg(a.lens + row / Hq) > 0) continue;
    const Joined j = join_prev(a, row, -CUDART_INF_F, 0.f);
    for (int d = lane; d < hd; d += 32) ((T*)a.o)[row * hd + d] = joined_value<T>(a, row, d, j, 0.f);
    __syncwarp();
    if (a.lse && lane == 0) a.lse[row] = j.lse;
  }
  grid_dependency();
  if (errors) {
    int bits = 0;
    for (int i = tid; i < a.n_cta; i += JT) bits |= __ldcg(a.cta_err + i);
    if (bits) atomicOr(&err, bits);
    __syncthreads();
    if (tid == 0) *a.err = err;
  }
  if (!mine) return;
  const Pieces pc = pieces_of(k);
  const size_t row = ((size_t)k.b * a.Hkv + k.h) * a.G + g;
  const int n = pc.n, ml = a.G * hd + g;
  const int cols = hd / 4, groups = JT / cols, col = tid % cols, group = tid / cols;
  auto values = [&](int i) {
    return __ldcg(reinterpret_cast<const float4*>(a.part + (size_t)pc.slot(i) * a.part_stride + g * hd) + col);
  };
  // a thread's first pieces are on their way before their weights are known
  constexpr int kAhead = 10;
  float4 v[kAhead];
#pragma unroll
  for (int x = 0; x < kAhead; ++x) {
    const int i = group + x * groups;
    v[x] = group < groups && i < n ? values(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float m = -CUDART_INF_F;
  for (int i = tid; i < n; i += JT) {
    const float* at = a.part + (size_t)pc.slot(i) * a.part_stride + ml;
    const float mi = __ldcg(at);
    sum_of[i] = __ldcg(at + 8);
    weight[i] = mi;
    m = fmaxf(m, mi);
  }
  m = warp_max(m);
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  const float ref = m == -CUDART_INF_F ? 0.f : m;
  float l = 0.f;
  for (int i = tid; i < n; i += JT) {
    const float w = exp2f(weight[i] - ref);
    weight[i] = w;
    l = fmaf(w, sum_of[i], l);
  }
  l = warp_sum(l);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  if (group < groups) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, const float4& x) {
      const float w = weight[i];
      s.x = fmaf(w, x.x, s.x);
      s.y = fmaf(w, x.y, s.y);
      s.z = fmaf(w, x.z, s.z);
      s.w = fmaf(w, x.w, s.w);
    };
#pragma unroll
    for (int x = 0; x < kAhead; ++x)
      if (group + x * groups < n) add(group + x * groups, v[x]);
#pragma unroll 4
    for (int i = group + kAhead * groups; i < n; i += groups) add(i, values(i));
    reinterpret_cast<float4*>(sums)[group * cols + col] = s;
  }
  const Joined j = join_prev(a, row, m, l);
  __syncthreads();  // lse may be lse_prev: every thread has read it
  for (int d = tid; d < hd; d += JT) {
    float acc = 0.f;
    for (int x = 0; x < groups; ++x) acc += sums[x * hd + d];
    ((T*)a.o)[row * hd + d] = joined_value<T>(a, row, d, j, acc);
  }
  if (a.lse && tid == 0) a.lse[row] = j.lse;
}

template <typename T>
cudaError_t launch_attn(const Kv8AttnArgs& a, const Kv8AttnPlan& plan, cudaStream_t st) {
  cudaError_t e;
  if (plan.tensor) {
    CUtensorMap mk, mv;
    if (!kv8_page_map(&mk, a.kc, a) || !kv8_page_map(&mv, a.vc, a)) return cudaErrorInvalidValue;
    e = launch_attn_tc(a, mk, mv, st);
  } else {
    e = launch_overlapped(attn_kernel(a.hd), dim3(plan.n_cta), NT, 0, st, a, sizeof(T) == 2);
  }
  if (e != cudaSuccess) return e;
  return launch_overlapped(kv8_join_kernel<T>, dim3(plan.n_cta, a.G), JT, 0, st, a);
}

}  // namespace
}  // namespace kv8

Kv8AttnPlan plan_kv8_attn(const lr_kv8_pages& kv, int n_q_heads, int sm_count) {
  Kv8AttnPlan p{};
  const int G = n_q_heads / kv.n_kv_heads;
  const long long most = (long long)kv.batch * kv.n_kv_heads * ((kv.max_pages + 1) / 2 + kv8::kSegmentUnits);  // units
  p.tensor = kv.dtype == LR_BF16 && kv.head_dim == 128;
  p.n_cta = (int)std::max(1LL, std::min<long long>(most, std::min((p.tensor ? 2 : kv8::resident(kv.head_dim)) * sm_count, kv8::kMaxCtas)));
  p.part_stride = G * kv.head_dim + 16;
  p.cta_err_off = 256;
  p.part_off = (256 + (size_t)p.n_cta * sizeof(int) + 255) & ~(size_t)255;
  p.ws_bytes = p.part_off + (((size_t)2 * p.n_cta * p.part_stride * sizeof(float) + 255) & ~(size_t)255);
  return p;
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, const Kv8AttnPlan& plan, lr_dtype dt, cudaStream_t st) {
  if (a.B == 0) return cudaMemsetAsync(a.err, 0, 256, st);
  return dt == LR_BF16 ? kv8::launch_attn<__nv_bfloat16>(a, plan, st) : kv8::launch_attn<float>(a, plan, st);
}

}  // namespace lr
