// Decode attention over the 8-bit paged cache: the choice of the kernel, the kernel for every storage type,
// head_dim and group size that the tcgen05 kernel does not take, and the joining of pieces.
//
// Products by mma.sync (m16n8k16, fp16 in, fp32 sums): codes are exact in fp16, one conversion for two of them,
// and what multiplies them is a sum of two fp16 numbers, the second one 2^11 times as fine:
//   q = 2^e (q0 + q1 / 2048),   p = (p0 + p1 / 2048) / 2^15,
// each right to 2^-23 (the second term rounds what the first leaves over, up to 2^-11 of it, to 11 bits), or to 2^-50 of
// the largest where it is an fp16 subnormal. The 16 rows of an operand are 8 query heads times two terms: row h
// and row h + 8, which the same lanes hold, so
//   S = Q K^T   (16 x 8 tokens): lane 4h + c has both terms of head h for tokens 2c and 2c + 1, and so
//   O = P V     (16 x 8 dims) takes the weights from the registers that the scores were in.
// The order of the dims is free: in S, lane 4t + c reads every fourth 16 bytes of token t's row, in O, lane 4d + c
// an eighth of the rows of its four tokens. Everything else is fp32.
//
// One CTA of 128 threads walks its share of the batch's tiles (kv8_common.cuh). Warp w takes the 32 tokens from
// 32 w on of every tile, by itself: its own maximum, sum and accumulators, joined with the other warps' at the
// segment's end. Its rows of a page are one piece of memory each for keys and values, copied as such to shared
// memory two tiles ahead, so a warp waits for nobody. Bound by its instructions' latency with two warps to a
// scheduler (about 900 instructions for a warp's 8 KB).
//
// Measured (B200, 60000 tokens of one sequence, 8 KV heads): fp32, head_dim 128, 36.5 us with 4 query heads per KV
// head, 38 with 8 (3.4 TB/s; on the CUDA cores, two multiply-adds to an instruction, 60 and 103); head_dim 64
// 25; bf16, head_dim 256, four sequences of 30000 tokens 114 us (4.3 TB/s).
#include <algorithm>

#include "kv8_common.cuh"
#include "sm100.cuh"

namespace lr {
namespace kv8 {
namespace {

using namespace sm100;

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

template <int kWords>
__device__ __forceinline__ void load_words(const uint8_t* smem, bool wide, uint32_t (&w)[kWords]) {
  if (kWords == 4 && wide) {
    const uint4 v = *reinterpret_cast<const uint4*>(smem);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < kWords; i += 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(smem + 4 * i);
    w[i] = v.x;
    w[i + 1] = v.y;
  }
}

template <int HD>
struct Ring {
  static constexpr int kStages = 3;
  static constexpr int kBatch = HD <= 128 ? 32 : 16;      // tokens of a stage
  static constexpr int kKeyParts = HD / 64;               // 16 bytes each, of a lane's quarter of a row
  static constexpr int kValueWords = HD == 64 ? 2 : 4;    // of a part of a lane's eighth of a row
  static constexpr int kValueParts = HD / 32 / kValueWords;
  static constexpr int kValues = kBatch * HD;             // offset of the values in a stage
  static constexpr int kStageBytes = 2 * kBatch * HD;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kBytes = kWarps * kWarpBytes;
};

// CTAs on an SM: what registers and rings allow.
constexpr int resident(int hd) { return hd <= 64 ? 3 : 2; }

template <int HD>  // head_dim <= HD
__global__ void __launch_bounds__(NT, resident(HD)) kv8_attn_kernel(Kv8AttnArgs a, bool bf16) {
  using R = Ring<HD>;
  constexpr int kBatch = R::kBatch, kBatches = 32 / kBatch, kSumStride = HD + 8;
  static_assert(8 * kSumStride * 4 <= R::kWarpBytes, "a warp's sums take the place of its ring");
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ long long scratch[NT + 4];
  __shared__ float ml[kWarps][2][8];
  __shared__ uint4 queries[HD / 16][32];  // the same for every warp
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hi = lane >> 2, c = lane & 3;
  const int hd = a.hd, G = a.G;
  const bool wide = hd % 16 == 0;
  uint8_t* const my_ring = ring + warp * R::kWarpBytes;
  __shared__ uint64_t full[kWarps][R::kStages];
  __shared__ volatile int gave_up;
  auto sums = [&](int w, int g) { return reinterpret_cast<float*>(ring + w * R::kWarpBytes) + g * kSumStride; };
  if (tid == 0) {
    err = 0;
    gave_up = 0;
    for (int i = 0; i < kWarps * R::kStages; ++i) mbar_init(&full[0][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  prefetch_inputs(a);
  grid_dependency();
  Walk<Kv8AttnArgs> k(a, a.cluster ? small_work(a, blockIdx.x) : find_work<NT>(a, scratch));
  if (blockIdx.x == 0 && k.wk.bad_len) atomicOr(&err, LR_DEVERR_LEN);
  if (tid == 0 && !a.cluster) reinterpret_cast<Pieces*>(a.split)[blockIdx.x] = pieces_of(a, k.wk, blockIdx.x);
  uint32_t stages = 0;  // copied to so far, by this warp
  bool ok = true;       // once a wait has failed the rest runs through without waiting: nobody is left at a barrier
  while (k.next()) {
    const int* table = a.table + (size_t)k.b * a.max_pages;
    const size_t row0 = ((size_t)k.b * a.Hkv + k.h) * G;

    // batch i of the range is batch i % kBatches of the warp's tokens of tile tile0 + i / kBatches
    const int n_batches = (k.tile1 - k.tile0) * kBatches;
    struct Part {  // a batch's page (-1: none) and the tokens that are attended, counted from its first: [from, to)
      int id, from, to;
      unsigned row;  // of its first token in the page
      float ks, vs;
    };
    // a page id is on its way a batch before it is looked at, the scales and rows two before they are used
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
    const uint32_t first_stage = stages;
    const unsigned batch_bytes = kBatch * hd;
    auto copy = [&](const Part& b) {
      __syncwarp();  // the stage's last batch has been read
      if (lane == 0) {
        const uint32_t s = stages % R::kStages;
        uint64_t* bar = &full[warp][s];
        if (b.to > b.from) {
          const size_t at = (size_t)b.id * a.page_stride + ((size_t)k.h * kBlock + b.row) * hd;
          mbar_arrive_expect_tx(bar, 2 * batch_bytes);
          bulk_load(my_ring + s * R::kStageBytes, a.kc + at, batch_bytes, bar);
          bulk_load(my_ring + s * R::kStageBytes + R::kValues, a.vc + at, batch_bytes, bar);
        } else {
          mbar_arrive(bar);
        }
      }
      ++stages;
    };
    Part now = part_of(0), next = part_of(1), after = part_of(2);
    fence_proxy_async_smem();
    __syncthreads();  // the last segment's queries and sums have been read

    // head `hi` of the queries, the dims of this lane's keys: scaled to [2^14, 2^15) and split
    float factor;
    {
      float x[HD / 4], top = 0.f;
#pragma unroll
      for (int d = 0; d < HD / 4; d += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const int dim = d / 16 * 64 + 16 * c + d % 16;
        const size_t at = (row0 + hi) * hd + dim;
        if (hi < G && dim < hd) {
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
      resolve(now);
      copy(now);
      resolve(next);
      copy(next);
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

    for (int i = 0; i < n_batches; ++i) {
      resolve(after);
      copy(after);
      const Part last = part_of(i + 3);
      const uint32_t at_stage = first_stage + i;
      if (ok && !(ok = mbar_wait(&full[warp][at_stage % R::kStages], (at_stage / R::kStages) & 1, &gave_up))) {
        gave_up = 1;
        atomicOr(&err, LR_DEVERR_TIMEOUT);
      }
      const uint8_t* stage = my_ring + at_stage % R::kStages * R::kStageBytes;
      const bool masked = now.from > 0 || now.to < kBatch;
      const bool any = now.to > now.from;  // else the stage holds what it held
      float x[kBatch / 8][2];  // scores of tokens 8 n + 2c and 8 n + 2c + 1
      {
        float s[kBatch / 8][4] = {};
#pragma unroll
        for (int y = 0; y < R::kKeyParts; ++y) {
          uint32_t w[kBatch / 8][4];
          const int d = 64 * y + 16 * c;
#pragma unroll
          for (int n = 0; n < kBatch / 8; ++n) {
            load_words(stage + (unsigned)((8 * n + hi) * hd + d), wide, w[n]);
            if (hd < HD) {  // what is behind the row may be a NaN code
              if (d >= hd) w[n][0] = w[n][1] = 0;
              if (d + 8 >= hd) w[n][2] = w[n][3] = 0;
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 q = queries[4 * y + j][lane];
#pragma unroll
            for (int n = 0; n < kBatch / 8; ++n) {
              mma_f16(s[n], q.x, q.y, q.z, q.w, code_pair(w[n][j]), code_pair(w[n][j] >> 16));
            }
          }
        }
#pragma unroll
        for (int n = 0; n < kBatch / 8; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) x[n][y] = fmaf(s[n][2 + y], 1.f / 2048.f, s[n][y]) * (factor * now.ks);
      }
      if (masked) {
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
      if (any) {
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
          const float p0 = exp2_ftz(x[2 * n + y][0] - ref), p1 = exp2_ftz(x[2 * n + y][1] - ref);
          l += p0 + p1;
          split(p0 * share * 32768.f, p1 * share * 32768.f, p[2 * y], p[2 * y + 1]);
        }
        if (!any) continue;
#pragma unroll
        for (int z = 0; z < R::kValueParts; ++z) {
          uint32_t r[4][R::kValueWords];  // of the rows 2c, 2c + 1, 2c + 8 and 2c + 9
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int t = 16 * n + 2 * c + (y & 1) + (y >> 1) * 8;
            load_words(stage + R::kValues + (unsigned)(t * hd + hi * (HD / 8) + 4 * R::kValueWords * z), wide, r[y]);
            if (masked && (t < now.from || t >= now.to)) {
#pragma unroll
              for (int w = 0; w < R::kValueWords; ++w) r[y][w] = 0;
            }
          }
#pragma unroll
          for (int w = 0; w < R::kValueWords; ++w) {  // four dims: pairs of tokens
            const uint32_t a0 = __byte_perm(r[0][w], r[1][w], 0x5140), a1 = __byte_perm(r[0][w], r[1][w], 0x7362);
            const uint32_t b0 = __byte_perm(r[2][w], r[3][w], 0x5140), b1 = __byte_perm(r[2][w], r[3][w], 0x7362);
            float(*to)[4] = acc + 4 * (z * R::kValueWords + w);
            mma_f16(to[0], p[0], p[1], p[2], p[3], code_pair(a0), code_pair(b0));
            mma_f16(to[1], p[0], p[1], p[2], p[3], code_pair(a0 >> 16), code_pair(b0 >> 16));
            mma_f16(to[2], p[0], p[1], p[2], p[3], code_pair(a1), code_pair(b1));
            mma_f16(to[3], p[0], p[1], p[2], p[3], code_pair(a1 >> 16), code_pair(b1 >> 16));
          }
        }
      }
      now = next;
      next = after;
      after = last;
    }
    __syncwarp();  // the ring has been read: the sums take its place
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (c == 0) {
      ml[warp][0][hi] = m;
      ml[warp][1][hi] = l;
    }
    // dim d of a head is at d % (HD / 8) * 8 + d / (HD / 8): no two lanes meet in a bank
    const float scale = unit * (1.f / 32768.f / kSumUnit);
#pragma unroll
    for (int j = 0; j < HD / 8; ++j)
      *reinterpret_cast<float2*>(sums(warp, hi) + 8 * j + 2 * c) =
          make_float2(fmaf(acc[j][2], 1.f / 2048.f, acc[j][0]) * scale, fmaf(acc[j][3], 1.f / 2048.f, acc[j][1]) * scale);
    __syncthreads();
    const bool whole = k.whole();
    float* slot = whole ? nullptr : a.part + (size_t)piece_slot(k.wk, blockIdx.x, k.seg_first) * a.part_stride;
    for (int g = warp; g < G; g += kWarps) {
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
      Joined j{0.f, 0.f, 0.f, 0.f};
      if (whole) {
        j = join_prev(a, row0 + g, top, sum);
        __syncwarp();  // lse may be lse_prev: every lane has read it
        if (a.lse && lane == 0) a.lse[row0 + g] = j.lse();
      } else if (lane == 0) {
        slot[G * hd + g] = top;
        slot[G * hd + 8 + g] = sum;
      }
      for (int at = lane; at < HD; at += 32) {
        const int d = at % 8 * (HD / 8) + at / 8;
        if (d >= hd) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v = fmaf(sums(w, g)[at], f[w], v);
        if (!whole) slot[g * hd + d] = v;
        else if (bf16) ((__nv_bfloat16*)a.o)[(row0 + g) * hd + d] = joined_value<__nv_bfloat16>(a, row0 + g, d, j, v);
        else ((float*)a.o)[(row0 + g) * hd + d] = joined_value<float>(a, row0 + g, d, j, v);
      }
    }
  }
  if (!ok)  // nothing may land in shared memory after the CTA has gone
    for (uint32_t j = stages > R::kStages ? stages - R::kStages : 0; j < stages; ++j)
      mbar_wait_drain(&full[warp][j % R::kStages], (j / R::kStages) & 1, kWaitCycles / 4);
  if (bf16) empty_rows<__nv_bfloat16>(a, blockIdx.x * kWarps + warp, gridDim.x * kWarps);
  else empty_rows<float>(a, blockIdx.x * kWarps + warp, gridDim.x * kWarps);
  if (a.cluster && blockIdx.x == 0) {
    const int bits = check_all(a, tid, NT);
    if (bits) atomicOr(&err, bits);
  }
  __syncthreads();
  if (a.cluster) {
    if (bf16) finish_small<__nv_bfloat16>(a, k.wk.pieces, err);
    else finish_small<float>(a, k.wk.pieces, err);
  } else if (tid == 0) {
    a.cta_err[blockIdx.x] = err;
  }
}

template <int HD>
cudaError_t launch_attn_hd(const Kv8AttnArgs& a, bool bf16, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kv8_attn_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<HD>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kv8_attn_kernel<HD>, dim3(a.n_cta), a.cluster, NT, Ring<HD>::kBytes, st, a, bf16);
}
cudaError_t launch_attn_any(const Kv8AttnArgs& a, bool bf16, cudaStream_t st) {
  return a.hd <= 64 ? launch_attn_hd<64>(a, bf16, st) : a.hd <= 128 ? launch_attn_hd<128>(a, bf16, st) : launch_attn_hd<256>(a, bf16, st);
}

// ------------------------------------------------------------------ joining the pieces
//
// CTA (c, g): query head g of the segment that CTA c of the attention kernel wrote down (none, most of the time).
// Four numbers to a thread, the pieces spread over the rest of the threads, so that all of
// them are under way at once; the order of the sums is fixed by the threads. CTA (0, 0) collects the
// device errors too.

constexpr int JT = 128;
constexpr int kMaxCtas = 1024;

template <typename T>
__global__ void __launch_bounds__(JT, 8) kv8_join_kernel(Kv8AttnArgs a) {
  __shared__ float weight[kMaxCtas], sum_of[kMaxCtas];
  __shared__ float red[2][JT / 32];
  __shared__ __align__(16) float sums[JT * 4];
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hd = a.hd;
  const bool errors = blockIdx.x == 0 && blockIdx.y == 0;
  if (errors && tid == 0) err = 0;
  grid_dependency();
  if (errors) {
    int bits = 0;
    for (int i = tid; i < a.n_cta; i += JT) bits |= __ldcg(a.cta_err + i);
    __syncthreads();
    if (bits) atomicOr(&err, bits);
    __syncthreads();
    if (tid == 0) *a.err = err;
  }
  const int4 said = __ldcg(reinterpret_cast<const int4*>(a.split) + blockIdx.x);
  const Pieces pc{said.x, said.y, said.z, said.w};
  const int n = min(pc.n, min(a.n_cta - pc.c0, kMaxCtas));
  if (n <= 0) return;
  const int cols = hd / 4, groups = JT / cols, col = tid % cols, group = tid / cols;
  const int g = blockIdx.y;
  const size_t row = (size_t)pc.head * a.G + g;
  const int ml = a.G * hd + g;
  auto values = [&](int i) {
    return __ldcg(reinterpret_cast<const float4*>(a.part + (size_t)pc.slot(i) * a.part_stride + g * hd) + col);
  };
  // a thread's first pieces are on their way before their weights are known
  constexpr int kAhead = 8;
  float4 v[kAhead];
#pragma unroll
  for (int x = 0; x < kAhead; ++x) {
    const int i = group + x * groups;
    v[x] = group < groups && i < n ? values(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float prev = prev_lse(a, row);
  float m = -CUDART_INF_F, l = 0.f;
  if (n <= 32) {  // every warp weighs all pieces, a lane for each
    const float* at = a.part + (size_t)pc.slot(min(lane, n - 1)) * a.part_stride + ml;
    const float mi = lane < n ? __ldcg(at) : -CUDART_INF_F, li = lane < n ? __ldcg(at + 8) : 0.f;
    m = warp_max(mi);
    const float w = exp2_ftz(mi - (m == -CUDART_INF_F ? 0.f : m));
    l = warp_sum(w * li);
    if (warp == 0 && lane < n) weight[lane] = w;
    __syncthreads();
  } else {
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
    for (int i = tid; i < n; i += JT) {
      const float w = exp2_ftz(weight[i] - ref);
      weight[i] = w;
      l = fmaf(w, sum_of[i], l);
    }
    l = warp_sum(l);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  }
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
  const Joined j = join_with(m, l, prev);
  __syncthreads();  // lse may be lse_prev, too: every thread has read it
  for (int d = tid; d < hd; d += JT) {
    float acc = 0.f;
    for (int x = 0; x < groups; ++x) acc += sums[x * hd + d];
    ((T*)a.o)[row * hd + d] = joined_value<T>(a, row, d, j, acc);
  }
  if (a.lse && tid == 0) a.lse[row] = j.lse();
}

template <typename T>
cudaError_t launch_attn(const Kv8AttnArgs& a, const Kv8AttnPlan& plan, cudaStream_t st) {
  cudaError_t e;
  if (plan.tensor) {
    CUtensorMap mk, mv;
    if (!kv8_page_map(&mk, a.kc, a) || !kv8_page_map(&mv, a.vc, a)) return cudaErrorInvalidValue;
    e = launch_attn_tc(a, mk, mv, st);
  } else {
    e = launch_attn_any(a, sizeof(T) == 2, st);
  }
  if (e != cudaSuccess || a.cluster) return e;
  return launch_overlapped(kv8_join_kernel<T>, dim3(plan.n_cta, a.G), 1, JT, 0, st, a);
}

}  // namespace
}  // namespace kv8

Kv8AttnPlan plan_kv8_attn(const lr_kv8_pages& kv, int n_q_heads, int sm_count) {
  Kv8AttnPlan p{};
  const int G = n_q_heads / kv.n_kv_heads;
  const long long most = (long long)kv.batch * kv.n_kv_heads * ((kv.max_pages + 1) / 2 + kv8::kSegmentUnits);  // units
  p.tensor = kv.dtype == LR_BF16 && kv.head_dim == 128;
  p.n_cta = (int)std::max(1LL, std::min<long long>(most, std::min((p.tensor ? 2 : kv8::resident(kv.head_dim)) * sm_count, kv8::kMaxCtas)));
  p.cluster = kv8::small_cluster(kv.batch, kv.n_kv_heads, kv.max_pages, p.tensor);
  if (p.cluster) p.n_cta = kv.batch * kv.n_kv_heads * p.cluster;
  p.part_stride = G * kv.head_dim + 16;
  p.split_off = 256;
  p.cta_err_off = p.split_off + (size_t)p.n_cta * sizeof(kv8::Pieces);
  p.part_off = (p.cta_err_off + (size_t)p.n_cta * sizeof(int) + 255) & ~(size_t)255;
  p.ws_bytes = p.part_off + (((size_t)2 * p.n_cta * p.part_stride * sizeof(float) + 255) & ~(size_t)255);
  return p;
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, const Kv8AttnPlan& plan, lr_dtype dt, cudaStream_t st) {
  if (a.B == 0) return cudaMemsetAsync(a.err, 0, 256, st);
  return dt == LR_BF16 ? kv8::launch_attn<__nv_bfloat16>(a, plan, st) : kv8::launch_attn<float>(a, plan, st);
}

}  // namespace lr
