// Decode attention over the 8-bit paged cache: the choice of the kernel, and the kernel on the CUDA
// cores for every storage type, head_dim and group size the entry point takes.
//
// One CTA of 128 threads walks its share of the batch's tiles (kv8_common.cuh). Warp w takes the 32 tokens from
// 32 w on of every tile, by itself: its own maximum, sum and accumulators, joined with the other warps' at the
// segment's end. A row is read by kLanes lanes, 16 bytes (8 for more than four query heads) each, so a lane has
// kDims dims of q of every query head in registers, and of the accumulators. Scores are summed across the lanes
// by exchanging heads, so each lane ends up with one head's; the weights go through shared memory to the lanes
// that need all heads'. Values of a batch and the keys of the next are on their way while scores and
// weights are worked out.
//
// Everything is fp32, two multiply-adds to an instruction. Bound by its instructions: about one per 7 bytes
// with four query heads.
#include <algorithm>

#include "kv8_common.cuh"

namespace lr {
namespace kv8 {
namespace {

constexpr int NT = 128, kWarps = NT / 32;
static_assert(kTileTokens == NT, "32 tokens of a tile to a warp");

// MG: query heads the registers hold; kLanes: lanes that share a row (head_dim <= kLanes * kDims).
template <int MG, int kLanes>
struct Shape {
  static constexpr int kDims = 64 / MG;
  static constexpr int kTokens = 32 / kLanes;                                    // of a step
  static constexpr int kSteps = kLanes < 128 / kDims ? kLanes : 128 / kDims;     // of a batch: 128 bytes a lane at most
  static constexpr int kBatch = kSteps * kTokens, kBatches = 32 / kBatch;
  static constexpr int kWords = kDims / 4;
};

// This lane's part of a row: `n` bytes of it (a multiple of 8) are there, the rest is 0.
template <int kWords>
__device__ __forceinline__ void load_row(const uint8_t* at, int n, bool wide, uint32_t (&w)[kWords]) {
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[i] = 0;
  if (kWords == 4 && wide && n >= 16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < kWords; i += 2)
    if (n > 4 * i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(at + 4 * i));
      w[i] = v.x;
      w[i + 1] = v.y;
    }
}
__device__ __forceinline__ Two code_pair(uint32_t codes) {
  const float2 v = e4m3x2_value(codes & 0xffffu);
  return Two(v.x, v.y);
}

template <int MG, int kLanes>
__global__ void __launch_bounds__(NT, 2) kv8_attn_kernel(Kv8AttnArgs a, bool bf16) {
  using S = Shape<MG, kLanes>;
  __shared__ long long scratch[NT + 4];
  __shared__ __align__(16) float ps[kWarps][S::kBatch][MG];  // weight times value scale
  __shared__ __align__(16) float olds[kWarps][MG];
  __shared__ float ml[kWarps][2][MG];
  __shared__ __align__(16) float sums[kWarps][MG][256];
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hd = a.hd, G = a.G;
  const int part = lane % kLanes, tg = lane / kLanes, d0 = part * S::kDims;
  const int n_dims = max(0, min(S::kDims, hd - d0));
  const bool wide = hd % 16 == 0;
  // the head whose scores this lane ends up with
  const int my_g = (part & 1) * (MG / 2) + ((part >> 1) & 1) * (MG / 4) + (MG == 8 ? (part >> 2) & 1 : 0);
  if (tid == 0) err = 0;
  grid_dependency();
  Walk k(a, find_work<NT>(a, scratch));
  auto number = [&](const void* p, size_t i) {
    return bf16 ? to_f32(((const __nv_bfloat16*)p)[i]) : ((const float*)p)[i];
  };
  while (k.next()) {
    const int* table = a.table + (size_t)k.b * a.max_pages;
    const size_t row0 = ((size_t)k.b * a.Hkv + k.h) * G;
    Two q[MG][S::kDims / 2];
#pragma unroll
    for (int g = 0; g < MG; ++g)
#pragma unroll
      for (int d = 0; d < S::kDims; d += 2) {
        const bool there = g < G && d < n_dims;
        const size_t at = (row0 + g) * hd + d0 + d;
        q[g][d / 2] = there ? Two(number(a.q, at) * a.scale, number(a.q, at + 1) * a.scale) : Two(0.f, 0.f);
      }
    Two acc[MG][S::kDims / 2];
#pragma unroll
    for (int g = 0; g < MG; ++g)
#pragma unroll
      for (int d = 0; d < S::kDims / 2; ++d) acc[g][d] = Two(0.f, 0.f);
    float m = -CUDART_INF_F, l = 0.f;  // of head my_g

    // batch i of the range is batch i % kBatches of the warp's tokens of tile tile0 + i / kBatches
    const int n_batches = (k.tile1 - k.tile0) * S::kBatches;
    auto first_token = [&](int i) {
      return (k.sp.page0 + (k.tile0 + i / S::kBatches) * kTilePages) * kBlock + warp * 32 + i % S::kBatches * S::kBatch;
    };
    auto page_of = [&](int i) {  // page of a batch, -1: none
      if (i >= n_batches) return -1;
      const int p = first_token(i) / kBlock;
      if (p * kBlock >= k.sp.n) return -1;
      int id = __ldg(table + p);
      if ((unsigned)id >= (unsigned)a.n_pages) {
        if (lane == 0) atomicOr(&err, LR_DEVERR_PAGE);
        id = -1;
      }
      return id;
    };
    // the tokens of a batch that are attended, counted from its first: [from, to)
    struct Part {
      int id, from, to;
    };
    auto part_of = [&](int i) {
      Part b{page_of(i), 0, 0};
      if (b.id >= 0) {
        const int t = first_token(i);
        b.from = max(0, k.sp.lo - t);
        b.to = min(S::kBatch, k.sp.n - t);
      }
      return b;
    };
    const unsigned step_bytes = S::kTokens * hd;
    auto load = [&](const uint8_t* codes, int i, const Part& b, uint32_t (&w)[S::kSteps][S::kWords]) {
      if (b.to <= b.from) {
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
          for (int x = 0; x < S::kWords; ++x) w[s][x] = 0;
        return;
      }
      const uint8_t* at = codes + (size_t)b.id * a.page_stride + (size_t)k.h * kBlock * hd +
                          (unsigned)((first_token(i) % kBlock + tg) * hd + d0);
      if (b.from == 0 && b.to == S::kBatch) {
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s) load_row(at + s * step_bytes, n_dims, wide, w[s]);
      } else {
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s) {
          const int t = s * S::kTokens + tg;
          load_row(at + s * step_bytes, t >= b.from && t < b.to ? n_dims : 0, wide, w[s]);
        }
      }
    };
    Part now = part_of(0), next = part_of(1);
    uint32_t kw[S::kSteps][S::kWords], vw[S::kSteps][S::kWords];
    load(a.kc, 0, now, kw);
    for (int i = 0; i < n_batches; ++i) {
      load(a.vc, i, now, vw);
      float ks = 0.f, vs = 0.f;
      if (now.id >= 0) {
        ks = __ldg(a.ks + (size_t)now.id * a.Hkv + k.h);
        vs = __ldg(a.vs + (size_t)now.id * a.Hkv + k.h);
      }
      float x[S::kSteps];
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) {
        Two dot[MG];
#pragma unroll
        for (int g = 0; g < MG; ++g) dot[g] = Two(0.f, 0.f);
#pragma unroll
        for (int d = 0; d < S::kDims / 2; ++d) {
          const Two v = code_pair(kw[s][d / 2] >> (d % 2 * 16));
#pragma unroll
          for (int g = 0; g < MG; ++g) dot[g] = fma(v, q[g][d], dot[g]);
        }
        float v[MG];
#pragma unroll
        for (int g = 0; g < MG; ++g) {
          float lo, hi;
          dot[g].get(lo, hi);
          v[g] = lo + hi;
        }
#pragma unroll
        for (int off = 1, n = MG; off < kLanes; off *= 2) {
          if (n > 1) {  // this lane keeps half of the heads and gives the other half away
            n /= 2;
            const bool upper = part & off;
#pragma unroll
            for (int g = 0; g < n; ++g) {
              const float give = upper ? v[g] : v[n + g], keep = upper ? v[n + g] : v[g];
              v[g] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
          } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
          }
        }
        x[s] = v[0] * ks;
      }
      if (now.from > 0 || now.to < S::kBatch) {
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s) {
          const int t = s * S::kTokens + tg;
          if (t < now.from || t >= now.to) x[s] = -CUDART_INF_F;
        }
      }
      load(a.kc, i + 1, next, kw);
      const Part after = part_of(i + 2);

      float top = x[0];
#pragma unroll
      for (int s = 1; s < S::kSteps; ++s) top = fmaxf(top, x[s]);
#pragma unroll
      for (int off = kLanes; off < 32; off *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      top = fmaxf(top, m);
      const float ref = top == -CUDART_INF_F ? 0.f : top, old = exp2f(m - ref);
      m = top;
      l *= old;
      __syncwarp();  // the last batch's weights have been read
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) {
        const float p = exp2f(x[s] - ref);
        l += p;
        if (part < MG) ps[warp][s * S::kTokens + tg][my_g] = x[s] == -CUDART_INF_F ? 0.f : p * vs;
      }
      if (part < MG && tg == 0) olds[warp][my_g] = old;
      __syncwarp();
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        const Two f(olds[warp][g], olds[warp][g]);
#pragma unroll
        for (int d = 0; d < S::kDims / 2; ++d) acc[g][d] = mul(acc[g][d], f);
      }
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) {
        Two w[MG];
#pragma unroll
        for (int g = 0; g < MG; g += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&ps[warp][s * S::kTokens + tg][g]);
          w[g] = Two(f.x, f.x);
          w[g + 1] = Two(f.y, f.y);
          w[g + 2] = Two(f.z, f.z);
          w[g + 3] = Two(f.w, f.w);
        }
#pragma unroll
        for (int d = 0; d < S::kDims / 2; ++d) {
          const Two v = code_pair(vw[s][d / 2] >> (d % 2 * 16));
#pragma unroll
          for (int g = 0; g < MG; ++g) acc[g][d] = fma(v, w[g], acc[g][d]);
        }
      }
      now = next;
      next = after;
    }
    // the token groups of the warp, then the warps
#pragma unroll
    for (int off = kLanes; off < 32; off *= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
    __syncthreads();
    if (part < MG && tg == 0) {
      ml[warp][0][my_g] = m;
      ml[warp][1][my_g] = l;
    }
#pragma unroll
    for (int g = 0; g < MG; ++g)
#pragma unroll
      for (int d = 0; d < S::kDims / 2; ++d) {
        float lo, hi;
        acc[g][d].get(lo, hi);
#pragma unroll
        for (int off = kLanes; off < 32; off *= 2) {
          lo += __shfl_xor_sync(0xffffffffu, lo, off);
          hi += __shfl_xor_sync(0xffffffffu, hi, off);
        }
        if (tg == 0 && 2 * d < n_dims) {
          sums[warp][g][d0 + 2 * d] = lo;
          sums[warp][g][d0 + 2 * d + 1] = hi;
        }
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

void (*attn_kernel(int G, int hd))(Kv8AttnArgs, bool) {
  if (G <= 4) return hd <= 64 ? kv8_attn_kernel<4, 4> : hd <= 128 ? kv8_attn_kernel<4, 8> : kv8_attn_kernel<4, 16>;
  return hd <= 64 ? kv8_attn_kernel<8, 8> : hd <= 128 ? kv8_attn_kernel<8, 16> : kv8_attn_kernel<8, 32>;
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
    e = launch_overlapped(attn_kernel(a.G, a.hd), dim3(plan.n_cta), NT, 0, st, a, sizeof(T) == 2);
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
  p.n_cta = (int)std::max(1LL, std::min<long long>(most, std::min(2 * sm_count, kv8::kMaxCtas)));
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
