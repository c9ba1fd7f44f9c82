// Decode attention over the 8-bit paged cache: the choice of the kernel, and the kernel on the CUDA
// cores for every storage type, head_dim and group size the entry point takes.
//
// One CTA of 128 threads walks its share of the batch's tiles (kv8_common.cuh), two pages of 64
// tokens at a time: thread t holds the score of token t for the G query heads of the KV head
// (q.k over the codes, times the page's key scale), the running maximum of the online softmax
// moves, and then thread d sums p v over the tokens for column d. Everything is fp32. Bound by
// its own instructions (a conversion and G multiply-adds per cached number).
#include <algorithm>

#include "kv8_common.cuh"

namespace lr {
namespace kv8 {
namespace {

constexpr int NT = kTileTokens;
static_assert(NT == 128, "thread t owns token t of a tile");

// Eight codes as fp32.
__device__ __forceinline__ void codes8(uint2 u, float (&v)[8]) {
  float2 f;
  f = e4m3x2_value(u.x & 0xffffu); v[0] = f.x; v[1] = f.y;
  f = e4m3x2_value(u.x >> 16);     v[2] = f.x; v[3] = f.y;
  f = e4m3x2_value(u.y & 0xffffu); v[4] = f.x; v[5] = f.y;
  f = e4m3x2_value(u.y >> 16);     v[6] = f.x; v[7] = f.y;
}

template <typename T, int MD>  // MD: columns of a thread (head_dim <= 128 MD)
__global__ void __launch_bounds__(NT) kv8_attn_kernel(Kv8AttnArgs a) {
  __shared__ long long scratch[NT + 4];
  __shared__ __align__(16) float qs[256][8];   // q * scale, head fastest
  __shared__ __align__(16) float ps[NT][8];    // p * value scale of the tile's tokens
  __shared__ float red[4][8];
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hd = a.hd, G = a.G;
  if (tid == 0) err = 0;
  grid_dependency();
  Walk k(a, find_work<NT>(a, scratch));
  while (k.next()) {
    const int* table = a.table + (size_t)k.b * a.max_pages;
    const size_t row0 = ((size_t)k.b * a.Hkv + k.h) * G;
    __syncthreads();
    for (int i = tid; i < 8 * hd; i += NT) {
      const int g = i / hd, d = i % hd;
      qs[d][g] = g < G ? to_f32(((const T*)a.q)[(row0 + g) * hd + d]) * a.scale : 0.f;
    }
    __syncthreads();
    float m[8], l[8], acc[MD][8];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      m[g] = -CUDART_INF_F;
      l[g] = 0.f;
#pragma unroll
      for (int x = 0; x < MD; ++x) acc[x][g] = 0.f;
    }
    for (int i = k.tile0; i < k.tile1; ++i) {
      const int p0 = k.sp.page0 + i * kTilePages;  // pages p0, p0 + 1 of the sequence
      const int t = p0 * kBlock + tid;
      int id[kTilePages];
#pragma unroll
      for (int x = 0; x < kTilePages; ++x) {
        id[x] = -1;
        if ((p0 + x) * kBlock < k.sp.n) {
          id[x] = __ldg(table + p0 + x);
          if ((unsigned)id[x] >= (unsigned)a.n_pages) {
            id[x] = -1;
            if (tid == 0) err |= LR_DEVERR_PAGE;
          }
        }
      }
      const int pg = tid < kBlock ? id[0] : id[1];
      const bool seen = t >= k.sp.lo && t < k.sp.n && pg >= 0;
      float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      float vs = 0.f;
      if (seen) {
        const uint8_t* row = a.kc + (size_t)pg * a.page_stride + ((size_t)k.h * kBlock + (tid & (kBlock - 1))) * hd;
        for (int d = 0; d < hd; d += 8) {
          float kv[8];
          codes8(__ldg(reinterpret_cast<const uint2*>(row + d)), kv);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 q0 = *reinterpret_cast<const float4*>(&qs[d + e][0]);
            s[0] = fmaf(kv[e], q0.x, s[0]);
            s[1] = fmaf(kv[e], q0.y, s[1]);
            s[2] = fmaf(kv[e], q0.z, s[2]);
            s[3] = fmaf(kv[e], q0.w, s[3]);
            if (G > 4) {
              const float4 q1 = *reinterpret_cast<const float4*>(&qs[d + e][4]);
              s[4] = fmaf(kv[e], q1.x, s[4]);
              s[5] = fmaf(kv[e], q1.y, s[5]);
              s[6] = fmaf(kv[e], q1.z, s[6]);
              s[7] = fmaf(kv[e], q1.w, s[7]);
            }
          }
        }
        const float ks = __ldg(a.ks + (size_t)pg * a.Hkv + k.h);
        vs = __ldg(a.vs + (size_t)pg * a.Hkv + k.h);
#pragma unroll
        for (int g = 0; g < 8; ++g) s[g] *= ks;
      }
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (!seen) s[g] = -CUDART_INF_F;
        const float top = warp_max(s[g]);
        if (lane == 0) red[warp][g] = top;
      }
      __syncthreads();
      float old[8];
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float top = fmaxf(fmaxf(fmaxf(red[0][g], red[1][g]), fmaxf(red[2][g], red[3][g])), m[g]);
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        old[g] = exp2f(m[g] - ref);
        const float p = exp2f(s[g] - ref);
        l[g] = fmaf(l[g], old[g], p);
        ps[tid][g] = seen ? p * vs : 0.f;
        m[g] = top;
      }
      __syncthreads();
      // rows [r0, r1) of the tile are attended; rows of pages that are left out are not read
      const int r0 = max(0, k.sp.lo - p0 * kBlock), r1 = min(kTileTokens, k.sp.n - p0 * kBlock);
#pragma unroll
      for (int x = 0; x < MD; ++x) {
        const int d = tid + x * NT;
        if (d < hd) {
#pragma unroll
          for (int g = 0; g < 8; ++g) acc[x][g] *= old[g];
#pragma unroll
          for (int half = 0; half < kTilePages; ++half) {
            if (id[half] < 0) continue;
            const uint8_t* col = a.vc + (size_t)id[half] * a.page_stride + (size_t)k.h * kBlock * hd + d;
            const int b0 = half * kBlock;
#pragma unroll 8
            for (int r = max(r0, b0); r < min(r1, b0 + kBlock); ++r) {
              const float v = e4m3x2_value(__ldg(col + (size_t)(r - b0) * hd)).x;
              const float4 w0 = *reinterpret_cast<const float4*>(&ps[r][0]);
              acc[x][0] = fmaf(w0.x, v, acc[x][0]);
              acc[x][1] = fmaf(w0.y, v, acc[x][1]);
              acc[x][2] = fmaf(w0.z, v, acc[x][2]);
              acc[x][3] = fmaf(w0.w, v, acc[x][3]);
              if (G > 4) {
                const float4 w1 = *reinterpret_cast<const float4*>(&ps[r][4]);
                acc[x][4] = fmaf(w1.x, v, acc[x][4]);
                acc[x][5] = fmaf(w1.y, v, acc[x][5]);
                acc[x][6] = fmaf(w1.z, v, acc[x][6]);
                acc[x][7] = fmaf(w1.w, v, acc[x][7]);
              }
            }
          }
        }
      }
    }
    // the sums of p are spread over the threads
    __syncthreads();
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const float x = warp_sum(l[g]);
      if (lane == 0) red[warp][g] = x;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < 8; ++g) l[g] = (red[0][g] + red[1][g]) + (red[2][g] + red[3][g]);

    if (!k.whole()) {
      float* slot = a.part + (size_t)piece_slot(k.wk, k.seg_first) * a.part_stride;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (g >= G) break;
#pragma unroll
        for (int x = 0; x < MD; ++x)
          if (tid + x * NT < hd) slot[g * hd + tid + x * NT] = acc[x][g];
        if (tid == 0) {
          slot[G * hd + g] = m[g];
          slot[G * hd + 8 + g] = l[g];
        }
      }
    } else {
      Joined j[8];
#pragma unroll
      for (int g = 0; g < 8; ++g)
        if (g < G) j[g] = join_prev(a, row0 + g, m[g], l[g]);
      __syncthreads();  // lse may be lse_prev: every thread has read it
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (g >= G) break;
#pragma unroll
        for (int x = 0; x < MD; ++x) {
          const int d = tid + x * NT;
          if (d < hd) ((T*)a.o)[(row0 + g) * hd + d] = joined_value<T>(a, row0 + g, d, j[g], acc[x][g]);
        }
        if (a.lse && tid == 0) a.lse[row0 + g] = j[g].lse;
      }
    }
  }
  if (tid == 0) a.cta_err[blockIdx.x] = err;
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
    e = launch_overlapped(a.hd <= 128 ? kv8_attn_kernel<T, 1> : kv8_attn_kernel<T, 2>, dim3(plan.n_cta), NT, 0, st, a);
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
