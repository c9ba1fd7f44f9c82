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
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hd = a.hd, G = a.G;
  empty_sequences<T>(a, tid, NT);
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
            if (tid == 0) flag_error(a.err, LR_DEVERR_PAGE);
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

    bool write = k.whole();
    if (!write) {
      const Pieces pc = pieces_of(k);
      float* slot = a.part + (size_t)pc.slot(blockIdx.x - pc.c0) * a.part_stride;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (g >= G) break;
#pragma unroll
        for (int x = 0; x < MD; ++x)
          if (tid + x * NT < hd) __stcg(slot + g * hd + tid + x * NT, acc[x][g]);
        if (tid == 0) {
          __stcg(slot + G * hd + g, m[g]);
          __stcg(slot + G * hd + 8 + g, l[g]);
        }
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) last = atomicAdd(a.count + pc.c0, 1u) == (unsigned)pc.n - 1;
      __syncthreads();
      write = last;
      if (write) {
        __threadfence();
#pragma unroll
        for (int x = 0; x < MD; ++x) join_pieces<8>(a, pc, tid + x * NT, tid + x * NT < hd, acc[x], m, l);
      }
    }
    if (write) {
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
}

}  // namespace
}  // namespace kv8

Kv8AttnPlan plan_kv8_attn(const lr_kv8_pages& kv, int n_q_heads, int sm_count) {
  Kv8AttnPlan p{};
  const int G = n_q_heads / kv.n_kv_heads;
  const long long most = (long long)kv.batch * kv.n_kv_heads * ((kv.max_pages + 1) / 2);  // tiles
  p.tensor = kv.dtype == LR_BF16 && kv.head_dim == 128;
  p.n_cta = (int)std::max(1LL, std::min(most, 2LL * sm_count));
  p.part_stride = G * kv.head_dim + 16;
  p.count_off = 256;
  p.part_off = (256 + (size_t)p.n_cta * sizeof(unsigned) + 255) & ~(size_t)255;
  p.ws_bytes = p.part_off + (((size_t)2 * p.n_cta * p.part_stride * sizeof(float) + 255) & ~(size_t)255);
  return p;
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, const Kv8AttnPlan& plan, lr_dtype dt, cudaStream_t st) {
  const cudaError_t e = cudaMemsetAsync(a.err, 0, plan.part_off, st);  // error word and piece counts
  if (e != cudaSuccess || a.B == 0) return e;
  if (plan.tensor) {
    CUtensorMap mk, mv;
    if (!kv8_page_map(&mk, a.kc, a) || !kv8_page_map(&mv, a.vc, a)) return cudaErrorInvalidValue;
    return kv8::launch_attn_tc(a, mk, mv, st);
  }
  if (dt == LR_BF16) {
    if (a.hd <= 128) kv8::kv8_attn_kernel<__nv_bfloat16, 1><<<plan.n_cta, kv8::NT, 0, st>>>(a);
    else kv8::kv8_attn_kernel<__nv_bfloat16, 2><<<plan.n_cta, kv8::NT, 0, st>>>(a);
  } else {
    if (a.hd <= 128) kv8::kv8_attn_kernel<float, 1><<<plan.n_cta, kv8::NT, 0, st>>>(a);
    else kv8::kv8_attn_kernel<float, 2><<<plan.n_cta, kv8::NT, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace lr
