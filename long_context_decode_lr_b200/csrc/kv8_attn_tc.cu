// Decode attention over the 8-bit paged cache on the tensor cores: bf16, head_dim 128, up to 8 query
// heads per KV head.
//
// The codes go from HBM into the matrix units as they are (tcgen05, kind::f8f6f4); a conversion to
// a wider type would cost more issue slots than the bytes cost time. What multiplies them is
// therefore written as a sum of e4m3 numbers too, each term taking four more bits of what the ones
// before leave over:
//   q = 2^e (q1 + q2 / 32)              exact for a bf16 number down to 2^-15 of the head's largest
//                                       (below that off by 2^-22 of it at most);
//   p = (p1 + p2 / 32 + p3 / 1024) / 256, relative error 2^-14 at most for p >= 2^-14, 2^-28 absolute
//                                       below, p relative to the largest of the tile.
// Every term is a column of its own, so a tile's products are
//   S  [128 tokens x 16]     = K q1 | K q2             (M 128, N 16, K 128)
//   O' [128 dims x 3 heads]  = V^T p1 | V^T p2 | V^T p3 (M 128, N 16 or 32, K 64) for each of the two pages,
// K as the K-major and V as the M-major operand, straight from the page rows (128 bytes, 128-byte
// swizzle). Thread t is token t in the softmax and dim t in the sum over the tiles: the maximum
// (one per head and tile, a warp reduction and four numbers in shared memory) is the only thing the
// threads exchange. Scales and the rescaling between tiles are fp32 factors in registers.
//
// Persistent, two CTAs per SM on an even share of the tiles (kv8_common.cuh): warps 0-3 softmax and
// sums, warp 4 loads (TMA, three stages of 32 KB), warp 5 issues the products. Bound by HBM: 256 bytes per token and KV head against about 2 cycles of the tensor pipe.
#include <algorithm>

#include "kv8_common.cuh"
#include "sm100.cuh"

namespace lr {
namespace kv8 {
namespace {

using namespace sm100;

constexpr int kHd = 128;
constexpr int kThreads = 192, kSoft = 128;
constexpr int kStages = 3, kQBufs = 4;
constexpr int kPageBytes = kBlock * kHd;
constexpr int kTileBytes = kTilePages * kPageBytes;  // of K, and of V
constexpr int kTmemCols = 128, kColS = 0, kColO = 32;

struct Meta {  // of a stage's two pages
  float ks[2], vs[2];
  int ok[2];
  int pad[2];
};

struct Layout {
  static constexpr int kOffRing = 0;  // stages of K, V
  static constexpr int kOffQ = kStages * 2 * kTileBytes;  // [kQBufs] of 16 rows of 128 bytes
  static constexpr int kOffP = kOffQ + kQBufs * 2048;     // [2][128 tokens][16 bytes]
  static constexpr int kOffMeta = kOffP + 4096;
  static constexpr int kOffMax = kOffMeta + kStages * (int)sizeof(Meta);  // [2][4 warps][8]
  static constexpr int kOffQs = kOffMax + 2 * 4 * 8 * 4;                  // [kQBufs][8]
  static constexpr int kOffBar = kOffQs + kQBufs * 32;
  static constexpr int kOffMisc = kOffBar + 192;
  static constexpr int kOffScratch = kOffMisc + 16;                       // find_work
  static constexpr int kBytes = kOffScratch + (kThreads + 4) * 8;
};
static_assert(Layout::kOffMeta % 16 == 0 && Layout::kOffBar % 8 == 0 && Layout::kOffScratch % 8 == 0, "alignment");
static_assert(2 * (Layout::kBytes + 1024) <= 227 * 1024, "two CTAs per SM");

enum Bar { K_FULL = 0, V_FULL = K_FULL + kStages, EMPTY = V_FULL + kStages, Q_READY = EMPTY + kStages, Q_FREE = Q_READY + kQBufs, S_FULL = Q_FREE + kQBufs, P_READY, O_FULL, DRAIN, kBars };
static_assert(kBars * 8 <= 192, "barriers");

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory"); }

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Operand without swizzle, M/N contiguous: 16 numbers of 8 K-rows are 128 bytes, K groups follow every
// `k_bytes`, blocks of 16 along N every `n_bytes`.
__device__ __forceinline__ uint64_t plain_mn_desc(uint32_t saddr, uint32_t k_bytes, uint32_t n_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(k_bytes >> 4) << 16) | ((uint64_t)(n_bytes >> 4) << 32) | (1ull << 46);
}

struct Shared {
  uint8_t* base;
  __device__ uint64_t* bar(int i) const { return reinterpret_cast<uint64_t*>(base + Layout::kOffBar) + i; }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(base + Layout::kOffMisc + 4); }
  __device__ int* err() const { return reinterpret_cast<int*>(base + Layout::kOffMisc + 8); }
  __device__ Meta* meta(int s) const { return reinterpret_cast<Meta*>(base + Layout::kOffMeta) + s; }
  __device__ uint8_t* queries(int i) const { return base + Layout::kOffQ + i * 2048; }
  __device__ float* factors(int i) const { return reinterpret_cast<float*>(base + Layout::kOffQs) + i * 8; }
  __device__ uint8_t* keys(int s) const { return base + Layout::kOffRing + s * 2 * kTileBytes; }
  __device__ uint8_t* values(int s) const { return keys(s) + kTileBytes; }
};

__device__ __forceinline__ void give_up(const Shared& sh) {
  *sh.abort_flag() = 1;
  atomicOr(sh.err(), LR_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------ loads (warp 4)

// The query heads as two e4m3 terms each: rows g and 8 + g of the K-major operand, and the factors
// that scores are multiplied by. A head with an infinite number gets a NaN factor. u: dims 4 lane .. 4 lane + 3 of
// every head, bf16.
template <int MG>
__device__ __forceinline__ void write_q(const Kv8AttnArgs& a, const uint2 (&u)[MG], uint8_t* q, float* factor) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int g = 0; g < MG; ++g) {
    if (g >= a.G) break;
    float x[4] = {__uint_as_float(u[g].x << 16), __uint_as_float(u[g].x & 0xffff0000u), __uint_as_float(u[g].y << 16),
                  __uint_as_float(u[g].y & 0xffff0000u)};
    const float top = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    // 2^e with top / 2^e in [128, 256); tiny heads share the smallest e, whose inverse is finite
    const int e = max((int)(__float_as_uint(top) >> 23) - 127 - 7, -120);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= inv;
    const uint32_t t1 = e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16);
    const float2 v0 = e4m3x2_value(t1 & 0xffffu), v1 = e4m3x2_value(t1 >> 16);
    const uint32_t t2 = e4m3x2((x[0] - v0.x) * 32.f, (x[1] - v0.y) * 32.f) |
                        (e4m3x2((x[2] - v1.x) * 32.f, (x[3] - v1.y) * 32.f) << 16);
    const int at = (((lane >> 2) ^ (g & 7)) << 4) + (lane & 3) * 4;  // 128-byte swizzle
    *reinterpret_cast<uint32_t*>(q + g * 128 + at) = t1;
    *reinterpret_cast<uint32_t*>(q + (8 + g) * 128 + at) = t2;
    if (lane == 0) factor[g] = top < CUDART_INF_F ? __uint_as_float((uint32_t)(127 + e) << 23) * a.scale : CUDART_NAN_F;
  }
}

// A batch is 32 pages: lane i has the id and the scales of page i. The next batch's ids are under
// way while one is loaded. A segment's queries follow its first tile, up to four segments ahead of the
// products, so that short sequences do not wait for them.
template <int MG>
__device__ void load_tiles(const Kv8AttnArgs& a, const Shared& sh, const CUtensorMap* mk, const CUtensorMap* mv, const Work& wk) {
  const int lane = threadIdx.x & 31;
  Walk k(a, wk);
  uint32_t it = 0, seg = 0;
  bool ok = true;
  for (; ok && k.next(); ++seg) {
    uint2 q[MG];
#pragma unroll
    for (int g = 0; g < MG; ++g)
      if (g < a.G)
        q[g] = __ldg(reinterpret_cast<const uint2*>((const __nv_bfloat16*)a.q + (((size_t)k.b * a.Hkv + k.h) * a.G + g) * kHd) + lane);
    const int* table = a.table + (size_t)k.b * a.max_pages;
    const int page_end = min(k.sp.page0 + k.tile1 * kTilePages, (k.sp.n + kBlock - 1) / kBlock);
    auto page_id = [&](int p) { return p < page_end ? __ldg(table + p) : -1; };
    int p0 = k.sp.page0 + k.tile0 * kTilePages;  // first page of the batch
    int id_next = page_id(p0 + lane);
    for (int i = k.tile0; ok && i < k.tile1; p0 += 32) {
      int id = id_next;
      id_next = page_id(p0 + 32 + lane);
      float ks = 0.f, vs = 0.f;
      if ((unsigned)id < (unsigned)a.n_pages) {
        ks = __ldg(a.ks + (size_t)id * a.Hkv + k.h);
        vs = __ldg(a.vs + (size_t)id * a.Hkv + k.h);
      } else {
        if (p0 + lane < page_end) atomicOr(sh.err(), LR_DEVERR_PAGE);
        id = -1;
      }
      for (int j = 0; j < 32 && i < k.tile1; j += kTilePages, ++i, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(sh.bar(EMPTY + s), ph ^ 1, sh.abort_flag())))) break;
        const int id0 = __shfl_sync(0xffffffffu, id, j), id1 = __shfl_sync(0xffffffffu, id, j + 1);
        if (lane == 0) {
          const uint32_t bytes = ((id0 >= 0) + (id1 >= 0)) * kPageBytes;
          mbar_arrive_expect_tx(sh.bar(K_FULL + s), bytes);
          if (id0 >= 0) tma_load_3d(sh.keys(s), mk, sh.bar(K_FULL + s), 0, k.h * kBlock, id0);
          if (id1 >= 0) tma_load_3d(sh.keys(s) + kPageBytes, mk, sh.bar(K_FULL + s), 0, k.h * kBlock, id1);
          mbar_arrive_expect_tx(sh.bar(V_FULL + s), bytes);
          if (id0 >= 0) tma_load_3d(sh.values(s), mv, sh.bar(V_FULL + s), 0, k.h * kBlock, id0);
          if (id1 >= 0) tma_load_3d(sh.values(s) + kPageBytes, mv, sh.bar(V_FULL + s), 0, k.h * kBlock, id1);
        }
        Meta m;
        m.ks[0] = __shfl_sync(0xffffffffu, ks, j);
        m.ks[1] = __shfl_sync(0xffffffffu, ks, j + 1);
        m.vs[0] = __shfl_sync(0xffffffffu, vs, j);
        m.vs[1] = __shfl_sync(0xffffffffu, vs, j + 1);
        if (lane == 0) {
          m.ok[0] = id0 >= 0;
          m.ok[1] = id1 >= 0;
          *sh.meta(s) = m;
          mbar_arrive(sh.bar(K_FULL + s));
        }
        if (i == k.tile0) {
          const uint32_t buf = seg % kQBufs;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(sh.bar(Q_FREE + buf), ((seg / kQBufs) & 1) ^ 1, sh.abort_flag())))) {
            ++it;  // its loads are under way
            break;
          }
          write_q<MG>(a, q, sh.queries(buf), sh.factors(buf));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(sh.bar(Q_READY + buf));
        }
      }
    }
  }
  if (!ok && lane == 0) {
    give_up(sh);
    // nothing may land in shared memory after the CTA has gone
    for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j) {
      mbar_wait_drain(sh.bar(K_FULL + j % kStages), (j / kStages) & 1, kWaitCycles / 4);
      mbar_wait_drain(sh.bar(V_FULL + j % kStages), (j / kStages) & 1, kWaitCycles / 4);
    }
  }
}

// ------------------------------------------------------------------ products (one thread of warp 5)
template <int MG>
__device__ void issue_products(const Kv8AttnArgs& a, const Shared& sh, const Work& wk, uint32_t tmem) {
  constexpr int NP = MG <= 4 ? 16 : 32;
  const uint32_t id_s = idesc_e4m3_f32(128, 16, false, false), id_o = idesc_e4m3_f32(128, NP, true, true);
  const uint32_t p = smem_u32(sh.base + Layout::kOffP);
  Walk k(a, wk);
  uint32_t it = 0, seg = 0;
  bool ok = true;
  for (; ok && k.next(); ++seg) {
    const uint32_t buf = seg % kQBufs, q = smem_u32(sh.queries(buf));
    ok = mbar_wait(sh.bar(Q_READY + buf), (seg / kQBufs) & 1, sh.abort_flag());
    for (int i = k.tile0; ok && i < k.tile1; ++i, ++it) {
      const uint32_t s = it % kStages, ph = (it / kStages) & 1;
      if (!(ok = mbar_wait(sh.bar(K_FULL + s), ph, sh.abort_flag()))) break;
      tc_fence_after();
      const uint32_t kb = smem_u32(sh.keys(s)), vb = smem_u32(sh.values(s));
#pragma unroll
      for (int x = 0; x < kHd / 32; ++x)
        mma_e4m3(tmem + kColS, sw128_desc(kb + x * 32, 16, 1024), sw128_desc(q + x * 32, 16, 1024), id_s, x != 0);
      mma_commit(sh.bar(S_FULL));
      if (!(ok = mbar_wait(sh.bar(V_FULL + s), ph, sh.abort_flag()))) break;
      if (!(ok = mbar_wait(sh.bar(P_READY), it & 1, sh.abort_flag()))) break;
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < kTileTokens / 32; ++x)  // two of K = 32 for each page
        mma_e4m3(tmem + kColO + (x >> 1) * NP, sw128_desc(vb + x * 4096, 0, 1024), plain_mn_desc(p + x * 512, 128, 2048), id_o,
                 x & 1);
      mma_commit(sh.bar(O_FULL));
      mma_commit(sh.bar(EMPTY + s));
    }
  }
  if (!ok) give_up(sh);
  mma_commit(sh.bar(DRAIN));  // every product has completed before shared memory and TMEM go
  mbar_wait_drain(sh.bar(DRAIN), 0, kWaitCycles / 4);
}

// ------------------------------------------------------------------ softmax and sums (warps 0-3)

template <int MG>
__device__ void attend(const Kv8AttnArgs& a, const Shared& sh, const Work& wk, uint32_t tmem) {
  constexpr int NP = MG <= 4 ? 16 : 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t tm = tmem + ((uint32_t)(warp * 32) << 16);
  float* wmax = reinterpret_cast<float*>(sh.base + Layout::kOffMax);
  const int G = a.G;
  Walk k(a, wk);
  uint32_t it = 0, seg = 0;
  bool ok = true;  // once a wait has failed the rest runs through without waiting: nobody is left at a barrier
  auto wait = [&](int bar, uint32_t parity) {
    if (ok && !(ok = mbar_wait(sh.bar(bar), parity, sh.abort_flag()))) give_up(sh);
  };
  for (; k.next(); ++seg) {
    const size_t row0 = ((size_t)k.b * a.Hkv + k.h) * G;
    const uint32_t buf = seg % kQBufs;
    wait(Q_READY + buf, (seg / kQBufs) & 1);
    float qs[MG], m[MG], l[MG], acc[MG];
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      qs[g] = g < G ? sh.factors(buf)[g] : 0.f;
      m[g] = -CUDART_INF_F;
      l[g] = acc[g] = 0.f;
    }
    for (int i = k.tile0; i < k.tile1; ++i, ++it) {
      const uint32_t s = it % kStages, ph = (it / kStages) & 1;
      const int t0 = (k.sp.page0 + i * kTilePages) * kBlock, t = t0 + tid, half = warp >> 1;
      wait(K_FULL + s, ph);
      const Meta* meta = sh.meta(s);
      const float ks = meta->ks[half], vs0 = meta->vs[0], vs1 = meta->vs[1];
      const bool both = meta->ok[0] & meta->ok[1];
      const bool seen = t >= k.sp.lo && t < k.sp.n && meta->ok[half];
      wait(S_FULL, it & 1);
      tc_fence_after();
      float x[MG];
      {
        uint32_t d[16];
        tmem_ld16(tm + kColS, d);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < MG; ++g) {
          const float dot = fmaf(__uint_as_float(d[8 + g]), 1.f / 32.f, __uint_as_float(d[g]));
          x[g] = seen ? dot * (qs[g] * ks) : -CUDART_INF_F;
        }
      }
      float* wm = wmax + (it & 1) * 32;
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        const float top = warp_max(x[g]);
        if (lane == g) wm[warp * 8 + g] = top;
      }
      soft_sync();
      float old[MG], now[MG], p[MG];
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        const float top = fmaxf(fmaxf(wm[g], wm[8 + g]), fmaxf(wm[16 + g], wm[24 + g]));
        const bool none = top == -CUDART_INF_F;
        p[g] = exp2f(x[g] - (none ? 0.f : top));
        const float mn = fmaxf(m[g], top);
        const float ref = mn == -CUDART_INF_F ? 0.f : mn;
        old[g] = exp2f(m[g] - ref);
        now[g] = none ? 0.f : exp2f(top - ref);
        m[g] = mn;
        l[g] = fmaf(l[g], old[g], p[g] * now[g]);
      }
      // the terms of p: two heads to a conversion
      uint32_t term[3][MG / 2];
#pragma unroll
      for (int g = 0; g < MG; g += 2) {
        float r0 = p[g] * 256.f, r1 = p[g + 1] * 256.f;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          term[e][g / 2] = e4m3x2(r0, r1);
          if (e < 2) {
            const float2 v = e4m3x2_value(term[e][g / 2]);
            r0 = (r0 - v.x) * 32.f;
            r1 = (r1 - v.y) * 32.f;
          }
        }
      }
      uint4* prow = reinterpret_cast<uint4*>(sh.base + Layout::kOffP) + tid;
      if constexpr (MG <= 4) {
        *prow = make_uint4(term[0][0] | (term[0][1] << 16), term[1][0] | (term[1][1] << 16),
                           term[2][0] | (term[2][1] << 16), 0u);
      } else {
        prow[0] = make_uint4(term[0][0] | (term[0][1] << 16), term[0][2] | (term[0][3] << 16),
                             term[1][0] | (term[1][1] << 16), term[1][2] | (term[1][3] << 16));
        prow[kTileTokens] = make_uint4(term[2][0] | (term[2][1] << 16), term[2][2] | (term[2][3] << 16), 0u, 0u);
      }
      if (t0 < k.sp.lo || t0 + kTileTokens > k.sp.n || !both) {
        // value rows outside the attended tokens may hold anything, NaN codes among it
        wait(V_FULL + s, ph);
        if (!seen) {
          uint4* row = reinterpret_cast<uint4*>(sh.values(s) + tid * kHd);
#pragma unroll
          for (int c = 0; c < kHd / 16; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.bar(P_READY));
      wait(O_FULL, it & 1);
      tc_fence_after();
      if constexpr (MG <= 4) {
        uint32_t d[32];
        tmem_ld32(tm + kColO, d);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < MG; ++g) {
          float o[2];
#pragma unroll
          for (int y = 0; y < 2; ++y)
            o[y] = fmaf(__uint_as_float(d[16 * y + 8 + g]), 1.f / 1024.f,
                        fmaf(__uint_as_float(d[16 * y + 4 + g]), 1.f / 32.f, __uint_as_float(d[16 * y + g])));
          acc[g] = fmaf(acc[g], old[g], fmaf(o[0], vs0, o[1] * vs1) * (now[g] * (1.f / 256.f)));
        }
      } else {
        float o[MG];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t d[32];
          tmem_ld32(tm + kColO + y * NP, d);
          tmem_ld_wait();
#pragma unroll
          for (int g = 0; g < MG; ++g) {
            const float v = fmaf(__uint_as_float(d[16 + g]), 1.f / 1024.f,
                                 fmaf(__uint_as_float(d[8 + g]), 1.f / 32.f, __uint_as_float(d[g])));
            if (y == 0) o[g] = v * vs0;
            else acc[g] = fmaf(acc[g], old[g], fmaf(v, vs1, o[g]) * (now[g] * (1.f / 256.f)));
          }
        }
      }
    }
    // the sums of p are spread over the threads
    float* red = wmax;
    soft_sync();
    if (tid == 0) mbar_arrive(sh.bar(Q_FREE + buf));
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const float v = warp_sum(l[g]);
      if (lane == 0) red[warp * 8 + g] = v;
    }
    soft_sync();
#pragma unroll
    for (int g = 0; g < MG; ++g) l[g] = (red[g] + red[8 + g]) + (red[16 + g] + red[24 + g]);

    if (!k.whole()) {
      float* slot = a.part + (size_t)piece_slot(k) * a.part_stride;
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        if (g >= G) break;
        slot[g * kHd + tid] = acc[g];
        if (tid == 0) {
          slot[G * kHd + g] = m[g];
          slot[G * kHd + 8 + g] = l[g];
        }
      }
    } else {
      Joined j[MG];
#pragma unroll
      for (int g = 0; g < MG; ++g)
        if (g < G) j[g] = join_prev(a, row0 + g, m[g], l[g]);
      soft_sync();  // lse may be lse_prev: every thread has read it
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        if (g >= G) break;
        ((__nv_bfloat16*)a.o)[(row0 + g) * kHd + tid] = joined_value<__nv_bfloat16>(a, row0 + g, tid, j[g], acc[g]);
        if (a.lse && tid == 0) a.lse[row0 + g] = j[g].lse;
      }
    }
  }
}

template <int MG>
__global__ void __launch_bounds__(kThreads, 2)
kv8_attn_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const Kv8AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) a.cta_err[blockIdx.x] = LR_DEVERR_LAUNCH;
    return;
  }
  const Shared sh{smem};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Layout::kOffMisc);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(sh.bar(K_FULL + i), 2);
      mbar_init(sh.bar(V_FULL + i), 1);
      mbar_init(sh.bar(EMPTY + i), 1);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(sh.bar(Q_READY + i), 1);
      mbar_init(sh.bar(Q_FREE + i), 1);
    }
    mbar_init(sh.bar(S_FULL), 1);
    mbar_init(sh.bar(P_READY), kSoft / 32);
    mbar_init(sh.bar(O_FULL), 1);
    mbar_init(sh.bar(DRAIN), 1);
    *sh.abort_flag() = 0;
    *sh.err() = 0;
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if (warp == 5) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  // rows of absent query heads stay zero
  for (int i = threadIdx.x; i < kQBufs * 2048 / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + Layout::kOffQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  grid_dependency();
  const Work wk = find_work<kThreads>(a, reinterpret_cast<long long*>(smem + Layout::kOffScratch));
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  if (warp < 4) {
    attend<MG>(a, sh, wk, tmem);
  } else if (warp == 4) {
    load_tiles<MG>(a, sh, &mk, &mv, wk);
  } else if (lane == 0) {
    issue_products<MG>(a, sh, wk, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kTmemCols);
  if (threadIdx.x == 0) a.cta_err[blockIdx.x] = *sh.err();
}

template <int MG>
cudaError_t launch(const Kv8AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kv8_attn_tc_kernel<MG>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout::kBytes);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kv8_attn_tc_kernel<MG>, dim3(a.n_cta), kThreads, Layout::kBytes, st, mk, mv, a);
}

}  // namespace

cudaError_t launch_attn_tc(const Kv8AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  return a.G <= 4 ? launch<4>(a, mk, mv, st) : launch<8>(a, mk, mv, st);
}

}  // namespace kv8
}  // namespace lr
