// Decode attention over the 8-bit paged cache on the tensor cores: bf16, head_dim 128, up to 8 query
// heads per KV head.
//
// The codes go from HBM into the matrix units as they are (tcgen05, kind::f8f6f4); a conversion to
// a wider type would cost more issue slots than the bytes cost time. What multiplies them is
// therefore written as a sum of e4m3 numbers too, each term taking four more bits of what the ones
// before leave over:
//   q = 2^e (q1 + q2 / 32)              exact for a bf16 number down to 2^-14 of the head's largest
//                                       (below that off by 2^-22 of it at most);
//   p = (p1 + p2 / 32 + p3 / 1024) / 256, p rounded to fp16 first: 2^-11 relative at most, and 2^-27 absolute
//                                       for p under 2^-17, p relative to the largest of the tile.
// Every term is a column of its own, so a tile's products are
//   S  [128 tokens x 16]     = K q1 | K q2             (M 128, N 16, K 128)
//   O' [128 dims x 3 heads]  = V^T p1 | V^T p2 | V^T p3 (M 128, N 16 or 32, K 64) for each of the two pages,
// K as the K-major and V as the M-major operand, straight from the page rows (128 bytes, 128-byte
// swizzle). Thread t is token t in the softmax and dim t in the sum over the tiles: the maximum
// (one per head and tile, a warp reduction and four numbers in shared memory) is the only thing the
// threads exchange. Scales and the rescaling between tiles are fp32 factors in registers.
//
// Persistent, two CTAs per SM on an even share of the tiles (kv8_common.cuh): one warp loads (TMA, three stages of
// 32 KB), one issues the products, four or eight do softmax and sums, four for every four query heads. Scores
// are a tile ahead of the softmax, value products a tile behind. Bound by HBM: 256 bytes per token and
// KV head, 12 cycles of an SM's share of the bandwidth, against 2 of shared memory into the tensor pipe.
//
// Measured (B200, 8 KV heads of 4 query heads): four sequences of 131072 tokens 169 us, 6.3 TB/s of codes; one of
// 262144 88 us; one of 32768 21 us, of which 5 us pass before the first tile is there and 5 us after the
// last. The loads run at 7.3 TB/s once they have begun; SMs of the larger GPCs end up to 10 % later.
#include <algorithm>

#include "kv8_common.cuh"
#include "sm100.cuh"

namespace lr {
namespace kv8 {
namespace {

using namespace sm100;

constexpr int kHd = 128;
constexpr int kSoft = 128;  // threads of a softmax group, which has up to four query heads
constexpr int kHeads = 4;
constexpr int threads_of(int groups) { return groups * kSoft + 64; }
constexpr int kStages = 3;
constexpr int kPageBytes = kBlock * kHd;
constexpr int kTileBytes = kTilePages * kPageBytes;  // of K, and of V
constexpr int kColS = 0, kColO = 32;  // TMEM: two S of 16 columns, two O' of 2 NP

// What the loading warp says of the tile in a stage.
enum Flag { OK0 = 1, OK1 = 2, FIRST = 4, LAST = 8, WHOLE = 16, END = 32 };
struct __align__(16) Meta {
  float ks[2], vs[2];    // scales of its two pages, of values for sums in units of kSumUnit with weights times 256
  int t0, lo, n, flags;  // its first token, the attended ones; which pages there are (OK0, OK1), first or last
                         // tile of the segment here, all of the segment here, no tile: the end
  int head, slot;        // b * Hkv + h, and where a piece of it goes
  int pad[2];
};

struct Layout {
  static constexpr int kOffRing = 0;                         // stages of K, V
  static constexpr int kOffQ = kStages * 2 * kTileBytes;     // [kStages][16 rows of 128 bytes]
  static constexpr int kOffP = kOffQ + kStages * 2048;             // [2][2][128 tokens][16 bytes]
  static constexpr int kOffMeta = kOffP + 2 * 4096;
  static constexpr int kOffMax = kOffMeta + kStages * (int)sizeof(Meta);  // [2 groups][2][4 warps][4]
  static constexpr int kOffRed = kOffMax + 2 * 4 * 8 * 4;    // [2 groups][4 warps][4]
  static constexpr int kOffQs = kOffRed + 4 * 8 * 4;         // [2][8]
  static constexpr int kOffBar = kOffQs + 64;
  static constexpr int kOffMisc = kOffBar + 160;
  static constexpr int kOffScratch = kOffP;                  // of find_work, before there are any weights
  static constexpr int kBytes = kOffMisc + 16;
};
static_assert(Layout::kOffMeta % 16 == 0 && Layout::kOffBar % 8 == 0, "alignment");
static_assert((threads_of(2) + 4) * 8 <= 2 * 4096, "scratch");
static_assert(2 * (Layout::kBytes + 1024) <= 227 * 1024, "two CTAs per SM");

enum Bar { K_FULL = 0, V_FULL = K_FULL + kStages, EMPTY = V_FULL + kStages, Q_READY = EMPTY + kStages, S_FULL = Q_READY + 2, P_READY = S_FULL + 2, O_FULL = P_READY + 2, DRAIN = O_FULL + 2, kBars };
static_assert(kBars * 8 <= 160, "barriers");

// Barriers of a softmax group; soft_all also says whether `ok` held in all of its threads.
__device__ __forceinline__ void soft_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kSoft) : "memory");
}
__device__ __forceinline__ bool soft_all(int group, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(1 + group), "n"(kSoft)
      : "memory");
  return r != 0;
}

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

template <int GROUPS>
__host__ __device__ constexpr int tmem_cols() { return GROUPS == 1 ? 128 : 256; }

struct Shared {
  uint8_t* base;
  __device__ uint64_t* bar(int i) const { return reinterpret_cast<uint64_t*>(base + Layout::kOffBar) + i; }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(base + Layout::kOffMisc + 4); }
  __device__ int* err() const { return reinterpret_cast<int*>(base + Layout::kOffMisc + 8); }
  __device__ Meta* meta(int s) const { return reinterpret_cast<Meta*>(base + Layout::kOffMeta) + s; }
  __device__ uint8_t* queries(int i) const { return base + Layout::kOffQ + i * 2048; }
  __device__ uint8_t* weights(int i) const { return base + Layout::kOffP + i * 4096; }
  __device__ float* factors(int i) const { return reinterpret_cast<float*>(base + Layout::kOffQs) + i * 8; }
  __device__ uint8_t* keys(int s) const { return base + Layout::kOffRing + s * 2 * kTileBytes; }
  __device__ uint8_t* values(int s) const { return keys(s) + kTileBytes; }
};

__device__ __forceinline__ void give_up(const Shared& sh) {
  *sh.abort_flag() = 1;
  atomicOr(sh.err(), LR_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------ loads (one warp)
//
// The CTA's units are taken 16 at a time: lanes 2j and 2j + 1 find the segment of unit j and have the ids
// and scales of its two pages, and lane 2j issues the loads of the tile. While one batch is loaded the ids
// and then the scales of the next are on their way, whatever segments they belong to.

struct Batch {
  Place at;
  int id;        // this lane's page, -1: none
  bool live;     // there is a tile
  bool page;     // and this page of it
  float ks, vs;
};

__device__ __forceinline__ void batch_ids(const Kv8AttnArgs& a, const Work& wk, long long unit, Batch& t) {
  t.live = t.page = false;
  t.id = -1;
  if (unit >= wk.end) return;
  t.at.seek(a, unit);
  t.live = t.at.tile < t.at.sp.tiles;
  const int p = t.at.sp.page0 + t.at.tile * kTilePages + (int)(threadIdx.x & 1);
  t.page = t.live && p * kBlock < t.at.sp.n;
  if (t.page) t.id = __ldg(a.table + (size_t)t.at.b * a.max_pages + p);
}
__device__ __forceinline__ void batch_scales(const Kv8AttnArgs& a, const Shared& sh, Batch& t) {
  t.ks = t.vs = 0.f;
  if ((unsigned)t.id < (unsigned)a.n_pages) {
    t.ks = __ldg(a.ks + (size_t)t.id * a.Hkv + t.at.h);
    t.vs = __ldg(a.vs + (size_t)t.id * a.Hkv + t.at.h);
  } else {
    if (t.page) atomicOr(sh.err(), LR_DEVERR_PAGE);
    t.id = -1;
  }
}

__device__ void load_tiles(const Kv8AttnArgs& a, const Shared& sh, const CUtensorMap* mk, const CUtensorMap* mv, const Work& wk) {
  const int lane = threadIdx.x & 31;
  uint32_t it = 0, seg = 0;
  bool ok = true;
  Batch next;
  long long unit = wk.begin + (lane >> 1);  // of this lane, in the batch under way
  if (wk.begin < wk.end) next.at.start(a, wk);
  batch_ids(a, wk, unit, next);
  batch_scales(a, sh, next);
  while (ok && unit - (lane >> 1) < wk.end) {
    const Batch t = next;
    const int id1 = __shfl_xor_sync(0xffffffffu, t.id, 1);
    float ks1, vs1;
    uint32_t live = __ballot_sync(0xffffffffu, t.live) & 0x55555555u;
    for (int x = 0; x < 16; ++x) {
      if (x == 8) batch_scales(a, sh, next);
      if (!live) {
        if (x == 0) batch_ids(a, wk, unit + 16, next);
        continue;
      }
      const int src = __ffs(live) - 1;
      live &= live - 1;
      const uint32_t s = it % kStages, ph = (it / kStages) & 1;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(sh.bar(EMPTY + s), ph ^ 1, sh.abort_flag())))) break;
      ++it;
      const bool first = t.at.tile == 0 || unit == wk.begin;
      seg += __shfl_sync(0xffffffffu, first, src);
      const bool last = t.at.tile == t.at.sp.tiles - 1 || unit == wk.end - 1;
      const int head = t.at.b * a.Hkv + t.at.h, row = t.at.h * kBlock;
      if (lane == src) {
        const uint32_t bytes = ((t.id >= 0) + (id1 >= 0)) * kPageBytes, q_bytes = a.G * kHd * 2;
        uint64_t *kf = sh.bar(K_FULL + s), *vf = sh.bar(V_FULL + s);
        mbar_arrive_expect_tx(kf, bytes + (first ? q_bytes : 0));
        if (t.id >= 0) tma_load_3d(sh.keys(s), mk, kf, 0, row, t.id);
        if (id1 >= 0) tma_load_3d(sh.keys(s) + kPageBytes, mk, kf, 0, row, id1);
        // the segment three before has no scores to come: the tile that was in this stage is behind its end
        if (first) bulk_load(sh.queries((seg - 1) % kStages), (const __nv_bfloat16*)a.q + (size_t)head * a.G * kHd, q_bytes, kf);
        mbar_arrive_expect_tx(vf, bytes);
        if (t.id >= 0) tma_load_3d(sh.values(s), mv, vf, 0, row, t.id);
        if (id1 >= 0) tma_load_3d(sh.values(s) + kPageBytes, mv, vf, 0, row, id1);
      }
      if (x == 0) {  // with the first tile on its way
        batch_ids(a, wk, unit + 16, next);
        ks1 = __shfl_xor_sync(0xffffffffu, t.ks, 1);
        vs1 = __shfl_xor_sync(0xffffffffu, t.vs, 1);
      }
      if (lane == src) {
        Meta m;
        m.ks[0] = t.ks;
        m.ks[1] = ks1;
        m.vs[0] = t.vs * (1.f / 256.f / kSumUnit);
        m.vs[1] = vs1 * (1.f / 256.f / kSumUnit);
        m.t0 = (t.at.sp.page0 + t.at.tile * kTilePages) * kBlock;
        m.lo = t.at.sp.lo;
        m.n = t.at.sp.n;
        m.flags = (t.id >= 0 ? OK0 : 0) | (id1 >= 0 ? OK1 : 0) | (first ? FIRST : 0) | (last ? LAST : 0) |
                  (t.at.seg_first >= wk.begin && t.at.seg_first + t.at.sp.tiles <= wk.end ? WHOLE : 0);
        m.head = head;
        m.slot = piece_slot(wk, blockIdx.x, t.at.seg_first);
        *sh.meta(s) = m;
        mbar_arrive(sh.bar(K_FULL + s));
      }
      __syncwarp();
    }
    unit += 16;
  }
  if (ok) {  // the end
    const uint32_t s = it % kStages, ph = (it / kStages) & 1;
    ok = __all_sync(0xffffffffu, mbar_wait(sh.bar(EMPTY + s), ph ^ 1, sh.abort_flag()));
    if (ok && lane == 0) {
      sh.meta(s)->flags = END;
      mbar_arrive(sh.bar(K_FULL + s));
      mbar_arrive(sh.bar(K_FULL + s));
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

// ------------------------------------------------------------------ products (one warp)

// The query heads, bf16 rows of 256 bytes at q, become two e4m3 terms each, rows g and 8 + g of the K-major
// operand in their place, and the factors that scores are multiplied by. A head with an infinite
// number gets a NaN factor. What is left in the rows of absent heads reaches columns that nobody reads.
template <int MG>
__device__ __forceinline__ void write_q(const Kv8AttnArgs& a, uint8_t* q, float* factors) {
  const int lane = threadIdx.x & 31;
  uint2 raw[MG];
#pragma unroll
  for (int g = 0; g < MG; ++g)
    if (g < a.G) raw[g] = reinterpret_cast<const uint2*>(q)[g * 32 + lane];
  __syncwarp();
#pragma unroll
  for (int g = 0; g < MG; ++g) {
    if (g >= a.G) break;
    const uint2 u = raw[g];
    float x[4] = {__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                  __uint_as_float(u.y & 0xffff0000u)};
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
    if (lane == 0) factors[g] = top < CUDART_INF_F ? __uint_as_float((uint32_t)(127 + e) << 23) * a.scale : CUDART_NAN_F;
  }
}

// The scores of the next tile go ahead of a tile's value product if its keys are there by the time the product
// would have to wait for the softmax, so that they are ready when the softmax is. (Polling for whichever is first
// took issue slots from the softmax: 98 us instead of 91 for 64 sequences of 8 query heads per KV head.)
// Lane 0 issues; the warp turns a segment's queries into an operand.
template <int GROUPS>
__device__ void issue_products(const Kv8AttnArgs& a, const Shared& sh, uint32_t tmem) {
  constexpr int NP = 16 * GROUPS;
  const uint32_t id_s = idesc_e4m3_f32(128, 16, false, false), id_o = idesc_e4m3_f32(128, NP, true, true);
  const int lane = threadIdx.x & 31;
  uint32_t qk = 0, pv = 0, seg = 0;  // tiles whose scores and whose value products are issued
  bool end = false, ok = true;
  while (!end || pv < qk) {
    if (!end && qk <= pv + 1) {
      const uint32_t s = qk % kStages, ph = (qk / kStages) & 1;
      bool there;
      if (qk <= pv) there = ok = __all_sync(0xffffffffu, mbar_wait(sh.bar(K_FULL + s), ph, sh.abort_flag()));
      else there = __all_sync(0xffffffffu, mbar_test(sh.bar(K_FULL + s), ph));
      if (!ok) break;
      if (there) {
        const int flags = sh.meta(s)->flags;
        if (flags & END) {
          end = true;
          continue;
        }
        if (flags & FIRST) {  // the factors of the segment before the last have been read
          write_q<kHeads * GROUPS>(a, sh.queries(seg % kStages), sh.factors(seg & 1));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(sh.bar(Q_READY + (seg & 1)));
          ++seg;
        }
        if (lane == 0) {
          tc_fence_after();
          const uint32_t kb = smem_u32(sh.keys(s)), q = smem_u32(sh.queries((seg - 1) % kStages));
#pragma unroll
          for (int x = 0; x < kHd / 32; ++x)
            mma_e4m3(tmem + kColS + (qk & 1) * 16, sw128_desc(kb + x * 32, 16, 1024), sw128_desc(q + x * 32, 16, 1024), id_s,
                     x != 0);
          mma_commit(sh.bar(S_FULL + (qk & 1)));
        }
        __syncwarp();
        ++qk;
        if (qk <= pv + 1) continue;
      }
    }
    const uint32_t s = pv % kStages;
    ok = mbar_wait(sh.bar(P_READY + (pv & 1)), (pv >> 1) & 1, sh.abort_flag()) &&
         mbar_wait(sh.bar(V_FULL + s), (pv / kStages) & 1, sh.abort_flag());
    if (!(ok = __all_sync(0xffffffffu, ok))) break;
    if (lane == 0) {
      tc_fence_after();
      const uint32_t vb = smem_u32(sh.values(s)), p = smem_u32(sh.weights(pv & 1));
#pragma unroll
      for (int x = 0; x < kTileTokens / 32; ++x)  // two of K = 32 for each page
        mma_e4m3(tmem + kColO + ((pv & 1) * 2 + (x >> 1)) * NP, sw128_desc(vb + x * 4096, 0, 1024),
                 plain_mn_desc(p + x * 512, 128, 2048), id_o, x & 1);
      mma_commit(sh.bar(O_FULL + (pv & 1)));
      mma_commit(sh.bar(EMPTY + s));
    }
    __syncwarp();
    ++pv;
  }
  if (lane == 0) {
    if (!ok) give_up(sh);
    mma_commit(sh.bar(DRAIN));  // every product has completed before shared memory and TMEM go
    mbar_wait_drain(sh.bar(DRAIN), 0, kWaitCycles / 4);
  }
}

// ------------------------------------------------------------------ softmax and sums (four or eight warps)

template <int GROUPS>
__device__ void attend(const Kv8AttnArgs& a, const Shared& sh, uint32_t tmem) {
  constexpr int NP = 16 * GROUPS;
  const int group = GROUPS == 1 ? 0 : threadIdx.x / kSoft;
  const int tid = threadIdx.x % kSoft, lane = tid & 31, warp = tid >> 5;
  const uint32_t tm = tmem + ((uint32_t)(warp * 32) << 16);
  float* wmax = reinterpret_cast<float*>(sh.base + Layout::kOffMax) + group * 32;
  float* red = reinterpret_cast<float*>(sh.base + Layout::kOffRed) + group * 16;
  const int g0 = group * kHeads, G = min(kHeads, a.G - g0);  // the group's query heads g0 .. g0 + G - 1
  uint32_t seg = 0;
  bool ok = true;
  auto wait = [&](int bar, uint32_t parity) {
    if (ok && !(ok = mbar_wait(sh.bar(bar), parity, sh.abort_flag()))) give_up(sh);
  };
  float qs[kHeads], m[kHeads], l[kHeads], acc[kHeads];
  float old[kHeads], now[kHeads], vs0, vs1;  // what the tile whose value product is under way is added with
  auto add_values = [&](uint32_t i) {
    wait(O_FULL + (i & 1), (i >> 1) & 1);
    tc_fence_after();
    uint32_t d[2][16];
#pragma unroll
    for (int y = 0; y < 2; ++y) tmem_ld16(tm + kColO + ((i & 1) * 2 + y) * NP + group * 16, d[y]);
    tmem_ld_wait();
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      float o[2];
#pragma unroll
      for (int y = 0; y < 2; ++y)
        o[y] = fmaf(__uint_as_float(d[y][8 + g]), 1.f / 1024.f,
                    fmaf(__uint_as_float(d[y][4 + g]), 1.f / 32.f, __uint_as_float(d[y][g])));
      acc[g] = fmaf(acc[g], old[g], fmaf(o[0], vs0, o[1] * vs1) * now[g]);
    }
  };
  for (uint32_t it = 0;; ++it) {
    const uint32_t s = it % kStages, ph = (it / kStages) & 1;
    wait(K_FULL + s, ph);
    Meta meta = *sh.meta(s);
    if (!ok) meta.flags = 0;
    if (meta.flags & END) {
      soft_all(group, ok);
      break;
    }
    if (meta.flags & FIRST) {
      const int buf = seg & 1;
      wait(Q_READY + buf, (seg >> 1) & 1);
      ++seg;
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        qs[g] = g < G ? sh.factors(buf)[g0 + g] : 0.f;
        m[g] = -CUDART_INF_F;
        l[g] = acc[g] = 0.f;
      }
    }
    {
      const int t = meta.t0 + tid, half = warp >> 1;
      const float ks = half ? meta.ks[1] : meta.ks[0];
      const bool both = (meta.flags & (OK0 | OK1)) == (OK0 | OK1);
      const bool seen = t >= meta.lo && t < meta.n && (meta.flags & (OK0 << half));
      wait(S_FULL + (it & 1), (it >> 1) & 1);
      tc_fence_after();
      float x[kHeads];
      {
        uint32_t d0[4], d1[4];
        tmem_ld4(tm + kColS + (it & 1) * 16 + g0, d0);
        tmem_ld4(tm + kColS + (it & 1) * 16 + 8 + g0, d1);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
          const float dot = fmaf(__uint_as_float(d1[g]), 1.f / 32.f, __uint_as_float(d0[g]));
          x[g] = seen ? dot * (qs[g] * ks) : -CUDART_INF_F;
        }
      }
      float* wm = wmax + (it & 1) * 16;
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        const float top = warp_max(x[g]);
        if (lane == g) wm[warp * 4 + g] = top;
      }
      if (!soft_all(group, ok)) break;  // after a failed wait all leave together: nobody is left at a barrier
      float p[kHeads], old_next[kHeads], now_next[kHeads], top[kHeads];
      {
        float4 w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) w[y] = reinterpret_cast<const float4*>(wm)[y];
        top[0] = fmaxf(fmaxf(w[0].x, w[1].x), fmaxf(w[2].x, w[3].x));
        top[1] = fmaxf(fmaxf(w[0].y, w[1].y), fmaxf(w[2].y, w[3].y));
        top[2] = fmaxf(fmaxf(w[0].z, w[1].z), fmaxf(w[2].z, w[3].z));
        top[3] = fmaxf(fmaxf(w[0].w, w[1].w), fmaxf(w[2].w, w[3].w));
      }
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        const bool none = top[g] == -CUDART_INF_F;
        p[g] = exp2_ftz(x[g] - (none ? 0.f : top[g]));
        const float mn = fmaxf(m[g], top[g]);
        const float ref = mn == -CUDART_INF_F ? 0.f : mn;
        old_next[g] = exp2_ftz(m[g] - ref);
        now_next[g] = none ? 0.f : exp2_ftz(top[g] - ref);
        m[g] = mn;
        l[g] = fmaf(l[g], old_next[g], p[g] * now_next[g]);
      }
      // the terms of p, two heads at a time: p to the 11 bits of fp16, of which each term takes four
      uint32_t term[3][kHeads / 2];
#pragma unroll
      for (int g = 0; g < kHeads; g += 2) {
        __half2 r = __floats2half2_rn(p[g] * 256.f, p[g + 1] * 256.f);
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          term[e][g / 2] = e4m3x2(r);
          if (e < 2) r = __hmul2(__hsub2(r, e4m3x2_half2(term[e][g / 2])), __float2half2_rn(32.f));  // both exact
        }
      }
      reinterpret_cast<uint4*>(sh.weights(it & 1))[group * kTileTokens + tid] =
          make_uint4(term[0][0] | (term[0][1] << 16), term[1][0] | (term[1][1] << 16), term[2][0] | (term[2][1] << 16), 0u);
      if (meta.t0 < meta.lo || meta.n - meta.t0 < kTileTokens || !both) {
        // value rows outside the attended tokens may hold anything, NaN codes among it
        wait(V_FULL + s, ph);
        if (!seen && group == 0) {
          uint4* row = reinterpret_cast<uint4*>(sh.values(s) + tid * kHd);
#pragma unroll
          for (int c = 0; c < kHd / 16; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.bar(P_READY + (it & 1)));
      if (!(meta.flags & FIRST)) add_values(it - 1);
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        old[g] = old_next[g];
        now[g] = now_next[g];
      }
      vs0 = meta.vs[0];
      vs1 = meta.vs[1];
    }
    if (!(meta.flags & LAST)) continue;
    const size_t row0 = (size_t)meta.head * a.G + g0;
    const bool whole = meta.flags & WHOLE;
    float prev[kHeads];  // the earlier partial result, on its way while the last product ends
#pragma unroll
    for (int g = 0; g < kHeads; ++g)
      prev[g] = whole && a.o_prev && g < G ? to_f32(((const __nv_bfloat16*)a.o_prev)[(row0 + g) * kHd + tid]) : 0.f;
    // the sums of p are spread over the threads: exchanging heads, a lane ends up with one head's
    const bool up1 = lane & 1, up2 = lane & 2;
    float v0 = (up1 ? l[2] : l[0]) + __shfl_xor_sync(0xffffffffu, up1 ? l[0] : l[2], 1);
    float v1 = (up1 ? l[3] : l[1]) + __shfl_xor_sync(0xffffffffu, up1 ? l[1] : l[3], 1);
    float sum = (up2 ? v1 : v0) + __shfl_xor_sync(0xffffffffu, up2 ? v0 : v1, 2);
#pragma unroll
    for (int off = 4; off < 32; off *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane < kHeads) red[warp * 4 + (lane & 1) * 2 + (lane >> 1)] = sum;
    add_values(it);
    soft_sync(group);
    const int mine = lane % kHeads;  // the head that this lane finishes
    sum = (red[mine] + red[4 + mine]) + (red[8 + mine] + red[12 + mine]);
    const float top = mine < 2 ? (mine == 0 ? m[0] : m[1]) : (mine == 2 ? m[2] : m[3]);
    if (!whole) {
      float* slot = a.part + (size_t)meta.slot * a.part_stride;
#pragma unroll
      for (int g = 0; g < kHeads; ++g)
        if (g < G) slot[(g0 + g) * kHd + tid] = acc[g];
      if (tid < G) {
        slot[a.G * kHd + g0 + tid] = top;
        slot[a.G * kHd + 8 + g0 + tid] = sum;
      }
    } else {
      Joined j{0.f, 0.f, 0.f, 0.f};
      if (mine < G) j = join_prev(a, row0 + mine, top, sum);
      if (a.lse_prev) soft_sync(group);  // it may be lse: every warp has read it
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        const float inv = __shfl_sync(0xffffffffu, j.inv, g), w = __shfl_sync(0xffffffffu, j.w_prev, g);
        if (g < G) ((__nv_bfloat16*)a.o)[(row0 + g) * kHd + tid] = from_f32<__nv_bfloat16>(join_value(acc[g], inv, prev[g], w));
      }
      if (a.lse && tid < G) a.lse[row0 + tid] = j.lse();
    }
  }
}

template <int GROUPS>
__global__ void __launch_bounds__(threads_of(GROUPS), 2)
kv8_attn_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const Kv8AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) {
      if (a.cluster && blockIdx.x == 0) *a.err = LR_DEVERR_LAUNCH;
      a.cta_err[blockIdx.x] = LR_DEVERR_LAUNCH;
      reinterpret_cast<Pieces*>(a.split)[blockIdx.x] = Pieces{0, 0, 0, 0};
    }
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh.bar(Q_READY + i), 1);
      mbar_init(sh.bar(S_FULL + i), 1);
      mbar_init(sh.bar(P_READY + i), GROUPS * kSoft / 32);
      mbar_init(sh.bar(O_FULL + i), 1);
    }
    mbar_init(sh.bar(DRAIN), 1);
    *sh.abort_flag() = 0;
    *sh.err() = 0;
    fence_mbar_init();
  }
  constexpr int kLoads = GROUPS * kSoft / 32, kIssue = kLoads + 1;
  if (warp == kLoads && lane == 0) {
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if (warp == kIssue) {
    tmem_alloc(tmem_holder, tmem_cols<GROUPS>());
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  prefetch_inputs(a);
  grid_dependency();
  const Work wk = a.cluster ? small_work(a, blockIdx.x) : find_work<threads_of(GROUPS)>(a, reinterpret_cast<long long*>(smem + Layout::kOffScratch));
  if (blockIdx.x == 0 && wk.bad_len) atomicOr(sh.err(), LR_DEVERR_LEN);
  if (warp < kLoads) {
    attend<GROUPS>(a, sh, tmem);
  } else if (warp == kLoads) {
    load_tiles(a, sh, &mk, &mv, wk);
    if (a.cluster) {
      const int bits = blockIdx.x == 0 ? check_all(a, lane, 32) : 0;
      if (bits) atomicOr(sh.err(), bits);
    } else if (lane == 0) {
      reinterpret_cast<Pieces*>(a.split)[blockIdx.x] = pieces_of(a, wk, blockIdx.x);
    }
    __syncwarp();
    empty_rows<__nv_bfloat16>(a, blockIdx.x, gridDim.x);
  } else {
    issue_products<GROUPS>(a, sh, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssue) tmem_dealloc(tmem, tmem_cols<GROUPS>());
  if (a.cluster) finish_small<__nv_bfloat16>(a, wk.pieces, *sh.err());
  else if (threadIdx.x == 0) a.cta_err[blockIdx.x] = *sh.err();
}

template <int GROUPS>
cudaError_t launch(const Kv8AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kv8_attn_tc_kernel<GROUPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout::kBytes);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kv8_attn_tc_kernel<GROUPS>, dim3(a.n_cta), a.cluster, threads_of(GROUPS), Layout::kBytes, st, mk, mv, a);
}

}  // namespace

cudaError_t launch_attn_tc(const Kv8AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  return a.G <= kHeads ? launch<1>(a, mk, mv, st) : launch<2>(a, mk, mv, st);
}

}  // namespace kv8
}  // namespace lr
