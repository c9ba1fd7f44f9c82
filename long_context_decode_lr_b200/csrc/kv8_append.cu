// Appending new keys and values to the 8-bit paged cache, keys and queries rotated by their
// position on the way (rotary embedding).
//
// A page of one KV head has one scale for its keys and one for its values, a power of two, so
// raising it when larger numbers arrive shifts the codes' exponents and loses nothing but what
// falls under the smallest code. Whoever writes a page therefore owns it: one CTA (or warp, with one
// token per sequence) takes all of a call's rows of a page and head, finds their largest
// magnitude, settles the scale and writes the codes. The rows are read from memory once and stay on the SM
// between the maximum and the rounding.
//
// Angles: a pair's frequency becomes a 64-bit fraction of a turn, so position * fraction wraps at
// whole turns by itself and stays right to 2^-32 of a turn at far positions; sine and cosine take the top 32 bits.
//
// Measured (B200, 32 query and 8 KV heads of 128 bf16 numbers, all rotated): 32K tokens of one sequence
// 127 us (132 in a long run), 5.8 TB/s of the 738 MB read and written; one token for each of 64 sequences 3.4 us.
// fp32 321 to 335 us, 4.2 to 4.4 TB/s, rotated or not: its warps wait for the memory queue, with the issue slots and HBM half idle.
// Lanes that exchange their 16-byte parts, so that an instruction covers whole sectors or lines, took 354 and 362.
#include <algorithm>

#include "kv8_common.cuh"
#include "kv8_rules.h"

namespace lr {
namespace kv8 {
namespace {

constexpr int kMinExp = -24;  // smallest scale 2^-24: numbers under 2^-34 become 0

// `radians` / 2 pi modulo 1, in 2^-64: off by one or two units, which at position 2^31 is 2^-32 of a turn (with 1 / 2 pi
// in one fp64 number it was 2^-22 of inv_freq there). 1 / 2 pi is the sum of two fp64 numbers and the product with the first
// is taken exactly, as a rounded product and what the rounding left.
__device__ __forceinline__ uint64_t turn_fraction(float radians) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18, k64 = 18446744073709551616.0;
  const double f = radians, t = __dmul_rn(f, kHi), rest = __fma_rn(f, kLo, __fma_rn(f, kHi, -t));
  return (uint64_t)__double2ll_rn((t - rint(t)) * k64) + (uint64_t)__double2ll_rn(rest * k64);
}
// Within 2^-22 for fp32: the angle, a number of half turns up to 1, is rounded to 24 bits (pi 2^-25), and sincospif to
// its last place. bf16 takes the hardware's sine and cosine, within 2^-20: 2^-21.2 on one turn, and the radians
// are rounded twice (half a step of bf16 is 2^-9; with sincospif the angles were a fifth of all instructions).
template <typename T>
__device__ __forceinline__ void sin_cos(uint64_t fraction, int pos, float& s, float& c) {
  const int32_t turns = (int32_t)((fraction * (uint64_t)(uint32_t)pos) >> 32);
  if constexpr (sizeof(T) == 2) {
    const float x = (float)turns * 1.4629180792671596e-9f;  // pi 2^-31: radians
    s = __sinf(x);
    c = __cosf(x);
  } else {
    sincospif((float)turns * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  }
}

// Exponent of the smallest power of two s >= 2^-24 with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kMinExp);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Magnitude bits of a finite number, 0 of any other: as integers they order like the numbers.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}
__device__ __forceinline__ float or_nan(float x) { return fabsf(x) <= 3.402823466e38f ? x : CUDART_NAN_F; }
__device__ __forceinline__ uint32_t codes2(float lo, float hi, float inv) {
  return e4m3x2(or_nan(lo) * inv, or_nan(hi) * inv);
}
// A page may hold a scale of the caller's that is no power of two, and then its fp32 reciprocal is a rounded one:
// numbers are divided. (Where no page does, that costs a call of one token under 0.1 us, 24 ragged sequences 2 of
// 71 us and 32K tokens nothing; with the division out of line 4 and 2 us, a product of fp64 numbers instead 3 and 2.)
__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// Four codes scaled again by `ratio`.
__device__ __forceinline__ uint32_t rescale4(uint32_t u, float ratio) {
  const float2 a = e4m3x2_value(u & 0xffffu), b = e4m3x2_value(u >> 16);
  return e4m3x2(a.x * ratio, a.y * ratio) | (e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

// The new tokens of sequence b: rows [start, start + n) go to positions p0 .. p0 + n - 1.
struct NewTokens {
  int start, n, p0;
  bool ok;
};
__device__ __forceinline__ NewTokens new_tokens(const Kv8AppendArgs& a, int b) {
  NewTokens t;
  const long long len = __ldg(a.lens + b);
  long long n;
  if (a.cu) {
    t.start = __ldg(a.cu + b);
    n = (long long)__ldg(a.cu + b + 1) - t.start;
  } else {
    t.start = b;
    n = len == 0 ? 0 : 1;
  }
  t.ok = t.start >= 0 && n >= 0 && t.start + n <= a.n_tokens && len >= n && len <= (long long)a.max_pages * kBlock;
  t.n = t.ok ? (int)n : 0;
  t.p0 = t.ok ? (int)(len - n) : 0;
  return t;
}

// ------------------------------------------------------------------ one token per sequence
//
// One warp per (sequence, head): a query head, or a KV head with its key and its value. A lane holds
// quads of two pairs (two neighbours in each half of the rotated dims), 4-byte loads of bf16: the
// work is latency, and this spreads the angles over all lanes.

constexpr int kOneWarps = 4;

template <typename T>
__device__ __forceinline__ void load2(const T* p, float& x, float& y);
template <>
__device__ __forceinline__ void load2<float>(const float* p, float& x, float& y) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  x = v.x;
  y = v.y;
}
template <>
__device__ __forceinline__ void load2<__nv_bfloat16>(const __nv_bfloat16* p, float& x, float& y) {
  const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  x = v.x;
  y = v.y;
}
__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}

// Dims of quad i: c0, c0 + 1 and c1, c1 + 1; pairs 2i and 2i + 1 of the rotation where rotated.
__device__ __forceinline__ void quad_dims(const Kv8AppendArgs& a, int i, int& c0, int& c1) {
  if (!a.interleaved && i < a.rot / 4) {
    c0 = 2 * i;
    c1 = a.rot / 2 + 2 * i;
  } else {
    c0 = 4 * i;
    c1 = 4 * i + 2;
  }
}
// x = {c0, c0 + 1, c1, c1 + 1}
__device__ __forceinline__ void rotate_quad(bool interleaved, float (&x)[4], const float (&s)[2], const float (&c)[2]) {
  const float x0 = x[0], x1 = x[1], x2 = x[2], x3 = x[3];
  if (interleaved) {
    x[0] = x0 * c[0] - x1 * s[0];
    x[1] = x1 * c[0] + x0 * s[0];
    x[2] = x2 * c[1] - x3 * s[1];
    x[3] = x3 * c[1] + x2 * s[1];
  } else {
    x[0] = x0 * c[0] - x2 * s[0];
    x[2] = x2 * c[0] + x0 * s[0];
    x[1] = x1 * c[1] - x3 * s[1];
    x[3] = x3 * c[1] + x1 * s[1];
  }
}

// A warp's row of one page and head (key or value): the scale, the codes held before, the new ones.
template <int Q>
__device__ __forceinline__ void append_one(const Kv8AppendArgs& a, uint8_t* codes, float* scale, int page, int h, int slot,
                                           const float (&x)[Q][4]) {
  const int lane = threadIdx.x & 31, quads = a.hd / 4;
  uint8_t* head = codes + (size_t)page * a.page_stride + (size_t)h * kBlock * a.hd;
  float* at = scale + (size_t)page * a.Hkv + h;
  const float held = slot > 0 ? *at : 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < Q; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, finite_bits(x[u][e]));
  const float fresh = pow2(scale_exp(__reduce_max_sync(0xffffffffu, top)));
  const float s = fmaxf(held, fresh);
  if (slot > 0 && s > held) {
    const float ratio = held / s;
    for (int i = lane; i < slot * a.hd / 4; i += 32) {
      uint32_t* w = reinterpret_cast<uint32_t*>(head) + i;
      *w = rescale4(*w, ratio);
    }
  }
  __syncwarp();
  if (lane == 0 && s != held) *at = s;
  uint8_t* row = head + (size_t)slot * a.hd;
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int u = 0; u < Q; ++u) {
    const int i = lane + 32 * u;
    if (i >= quads) continue;
    int c0, c1;
    quad_dims(a, i, c0, c1);
    if (is_pow2(s)) {
      *reinterpret_cast<uint16_t*>(row + c0) = (uint16_t)codes2(x[u][0], x[u][1], inv);
      *reinterpret_cast<uint16_t*>(row + c1) = (uint16_t)codes2(x[u][2], x[u][3], inv);
    } else {
      *reinterpret_cast<uint16_t*>(row + c0) = (uint16_t)codes2(__fdiv_rn(x[u][0], s), __fdiv_rn(x[u][1], s), 1.f);
      *reinterpret_cast<uint16_t*>(row + c1) = (uint16_t)codes2(__fdiv_rn(x[u][2], s), __fdiv_rn(x[u][3], s), 1.f);
    }
  }
}

template <typename T, int Q>  // Q: quads of a lane (head_dim <= 128 Q)
__global__ void __launch_bounds__(32 * kOneWarps) kv8_append_one_kernel(Kv8AppendArgs a) {
  if (blockIdx.x == gridDim.x - 1) {  // the device checks; the word is written, not or-ed: no clearing before
    __shared__ int bits;
    if (threadIdx.x == 0) bits = 0;
    __syncthreads();
    int mine = 0;
    for (int b = threadIdx.x; b < a.B; b += 32 * kOneWarps) {
      const NewTokens t = new_tokens(a, b);
      if (!t.ok) mine |= LR_DEVERR_LEN;
      else if (t.n && (unsigned)__ldg(a.table + (size_t)b * a.max_pages + t.p0 / kBlock) >= (unsigned)a.n_pages)
        mine |= LR_DEVERR_PAGE;
    }
    if (mine) atomicOr(&bits, mine);
    __syncthreads();
    if (threadIdx.x == 0) *a.err = bits;
    return;
  }
  const int jobs = a.Hkv + a.Hq;
  const long long job = (long long)blockIdx.x * kOneWarps + (threadIdx.x >> 5);
  if (job >= (long long)a.B * jobs) return;
  const int b = (int)(job / jobs), j = (int)(job % jobs), lane = threadIdx.x & 31, quads = a.hd / 4;
  const NewTokens t = new_tokens(a, b);
  if (!t.n) return;
  const bool query = j >= a.Hkv;
  const T* src = query ? (const T*)a.q + (size_t)t.start * a.q_stride + (size_t)(j - a.Hkv) * a.hd
                       : (const T*)a.k + (size_t)t.start * a.k_stride + (size_t)j * a.hd;
  float x[Q][4], v[Q][4];
#pragma unroll
  for (int u = 0; u < Q; ++u) {
    const int i = lane + 32 * u;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[u][e] = v[u][e] = 0.f;
    if (i >= quads) continue;
    int c0, c1;
    quad_dims(a, i, c0, c1);
    load2<T>(src + c0, x[u][0], x[u][1]);
    load2<T>(src + c1, x[u][2], x[u][3]);
    if (!query) {
      const T* vr = (const T*)a.v + (size_t)t.start * a.v_stride + (size_t)j * a.hd;
      load2<T>(vr + c0, v[u][0], v[u][1]);
      load2<T>(vr + c1, v[u][2], v[u][3]);
    }
    if (i < a.rot / 4) {
      float s[2], c[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) sin_cos<T>(turn_fraction(__ldg(a.inv_freq + 2 * i + e)), t.p0, s[e], c[e]);
      rotate_quad(a.interleaved, x[u], s, c);
    }
  }
  if (query) {
    T* out = (T*)a.q_out + ((size_t)t.start * a.Hq + (j - a.Hkv)) * a.hd;
#pragma unroll
    for (int u = 0; u < Q; ++u) {
      const int i = lane + 32 * u;
      if (i >= quads) continue;
      int c0, c1;
      quad_dims(a, i, c0, c1);
      store2(out + c0, x[u][0], x[u][1]);
      store2(out + c1, x[u][2], x[u][3]);
    }
    return;
  }
  const int page = __ldg(a.table + (size_t)b * a.max_pages + t.p0 / kBlock);
  if ((unsigned)page >= (unsigned)a.n_pages) return;
  append_one<Q>(a, a.kc, a.ks, page, j, t.p0 % kBlock, x);
  append_one<Q>(a, a.vc, a.vs, page, j, t.p0 % kBlock, v);
}

// ------------------------------------------------------------------ ranges of tokens
//
// One CTA per page that receives tokens, for a share (blockIdx.y) of the heads. A thread has one row of the
// page (64 rows x hd / 16 threads) and, of each head's row, the two chunks of 8 numbers that its rotation
// pairs up. The angles depend on row and chunk alone, so a thread finds its 8 sines and cosines once and
// uses them for every head.
//
// Bound by memory (rows with few query heads by issue slots: a KV head costs a thread about 440
// instructions, the angles 500, a query head 90), if enough of it is asked for in time: a thread copies its own chunks to shared memory
// with cp.async, kAhead heads ahead (query heads first, then a key and a value row per KV head), and reads
// them back without a barrier. Keys and values meet at one barrier per KV head, for the largest magnitude.
// That maximum is taken without a look at what is infinite (NaN drops out by itself); only a page where it
// comes out infinite is gone through again.

template <typename T>
struct Row8;  // 8 consecutive numbers
template <>
struct Row8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {  // numbers or NaN, no infinities
  uint2 u;
  const Two f(inv, inv);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) mul(Two(v[i], v[i + 1]), f).get(x[i], x[i + 1]);
  u.x = e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16);
  u.y = e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16);
  return u;
}

// Sines, negative sines and cosines of a thread's 8 angles.
struct Angles {
  Two s[4], n[4], c[4];
};
// Two pairs (x, y) turned by angles 2i and 2i + 1.
__device__ __forceinline__ void turn(const Angles& t, int i, float& x0, float& x1, float& y0, float& y1) {
  const Two x(x0, x1), y(y0, y1);
  fma(x, t.c[i], mul(y, t.n[i])).get(x0, x1);
  fma(y, t.c[i], mul(x, t.s[i])).get(y0, y1);
}
// Rotates across two chunks (halves of the rotated dims), or the pairs within one (interleaved).
__device__ __forceinline__ void rotate_across(float (&x)[8], float (&y)[8], const Angles& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) turn(t, i, x[2 * i], x[2 * i + 1], y[2 * i], y[2 * i + 1]);
}
template <int AT>
__device__ __forceinline__ void rotate_within(float (&x)[8], const Angles& t) {
#pragma unroll
  for (int i = 0; i < 2; ++i) turn(t, AT / 2 + i, x[4 * i], x[4 * i + 2], x[4 * i + 1], x[4 * i + 3]);
}

// The device checks of every sequence and page, by one CTA: the word is written, so nothing has to clear it
// before.
__device__ void check_ranges(const Kv8AppendArgs& a, int n_units, int* bits) {
  if (threadIdx.x == 0) *bits = 0;
  __syncthreads();
  int mine = 0;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x)
    if (!new_tokens(a, b).ok) mine |= LR_DEVERR_LEN;
  for (int u = threadIdx.x; u < n_units; u += blockDim.x) {
    const int b = sequence_of_unit(a, u);
    const NewTokens t = new_tokens(a, b);
    PageRows pr;
    if (page_rows(t.p0, t.n, u - unit_of(a, b), pr) &&
        (unsigned)__ldg(a.table + (size_t)b * a.max_pages + pr.page) >= (unsigned)a.n_pages)
      mine |= LR_DEVERR_PAGE;
  }
  if (mine) atomicOr(bits, mine);
  __syncthreads();
  if (threadIdx.x == 0) *a.err = *bits;
}

// Largest magnitude of 8 numbers, and of the finite ones alone.
__device__ __forceinline__ float top8(const Row8<__nv_bfloat16>& v) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v.u);
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 m = __hmax2(__hmax2(__hmax2(zero, __habs2(h[0])), __hmax2(zero, __habs2(h[1]))),
                                   __hmax2(__hmax2(zero, __habs2(h[2])), __hmax2(zero, __habs2(h[3]))));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float top8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
__device__ __forceinline__ float top8(const Row8<float>& v) {
  float f[8];
  v.get(f);
  return top8(f);
}
__device__ __forceinline__ uint32_t finite_top8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[i]));
  return m;
}

__device__ __forceinline__ void copy16(uint32_t smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(global) : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t smem) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem) : "memory");
  return v;
}

// Items in shared memory, under way or at work. A key and its value are at work together; four fp32 items
// would not fit at head_dim 256.
template <typename T>
constexpr int ahead() { return sizeof(T) == 2 ? 4 : 3; }
constexpr int kMaxWarps = 32;

// What the rotation does to a thread's chunks. One kernel per answer: asked of every thread and chunk, the
// question alone was most of the instructions.
enum class Turn { kNone, kAcross, kWithin, kMixed };  // kMixed: part of the row, or a chunk alone

template <typename T, Turn kTurn>
__global__ void __launch_bounds__(1024) kv8_append_kernel(Kv8AppendArgs a, int n_units) {
  constexpr int kAhead = ahead<T>();
  extern __shared__ __align__(16) uint8_t ring[];  // [kAhead][2 chunks][16-byte parts][thread]
  __shared__ uint32_t top[2][2][kMaxWarps];        // [parity][key, value][warp]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  const int u = blockIdx.x;
  if (u == n_units) {
    if (blockIdx.y == 0) check_ranges(a, n_units, (int*)top);
    return;
  }
  // the sequence of this unit, as sequence_of_unit finds it, 32 candidates a round
  int b = 0, len = a.B;
  while (len > 1) {
    const int step = (len + 31) / 32, at = b + lane * step;
    const bool below = lane * step < len && (lane == 0 || unit_of(a, at) <= u);
    const int n = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // the last candidate below (they ascend)
    b += n * step;
    len = min(step, len - n * step);
  }
  const NewTokens t = new_tokens(a, b);
  PageRows pr;
  if (!page_rows(t.p0, t.n, u - unit_of(a, b), pr)) return;
  const int pg = pr.page, first = pr.first;
  const int slot0 = first - pg * kBlock, rows = pr.end - first;  // new rows slot0 .. slot0 + rows - 1
  const int token0 = t.start + (first - t.p0);
  int page = __ldg(a.table + (size_t)b * a.max_pages + pg);
  if ((unsigned)page >= (unsigned)a.n_pages) page = -1;
  const int hd = a.hd, P = (hd + 15) / 16;  // chunk pairs of a row
  const int r = tid / P, p = tid % P;
  // The thread's chunks, as first dims, so that neighbours in the row are neighbours in the warp: the halves'
  // pairs and then the rest of the row in two halves, or all of it in two halves.
  int c0 = 8 * p, c1 = 8 * (P + p);
  bool across = kTurn == Turn::kAcross, within0 = kTurn == Turn::kWithin, within1 = within0, two = true;
  if (kTurn == Turn::kMixed) {
    if (!a.interleaved) {
      const int pairs = a.rot / 16;
      across = p < pairs;
      c0 = across ? 8 * p : a.rot + 8 * (p - pairs);
      c1 = across ? a.rot / 2 + 8 * p : a.rot + 8 * (P - pairs + p - pairs);
    }
    two = c1 < hd;  // head_dim an odd multiple of 8: one chunk is alone
    within0 = a.interleaved && c0 < a.rot;
    within1 = a.interleaved && c1 < a.rot;
  }
  const bool in = r < rows;
  const size_t token = (size_t)(token0 + (in ? r : 0));

  // items: this share's query heads, then key and value of its KV heads
  const int y = blockIdx.y, ny = gridDim.y;
  const int n_q = a.Hq > y ? (a.Hq - y - 1) / ny + 1 : 0, n_kv = page >= 0 && a.Hkv > y ? (a.Hkv - y - 1) / ny + 1 : 0;
  constexpr int kParts = sizeof(T) == 2 ? 1 : 2;  // 16 bytes each
  const uint32_t part_bytes = blockDim.x * 16, slot_bytes = 2 * kParts * part_bytes;
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(ring) + tid * 16;
  auto copy = [&](int slot, const T* src) {
    const uint32_t to = slots + slot * slot_bytes;
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
      copy16(to + x * part_bytes, reinterpret_cast<const uint4*>(src + c0) + x);
      if (two) copy16(to + (kParts + x) * part_bytes, reinterpret_cast<const uint4*>(src + c1) + x);
    }
  };
  auto take = [&](int slot, int chunk) {
    const uint32_t from = slots + slot * slot_bytes + chunk * kParts * part_bytes;
    Row8<T> v;
    uint4* to = reinterpret_cast<uint4*>(&v);
#pragma unroll
    for (int x = 0; x < kParts; ++x) to[x] = load16(from + x * part_bytes);
    return v;
  };
  // the next item to copy; the queries are counted up to whole rings, so that an item's slot is known
  const int n_q_ring = (n_q + kAhead - 1) / kAhead * kAhead, n_items = n_q_ring + 2 * n_kv, step = ny * hd;
  const T* q_next = (const T*)a.q + token * a.q_stride + y * hd;
  const T* k_next = (const T*)a.k + token * a.k_stride + y * hd;
  const T* v_next = (const T*)a.v + token * a.v_stride + y * hd;
  int next = 0;
  auto copy_next = [&](int slot) {
    if (next < n_q) {
      copy(slot, q_next);
      q_next += step;
    } else if (next >= n_q_ring && next < n_items) {
      copy(slot, (next - n_q_ring) & 1 ? v_next : k_next);
      if ((next - n_q_ring) & 1) v_next += step;
      else k_next += step;
    }
    ++next;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Angles angles;
  auto rotate = [&](float (&x0)[8], float (&x1)[8]) {
    if (across) rotate_across(x0, x1, angles);
    if (within0) rotate_within<0>(x0, angles);
    if (within1) rotate_within<4>(x1, angles);
  };
  if (in) {
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) copy_next(i);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      if (!(across || (i < 4 ? within0 : within1))) continue;
      const int pair = across ? c0 + i : i < 4 ? c0 / 2 + i : c1 / 2 + i - 4;
      const float2 f = __ldg(reinterpret_cast<const float2*>(a.inv_freq + pair));
      float s0, c0_, s1, c1_;
      sin_cos<T>(turn_fraction(f.x), first + r, s0, c0_);
      sin_cos<T>(turn_fraction(f.y), first + r, s1, c1_);
      angles.s[i / 2] = Two(s0, s1);
      angles.n[i / 2] = Two(-s0, -s1);
      angles.c[i / 2] = Two(c0_, c1_);
    }
    // queries
    T* out = (T*)a.q_out + (token * a.Hq + y) * hd;
    for (int i0 = 0; i0 < n_q_ring; i0 += kAhead) {
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
        if (i0 + x < n_q) {
          float v0[8], v1[8] = {};
          take(x, 0).get(v0);
          if (two) take(x, 1).get(v1);
          rotate(v0, v1);
          store8(out + c0, v0);
          if (two) store8(out + c1, v1);
          out += step;
        }
        copy_next((x + kAhead - 1) % kAhead);
      }
    }
  }

  // keys and values
  int ks = 0;  // slot of the key
  uint8_t* head[2];
  float* scale[2];
  if (n_kv > 0) {
    const size_t at = (size_t)page * a.page_stride + (size_t)y * kBlock * hd, sc = (size_t)page * a.Hkv + y;
    head[0] = a.kc + at;
    head[1] = a.vc + at;
    scale[0] = a.ks + sc;
    scale[1] = a.vs + sc;
  }
  const unsigned row = (unsigned)(slot0 + r) * hd;
  for (int j = 0; j < n_kv; ++j) {
    const int parity = j & 1, vs = ks + 1 < kAhead ? ks + 1 : 0;
    float held[2] = {0.f, 0.f};
    if (slot0 > 0) {
      held[0] = *scale[0];
      held[1] = *scale[1];
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 3) : "memory");  // both items
    float kx[2][8] = {};
    uint32_t mk = 0, mv = 0;
    if (in) {
      take(ks, 0).get(kx[0]);
      float m = top8(take(vs, 0));
      if (two) {
        take(ks, 1).get(kx[1]);
        m = fmaxf(m, top8(take(vs, 1)));
      }
      rotate(kx[0], kx[1]);
      mk = __float_as_uint(fmaxf(top8(kx[0]), top8(kx[1])));
      mv = __float_as_uint(m);
    }
    auto largest = [&](uint32_t (&row)[2][kMaxWarps], bool again) {
      mk = __reduce_max_sync(0xffffffffu, mk);
      mv = __reduce_max_sync(0xffffffffu, mv);
      if (again) __syncthreads();  // the first maxima have been read
      if (lane == 0) {
        row[0][warp] = mk;
        row[1][warp] = mv;
      }
      __syncthreads();
      mk = __reduce_max_sync(0xffffffffu, lane < n_warps ? row[0][lane] : 0u);
      mv = __reduce_max_sync(0xffffffffu, lane < n_warps ? row[1][lane] : 0u);
    };
    largest(top[parity], false);
    constexpr uint32_t kInf = 0x7f800000u;
    const bool infinite = mk >= kInf || mv >= kInf;
    if (infinite) {  // rare
      mk = mv = 0;
      if (in) {
        float v[8];
        mk = max(finite_top8(kx[0]), finite_top8(kx[1]));
        take(vs, 0).get(v);
        mv = finite_top8(v);
        if (two) {
          take(vs, 1).get(v);
          mv = max(mv, finite_top8(v));
        }
      }
      largest(top[parity], true);
    }
    const float now[2] = {fmaxf(held[0], pow2(scale_exp(mk))), fmaxf(held[1], pow2(scale_exp(mv)))};
    if (slot0 > 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (!(now[e] > held[e])) continue;  // the codes held before move to the new scale
        const float ratio = held[e] / now[e];
        for (int i = tid; i < slot0 * hd / 4; i += blockDim.x) {
          uint32_t* w = reinterpret_cast<uint32_t*>(head[e]) + i;
          *w = rescale4(*w, ratio);
        }
      }
    }
    if (tid < 2) *(tid ? scale[1] : scale[0]) = tid ? now[1] : now[0];
    if (in) {
      const bool dk = !is_pow2(now[0]), dv = !is_pow2(now[1]);
      const float ik = dk ? 1.f : __frcp_rn(now[0]), iv = dv ? 1.f : __frcp_rn(now[1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x && !two) break;
        float v[8];
        take(vs, x).get(v);
        const int at = x ? c1 : c0;
        if (infinite) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] = or_nan(v[i]);
            kx[x][i] = or_nan(kx[x][i]);
          }
        }
        if (dk) {
#pragma unroll
          for (int i = 0; i < 8; ++i) kx[x][i] = __fdiv_rn(kx[x][i], now[0]);
        }
        if (dv) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], now[1]);
        }
        *reinterpret_cast<uint2*>(head[0] + row + at) = codes8(kx[x], ik);
        *reinterpret_cast<uint2*>(head[1] + row + at) = codes8(v, iv);
      }
    }
    if (in) {
      copy_next(ks ? ks - 1 : kAhead - 1);
      copy_next(ks);
    }
    ks = vs + 1 < kAhead ? vs + 1 : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      head[e] += step * kBlock;
      scale[e] += ny;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T>
cudaError_t launch_append(const Kv8AppendArgs& a, int sm_count, cudaStream_t st) {
  if (!a.cu) {
    const long long warps = (long long)a.B * (a.Hkv + a.Hq);
    const unsigned grid = (unsigned)((warps + kOneWarps - 1) / kOneWarps) + 1;
    if (a.hd <= 128) kv8_append_one_kernel<T, 1><<<grid, 32 * kOneWarps, 0, st>>>(a);
    else kv8_append_one_kernel<T, 2><<<grid, 32 * kOneWarps, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int threads = kBlock * ((a.hd + 15) / 16);
  const int units = n_units(a);
  const int smem = ahead<T>() * 2 * 8 * (int)sizeof(T) * threads;
  const int ny = append_shares(a, threads, sm_count);
  void (*kernel)(Kv8AppendArgs, int) = kv8_append_kernel<T, Turn::kMixed>;
  if (a.hd % 16 == 0 && a.rot == 0) kernel = kv8_append_kernel<T, Turn::kNone>;
  else if (a.hd % 16 == 0 && a.rot == a.hd)
    kernel = a.interleaved ? kv8_append_kernel<T, Turn::kWithin> : kv8_append_kernel<T, Turn::kAcross>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)units + 1, (unsigned)ny);  // the last one checks
  kernel<<<grid, threads, smem, st>>>(a, units);
  return cudaGetLastError();
}

}  // namespace
}  // namespace kv8

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, lr_dtype dt, int sm_count, cudaStream_t st) {
  if (a.B == 0) return cudaMemsetAsync(a.err, 0, 256, st);
  return dt == LR_BF16 ? kv8::launch_append<__nv_bfloat16>(a, sm_count, st) : kv8::launch_append<float>(a, sm_count, st);
}

}  // namespace lr
