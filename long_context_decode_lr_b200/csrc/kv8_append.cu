// Appending new keys and values to the 8-bit paged cache, keys and queries rotated by their
// position on the way (rotary embedding).
//
// A page of one KV head has one scale for its keys and one for its values, a power of two, so
// raising it when larger numbers arrive shifts the codes' exponents and loses nothing but what
// falls under the smallest code. Whoever writes a page therefore owns it: one CTA (or warp, with one
// token per sequence) takes all of a call's rows of a page and head, finds their largest
// magnitude, settles the scale and writes the codes. Bound by memory: the rows are read once and
// stay in registers between the maximum and the rounding.
//
// Angles: a pair's frequency becomes a 64-bit fraction of a turn, so position * fraction wraps at
// whole turns by itself and far positions lose nothing; sincospif takes the top 32 bits.
#include <algorithm>

#include "kv8_common.cuh"

namespace lr {
namespace kv8 {
namespace {

constexpr int kMinExp = -24;  // smallest scale 2^-24: numbers under 2^-34 become 0

__device__ __forceinline__ uint64_t turn_fraction(float radians) {
  double t = (double)radians * 0.15915494309189533577;  // / 2 pi
  t -= floor(t);
  return (uint64_t)(t * 18446744073709551616.0);
}
__device__ __forceinline__ void sin_cos(uint64_t fraction, int pos, float& s, float& c) {
  const int32_t turns = (int32_t)((fraction * (uint64_t)(uint32_t)pos) >> 32);
  sincospif((float)turns * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
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
  const float s = fmaxf(held, fresh), inv = 1.f / s;
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
#pragma unroll
  for (int u = 0; u < Q; ++u) {
    const int i = lane + 32 * u;
    if (i >= quads) continue;
    int c0, c1;
    quad_dims(a, i, c0, c1);
    *reinterpret_cast<uint16_t*>(row + c0) = (uint16_t)codes2(x[u][0], x[u][1], inv);
    *reinterpret_cast<uint16_t*>(row + c1) = (uint16_t)codes2(x[u][2], x[u][3], inv);
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
      for (int e = 0; e < 2; ++e) sin_cos(turn_fraction(__ldg(a.inv_freq + 2 * i + e)), t.p0, s[e], c[e]);
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
// One CTA per page that receives tokens, for a share (blockIdx.y) of the heads. The CTA's threads are
// 32 rows x hd / 16 pairs of 8-number chunks; a thread has two rows of the page (r and r + 32) and
// two chunks of each head's row that its rotation pairs up. The angles depend on row and chunk
// alone, so a thread finds its 16 sines and cosines once and uses them for every head.
//
// Sequence b's pages are the units from cu[b] / 64 + 2 b on: always enough of them (n tokens touch
// at most n / 64 + 2 pages), without a scan over the batch.

template <typename T>
struct Row8;  // 8 consecutive numbers
template <>
struct Row8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
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
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
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
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  uint2 u;
  u.x = codes2(v[0], v[1], inv) | (codes2(v[2], v[3], inv) << 16);
  u.y = codes2(v[4], v[5], inv) | (codes2(v[6], v[7], inv) << 16);
  return u;
}

// Rotates a thread's two chunks: across them (halves) or within each (interleaved).
__device__ __forceinline__ void rotate8(bool interleaved, float (&x)[8], float (&y)[8], const float (&s)[8],
                                        const float (&c)[8]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = x[2 * i], a1 = x[2 * i + 1], b0 = y[2 * i], b1 = y[2 * i + 1];
      x[2 * i] = a0 * c[i] - a1 * s[i];
      x[2 * i + 1] = a1 * c[i] + a0 * s[i];
      y[2 * i] = b0 * c[4 + i] - b1 * s[4 + i];
      y[2 * i + 1] = b1 * c[4 + i] + b0 * s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a0 = x[i], a1 = y[i];
      x[i] = a0 * c[i] - a1 * s[i];
      y[i] = a1 * c[i] + a0 * s[i];
    }
  }
}

__device__ __forceinline__ int unit_of(const Kv8AppendArgs& a, int b) { return __ldg(a.cu + b) / kBlock + 2 * b; }

template <typename T>
__global__ void __launch_bounds__(512) kv8_append_kernel(Kv8AppendArgs a, int n_units) {
  __shared__ uint32_t top[2][2][16];  // [parity][key, value][warp]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  const int u = blockIdx.x;
  if (u >= n_units) {  // the device checks of the sequences
    const int b = (u - n_units) * blockDim.x + tid;
    if (blockIdx.y == 0 && b < a.B && !new_tokens(a, b).ok) flag_error(a.err, LR_DEVERR_LEN);
    return;
  }
  // the sequence of this unit: largest b with unit_of(b) <= u, 32 candidates a round
  int b = 0, len = a.B;
  while (len > 1) {
    const int step = (len + 31) / 32, at = b + lane * step;
    const bool below = lane * step < len && (lane == 0 || unit_of(a, at) <= u);
    const int n = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // the last candidate below (they ascend)
    b += n * step;
    len = min(step, len - n * step);
  }
  const int page_i = u - unit_of(a, b);
  const NewTokens t = new_tokens(a, b);
  if (page_i < 0 || !t.n) return;
  const int pg = t.p0 / kBlock + page_i;                      // page of the sequence
  const int first = max(t.p0, pg * kBlock), end = min(t.p0 + t.n, (pg + 1) * kBlock);
  if (first >= end) return;
  const int slot0 = first - pg * kBlock, rows = end - first;  // new rows slot0 .. slot0 + rows - 1
  const int token0 = t.start + (first - t.p0);
  int page = __ldg(a.table + (size_t)b * a.max_pages + pg);
  if ((unsigned)page >= (unsigned)a.n_pages) {
    if (tid == 0 && blockIdx.y == 0) flag_error(a.err, LR_DEVERR_PAGE);
    page = -1;
  }
  const int hd = a.hd, P = (hd + 15) / 16;  // chunk pairs of a row
  const int r0 = tid / P, p = tid % P;
  const int rot_pairs = a.rot / 16;
  int c0, c1;  // the thread's chunks, as first dims
  if (!a.interleaved && p < rot_pairs) {
    c0 = 8 * p;
    c1 = a.rot / 2 + 8 * p;
  } else {
    c0 = 16 * p;
    c1 = 16 * p + 8;
  }
  const bool rotated = p < rot_pairs, two = c1 < hd;  // head_dim an odd multiple of 8: the last chunk is alone
  float s[2][8], c[2][8];
  if (rotated) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t f = turn_fraction(__ldg(a.inv_freq + 8 * p + i));
#pragma unroll
      for (int x = 0; x < 2; ++x) sin_cos(f, first + r0 + 32 * x, s[x][i], c[x][i]);
    }
  }
  const bool in[2] = {r0 < rows, r0 + 32 < rows};

  // queries
  for (int h = blockIdx.y; h < a.Hq; h += gridDim.y) {
    Row8<T> raw[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!in[x]) continue;
      const T* src = (const T*)a.q + (size_t)(token0 + r0 + 32 * x) * a.q_stride + (size_t)h * hd;
      raw[x][0].load(src + c0);
      if (two) raw[x][1].load(src + c1);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!in[x]) continue;
      float v0[8], v1[8] = {};
      raw[x][0].get(v0);
      if (two) raw[x][1].get(v1);
      if (rotated) rotate8(a.interleaved, v0, v1, s[x], c[x]);
      T* out = (T*)a.q_out + ((size_t)(token0 + r0 + 32 * x) * a.Hq + h) * hd;
      store8(out + c0, v0);
      if (two) store8(out + c1, v1);
    }
  }
  if (page < 0) return;

  // keys and values
  int parity = 0;
  for (int h = blockIdx.y; h < a.Hkv; h += gridDim.y, parity ^= 1) {
    Row8<T> rk[2][2], rv[2][2];
    const size_t sc = (size_t)page * a.Hkv + h;
    float held[2] = {0.f, 0.f};
    if (slot0 > 0) {
      held[0] = a.ks[sc];
      held[1] = a.vs[sc];
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rk[x][e].zero();
        rv[x][e].zero();
      }
      if (!in[x]) continue;
      const size_t tok = (size_t)(token0 + r0 + 32 * x);
      const T* ksrc = (const T*)a.k + tok * a.k_stride + (size_t)h * hd;
      const T* vsrc = (const T*)a.v + tok * a.v_stride + (size_t)h * hd;
      rk[x][0].load(ksrc + c0);
      rv[x][0].load(vsrc + c0);
      if (two) {
        rk[x][1].load(ksrc + c1);
        rv[x][1].load(vsrc + c1);
      }
    }
    float kx[2][2][8];
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      rk[x][0].get(kx[x][0]);
      rk[x][1].get(kx[x][1]);
      if (rotated) rotate8(a.interleaved, kx[x][0], kx[x][1], s[x], c[x]);
      float v[8];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rv[x][e].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mv = max(mv, finite_bits(v[i]));
          mk = max(mk, in[x] ? finite_bits(kx[x][e][i]) : 0u);
        }
      }
    }
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if (lane == 0) {
      top[parity][0][warp] = mk;
      top[parity][1][warp] = mv;
    }
    __syncthreads();
    for (int w = 0; w < n_warps; ++w) {
      mk = max(mk, top[parity][0][w]);
      mv = max(mv, top[parity][1][w]);
    }
    const float now[2] = {fmaxf(held[0], pow2(scale_exp(mk))), fmaxf(held[1], pow2(scale_exp(mv)))};
    uint8_t* const head[2] = {a.kc + (size_t)page * a.page_stride + (size_t)h * kBlock * hd,
                              a.vc + (size_t)page * a.page_stride + (size_t)h * kBlock * hd};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (slot0 > 0 && now[e] > held[e]) {  // the codes held before move to the new scale
        const float ratio = held[e] / now[e];
        for (int i = tid; i < slot0 * hd / 4; i += blockDim.x) {
          uint32_t* w = reinterpret_cast<uint32_t*>(head[e]) + i;
          *w = rescale4(*w, ratio);
        }
      }
      if (tid == e) (e ? a.vs : a.ks)[sc] = now[e];
    }
    const float ik = 1.f / now[0], iv = 1.f / now[1];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!in[x]) continue;
      const size_t off = (size_t)(slot0 + r0 + 32 * x) * hd;
      float v[8];
      *reinterpret_cast<uint2*>(head[0] + off + c0) = codes8(kx[x][0], ik);
      rv[x][0].get(v);
      *reinterpret_cast<uint2*>(head[1] + off + c0) = codes8(v, iv);
      if (two) {
        *reinterpret_cast<uint2*>(head[0] + off + c1) = codes8(kx[x][1], ik);
        rv[x][1].get(v);
        *reinterpret_cast<uint2*>(head[1] + off + c1) = codes8(v, iv);
      }
    }
  }
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
  const cudaError_t e = cudaMemsetAsync(a.err, 0, 256, st);
  if (e != cudaSuccess) return e;
  const int threads = 32 * ((a.hd + 15) / 16);
  const int units = a.n_tokens / kBlock + 2 * a.B;
  // heads are shared out among CTAs until the grid fills the SMs four times over
  const int ny = std::min(a.Hkv, std::max(1, 4 * sm_count / std::max(1, units)));
  const dim3 grid((unsigned)(units + (a.B + threads - 1) / threads), (unsigned)ny);
  kv8_append_kernel<T><<<grid, threads, 0, st>>>(a, units);
  return cudaGetLastError();
}

}  // namespace
}  // namespace kv8

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, lr_dtype dt, int sm_count, cudaStream_t st) {
  if (a.B == 0) return cudaMemsetAsync(a.err, 0, 256, st);
  return dt == LR_BF16 ? kv8::launch_append<__nv_bfloat16>(a, sm_count, st) : kv8::launch_append<float>(a, sm_count, st);
}

}  // namespace lr
