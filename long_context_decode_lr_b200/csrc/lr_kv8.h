// Launch arguments of the 8-bit paged cache (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "lowram.h"

namespace lr {

struct Kv8AppendArgs {
  int B, Hkv, Hq, hd, n_pages, max_pages, n_tokens;
  long long page_stride;  // bytes
  uint8_t* kc;            // [n_pages] x [Hkv, 64, hd]
  uint8_t* vc;
  float* ks;              // [n_pages, Hkv]
  float* vs;
  const int* table;       // [B, max_pages]
  const int* lens;        // [B], the new tokens counted
  const int* cu;          // [B + 1] or null (one token per sequence)
  const void* q;          // [n_tokens, Hq, hd] rows q_stride elements apart, or null
  const void* k;          // [n_tokens, Hkv, hd]
  const void* v;
  long long q_stride, k_stride, v_stride;
  void* q_out;            // [n_tokens, Hq, hd] dense
  const float* inv_freq;  // [rot / 2]
  int rot, interleaved;
  int* err;
};
cudaError_t launch_kv8_append(const Kv8AppendArgs& a, lr_dtype dt, int sm_count, cudaStream_t st);

struct Kv8AttnArgs {
  int B, Hkv, G, hd, n_pages, max_pages, window;
  long long page_stride;
  float scale;            // times log2(e): scores in units of 2^x
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  const int* table;
  const int* lens;
  const void* q;          // [B, Hq, hd]
  const void* o_prev;     // [B, Hq, hd] or null
  const float* lse_prev;  // [B, Hq]
  void* o;                // [B, Hq, hd]
  float* lse;             // [B, Hq] or null
  int* err;
  int* cta_err;           // [n_cta] device error bits of each CTA, joined into *err
  void* split;            // [n_cta] kv8::Pieces: the split segment that each CTA wrote down
  float* part;            // [2 n_cta] slots of part_stride floats: acc [G, hd] (in units of kv8::kSumUnit), max [8], sum [8]
  int n_cta;
  int part_stride;
  int cluster;            // 0, or CTAs of a cluster that has a segment to itself and joins it (small calls)
};
struct Kv8AttnPlan {
  bool tensor;            // the tcgen05 kernel (bf16, head_dim 128)
  int cluster;
  int n_cta;
  int part_stride;
  size_t split_off, cta_err_off, part_off, ws_bytes;
};
Kv8AttnPlan plan_kv8_attn(const lr_kv8_pages& kv, int n_q_heads, int sm_count);
// Tensor map of a pool of pages with head_dim 128, a box one page of one head (plan.cu).
bool kv8_page_map(CUtensorMap* m, const uint8_t* codes, const Kv8AttnArgs& a);
cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, const Kv8AttnPlan& plan, lr_dtype dt, cudaStream_t st);

namespace kv8 {
cudaError_t launch_attn_tc(const Kv8AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st);
}

}  // namespace lr
