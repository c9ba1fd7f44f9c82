// Integer rules of the 8-bit paged cache, for the kernels and for host code alike (no CUDA needed).
#pragma once

#include "lowram.h"

#ifdef __CUDACC__
#define LR_HD __host__ __device__ __forceinline__
#else
#define LR_HD inline
#endif

namespace lr {
namespace kv8 {

constexpr int kPage = LR_BLOCK_TOKENS;  // tokens of a page

// The positions [first, end) of a page of a sequence that receive new tokens.
struct PageRows {
  int page;  // index in the sequence
  int first, end;
};
// Page i, counted from 0, of those that n new tokens from position p0 on go to; false behind the last one. A
// sequence may end at the last page boundary that an int holds: page indices are compared, and no position behind
// the sequence is formed.
LR_HD bool page_rows(int p0, int n, int i, PageRows& r) {
  if (n < 1 || i < 0) return false;
  const int page0 = p0 / kPage, last = (p0 + n - 1) / kPage;
  if (i > last - page0) return false;
  r.page = page0 + i;
  r.first = i == 0 ? p0 : r.page * kPage;
  r.end = r.page == last ? p0 + n : (r.page + 1) * kPage;
  return true;
}

}  // namespace kv8
}  // namespace lr
