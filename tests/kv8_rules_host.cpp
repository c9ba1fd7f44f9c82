// The integer rules of the 8-bit paged cache as the kernels are compiled with them, for the host tests.
#include "kv8_rules.h"

using namespace lr::kv8;

extern "C" int kv8_page_rows(int p0, int n, int i, int* out) {
  PageRows r;
  if (!page_rows(p0, n, i, r)) return 0;
  out[0] = r.page;
  out[1] = r.first;
  out[2] = r.end;
  return 1;
}
