// The integer rules of the 8-bit paged cache as the kernels are compiled with them, for the host tests. What the
// kernels do with a warp's or a CTA's threads together (the scan over the lengths, the search for a unit's sequence)
// is a plain loop here.
#include "kv8_rules.h"

using namespace lr::kv8;

extern "C" {

// ---- append

int kv8_page_rows(int p0, int n, int i, int* out) {
  PageRows r;
  if (!page_rows(p0, n, i, r)) return 0;
  out[0] = r.page;
  out[1] = r.first;
  out[2] = r.end;
  return 1;
}

struct Append {
  int B, n_tokens, Hkv, Hq;
  const int* cu;
};
int kv8_units(int B, int n_tokens) { return n_units(Append{B, n_tokens, 1, 1, nullptr}); }
int kv8_unit_of(const int* cu, int B, int b) { return unit_of(Append{B, cu[B], 1, 1, cu}, b); }
int kv8_sequence_of_unit(const int* cu, int B, int u) { return sequence_of_unit(Append{B, cu[B], 1, 1, cu}, u); }
int kv8_append_shares(int B, int n_tokens, int Hkv, int Hq, int threads, int sm_count) {
  return append_shares(Append{B, n_tokens, Hkv, Hq, nullptr}, threads, sm_count);
}

// ---- attention

struct Attn {
  int B, Hkv, max_pages, window, n_cta, cluster;
  const int* lens;
};

int kv8_small_cluster(int batch, int n_kv_heads, int max_pages, int tensor) {
  return small_cluster(batch, n_kv_heads, max_pages, tensor);
}

// Tiles and units of a sequence of len tokens: out = lo, n, page0, tiles, units.
void kv8_span(int max_pages, int window, int len, int* out) {
  const Span s = span_of(Attn{1, 1, max_pages, window, 1, 0, nullptr}, len);
  out[0] = s.lo;
  out[1] = s.n;
  out[2] = s.page0;
  out[3] = s.tiles;
  out[4] = s.units;
}

static Work work_of(const Attn& a, int c) {
  if (a.cluster) return small_work(a, c);
  Work w{};
  for (int b = 0; b < a.B; ++b) w.total += (long long)seq_span(a, b).units * a.Hkv;
  w.active = (int)least((long long)a.n_cta, w.total);
  if (c >= w.active) return w;
  w.begin = range_begin(w.total, c, w.active);
  w.end = range_begin(w.total, c + 1, w.active);
  for (long long first = 0; w.b < a.B; ++w.b) {
    const long long n = (long long)seq_span(a, w.b).units * a.Hkv;
    if (w.begin < first + n) {
      w.b_first = first;
      break;
    }
    first += n;
  }
  return w;
}

// What CTA c does: for each of its segments b, h, first tile, last + 1, whole, slot of a piece (at most `room`
// rows of 6); returns their number. record = the segment it writes down: head, n, then the slots of the pieces
// (at most `slots`). `visit` >= 0: every unit of the range is also looked up from the one `visit` units before it, as
// the loading warp does, and the tiles that it finds are counted into *seen.
int kv8_cta(const int* lens, int B, int Hkv, int max_pages, int window, int n_cta, int cluster, int c, int* out, int room,
            int* record, int slots, int visit, long long* seen) {
  const Attn a{B, Hkv, max_pages, window, n_cta, cluster, lens};
  const Work w = work_of(a, c);
  Walk<Attn> k(a, w);
  int n = 0;
  while (k.next() && n < room) {
    int* o = out + 6 * n++;
    o[0] = k.b;
    o[1] = k.h;
    o[2] = k.tile0;
    o[3] = k.tile1;
    o[4] = k.whole();
    o[5] = piece_slot(w, c, k.seg_first);
  }
  const Pieces p = cluster ? Pieces{0, 0, 0, 0} : pieces_of(a, w, c);
  record[0] = p.head;
  record[1] = p.n;
  for (int i = 0; i < p.n && i < slots; ++i) record[2 + i] = p.slot(i);
  if (visit >= 0 && w.begin < w.end) {
    for (int first = 0; first < most(visit, 1); ++first) {
      Place at;
      at.start(a, w);
      for (long long u = w.begin + first; u < w.end; u += most(visit, 1)) {
        at.seek(a, u);
        if (at.tile >= at.sp.tiles) continue;
        for (int i = 0; i < n; ++i)
          if (out[6 * i] == at.b && out[6 * i + 1] == at.h && at.tile >= out[6 * i + 2] && at.tile < out[6 * i + 3]) ++*seen;
      }
    }
  }
  return n;
}

}  // extern "C"
