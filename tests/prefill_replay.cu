// Host entries over the parts of the prefill kernel that deal out its work, for tests without a GPU.
#include "../mxfp4_routed_expert_latentmoe_gb300/csrc/attn/k3_prefill.cuh"

namespace {
using namespace k3;

PrefillParams params(const int32_t* starts, const int32_t* lens, int B, int T, int Hkv, int G, int window, int sinks, int rows,
                     int longest) {
  PrefillParams p{};
  p.starts = starts;
  p.lens = lens;
  p.B = B;
  p.T = T;
  p.Hkv = Hkv;
  p.G = G;
  p.window = window;
  p.sinks = sinks;
  p.table_width = longest;
  p.c.page_size = 1;
  p.groups = (G + rows - 1) / rows;
  p.heads = (G + p.groups - 1) / p.groups;
  p.tokens = rows / p.heads;
  return p;
}
}  // namespace

extern "C" {

// The items of one block of `blocks`, 17 numbers each in the struct's order; returns their number (at most
// `most` are written), the total of places in *total.
int replay_items(const int32_t* starts, const int32_t* lens, int B, int T, int Hkv, int G, int window, int sinks, int rows,
                 int longest, int bn, int blocks, int block, int64_t* total, int32_t* items, int most) {
  const PrefillParams p = params(starts, lens, B, T, Hkv, G, window, sinks, rows, longest);
  const int HR = Hkv * p.groups;
  *total = 0;
  for (int b = 0; b < B; ++b) {
    int32_t s0, n, len;
    pre_bounds(p, b, s0, n, len);
    const PreSeq s = pre_seq(p, n, len);
    *total += s.place(s.tiles()) * HR;
  }
  const int64_t chunk = pre_chunk(*total, blocks), first = block * chunk;
  if (first >= *total) return 0;
  PreWalk w;
  w.bn = bn;
  w.chunk = chunk;
  w.end = first + chunk;
  int64_t before = 0;
  for (w.b = 0;; ++w.b) {
    int32_t s0, n, len;
    pre_bounds(p, w.b, s0, n, len);
    const PreSeq s = pre_seq(p, n, len);
    const int64_t here = s.place(s.tiles()) * HR;
    if (first < before + here) break;
    before += here;
  }
  w.land(p, first - before);
  PreItem it;
  int n = 0;
  for (; w.item(p, it); ++n)
    if (n < most) {
      const int32_t* x = reinterpret_cast<const int32_t*>(&it);
      for (int i = 0; i < 17; ++i) items[17 * n + i] = x[i];
    }
  return n;
}

// Places of a sequence's first m tiles: in closed form, and one by one.
void replay_place(int64_t n, int64_t old, int64_t window, int64_t sinks, int tokens, int64_t m, int64_t* got) {
  const PreSeq s{n, old, window, sinks, tokens};
  got[0] = s.place(m);
  got[1] = 0;
  for (int64_t i = 0; i < m; ++i) got[1] += s.keys(i) + PRE_START;
}

void replay_constants(int* x) {
  x[0] = PRE_START;
  x[1] = PRE_LEAST;
  x[2] = PRE_WHOLE;
}

}  // extern "C"
