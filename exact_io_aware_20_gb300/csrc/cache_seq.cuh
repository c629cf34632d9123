// Lengths of the sequences of a cache call, read on the device, and the flat
// order of its work (shared by the kernels of fa_cache_fwd.cu).
#pragma once

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

struct SeqParams {
  const int *seq_lens, *new_lens;
  int B, G, Nq, causal;
  long long capacity;   // tokens that a table row can map
  unsigned int* err;
};

// Tokens of sequence b and the query rows among them; both 0 when a length is
// out of range (*bad is set).
struct Sequence {
  int len, n;
};
__device__ __forceinline__ Sequence sequence_at(const SeqParams& p, int b, bool* bad) {
  Sequence s;
  s.len = p.seq_lens[b];
  s.n = p.new_lens != nullptr ? p.new_lens[b] : p.Nq;
  if (s.len < 0 || s.len > p.capacity || s.n < 0 || s.n > p.Nq) {
    *bad = true;
    s.len = s.n = 0;
  }
  return s;
}

// Rows of a key/value head are taken token by token, row r = i * G + g being
// query head g of token i, so that a tile of consecutive rows spans few
// tokens and a causal tile ends early.  `lim`: the keys that any row of the
// tile [r0, r1) sees; `full`: the keys that every one of its live rows sees.
struct TileLimits {
  int lim, full;
};
__device__ __forceinline__ TileLimits tile_limits(const SeqParams& p, const Sequence& s, int r0,
                                                  int r1) {
  const int i0 = r0 / p.G, i1 = min(s.n - 1, (r1 - 1) / p.G);
  TileLimits t;
  if (i0 > i1) {
    t.lim = t.full = 0;
  } else if (p.causal) {
    t.lim = max(0, s.len - s.n + i1 + 1);
    t.full = max(0, s.len - s.n + i0 + 1);
  } else {
    t.lim = t.full = s.len;
  }
  return t;
}

}  // namespace fa
