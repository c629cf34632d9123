// Rotary positions: angles, and the rotation of one 16-element slot of a row
// (the device side shared by fa_rope.cu and fa_cache_append.cu).
//
// The angle t * freq of a pair is kept as a 64-bit fraction of a turn: with
// F = freq / 2 pi * 2^64 modulo 2^64 (a whole number, off by less than one; the
// host forms it in more than a double), t * F in 64-bit integers is the angle
// modulo one turn to t * 2^-64 turns, where a product in fp32 loses t * 2^-24
// radians.  The quadrant is taken off in integers as well, and sin and cos of
// what is left, |a| <= pi / 4, are their Taylor polynomials (the first terms
// left out are a^11 / 11! < 1.8e-9 and a^12 / 12! < 1.2e-10, below half an fp32
// step): about 32 instructions a pair, no tables, no double precision, errors
// below 7.4e-8 (over all 2^32 angles that a quarter turn is cut into; 1.2e-8 and
// 1.9e-8 in the mean; the rounding of an exact value to fp32 is 1.1e-8 and
// 1.7e-8).
#pragma once

#include <cstdint>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

// cos and sin of `phase` / 2^64 turns (on the host too, where a test sweeps it).
__host__ __device__ __forceinline__ void turn_cos_sin(uint64_t phase, float& c, float& s) {
  const uint64_t quarter = phase + (1ull << 61);          // nearest quarter turn, in the top 2 bits
  const int q = static_cast<int>(quarter >> 62);
  const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(q) << 62));   // +- 2^61
  // a = n * 2 pi / 2^34, as an fp32 value and what its rounding left: without
  // the latter sin and cos are off by twice as much, which shows in how often a
  // key next to a border of two codes falls on the other side
  const int n = static_cast<int>(rest >> 30);
  // (the last 64 of them would round up to 2^31, which no int holds)
  const float fn = fminf(static_cast<float>(n), 2147483520.f);
  constexpr float kUnit = 3.65729529994141e-10f, kUnitRest = -1.0177350669805e-17f;
  const float a = fn * kUnit;
  float lo = fmaf(fn, kUnit, -a);
  lo = fmaf(fn, kUnitRest, lo);
  lo = fmaf(static_cast<float>(n - static_cast<int>(fn)), kUnit, lo);
  const float z = a * a;
  float ps = fmaf(z, 2.7557319224e-6f, -1.9841269841e-4f);   // 1/9!, -1/7!
  ps = fmaf(z, ps, 8.3333333333e-3f);                        // 1/5!
  ps = fmaf(z, ps, -1.6666666667e-1f);                       // -1/3!
  ps = a + fmaf(z * a, ps, lo);
  float pc = fmaf(z, -2.7557319224e-7f, 2.4801587302e-5f);   // -1/10!, 1/8!
  pc = fmaf(z, pc, -1.3888888889e-3f);                       // -1/6!
  pc = fmaf(z, pc, 4.1666666667e-2f);                        // 1/4!
  pc = fmaf(z, pc, -0.5f);
  pc = 1.0f + fmaf(z, pc, -(lo * a));
  const float x = (q & 1) ? ps : pc, y = (q & 1) ? pc : ps;
  c = (q == 1 || q == 2) ? -x : x;
  s = (q >= 2) ? -y : y;
}

// A row of d columns is d / 16 slots of two 8-element chunks each.  A rotated
// slot holds 8 pairs (interleaved: 16 consecutive columns; half-split: 8
// columns of each half), the others 16 consecutive columns that are copied.
struct Slot {
  int col_a, col_b;   // first columns of the chunks
  bool turns;
};
__device__ __forceinline__ Slot slot_of(const RopeArgs& r, int slot) {
  const int turning = r.pairs >> 3;
  Slot s;
  s.turns = slot < turning;
  const bool halves = s.turns && !r.interleaved;
  s.col_a = halves ? 8 * slot : 16 * slot;
  s.col_b = halves ? r.pairs + 8 * slot : 16 * slot + 8;
  return s;
}

// cos and sin of a rotated slot's 8 pairs for a token at `pos` (one entry an axis).
__device__ __forceinline__ void slot_cos_sin(const RopeArgs& r, int slot, const int (&pos)[4],
                                             float (&c)[8], float (&s)[8]) {
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int pair = 8 * slot + j;
    const int ax = r.axis[pair];
    const int t = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
    turn_cos_sin(static_cast<uint64_t>(static_cast<int64_t>(t)) * r.turn[pair], c[j], s[j]);
    s[j] = r.inverse ? -s[j] : s[j];
  }
}

// The positions of token n of sequence b on every axis; `own` where there are
// no positions.
__device__ __forceinline__ void load_positions(const RopeArgs& r, int b, int n, int N, int own,
                                               int (&pos)[4]) {
  #pragma unroll
  for (int a = 0; a < 4; ++a) {
    pos[a] = own;
    if (r.positions != nullptr && a < r.axes)
      pos[a] = r.positions[(static_cast<long long>(a) * r.pos_batch + (r.pos_batch > 1 ? b : 0)) * N + n];
  }
}

// The 16 values of a slot as pairs x1[8], x2[8] (chunks a and b as loaded).
template <bool BF16>
__device__ __forceinline__ void unpack_slot(uint4 a, uint4 b, bool by_pairs, float (&x1)[8],
                                            float (&x2)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = unpack2<BF16>(w[i]), hi = unpack2<BF16>(w[4 + i]);
    // by pairs: word i is pair i of the slot's first four, word 4 + i of its last four
    x1[by_pairs ? i : 2 * i] = lo.x;
    if (by_pairs) x2[i] = lo.y; else x1[2 * i + 1] = lo.y;
    if (by_pairs) x1[4 + i] = hi.x; else x2[2 * i] = hi.x;
    x2[by_pairs ? 4 + i : 2 * i + 1] = hi.y;
  }
}

__device__ __forceinline__ void turn_pairs(float (&x1)[8], float (&x2)[8], const float (&c)[8],
                                           const float (&s)[8]) {
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = x1[j], b = x2[j];
    x1[j] = fmaf(a, c[j], -(b * s[j]));
    x2[j] = fmaf(b, c[j], a * s[j]);
  }
}

// Rotates the 16 values of a slot, rounding each once.
template <bool BF16, bool BY_PAIRS>
__device__ __forceinline__ void turn_slot(uint4& a, uint4& b, const float (&c)[8],
                                          const float (&s)[8]) {
  float x1[8], x2[8];
  unpack_slot<BF16>(a, b, BY_PAIRS, x1, x2);
  turn_pairs(x1, x2, c, s);
  uint32_t w[8];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = BY_PAIRS ? pack2<BF16>(x1[i], x2[i]) : pack2<BF16>(x1[2 * i], x1[2 * i + 1]);
    w[4 + i] = BY_PAIRS ? pack2<BF16>(x1[4 + i], x2[4 + i]) : pack2<BF16>(x2[2 * i], x2[2 * i + 1]);
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}

// Rotates (or, without a rotation, copies) one slot of heads [h0, h1) of one
// token: heads below H are q's, the others k's.  Loads of kAhead heads are in
// flight together, the first ahead of the angles and each next one as soon as
// its registers are stored.  `live` false: zeros are written instead.
struct RopeRows {
  const uint16_t *q, *k;         // of this token's sequence and row (head 0, column 0)
  uint16_t *q_out, *k_out;
  long long q_h, k_h, q_out_h, k_out_h;   // head strides
  int H;
};
template <bool BF16, int kAhead>
__device__ __forceinline__ void rope_heads(const RopeArgs& r, const RopeRows& w, int slot, int h0,
                                           int h1, const int (&pos)[4], bool live) {
  const Slot at = slot_of(r, slot);
  uint4 a[kAhead], b[kAhead];
  auto load = [&](int u, int h) {
    a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
    if (h < h1 && live) {
      const uint16_t* src = h < w.H ? w.q + h * w.q_h : w.k + (h - w.H) * w.k_h;
      a[u] = *reinterpret_cast<const uint4*>(src + at.col_a);
      b[u] = *reinterpret_cast<const uint4*>(src + at.col_b);
    }
  };
  #pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, h0 + u);
  float c[8], s[8];
  if (at.turns) slot_cos_sin(r, slot, pos, c, s);
  for (int h = h0; h < h1; h += kAhead) {
    #pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (h + u < h1) {
        if (at.turns) {
          if (r.interleaved) turn_slot<BF16, true>(a[u], b[u], c, s);
          else turn_slot<BF16, false>(a[u], b[u], c, s);
        }
        uint16_t* dst = h + u < w.H ? w.q_out + (h + u) * w.q_out_h : w.k_out + (h + u - w.H) * w.k_out_h;
        *reinterpret_cast<uint4*>(dst + at.col_a) = a[u];
        *reinterpret_cast<uint4*>(dst + at.col_b) = b[u];
      }
      load(u, h + u + kAhead);
    }
  }
}

}  // namespace fa
