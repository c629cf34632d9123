// Appending keys and values to the paged 8-bit cache, the keys rotated on the
// way, and q rotated for the attention that follows (fa_cache_append).
//
// A unit is one page of one head of K or of V that receives tokens: its
// threads read the new rows once (rotating keys in fp32 registers), find the
// largest magnitude, settle the page's scale, and round the rows to e4m3.
// Tokens that the page holds already keep their codes unless the scale grows;
// scales are powers of two, so that rounding them again is a shift of the
// exponent, exact for all but subnormal codes, and so that the power of two
// costs no precision (e4m3 has the same three mantissa bits in every octave).
//
// What bounds it: memory for prompts (2 bytes read and 1 written an element of
// k and v, 4 an element of q), latency for single tokens.  Everything is one
// launch: the first blocks hold the units, the rest walk q's heads.
#include <algorithm>

#include <cuda_fp8.h>

#include "rope.cuh"

namespace fa {
namespace {

struct AppendParams {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  Strides qs, ks, vs, qos;
  Cache cache;
  int B, H, N;
  int slots;            // of a row
  int page_log2;
  int span;             // pages that N tokens can touch
  int units, unit_blocks;
  int q_heads_per;      // heads of a thread of q's blocks
  long long q_items;    // B * N * slots
  const int *seq_lens, *new_lens;
  unsigned int* err;
  RopeArgs r;
};

// The new tokens of sequence b; false (and the error word) when its lengths
// are out of range.
struct Sequence {
  int len, n;
};
__device__ __forceinline__ bool sequence_of(const AppendParams& p, int b, Sequence& s) {
  s.len = p.seq_lens[b];
  s.n = p.new_lens != nullptr ? p.new_lens[b] : p.N;
  return s.n >= 0 && s.n <= p.N && s.len >= s.n &&
         s.len <= (static_cast<long long>(p.cache.width) << p.page_log2);
}

// The smallest 2^e >= 2^-100 with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -100) + 127) << 23);
}

// Eight values over the scale (inv = 1 / scale) as codes; NaN and infinities
// become NaN.
__device__ __forceinline__ uint2 to_codes(const float* x, float inv) {
  uint32_t w[2];
  #pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 v = make_float2(x[4 * i + 2 * j] * inv, x[4 * i + 2 * j + 1] * inv);
      if (!(fabsf(v.x) < __uint_as_float(0x7f800000u))) v.x = __uint_as_float(0x7fffffffu);
      if (!(fabsf(v.y) < __uint_as_float(0x7f800000u))) v.y = __uint_as_float(0x7fffffffu);
      w[i] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3))
              << (16 * j);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Sixteen codes for a scale `ratio` (<= 1) times their own.
__device__ __forceinline__ uint4 rescaled(uint4 v, float ratio) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t out = 0;
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(w[i] >> (16 * j));
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
      out |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                 make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE, __NV_E4M3))
             << (16 * j);
    }
    w[i] = out;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One slot of one new row: its 16 values in fp32 (keys rotated), in the order
// of its two chunks.
template <bool BF16>
__device__ __forceinline__ void slot_values(const AppendParams& p, const uint16_t* rows,
                                            long long row_stride, bool key, int b, int start,
                                            int i, int slot, const Slot& at, float (&x)[16]) {
  const uint16_t* src = rows + i * row_stride;
  const uint4 a = *reinterpret_cast<const uint4*>(src + at.col_a);
  const uint4 c = *reinterpret_cast<const uint4*>(src + at.col_b);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = unpack2<BF16>(w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
  if (key && at.turns) {
    int pos[4];
    load_positions(p.r, b, i, p.N, start + i, pos);
    float cs[8], sn[8];
    slot_cos_sin(p.r, slot, pos, cs, sn);
    if (p.r.interleaved) {
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = x[2 * j], v = x[2 * j + 1];
        x[2 * j] = fmaf(u, cs[j], -(v * sn[j]));
        x[2 * j + 1] = fmaf(v, cs[j], u * sn[j]);
      }
    } else {
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = x[j], v = x[8 + j];
        x[j] = fmaf(u, cs[j], -(v * sn[j]));
        x[8 + j] = fmaf(v, cs[j], u * sn[j]);
      }
    }
  }
}

__device__ __forceinline__ float finite_max(float m, const float (&x)[16]) {
  #pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float a = fabsf(x[j]);
    m = a < __uint_as_float(0x7f800000u) ? fmaxf(m, a) : m;
  }
  return m;
}

// GROUP threads do a unit (32: four units a block, no block barrier).  HOLD:
// slots that a thread keeps in registers between the two passes over the new
// rows; 0: it reads (from L2) and rotates them again, for pages of more slots
// than registers.
template <bool BF16, int GROUP, int HOLD>
__global__ void __launch_bounds__(GROUP == 32 ? 128 : GROUP)
append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kThreads = GROUP == 32 ? 128 : GROUP;
  constexpr int kUnits = kThreads / GROUP;
  __shared__ float red[32];
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= p.unit_blocks) {
    // q: rotated (or copied), zeros behind a sequence's new tokens
    const long long item =
        (static_cast<long long>(blockIdx.x) - p.unit_blocks) * kThreads + tid;
    const int groups = (p.H + p.q_heads_per - 1) / p.q_heads_per;
    if (item >= p.q_items * groups) return;
    const int slot = static_cast<int>(item % p.slots);
    const long long rest = item / p.slots;
    const int n = static_cast<int>(rest % p.N);
    const int group = static_cast<int>(rest / p.N % groups);
    const int b = static_cast<int>(rest / p.N / groups);
    Sequence s;
    const bool ok = sequence_of(p, b, s);
    int pos[4];
    load_positions(p.r, b, n, p.N, s.len - s.n + n, pos);
    RopeRows w;
    w.in[0] = w.in[1] = p.q + b * p.qs.b + n * p.qs.n;
    w.out[0] = w.out[1] = p.q_out + b * p.qos.b + n * p.qos.n;
    w.in_h[0] = w.in_h[1] = p.qs.h;
    w.out_h[0] = w.out_h[1] = p.qos.h;
    w.H = p.H;
    const int h0 = group * p.q_heads_per;
    rope_heads<BF16>(p.r, w, slot, h0, min(p.H, h0 + p.q_heads_per), pos, ok && n < s.n);
    return;
  }
  const int unit = blockIdx.x * kUnits + tid / GROUP;
  const int t = tid % GROUP;
  if (unit >= p.units) return;   // (whole groups; a block-wide group never has one left over)
  // units in the order (b, page of the span, K or V, head)
  const Cache& ca = p.cache;
  const int h = unit % ca.Hkv;
  const bool key = (unit / ca.Hkv & 1) == 0;
  const int j = unit / (2 * ca.Hkv) % p.span;
  const int b = unit / (2 * ca.Hkv) / p.span;
  Sequence s;
  if (!sequence_of(p, b, s)) {
    if (t == 0 && j == 0) atomicOr(p.err, kErrCache);
    return;
  }
  const int start = s.len - s.n, page = 1 << p.page_log2;
  const int number = (start >> p.page_log2) + j;      // page of the sequence
  const long long first = static_cast<long long>(number) << p.page_log2;   // its first token
  if (first >= s.len || s.n == 0) return;
  const int phys = ca.table[static_cast<long long>(b) * ca.width + number];
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(ca.pages)) {
    if (t == 0) atomicOr(p.err, kErrCache);
    return;
  }
  const int r0 = first < start ? start - static_cast<int>(first) : 0;      // rows that stay
  const int rows = min(page, s.len - static_cast<int>(first)) - r0;        // new rows
  const int i0 = static_cast<int>(first) + r0 - start;                     // the first of them in k, v
  const Strides in = key ? p.ks : p.vs, to = key ? ca.ks : ca.vs;
  const uint16_t* src = (key ? p.k : p.v) + b * in.b + h * in.h;
  unsigned char* dst = (key ? ca.k : ca.v) + phys * to.b + h * to.h;
  float* scale = (key ? ca.k_scale : ca.v_scale) + static_cast<long long>(phys) * ca.Hkv + h;
  const float was = r0 > 0 ? *scale : 0.f;
  const int count = rows * p.slots;
  const bool turn = key && p.r.pairs > 0;
  auto slot_at = [&](int slot) -> Slot {
    if (turn) return slot_of(p.r, slot);
    return {16 * slot, 16 * slot + 8, false};
  };

  float amax = 0.f;
  float held[HOLD > 0 ? HOLD : 1][16];
  if constexpr (HOLD > 0) {
    #pragma unroll
    for (int u = 0; u < HOLD; ++u) {
      const int at = t + u * GROUP;
      if (at < count) {
        const int slot = at % p.slots;
        slot_values<BF16>(p, src, in.n, turn, b, start, i0 + at / p.slots, slot, slot_at(slot),
                          held[u]);
        amax = finite_max(amax, held[u]);
      }
    }
  } else {
    for (int at = t; at < count; at += GROUP) {
      const int slot = at % p.slots;
      float x[16];
      slot_values<BF16>(p, src, in.n, turn, b, start, i0 + at / p.slots, slot, slot_at(slot), x);
      amax = finite_max(amax, x);
    }
  }
  #pragma unroll
  for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  if constexpr (GROUP > 32) {
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();   // (and every thread has read the old scale)
    #pragma unroll
    for (int i = 0; i < GROUP / 32; ++i) amax = fmaxf(amax, red[i]);
  } else {
    __syncwarp();
  }
  const float now = fmaxf(scale_for(amax), was);
  const float inv = 1.f / now;
  if (t == 0) *scale = now;
  if (r0 > 0 && now > was) {
    const float ratio = was * inv;
    for (int at = t; at < r0 * p.slots; at += GROUP) {
      uint4* code = reinterpret_cast<uint4*>(dst + (at / p.slots) * to.n + (at % p.slots) * 16);
      *code = rescaled(*code, ratio);
    }
  }
  auto put = [&](int at, const float (&x)[16]) {
    const int slot = at % p.slots;
    const Slot where = slot_at(slot);
    unsigned char* row = dst + (r0 + at / p.slots) * to.n;
    const uint2 a = to_codes(x, inv), c = to_codes(x + 8, inv);
    if (where.col_b == where.col_a + 8) {
      *reinterpret_cast<uint4*>(row + where.col_a) = make_uint4(a.x, a.y, c.x, c.y);
    } else {
      *reinterpret_cast<uint2*>(row + where.col_a) = a;
      *reinterpret_cast<uint2*>(row + where.col_b) = c;
    }
  };
  if constexpr (HOLD > 0) {
    #pragma unroll
    for (int u = 0; u < HOLD; ++u)
      if (t + u * GROUP < count) put(t + u * GROUP, held[u]);
  } else {
    for (int at = t; at < count; at += GROUP) {
      const int slot = at % p.slots;
      float x[16];
      slot_values<BF16>(p, src, in.n, turn, b, start, i0 + at / p.slots, slot, slot_at(slot), x);
      put(at, x);
    }
  }
}

template <int GROUP, int HOLD>
cudaError_t launch(AppendParams& p, int bf16, cudaStream_t stream) {
  constexpr int kThreads = GROUP == 32 ? 128 : GROUP;
  p.unit_blocks = (p.units + kThreads / GROUP - 1) / (kThreads / GROUP);
  long long blocks = p.unit_blocks;
  if (p.q != nullptr) {
    const long long groups = (p.H + p.q_heads_per - 1) / p.q_heads_per;
    blocks += (p.q_items * groups + kThreads - 1) / kThreads;
  }
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (bf16) append_kernel<true, GROUP, HOLD><<<grid, kThreads, 0, stream>>>(p);
  else append_kernel<false, GROUP, HOLD><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const Cache& cache, const AppendCall& c, const RopeArgs& r,
                                cudaStream_t stream) {
  AppendParams p = {};
  p.q = static_cast<const uint16_t*>(c.q);
  p.k = static_cast<const uint16_t*>(c.k);
  p.v = static_cast<const uint16_t*>(c.v);
  p.q_out = static_cast<uint16_t*>(c.q_out);
  p.qs = c.qs;
  p.ks = c.ks;
  p.vs = c.vs;
  p.qos = c.qos;
  p.cache = cache;
  p.B = c.B;
  p.H = c.H;
  p.N = c.N;
  p.slots = cache.d / 16;
  while ((1 << p.page_log2) < cache.page) ++p.page_log2;
  p.span = (c.N - 1 + cache.page - 1) / cache.page + 1;
  const long long units = 2ll * c.B * p.span * cache.Hkv;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  p.units = static_cast<int>(units);
  p.q_items = static_cast<long long>(c.B) * c.N * p.slots;
  const long long groups =
      std::max(1ll, std::min<long long>(std::max(c.H, 1), 2048ll * 152 / p.q_items));
  p.q_heads_per = (std::max(c.H, 1) + groups - 1) / groups;
  p.seq_lens = c.seq_lens;
  p.new_lens = c.new_lens;
  p.err = c.err;
  p.r = r;
  // The slots of the new rows of a page: a warp holds up to 64 of them, 256
  // threads 512, 512 threads 1024; larger pages are read twice.
  const int count = std::min(c.N, cache.page) * p.slots;
  if (count <= 64) return launch<32, 2>(p, c.bf16, stream);
  if (count <= 512) return launch<256, 2>(p, c.bf16, stream);
  if (count <= 1024) return launch<512, 2>(p, c.bf16, stream);
  return launch<512, 0>(p, c.bf16, stream);
}

}  // namespace fa
