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
// k and v, 4 an element of q; 4 x 4099 tokens of 32 + 2 x 8 heads, d = 128: 73 us,
// 5.1 TB/s, 76% of what a copy reaches), latency for single tokens (64
// sequences: 5.0 us).  Everything is one launch: the first blocks hold the
// units, the rest walk q's heads.
#include <algorithm>

#include <cuda_fp8.h>

#include "rope.cuh"

namespace fa {
namespace {

// Block-wide units to aim at: without q they have to fill the chip by
// themselves; with it few and long ones leave the memory to q's blocks (prompts
// of 4 x 4099 tokens, 2 / 4 / 8 an SM: 72 / 77 / 81 us with q, 57 / 48 / 51
// without).
inline int units_wanted(bool q, int sms) { return (q ? 2 : 4) * sms; }

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
  int unit_heads;       // heads that a block-wide unit does one after another
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

__device__ __forceinline__ float finite_max(float m, const float (&x)[16]) {
  #pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float a = fabsf(x[j]);
    m = a < __uint_as_float(0x7f800000u) ? fmaxf(m, a) : m;
  }
  return m;
}

// The 16 values of a slot from its two chunks as loaded.
template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& c, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = unpack2<BF16>(w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}
__device__ __forceinline__ void turn16(float (&x)[16], const float (&c)[8], const float (&s)[8],
                                       bool interleaved) {
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (interleaved) {
      const float u = x[2 * j], v = x[2 * j + 1];
      x[2 * j] = fmaf(u, c[j], -(v * s[j]));
      x[2 * j + 1] = fmaf(v, c[j], u * s[j]);
    } else {
      const float u = x[j], v = x[8 + j];
      x[j] = fmaf(u, c[j], -(v * s[j]));
      x[8 + j] = fmaf(v, c[j], u * s[j]);
    }
  }
}

// What a unit's threads know of its page.
struct Target {
  int r0, rows;         // rows that stay, and new rows behind them
  int i0, start;        // the first new row's number in k and v, and the sequence's first new token
  int phys;             // the page
};
__device__ __forceinline__ bool target_of(const AppendParams& p, int b, int j, bool report, Target& t) {
  Sequence s;
  if (!sequence_of(p, b, s)) {
    if (report && j == 0) atomicOr(p.err, kErrCache);
    return false;
  }
  t.start = s.len - s.n;
  const int number = (t.start >> p.page_log2) + j;      // page of the sequence
  const long long first = static_cast<long long>(number) << p.page_log2;   // its first token
  if (first >= s.len || s.n == 0) return false;
  t.phys = p.cache.table[static_cast<long long>(b) * p.cache.width + number];
  if (static_cast<unsigned>(t.phys) >= static_cast<unsigned>(p.cache.pages)) {
    if (report) atomicOr(p.err, kErrCache);
    return false;
  }
  t.r0 = first < t.start ? t.start - static_cast<int>(first) : 0;
  t.rows = min(1 << p.page_log2, s.len - static_cast<int>(first)) - t.r0;
  t.i0 = static_cast<int>(first) + t.r0 - t.start;
  return true;
}

// Codes of a slot's 16 values, at its two places in a row.
__device__ __forceinline__ void put16(unsigned char* row, const Slot& where, const float (&x)[16],
                                      float inv) {
  const uint2 a = to_codes(x, inv), c = to_codes(x + 8, inv);
  if (where.col_b == where.col_a + 8) {
    *reinterpret_cast<uint4*>(row + where.col_a) = make_uint4(a.x, a.y, c.x, c.y);
  } else {
    *reinterpret_cast<uint2*>(row + where.col_a) = a;
    *reinterpret_cast<uint2*>(row + where.col_b) = c;
  }
}

// A unit: one page, K or V, of one head for a warp (GROUP 32, four units a
// block) and of unit_heads heads, one after another, for a block.  A thread
// keeps up to HOLD slots of the new rows between the two passes over them, as
// they were loaded; a block's keeps the angles' cos and sin, which every head
// shares, in shared memory of its own (16 floats a slot: with them in
// registers too few threads were resident to keep memory busy, and worked out
// anew for each head they took as long as the loads), and has the next head's
// rows in flight.  HOLD 0: rows are read (from L2) and rotated again, for
// pages of more slots than that.
template <bool BF16, int GROUP, int HOLD>
__global__ void __launch_bounds__(GROUP == 32 ? 128 : GROUP, GROUP == 256 || GROUP == 32 ? 4 : 2)
append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kThreads = GROUP == 32 ? 128 : GROUP;
  constexpr int kUnits = kThreads / GROUP;
  constexpr bool kAngles = GROUP > 32 && HOLD > 0;     // in shared memory
  __shared__ float red[2][GROUP > 32 ? GROUP / 32 : 1];
  extern __shared__ float4 angles[];                   // [HOLD][4][thread]
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
    uint16_t* to = p.q_out + b * p.qos.b + n * p.qos.n;
    const uint16_t* from = p.q + b * p.qs.b + n * p.qs.n;
    const RopeRows w = {from, from, to, to, p.qs.h, p.qs.h, p.qos.h, p.qos.h, p.H};
    const int h0 = group * p.q_heads_per;
    rope_heads<BF16, 2>(p.r, w, slot, h0, min(p.H, h0 + p.q_heads_per), pos, ok && n < s.n);
    return;
  }
  const int unit = blockIdx.x * kUnits + tid / GROUP;
  const int t = tid % GROUP;
  if (unit >= p.units) return;   // (whole groups; a block-wide group never has one left over)
  // units in the order (b, page of the span, K or V, head group)
  const Cache& ca = p.cache;
  const int groups = (ca.Hkv + p.unit_heads - 1) / p.unit_heads;
  const int h0 = unit % groups * p.unit_heads, h1 = min(ca.Hkv, h0 + p.unit_heads);
  const bool key = (unit / groups & 1) == 0;
  const int b = unit / (2 * groups) / p.span;
  Target at;
  if (!target_of(p, b, unit / (2 * groups) % p.span, t == 0, at)) return;
  const Strides in = key ? p.ks : p.vs, to = key ? ca.ks : ca.vs;
  const uint16_t* src = (key ? p.k : p.v) + b * in.b + at.i0 * in.n;
  unsigned char* page = (key ? ca.k : ca.v) + at.phys * to.b;
  float* scales = (key ? ca.k_scale : ca.v_scale) + static_cast<long long>(at.phys) * ca.Hkv;
  const int count = at.rows * p.slots;
  const bool turn = key && p.r.pairs > 0;
  auto slot_at = [&](int slot) -> Slot {
    if (turn) return slot_of(p.r, slot);
    return {16 * slot, 16 * slot + 8, false};
  };
  auto cos_sin = [&](int i, int slot, float (&c)[8], float (&s)[8]) {
    int pos[4];
    load_positions(p.r, b, at.i0 + i, p.N, at.start + at.i0 + i, pos);
    slot_cos_sin(p.r, slot, pos, c, s);
  };
  // one slot of one new row of head h, rotated
  auto values = [&](int h, int n, float (&x)[16]) {
    const int i = n / p.slots, slot = n % p.slots;
    const Slot w = slot_at(slot);
    const uint16_t* row = src + h * in.h + i * in.n;
    unpack16<BF16>(*reinterpret_cast<const uint4*>(row + w.col_a),
                   *reinterpret_cast<const uint4*>(row + w.col_b), x);
    if (w.turns) {
      float c[8], s[8];
      cos_sin(i, slot, c, s);
      turn16(x, c, s, p.r.interleaved);
    }
  };

  constexpr int kHold = HOLD > 0 ? HOLD : 1;
  uint4 raw[kHold][2];
  auto load = [&](int h) {
    #pragma unroll
    for (int u = 0; u < kHold; ++u) {
      const int n = t + u * GROUP;
      if (n < count) {
        const Slot w = slot_at(n % p.slots);
        const uint16_t* row = src + h * in.h + (n / p.slots) * in.n;
        raw[u][0] = *reinterpret_cast<const uint4*>(row + w.col_a);
        raw[u][1] = *reinterpret_cast<const uint4*>(row + w.col_b);
      }
    }
  };
  if constexpr (HOLD > 0) load(h0);
  if constexpr (kAngles) {
    if (turn) {
      #pragma unroll
      for (int u = 0; u < kHold; ++u) {
        const int n = t + u * GROUP;
        if (n < count && slot_at(n % p.slots).turns) {
          float c[8], s[8];
          cos_sin(n / p.slots, n % p.slots, c, s);
          #pragma unroll
          for (int i = 0; i < 2; ++i) {
            angles[(4 * u + i) * GROUP + t] = make_float4(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]);
            angles[(4 * u + 2 + i) * GROUP + t] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
          }
        }
      }
    }
  }
  // slot u of the head held, rotated
  auto held = [&](const uint4 (&v)[2], int u, float (&x)[16]) {
    unpack16<BF16>(v[0], v[1], x);
    const int n = t + u * GROUP;
    if (turn && slot_at(n % p.slots).turns) {
      float c[8], s[8];
      if constexpr (kAngles) {
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 a = angles[(4 * u + i) * GROUP + t], e = angles[(4 * u + 2 + i) * GROUP + t];
          c[4 * i] = a.x, c[4 * i + 1] = a.y, c[4 * i + 2] = a.z, c[4 * i + 3] = a.w;
          s[4 * i] = e.x, s[4 * i + 1] = e.y, s[4 * i + 2] = e.z, s[4 * i + 3] = e.w;
        }
      } else {
        cos_sin(n / p.slots, n % p.slots, c, s);
      }
      turn16(x, c, s, p.r.interleaved);
    }
  };
  for (int h = h0; h < h1; ++h) {
    uint4 now_raw[kHold][2];
    float kept[kHold][16];      // a warp's unit has one head: its rows stay as rotated
    const float was = at.r0 > 0 ? scales[h] : 0.f;
    float amax = 0.f;
    if constexpr (HOLD > 0) {
      #pragma unroll
      for (int u = 0; u < kHold; ++u) {
        now_raw[u][0] = raw[u][0];
        now_raw[u][1] = raw[u][1];
      }
      if (h + 1 < h1) load(h + 1);
      #pragma unroll
      for (int u = 0; u < kHold; ++u)
        if (t + u * GROUP < count) {
          held(now_raw[u], u, kept[u]);
          amax = finite_max(amax, kept[u]);
        }
    } else {
      for (int n = t; n < count; n += GROUP) {
        float x[16];
        values(h, n, x);
        amax = finite_max(amax, x);
      }
    }
    #pragma unroll
    for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    if constexpr (GROUP > 32) {
      // (two places by turns: one barrier a head; it also says that every
      // thread has read the old scale)
      float* mine = red[(h - h0) & 1];
      if ((tid & 31) == 0) mine[tid >> 5] = amax;
      __syncthreads();
      #pragma unroll
      for (int i = 0; i < GROUP / 32; ++i) amax = fmaxf(amax, mine[i]);
    } else {
      __syncwarp();
    }
    const float now = fmaxf(scale_for(amax), was);
    const float inv = 1.f / now;
    unsigned char* dst = page + h * to.h;
    if (t == 0) scales[h] = now;
    if (at.r0 > 0 && now > was) {
      const float ratio = was * inv;
      for (int n = t; n < at.r0 * p.slots; n += GROUP) {
        uint4* code = reinterpret_cast<uint4*>(dst + (n / p.slots) * to.n + (n % p.slots) * 16);
        *code = rescaled(*code, ratio);
      }
    }
    if constexpr (HOLD > 0) {
      #pragma unroll
      for (int u = 0; u < kHold; ++u) {
        const int n = t + u * GROUP;
        if (n < count) {
          if constexpr (kAngles) held(now_raw[u], u, kept[u]);
          put16(dst + (at.r0 + n / p.slots) * to.n, slot_at(n % p.slots), kept[u], inv);
        }
      }
    } else {
      for (int n = t; n < count; n += GROUP) {
        float x[16];
        values(h, n, x);
        put16(dst + (at.r0 + n / p.slots) * to.n, slot_at(n % p.slots), x, inv);
      }
    }
  }
}

template <int GROUP, int HOLD>
cudaError_t launch(AppendParams& p, int bf16, int sms, cudaStream_t stream) {
  constexpr int kThreads = GROUP == 32 ? 128 : GROUP;
  // Heads of a unit: all of them when there are pages enough to fill the chip
  // without (angles are then worked out once a page), one when there are few.
  const long long pages = 2ll * p.B * p.span;
  p.unit_heads = GROUP == 32 || HOLD == 0
                     ? 1
                     : static_cast<int>(std::max(1ll, std::min<long long>(
                           p.cache.Hkv, pages * p.cache.Hkv / units_wanted(p.q != nullptr, sms))));
  const int groups = (p.cache.Hkv + p.unit_heads - 1) / p.unit_heads;
  p.unit_heads = (p.cache.Hkv + groups - 1) / groups;      // evenly
  const long long units = pages * groups;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  p.units = static_cast<int>(units);
  p.unit_blocks = (p.units + kThreads / GROUP - 1) / (kThreads / GROUP);
  long long blocks = p.unit_blocks;
  if (p.q != nullptr) {
    const long long q_groups = (p.H + p.q_heads_per - 1) / p.q_heads_per;
    blocks += (p.q_items * q_groups + kThreads - 1) / kThreads;
  }
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  constexpr size_t smem = GROUP > 32 ? HOLD * 64 * GROUP : 0;
  auto kern = bf16 ? append_kernel<true, GROUP, HOLD> : append_kernel<false, GROUP, HOLD>;
  if constexpr (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const Cache& cache, const AppendCall& c, const RopeArgs& r,
                                int sms, cudaStream_t stream) {
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
  p.q_items = static_cast<long long>(c.B) * c.N * p.slots;
  // q's heads of a thread: fewer threads than the rotary kernel's, beside the
  // units' (256 / 512 / 1024 an SM: 6 x 333 padded tokens of 16 + 2 x 16 heads on
  // three axes 9.6 / 10.5 / 12.8 us, 512 tokens of 32 + 2 x 8 heads 8.4 / 9.3 /
  // 10.1, long prompts the same).
  const long long groups =
      std::max(1ll, std::min<long long>(std::max(c.H, 1), 256ll * sms / p.q_items));
  p.q_heads_per = std::min<long long>(16, (std::max(c.H, 1) + groups - 1) / groups);
  p.seq_lens = c.seq_lens;
  p.new_lens = c.new_lens;
  p.err = c.err;
  p.r = r;
  // The slots of the new rows of a page: a warp holds up to 64 of them, 256
  // threads 512, 512 threads 1024; larger pages are read twice, their angles
  // worked out for every head and both times, which shows (4 x 4099 tokens behind
  // 300, floor 55 us: 32 + 2 x 8 heads at d = 128, pages of 64 / 128 / 256 take
  // 73 / 81 / 120 us; 16 + 2 x 4 heads at d = 256, pages of 64 / 128 90 / 175).
  const int count = std::min(c.N, cache.page) * p.slots;
  if (count <= 64) return launch<32, 2>(p, c.bf16, sms, stream);
  if (count <= 512) return launch<256, 2>(p, c.bf16, sms, stream);
  if (count <= 1024) return launch<512, 2>(p, c.bf16, sms, stream);
  return launch<512, 0>(p, c.bf16, sms, stream);
}

}  // namespace fa
