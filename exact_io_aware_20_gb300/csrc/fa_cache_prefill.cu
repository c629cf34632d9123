// Attention over the paged 8-bit cache for many query rows (chunks of prompts,
// and whole ones): the same formulas as fa_cache_fwd.cu on the tensor cores of
// tcgen05, tiles of 128 query rows x 128 keys.
//
// Scores.  The keys' codes are the products' operand as they are: TMA copies
// them from the pages into the swizzled layout, and q becomes 8-bit parts
// q 2^e = q1 + q2 (+ q3), each what the ones before have left, the largest
// element in [2^7, 2^8); S is their sum in fp32.  An e4m3 part takes four
// significant bits, so two hold a bf16 (8 bits) and three an f16 (11).  The last
// part is e5m2: what is left by then has at most three bits, which is all that
// e5m2 holds, and its steps go down to 2^-16, where those of e4m3 end at 2^-9.
// So q is exact but for elements below 2^-13 (f16: 2^-10) of the row's largest,
// which are off by 2^-21 of it at most, less than the fp32 sums (with e4m3
// throughout it was 2^-17 for those below 2^-6, which showed in rows with one
// column far above the rest).  8-bit products run at twice the rate of 16-bit
// ones, so two parts cost what one f16 product of widened keys would, and no
// key passes through a register (the change from keys widened to f16 as
// well took a chunk from 325 to 282 us).
//
// Values are widened to f16 (exact) by warps of their own, which follow the
// page table row by row and write swizzled shared memory, the next tile's loads
// in flight: 64 conversions a clock an SM, an eighth of a tile's time at
// d <= 128, where one conversion serves two tiles of query rows (256 rows,
// every head of a key/value head's group among them).  At d = 256 TMEM holds
// one tile's O.
//
// The keys' scale multiplies the scores and the values' scale goes into the
// exponent, both by groups of keys that a page holds for certain (64, 32 or 16
// by the page size): the group's largest raw score is scaled, not each score,
// and the exponent's multiply-add takes the scales for the rest (the chunk
// below with pages of 64 takes 173 us, with pages of 16 195).
//
// Roles: warps 0-3 softmax of tile A, 4-7 of tile B (d = 256: conversion),
// 8-11 conversion and q, 12 issues the products, 13 walks the share and
// describes its pieces to the others, 14 finds the pages and scales of the
// tiles to come, 15 copies the keys.  512 threads start with 128 registers
// each, which the groups then share out by their need.  With 210 KB of tiles
// next to none of the SM's storage is left as L1, so a register that spills
// costs a trip to L2, and what is in nobody's loop is fetched anew each time:
// the walk lives in one warp, and a piece's start and end are small loops (O
// rescaled by 16 columns in a loop instead of by 32 unrolled: pages of 16, 240
// -> 222 us; eight lanes' results brought together by shuffles so that they
// fill lines, in more code: d = 256 308 -> 315 us, not kept).
//
// Measured (2 chunks of 512 tokens against up to 16384, 32 heads on 8, d = 128,
// bf16): 173 us, 1260 TFLOP/s; d = 256, f16, four causal prompts of 4096
// tokens, 8 heads: 300 us, 915 TFLOP/s.  What bounds it: at d <= 128 a tile pair
// takes about 2900 clocks for 2048 of products, the softmax of each row tile
// (400 for the maximum, 950 for the weights) and the products of the other by
// turns; at d = 256 about 3800 for 2560, where one softmax group has nothing to
// take turns with, and a piece's start and end, when O is read out and the
// next q is taken apart (copies for timing without q, without the
// results and without the join: 19, 18 and 17 us less of then 302).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache_work.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;

template <int D>
struct Pre {
  static constexpr int kTiles = D == 256 ? 1 : 2;
  static constexpr int kRows = 128 * kTiles;        // of a unit
  // A unit's cost besides its steps, in steps.  d = 256, 3 / 4 / 5 / 6 / 7 / 8:
  // causal prompts of 4 x 4096 take 322 / 311 / 301 / 305 / 321 / 326 us, of
  // 8 x 1024 135 / 135 / 132 / 136 / 138 / 144, of 8192 249 / 238 / 236 / 237 /
  // 240 / 243, ragged chunks of 1500 82 / 82 / 77 / 78 / 80 / 80.  d = 128, 4 / 5 /
  // 6 / 8 / 10 / 12: 4 x 2048 121 / 124 / 117 / 117 / 115 / 119, 8 x 1000 158 / 156 /
  // 154 / 154 / 162 / 155, 8192 265 / 246 / 240 / 244 / 244 / 248; d = 64,
  // 4 x 2048: 90 / 97 / 89 / 96 / 90 / 98.  (How shares fall on a shape moves a
  // time by up to 8% either way; 5 and 6 are within 2% of the best on each.)
  static constexpr int kOver = kTiles == 1 ? 5 : 6;
  static constexpr int kSoftWarps = 4 * kTiles;
  static constexpr int kConvWarps = 12 - kSoftWarps;
  static constexpr int kConvRows = 128 / kConvWarps;   // keys of a tile that a warp converts
  static constexpr int kChunks = D / 64;            // 64-column parts
  static constexpr int kQParts = 3;                 // 8-bit parts of q at most
  static constexpr int kQPart = 128 * D;            // one part of a tile of rows
  static constexpr int kQTile = kQParts * kQPart;
  static constexpr int kKCols = D < 128 ? D : 128;  // K: 128 keys x kKCols codes
  static constexpr int kKParts = D / kKCols;
  static constexpr int kKPiece = 128 * kKCols;
  static constexpr int kKStages = D == 64 ? 4 : 3;
  static constexpr int kVKeys = D == 256 ? 64 : 128;   // V: kVKeys keys x D columns, f16
  static constexpr int kVParts = 128 / kVKeys;
  static constexpr int kVPiece = kVKeys * D * 2;
  static constexpr int kVStages = D == 64 ? 4 : 2;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kTiles * kQTile;
  static constexpr int kVOff = kKOff + kKStages * kKPiece;
  // By 16-key group, of eight tiles: the scales (ks, log2 vs, 2^-7 / vs); where
  // the group's V begins, its page and its first row there
  static constexpr int kMetaOff = kVOff + kVStages * kVPiece;
  static constexpr int kWhereOff = kMetaOff + 8 * 8 * 16;
  static constexpr int kPowOff = kWhereOff + 8 * 8 * 16;        // [2 pieces][rows] of q
  static constexpr int kRecOff = kPowOff + 2 * kRows * 4;       // [4 pieces] (Piece)
  static constexpr int kBarOff = kRecOff + 4 * 64;
  static constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kKEmpty = kKFull + kKStages,
                       kVFull = kKEmpty + kKStages, kVEmpty = kVFull + kVStages,
                       kSFull = kVEmpty + kVStages, kPFull = kSFull + 2, kODone = kPFull + 2,
                       kDrain = kODone + 2, kRecFull = kDrain + 1, kRecEmpty = kRecFull + 4,
                       kTileFull = kRecEmpty + 4, kTileEmpty = kTileFull + 8,
                       kNumBars = kTileEmpty + 8;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kRedOff = (kMiscOff + 48 + 15) / 16 * 16;   // start: sums and the found entry
  static constexpr int kBytes = kRedOff + 2 * 16 * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kTS = 0, kTO = 256, kTmemCols = 512;
  // registers a thread: the launch's 4 * 128 among the four warpgroups
  static constexpr int kRegSoft = 176;
  static constexpr int kRegMisc = kTiles == 1 ? 80 : 64;
  static constexpr int kRegConv = (512 - kTiles * kRegSoft - kRegMisc) / (3 - kTiles);
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
  static_assert(256 + kTiles * D <= 512, "TMEM budget");
};

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 bytes of global memory (where `on` is false: zeros).  Kept in program
// order with the other volatile asm, so that a load is issued where it stands,
// a tile ahead of its use: left to the compiler the loads of a tile were
// waited for one by one.
__device__ __forceinline__ void load_16(uint4& x, const void* src) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(src));
}
__device__ __forceinline__ void load_16_if(uint4& x, const void* src, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
      : "l"(src), "r"(static_cast<uint32_t>(on)));
}

// Reads of shared memory by its own address: through a generic pointer they
// queue with the loads of global memory (the eight scales of a tile's first
// pass took 600 clocks instead of 100).
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ const unsigned char* ld_shared_ptr(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(addr));
  return reinterpret_cast<const unsigned char*>(v);
}

// A piece of a unit, as the scheduling warp describes it to the others.
struct Piece {
  int s0, s1;          // its steps; s1 < 0: there are no more pieces
  int end[2];          // end of each row tile's steps
  int full[2];         // the keys that every live row of the tile sees
  int all;             // ... that every live row of both tiles sees
  int lim;             // the keys that any row sees
  int b, h, row0;      // sequence, key/value head, first row
  int len, n;          // of the sequence
  int whole;           // the piece is a whole unit
};
static_assert(sizeof(Piece) <= 64, "a record's place");
struct __align__(16) Where {
  const unsigned char* v;
  int page, row;
};

// D[tmem] (+)= A[smem] * B[smem], both 8 bits: kSteps products of 32 columns, one
// after another along a row of both.  One election and one predicate for all of
// them: the warp that issues is what the tensor pipe waits for.
template <int kSteps>
__device__ __forceinline__ void mma_rows_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  static_assert(kSteps == 2 || kSteps == 4, "columns of a row");
  if constexpr (kSteps == 2)
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], f16: four products of 16 keys (8 columns of A,
// 2048 bytes of B each).
__device__ __forceinline__ void mma_64_keys(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f8f6f4: fp32 sums, both operands K-major, A e4m3
// (type 0) or e5m2 (type 1), B e4m3.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_e5m2) {
  return (1u << 4) | (static_cast<uint32_t>(a_e5m2) << 7) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// Shared-memory descriptor of K-major rows of COLS bytes (128: 128-byte
// swizzle, 64: 64-byte swizzle), eight rows after eight.
template <int COLS>
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr) {
  uint64_t d = smem_desc_sw128(addr, 16, 8 * COLS);
  if constexpr (COLS == 64) d = (d & ~(7ull << 61)) | (4ull << 61);
  return d;
}
// Byte offset of 16-byte chunk c of row r there.
template <int COLS>
__device__ __forceinline__ uint32_t row_chunk(int r, int c) {
  return COLS == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// The larger of two pairs of 16-bit patterns without sign (of bf16 and f16
// magnitudes: NaN is the largest).
__device__ __forceinline__ uint32_t max_16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Two f16 -> two e4m3 codes (the low 16 bits); x becomes what the codes leave
// of it (exact in f16).
__device__ __forceinline__ uint32_t take_e4m3(uint32_t& x) {
  uint16_t two;
  uint32_t back;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(two) : "r"(x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(two));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(back));
  return two;
}
// Two f16 -> two e5m2 codes (the low 16 bits).
__device__ __forceinline__ uint32_t to_e5m2(uint32_t x) {
  uint16_t two;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(two) : "r"(x));
  return two;
}

// This thread's row of O in TMEM times alpha.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t tO, float alpha) {
  tc_fence_after();
  #pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint32_t o[16];
    tmem_ld16(tO + 16 * c, o);
    tmem_ld_wait();
    reg_fence(o);
    #pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st16(tO + 16 * c, o);
  }
  tmem_st_wait();
}

// SEG: keys that share their scales for certain (a page's, 64 at most).
template <int D, int SEG>
__global__ void __launch_bounds__(kThreads, 1)
cache_prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ FwdCacheParams p) {
  using L = Pre<D>;
  using W = Walk<L::kRows, 128, L::kOver>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  volatile int* nan_seen = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 8);   // [8 pieces]
  long long* red = reinterpret_cast<long long*>(smem + L::kRedOff);
  longlong2* found = reinterpret_cast<longlong2*>(smem + L::kRedOff + 256);
  float4* meta = reinterpret_cast<float4*>(smem + L::kMetaOff);
  Where* where = reinterpret_cast<Where*>(smem + L::kWhereOff);
  float* q_pow = reinterpret_cast<float*>(smem + L::kPowOff);
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBarOff + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(bar(L::kQFull), L::kConvWarps);
    mbar_init(bar(L::kQEmpty), 1);
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(bar(L::kKFull + s), 1);
      mbar_init(bar(L::kKEmpty + s), 1);
    }
    for (int s = 0; s < L::kVStages; ++s) {
      mbar_init(bar(L::kVFull + s), L::kConvWarps / L::kVParts);   // (a warp's rows lie in one piece)
      mbar_init(bar(L::kVEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::kSFull + s), 1);
      mbar_init(bar(L::kPFull + s), 4);   // one arrival per softmax warp
      mbar_init(bar(L::kODone + s), 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(L::kRecFull + s), 1);
      // (read by the products, pages and keys warps, the converters and softmax)
      mbar_init(bar(L::kRecEmpty + s), 3 + L::kConvWarps + L::kSoftWarps);
    }
    for (int s = 0; s < 8; ++s) {
      nan_seen[s] = 0;
      mbar_init(bar(L::kTileFull + s), 1);
      mbar_init(bar(L::kTileEmpty + s), 1);
    }
    mbar_init(bar(L::kDrain), 1);
    *abort = 0;
    fence_barrier_init();
  }
  bool bad = false;
  long long lo = 0, hi = 0, share = 0;
  find_place<L::kRows, 128, L::kOver, kThreads>(p, red, found, &bad, [&](long long count) {
    const long long total = count * p.Hkv;
    share = (total + p.ctas - 1) / p.ctas;
    lo = blockIdx.x * share;
    hi = min(total, lo + share);
    return lo < hi ? lo / p.Hkv : -1ll;
  });
  if (bad && blockIdx.x == 0) atomicOr(p.seq.err, kErrCache);
  if (threadIdx.x == 0) p.joins[blockIdx.x] = make_int4(0, 0, -1, 0);
  if (lo >= hi) return;
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_holder), L::kTmemCols);
    tmem_relinquish();
  }
  W at;
  if (warp == 13) at.start(p, found, lo, hi - lo);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // piece np, once it is there; and this warp has no more need of it
  auto piece = [&](int np) { return reinterpret_cast<const volatile Piece*>(smem + L::kRecOff + (np & 3) * 64); };
  auto piece_wait = [&](int np) { return wait_uniform(bar(L::kRecFull + (np & 3)), (np >> 2) & 1, abort); };
  auto piece_done = [&](int np) { mbar_arrive_warp(bar(L::kRecEmpty + (np & 3))); };

  if (warp >= 12) {
    fewer_registers<L::kRegMisc>();
    if (warp == 13) {
      // -------------------------------------------------------- schedule
      for (int np = 0;; ++np) {
        if (np >= 4 && !wait_uniform(bar(L::kRecEmpty + (np & 3)), ((np >> 2) + 1) & 1, abort)) break;
        volatile Piece* w = reinterpret_cast<volatile Piece*>(smem + L::kRecOff + (np & 3) * 64);
        const int s1 = at.next(p) ? at.s1 : -1;
        if (lane == 0) {
          w->s0 = at.s0;
          w->s1 = s1;
          if (s1 >= 0) {
            const int row0 = at.e % p.row_tiles * L::kRows;
            int all = 0x7fffffff;
            #pragma unroll
            for (int u = 0; u < L::kTiles; ++u) {
              const int r0 = row0 + 128 * u, r1 = min(p.rows, r0 + 128);
              TileLimits t = {0, 0};
              if (r0 < r1) t = tile_limits(p.seq, at.seq, r0, r1);
              const int end = min(s1, (t.lim + 127) / 128);
              w->end[u] = end;
              w->full[u] = t.full;
              if (end > at.s0) all = min(all, t.full);
            }
            w->all = all;
            w->lim = at.lim;
            w->b = at.e / p.row_tiles;
            w->h = at.h;
            w->row0 = row0;
            w->len = at.seq.len;
            w->n = at.seq.n;
            w->whole = at.s0 == 0 && s1 == at.steps;
            // the unit begins here and goes on behind this share, which ends
            // where the piece does: its last place, and whose that is
            if (at.s0 == 0 && s1 < at.steps)
              p.joins[blockIdx.x] =
                  make_int4(at.e, at.h, static_cast<int>((hi - 1 + at.steps - s1) / share), at.seq.n);
          }
        }
        __syncwarp();
        if (elect_one()) mbar_arrive(bar(L::kRecFull + (np & 3)));
        __syncwarp();
        if (s1 < 0) break;
      }
    } else if (warp == 14) {
      // ----------------------------------------------------------- pages
      // Of every tile, up to eight ahead of the products.  Four tiles at a
      // time: lane 8 t + i finds the page and scales of group i of tile t.
      int g = 0;
      bool ok = true;
      for (int np = 0; ok; ++np) {
        if (!piece_wait(np)) break;
        const int s0 = piece(np)->s0, s1 = piece(np)->s1, lim = piece(np)->lim, h = piece(np)->h;
        const int* row = p.table + static_cast<long long>(piece(np)->b) * p.width;
        piece_done(np);
        if (s1 < 0) break;
        for (int j = s0; ok && j < s1; j += 4) {
          const int key = j * 128 + 16 * lane;
          const bool on = key < lim;
          int page = 0;
          if (on) {
            page = row[key >> p.page_log2];
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) {
              atomicOr(p.seq.err, kErrCache);
              page = 0;
            }
          }
          const long long sc = static_cast<long long>(page) * p.Hkv + h;
          const float ks = on ? p.k_scale[sc] : 1.f, lv = on ? log2f(p.v_scale[sc]) : 0.f;
          const int r = key & ((1 << p.page_log2) - 1), i = lane & 7;
          for (int t = 0; t < min(4, s1 - j); ++t, ++g) {
            if (g >= 8 && !wait_uniform(bar(L::kTileEmpty + (g & 7)), ((g >> 3) + 1) & 1, abort)) {
              ok = false;
              break;
            }
            if (lane >> 3 == t) {
              meta[(g & 7) * 8 + i] = make_float4(ks, lv, ex2_approx(-lv) * kHeadInv, 0.f);
              Where* w = where + (g & 7) * 8 + i;
              w->v = p.v + page * p.vs.b + h * p.vs.h + r * p.vs.n;
              w->page = page;
              w->row = r;
            }
            mbar_arrive_warp(bar(L::kTileFull + (g & 7)));
          }
        }
      }
    } else if (warp == 15) {
      // ------------------------------------------------------------ keys
      // Codes as they are, a box of a page (at most 128 rows) at a time; rows
      // past the keys that any row sees are left as they were (their scores
      // are masked).
      if (elect_one()) tma_prefetch_desc(&tm_k);
      __syncwarp();
      const int box_log2 = min(p.page_log2, 7);
      int g = 0, kp = 0;
      bool ok = true;
      for (int np = 0; ok; ++np) {
        if (!piece_wait(np)) break;
        const int s0 = piece(np)->s0, s1 = piece(np)->s1, lim = piece(np)->lim, h = piece(np)->h;
        piece_done(np);
        if (s1 < 0) break;
        for (int j = s0; ok && j < s1; ++j, ++g) {
          if (!wait_uniform(bar(L::kTileFull + (g & 7)), (g >> 3) & 1, abort)) { ok = false; break; }
          const int boxes = min(128 >> box_log2, (lim - j * 128 + (1 << box_log2) - 1) >> box_log2);
          #pragma unroll 1
          for (int c = 0; c < L::kKParts; ++c) {
            const int s = kp % L::kKStages;
            if (kp >= L::kKStages && !wait_uniform(bar(L::kKEmpty + s), (kp / L::kKStages + 1) & 1, abort)) {
              ok = false;
              break;
            }
            if (elect_one()) {
              const uint32_t full = bar(L::kKFull + s), dst = sbase + L::kKOff + s * L::kKPiece;
              mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes * L::kKCols) << box_log2);
              for (int i = 0; i < boxes; ++i) {
                const Where* w = where + (g & 7) * 8 + (i << (box_log2 - 4));
                tma_load_4d(dst + (static_cast<uint32_t>(i * L::kKCols) << box_log2), &tm_k, full,
                            c * L::kKCols, w->row, h, w->page);
              }
            }
            __syncwarp();
            ++kp;
          }
        }
      }
      for (int i = max(0, kp - L::kKStages); i < kp; ++i)
        drain_wait(bar(L::kKFull + i % L::kKStages), (i / L::kKStages) & 1);
    } else if (warp == 12) {
      // ---------------------------------------------------------- products
      constexpr uint32_t kIdS = idesc_f8(128, 128, 0), kIdLast = idesc_f8(128, 128, 1);
      constexpr uint32_t kIdO = idesc_f16(128, D, 0, 0, 1);
      const uint64_t q_desc = rows_desc<L::kKCols>(sbase + L::kQOff);
      const uint64_t k_desc = rows_desc<L::kKCols>(sbase + L::kKOff);
      const int q_parts = p.bf16 ? 2 : 3;
      const uint64_t v_desc = smem_desc_sw128(sbase + L::kVOff, L::kVKeys * 128, 1024);
      int kp = 0, vp = 0;                 // pieces of K and V consumed
      int pf[2] = {0, 0};                 // P_FULL phases consumed, by score buffer
      bool ok = true;
      // Products are issued by small loops: a tile's run of them unrolled does
      // not stay in the instruction cache beside the other roles' loops, and
      // issuing took longer than the products.
      // S (+)= part c of Q K^T of row tile u, into score buffer `buf`, from the
      // K piece in place s
      auto scores = [&](int u, int buf, int c, int s) {
        uint64_t qs = desc_add(q_desc, u * L::kQTile + c * (128 * L::kKCols));
        const uint64_t ks = desc_add(k_desc, s * L::kKPiece);
        uint32_t more = c > 0;
        #pragma unroll 1
        for (int q = 0; q < q_parts; ++q) {
          mma_rows_f8<L::kKCols / 32>(tmem + L::kTS + 128 * buf, qs, ks, q + 1 < q_parts ? kIdS : kIdLast, more);
          qs = desc_add(qs, L::kQPart);
          more = 1;
        }
      };
      // O (+)= part h of P V of row tile u, P from score buffer `buf`, from the
      // V piece in place s
      auto values = [&](int u, int buf, int h, int s, bool fresh) {
        uint64_t vs = desc_add(v_desc, s * L::kVPiece);
        uint32_t from = tmem + L::kTS + 128 * buf + h * (L::kVKeys / 2);
        uint32_t more = !fresh || h > 0;
        #pragma unroll
        for (int w = 0; w < L::kVKeys / 64; ++w) {
          mma_64_keys(tmem + L::kTO + D * u, from, vs, kIdO, more);
          vs = desc_add(vs, 64 * 128);
          from += 32;
          more = 1;
        }
      };
      auto k_wait = [&](int n) { return wait_uniform(bar(L::kKFull + n % L::kKStages), (n / L::kKStages) & 1, abort); };
      auto v_wait = [&](int n) { return wait_uniform(bar(L::kVFull + n % L::kVStages), (n / L::kVStages) & 1, abort); };
      auto lane0 = [&](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      int g = 0;   // tiles so far
      for (int np = 0; ok; ++np) {
        if (!piece_wait(np)) break;
        struct { int s0, s1, end[2]; } w;
        w.s0 = lane0(piece(np)->s0);
        w.s1 = lane0(piece(np)->s1);
        w.end[0] = lane0(piece(np)->end[0]);
        w.end[1] = lane0(piece(np)->end[1]);
        piece_done(np);
        if (w.s1 < 0) break;
        ok = wait_uniform(bar(L::kQFull), np & 1, abort);
        if (!ok) break;
        tc_fence_after();
        if constexpr (L::kTiles == 1) {
          // one row tile, its scores a tile ahead in the other buffer
          auto next_scores = [&](int buf) -> bool {
            #pragma unroll 1
            for (int c = 0; c < L::kKParts; ++c, ++kp) {
              if (!k_wait(kp)) return false;
              tc_fence_after();
              const int s = lane0(kp % L::kKStages);
              scores(0, buf, c, s);
              mma_commit(bar(L::kKEmpty + s));
            }
            mma_commit(bar(L::kSFull + buf));
            return true;
          };
          ok = next_scores(lane0(g & 1));
          for (int j = w.s0; ok && j < w.s1; ++j, ++g) {
            if (j + 1 < w.s1) {
              if (!next_scores(lane0((g + 1) & 1))) { ok = false; break; }
            } else {
              mma_commit(bar(L::kQEmpty));
            }
            const int buf = lane0(g & 1);
            if (!wait_uniform(bar(L::kPFull + buf), (g >> 1) & 1, abort)) { ok = false; break; }
            #pragma unroll 1
            for (int h = 0; h < L::kVParts; ++h, ++vp) {
              if (ok) ok = v_wait(vp);
              if (!ok) break;
              tc_fence_after();
              const int s = lane0(vp % L::kVStages);
              values(0, buf, h, s, j == w.s0);
              mma_commit(bar(L::kVEmpty + s));
            }
            if (!ok) break;
            mma_commit(bar(L::kODone));
            mma_commit(bar(L::kTileEmpty + (g & 7)));
          }
        } else {
          // two row tiles by turns, P V of a tile and its next scores together
          const bool a0 = w.s0 < w.end[0], b0 = w.s0 < w.end[1];
          ok = k_wait(kp);
          if (!ok) break;
          tc_fence_after();
          {
            const int s = lane0(kp % L::kKStages);
            if (a0) {
              scores(0, 0, 0, s);
              mma_commit(bar(L::kSFull));
            }
            if (b0) {
              scores(1, 1, 0, s);
              mma_commit(bar(L::kSFull + 1));
            }
            mma_commit(bar(L::kKEmpty + s));
            ++kp;
          }
          if (w.s1 - w.s0 == 1) mma_commit(bar(L::kQEmpty));
          for (int j = w.s0; ok && j < w.s1; ++j, ++g, ++vp) {
            // the tile's V and the next tile's K before the waits for P, so
            // that none sits between P V and the next scores
            const bool next = j + 1 < w.s1;
            ok = v_wait(vp) && (!next || k_wait(kp));
            if (!ok) break;
            const int sv = lane0(vp % L::kVStages), sk = lane0(kp % L::kKStages);
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (!ok || j >= w.end[u]) continue;
              if (!wait_uniform(bar(L::kPFull + u), pf[u] & 1, abort)) { ok = false; continue; }
              ++pf[u];
              tc_fence_after();
              values(u, u, 0, sv, j == w.s0);
              if (j + 1 == w.end[u]) {
                mma_commit(bar(L::kODone + u));
              } else {
                scores(u, u, 0, sk);
                mma_commit(bar(L::kSFull + u));
              }
            }
            if (!ok) break;
            mma_commit(bar(L::kVEmpty + sv));
            mma_commit(bar(L::kTileEmpty + (g & 7)));
            if (next) {
              mma_commit(bar(L::kKEmpty + sk));
              ++kp;
              if (j + 2 == w.s1) mma_commit(bar(L::kQEmpty));
            }
          }
        }
      }
      mma_commit(bar(L::kDrain));
      drain_wait(bar(L::kDrain), 0);
    }
  } else if (warp >= L::kSoftWarps) {
    // ------------------------------------------------------------ conversion
    if constexpr (L::kRegConv > 128) more_registers<L::kRegConv>();
    else fewer_registers<L::kRegConv>();
    const int cw = warp - L::kSoftWarps;
    const int r8 = lane >> 2, c16 = lane & 3;   // row of eight, 16-column part of 64
    constexpr int kI = L::kConvRows / 8;
    // Codes of one tile: rows kConvRows cw + 8 i + r8, 16 columns of each
    // 64-column part.  Each part's registers are loaded again, for the next
    // tile, as soon as it has been written: a tile's time hides the latency.
    uint4 vr[L::kChunks][kI];
    int tile = 0, lim = 0, b = 0, h = 0;      // the tile that is loaded next, and its piece
    auto enter = [&](int np) {
      tile = piece(np)->s0;
      lim = piece(np)->lim;
      b = piece(np)->b;
      h = piece(np)->h;
    };
    // Rows past the keys that any row sees are zeros.  at: this thread's place
    // in the first of the warp's groups (of tile gn), by group and 8-row half.
    const long long v_row = r8 * p.vs.n + 16 * c16, v_half = 8 * p.vs.n;
    auto load = [&](int gn, int c) {
      const uint32_t w = sbase + L::kWhereOff + ((gn & 7) * 8 + (kI / 2) * cw) * 16;
      const bool whole = tile * 128 + 128 <= lim;
      #pragma unroll
      for (int i = 0; i < kI; ++i) {
        const unsigned char* src = ld_shared_ptr(w + 16 * (i / 2)) + v_row + (i & 1 ? v_half : 0) + 64 * c;
        if (whole) load_16(vr[c][i], src);
        else load_16_if(vr[c][i], src, tile * 128 + L::kConvRows * cw + 8 * i + r8 < lim);
      }
    };
    auto tile_wait = [&](int gn) {
      return wait_uniform(bar(L::kTileFull + (gn & 7)), (gn >> 3) & 1, abort);
    };
    // this thread's two 16-byte places in a row of 64 f16 columns
    const uint32_t place0 = r8 * 128 + (((2 * c16) ^ r8) << 4);
    const uint32_t place1 = r8 * 128 + (((2 * c16 + 1) ^ r8) << 4);
    auto put = [&](uint32_t rows, const uint4& x) {     // rows: of eight rows
      uint32_t w[8];
      widen4(x.x, w[0], w[1]);
      widen4(x.y, w[2], w[3]);
      widen4(x.z, w[4], w[5]);
      widen4(x.w, w[6], w[7]);
      st_shared_v4(rows + place0, w[0], w[1], w[2], w[3]);
      st_shared_v4(rows + place1, w[4], w[5], w[6], w[7]);
    };
    bool ok = piece_wait(0);
    bool more = ok && piece(0)->s1 >= 0;
    int vp = 0, g = 0;
    for (int np = 0; ok && more; ++np) {
      enter(np);
      // ---- q, once the last scores of the piece before are done.  A row is
      // scaled by a power of two to [2^7, 2^8) and becomes 8-bit parts, each
      // what the ones before have left, the last of them e5m2.
      // Four lanes to a row, each 16 of a part's 64 columns, so that eight
      // lanes' load touches two lines (with a thread a row it touched eight, and
      // the look-ups of those were most of a piece's start).  A warp does eight
      // rows at a time, the next eight's loads in flight, and converts them in a
      // loop small enough to stay in the instruction cache (the registers move
      // on instead of an index).
      // Odd rows take the parts of a pair the other way round: the codes of two
      // rows then lie in banks of their own.
      const int live = piece(np)->n, row0 = piece(np)->row0;
      const int flip = L::kChunks > 1 ? r8 & 1 : 0;
      uint4 ahead[2 * L::kChunks];        // [64-column part][half]
      auto load_q = [&](int n) {
        const int r = row0 + n + r8, i = r / p.seq.G;
        const bool on = r < p.rows && i < live;
        const uint16_t* src = p.q + b * p.qs.b + (h * p.seq.G + r - i * p.seq.G) * p.qs.h + i * p.qs.n + 16 * c16;
        #pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          #pragma unroll
          for (int k = 0; k < 2; ++k)
            load_16_if(ahead[2 * c + k], src + 64 * (c ^ flip) + 8 * k, on);
      };
      load_q(8 * cw);
      if (np > 0 && !wait_uniform(bar(L::kQEmpty), (np - 1) & 1, abort)) break;
      // The next piece's flag: no converting warp is there before this one has
      // announced this piece's q.  A softmax group whose row tile has no keys in
      // the pieces between may be as far behind as the records let it, at piece
      // np - 3: eight flags.
      if (cw == 0 && lane == 0) nan_seen[(np + 1) & 7] = 0;
      #pragma unroll 1
      for (int n = 8 * cw; n < L::kRows; n += 8 * L::kConvWarps) {
        uint4 x[2 * L::kChunks];
        #pragma unroll
        for (int k = 0; k < 2 * L::kChunks; ++k) x[k] = ahead[k];
        if (n + 8 * L::kConvWarps < L::kRows) load_q(n + 8 * L::kConvWarps);
        uint32_t top = 0;    // of the magnitudes, two lanes of 16 bits
        #pragma unroll
        for (int k = 0; k < 2 * L::kChunks; ++k)
          top = max_16x2(top, max_16x2(max_16x2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu),
                                       max_16x2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu)));
        top = max_16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max_16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t top1 = max(top & 0xffffu, top >> 16);
        float up, down;
        const float amax = p.bf16 ? __uint_as_float(top1 << 16) : unpack2<false>(top1).x;
        row_power<7>(amax, &up, &down);
        // (infinities have no code: their row is NaN, as its scores are)
        if (!(amax < __uint_as_float(0x7f800000u))) down = __uint_as_float(0x7fffffffu);
        const int rr = n + r8;
        if (c16 == 0) q_pow[(np & 1) * L::kRows + rr] = up;
        #pragma unroll 1
        for (int t = 0; t < L::kChunks; ++t) {
          const uint32_t y[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
          uint32_t f[8];      // (below 256 every f16 and bf16 is an f16 to 2^-25)
          #pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 v = p.bf16 ? unpack2<true>(y[k]) : unpack2<false>(y[k]);
            f[k] = pack2<false>(v.x * down, v.y * down);
          }
          const int chunk = 4 * (t ^ flip) + c16;     // 16 columns of the row
          constexpr int kRowChunks = L::kKCols / 16;
          const uint32_t at = sbase + L::kQOff + (rr >> 7) * L::kQTile + chunk / kRowChunks * (128 * L::kKCols) +
                              row_chunk<L::kKCols>(rr & 127, chunk % kRowChunks);
          auto part = [&](uint32_t to, auto code) {
            uint32_t w[4];
            #pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __byte_perm(code(f[2 * k]), code(f[2 * k + 1]), 0x5410);
            st_shared_v4(to, w[0], w[1], w[2], w[3]);
          };
          // (the first part in either branch, not ahead of them: that way a
          // register spilled at d = 256)
          if (p.bf16) {
            part(at, take_e4m3);
            part(at + L::kQPart, to_e5m2);
          } else {
            part(at, take_e4m3);
            part(at + L::kQPart, take_e4m3);
            part(at + 2 * L::kQPart, to_e5m2);
          }
          #pragma unroll
          for (int k = 0; k + 2 < 2 * L::kChunks; ++k) x[k] = x[k + 2];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(bar(L::kQFull));
      // the first tile's values (they are not needed before its scores and
      // weights are done)
      ok = tile_wait(g);
      if (!ok) break;
      #pragma unroll
      for (int c = 0; c < L::kChunks; ++c) load(g, c);
      const int full = piece(np)->all, s1 = piece(np)->s1;
      for (int j = piece(np)->s0; j < s1; ++j, ++g) {
        const bool next = j + 1 < s1;      // the piece has another tile
        ++tile;
        if (next) ok = tile_wait(g + 1);
        if (!ok) break;
        // V: this warp's rows lie in one piece of the tile
        const int n = vp + L::kConvRows * cw / L::kVKeys, s = n % L::kVStages;
        vp += L::kVParts;
        if (n >= L::kVStages && ok)
          ok = wait_uniform(bar(L::kVEmpty + s), (n / L::kVStages + 1) & 1, abort);
        if (!ok) break;
        if (j * 128 + 128 > full) {
          // NaN in a place that some row may not see: 0 instead, and the rows
          // that see it are mended when they are written
          uint32_t any = 0;
          #pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
            #pragma unroll
            for (int i = 0; i < kI; ++i) {
              uint32_t x[4] = {vr[c][i].x, vr[c][i].y, vr[c][i].z, vr[c][i].w};
              #pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t nan = nan_bytes(x[k]);
                any |= nan;
                x[k] &= ~nan;
              }
              vr[c][i] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          if (any != 0) nan_seen[np & 7] = 1;
        }
        #pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          #pragma unroll
          for (int i = 0; i < kI; ++i)
            put(sbase + L::kVOff + s * L::kVPiece + c * (L::kVKeys * 128) +
                    ((L::kConvRows * cw + 8 * i) & (L::kVKeys - 1)) * 128,
                vr[c][i]);
          if (c + 1 == L::kChunks) {
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(L::kVFull + s));
          }
          if (next) load(g + 1, c);
        }
      }
      if (!ok) break;
      piece_done(np);
      ok = piece_wait(np + 1);
      more = ok && piece(np + 1)->s1 >= 0;
    }
  } else {
    // ------------------------------------------------------------ softmax
    more_registers<L::kRegSoft>();
    const int u = warp >> 2;                      // row tile of this warpgroup
    const int r_tile = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + L::kTO + (L::kTiles == 2 ? D * u : 0) + lane_off;
    int cs = 0, od = 0;     // S_FULL phases (d = 256: tiles), O_DONE phases consumed
    int g = 0;              // tiles of the CTA so far
    bool ok = true;
    for (int np = 0; ok; ++np) {
      if (!piece_wait(np)) break;
      const int s0 = piece(np)->s0;
      if (piece(np)->s1 < 0) break;
      const int end = piece(np)->end[u], full = piece(np)->full[u];
      int sees;       // the keys that this thread's row sees
      {
        const int r = piece(np)->row0 + 128 * u + r_tile;
        const Sequence seq = {piece(np)->len, piece(np)->n};
        sees = r < p.rows ? max(0, row_limit(p.seq, seq, r)) : 0;
      }
      float m = kNoMax, l = 0.f, row_scale = 0.f;
      for (int j = s0; j < end; ++j) {
        const int buf = L::kTiles == 2 ? u : cs & 1;
        const uint32_t tS = tmem + L::kTS + 128 * buf + lane_off;
        if (!wait_uniform(bar(L::kSFull + buf), (L::kTiles == 2 ? cs : cs >> 1) & 1, abort)) {
          ok = false;
          break;
        }
        ++cs;
        tc_fence_after();
        if (j == s0) row_scale = q_pow[(np & 1) * L::kRows + 128 * u + r_tile] * p.scale_log2;
        uint32_t sr[128];
        #pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
        tmem_ld_wait();
        reg_fence(sr);
        float* s = reinterpret_cast<float*>(sr);
        if (j * 128 + 128 > full) {
          const int lim = sees - j * 128;
          #pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= lim) s[i] = -INFINITY;
        }
        const uint32_t mt = sbase + L::kMetaOff + ((g + j - s0) & 7) * 128;
        float top = kNoMax;
        #pragma unroll
        for (int c = 0; c < 128 / SEG; ++c) {
          float part[4];
          #pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* x = s + SEG * c + SEG / 4 * k;
            part[k] = fmax3(x[0], x[1], fmaxf(x[2], x[3]));
            #pragma unroll
            for (int i = 4; i < SEG / 4; i += 2) part[k] = fmax3(part[k], x[i], x[i + 1]);
          }
          const float4 sc = ld_shared_f4(mt + 16 * (SEG / 16) * c);
          top = fmaxf(top, fmaf(fmax3(part[0], part[1], fmaxf(part[2], part[3])), row_scale * sc.x, sc.y));
        }
        const bool grow = top > m + (kHead + kGrow);
        const bool any = __any_sync(0xffffffffu, grow);
        float alpha = 1.f;
        if (any) {
          const float now = fmaxf(m, top - kHead);
          alpha = ex2_approx(m - now);
          m = now;
          l *= alpha;
        }
        // O follows the maximum.  d <= 128: S of this tile was issued after P V of
        // the tile before on the same rows, and its completion tells of that as
        // well.  With scales by 16 keys ahead of the weights, which leaves more
        // registers to them (d = 128, pages of 16: 209.5 -> 197 us), otherwise
        // behind them (pages of 64: 176.5, ahead 178.7).
        constexpr bool kScaleFirst = L::kTiles == 2 && SEG == 16;
        if (kScaleFirst && any && j > s0) scale_o<D>(tO, alpha);
        // the weights over S as f16
        #pragma unroll
        for (int seg = 0; seg < 128 / SEG; ++seg) {
          const float4 sc = ld_shared_f4(mt + 16 * (SEG / 16) * seg);
          // (a product that underflows to 0 would make a masked score, -inf, NaN)
          const float ksr = fmaxf(row_scale * sc.x, 1.17549435e-38f), sub = sc.y - m;
          const f2 k2 = {ksr, ksr}, m2 = {sub, sub};
          f2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
          #pragma unroll
          for (int c = 0; c < SEG / 16; ++c) {
            uint32_t pk[8];
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float* x = s + SEG * seg + 16 * c + 2 * i;
              const f2 arg = ffma2(f2{x[0], x[1]}, k2, m2);
              const f2 pe = {ex2_approx(arg.x), ex2_approx(arg.y)};
              pk[i] = pack2<false>(pe.x, pe.y);
              sum[i & 1] = fadd2(sum[i & 1], pe);
            }
            tmem_st8(tS + SEG / 2 * seg + 8 * c, pk);
          }
          const f2 all = fadd2(sum[0], sum[1]);
          l = fmaf(all.x + all.y, sc.z, l);
        }
        tmem_st_wait();
        if constexpr (L::kTiles == 1) {
          // P V of the tile before has to be done before O may be rescaled
          // (the scores waited for above were issued ahead of it)
          if (j > s0) {
            if (!wait_uniform(bar(L::kODone), od & 1, abort)) { ok = false; break; }
            ++od;
            tc_fence_after();
          }
        }
        if (!kScaleFirst && any && j > s0) scale_o<D>(tO, alpha);
        tc_fence_before();
        mbar_arrive_warp(bar(L::kPFull + buf));
      }
      if (!ok) break;
      // ---------------------------------------------------------- results
      const bool some = end > s0;     // the tile has keys in this piece
      if (some) {
        if (!wait_uniform(bar(L::kODone + (L::kTiles == 2 ? u : 0)), od & 1, abort)) { ok = false; break; }
        ++od;
        tc_fence_after();
      }
      const volatile Piece* w = piece(np);
      const int r = w->row0 + 128 * u + r_tile, b = w->b, kh = w->h, s1 = w->s1;
      const int i = r / p.seq.G, head = kh * p.seq.G + r % p.seq.G;
      const bool in = r < p.rows, whole = w->whole != 0;
      const float sum = (in && i < w->n) ? l : 0.f;
      const long long slot = 2ll * blockIdx.x + (s0 > 0 ? 0 : 1);
      const float inv = whole ? (sum == 0.f ? 0.f : kHeadInv / sum) : 1.f;
      // (a tile without keys in this piece may be here before the flag is reset)
      const bool nans = some && nan_seen[np & 7] != 0;
      const int nan_from = max(s0, w->all / 128) * 128, nan_to = min(s1 * 128, sees);
      piece_done(np);
      auto write = [&](auto with_nans, int c) {
        uint32_t o[32];
        #pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
        if (some) {
          tmem_ld32(tO + 32 * c, o);
          tmem_ld_wait();
          reg_fence(o);
        }
        if constexpr (decltype(with_nans)::value) {
          // NaN codes among the values that this row sees in tiles where the
          // conversion left them out (rare: a loop over those keys)
          for (int key = nan_from; in && key < nan_to; ++key) {
            int page = p.table[static_cast<long long>(b) * p.width + (key >> p.page_log2)];
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) page = 0;
            const uint32_t* row = reinterpret_cast<const uint32_t*>(
                p.v + page * p.vs.b + kh * p.vs.h + (key & ((1 << p.page_log2) - 1)) * p.vs.n + 32 * c);
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t n = nan_bytes(row[k]);
              #pragma unroll
              for (int x = 0; x < 4; ++x)
                if (n >> (8 * x) & 1) o[4 * k + x] = 0x7fffffffu;
            }
          }
        }
        if (in) {
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + b * p.os.b + head * p.os.h + i * p.os.n + 32 * c);
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
              #pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float lo2 = __uint_as_float(o[8 * k + 2 * x]) * inv;
                const float hi2 = __uint_as_float(o[8 * k + 2 * x + 1]) * inv;
                w[x] = sum == 0.f ? 0u : p.bf16 ? pack2<true>(lo2, hi2) : pack2<false>(lo2, hi2);
              }
              dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (sum != 0.f) {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + (slot * L::kRows + 128 * u + r_tile) * D + 32 * c);
            #pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      };
      if (nans) {     // (the same for the whole warp)
        #pragma unroll 1
        for (int c = 0; c < D / 32; ++c) write(std::true_type{}, c);
      } else {
        #pragma unroll 1
        for (int c = 0; c < D / 32; ++c) write(std::false_type{}, c);
      }
      if (in) {
        if (whole)
          p.lse[(static_cast<long long>(b) * p.H + head) * p.seq.Nq + i] =
              sum == 0.f ? -INFINITY : (m + kHead + log2f(sum)) * kLogE2;
        else
          p.part_ml[slot * L::kRows + 128 * u + r_tile] = make_float2(m, sum);
      }
      tc_fence_before();   // O has been read out before the next P_FULL allows P V over it
      g += s1 - s0;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort == 2) atomicOr(p.seq.err, kErrTimeout);
  if (warp == 12) {
    __syncwarp();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

template <int D, int SEG>
cudaError_t launch_seg(const Cache& cache, FwdCacheParams& p, int sms, cudaStream_t stream) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kern = cache_prefill_kernel<D, SEG>;
  if (!set[dev & 63]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pre<D>::kAlloc);
    if (e != cudaSuccess) return e;
    // the warpgroups share out the registers that the launch comes with: with
    // fewer of them, those that ask for more would wait for ever
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return e;
    if (attr.numRegs != 128) return cudaErrorInvalidConfiguration;
    set[dev & 63] = true;
  }
  CUtensorMap tk;
  if ((e = make_tmap_u8_4d(&tk, cache.k, D, cache.page, cache.Hkv, cache.pages, cache.ks,
                           Pre<D>::kKCols, std::min(cache.page, 128))) != cudaSuccess)
    return e;
  p.ctas = sms;
  kern<<<p.ctas, kThreads, Pre<D>::kAlloc, stream>>>(tk, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_cache_merge<D, Pre<D>::kRows, 128, Pre<D>::kOver, true>(p, stream);
}

template <int D>
cudaError_t launch(const Cache& cache, FwdCacheParams& p, int sms, cudaStream_t stream) {
  return cache.page >= 64   ? launch_seg<D, 64>(cache, p, sms, stream)
         : cache.page == 32 ? launch_seg<D, 32>(cache, p, sms, stream)
                            : launch_seg<D, 16>(cache, p, sms, stream);
}

}  // namespace

int cache_prefill_rows(int d) { return d == 256 ? Pre<256>::kRows : Pre<128>::kRows; }

cudaError_t launch_cache_prefill(const Cache& cache, FwdCacheParams& p, int sms,
                                 cudaStream_t stream) {
  switch (cache.d) {
    case 64: return launch<64>(cache, p, sms, stream);
    case 128: return launch<128>(cache, p, sms, stream);
    case 256: return launch<256>(cache, p, sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
