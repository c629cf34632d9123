// Attention over the paged 8-bit cache for many query rows (chunks of prompts,
// and whole ones): the same formulas as fa_cache_fwd.cu on the tensor cores of
// tcgen05, tiles of 128 query rows x 128 keys.
//
// What bounds it: the tensor pipe and, next to it, the exponentials, as in the
// 16-bit forward kernel; on top of those every 8-bit key and value has to
// become f16 in the layout the products read.  A warpgroup of its own does
// that: it reads the codes from memory (pages may lie anywhere, so each thread
// follows the table for its rows; the next piece's loads are in flight while a
// piece is converted), widens them (64 conversions a clock an SM, a quarter of
// a tile's time) and writes them to swizzled shared memory.  A piece converted
// once serves two tiles of query rows at d <= 128 (256 rows; every head of a
// key/value head's group is among them), so the conversion is half of what one
// tile would cost; at d = 256 TMEM holds one tile's O.
//
// The keys' scale multiplies the scores and the values' scale goes into the
// exponent, both by 16-key groups (a page has at least 16): the group's
// largest raw score is scaled, not each score, so that the scales cost eight
// multiplications a row and tile, and the exponent's multiply-add takes them
// for the rest.
//
// Roles: warps 0-3 softmax of tile A, 4-7 of tile B (d = 256: conversion),
// 8-11 conversion and q, 12 issues the products, 13 walks the share and
// describes its pieces to the others.  512 threads start with 128 registers
// each, which the groups then share out by their need.  With 192 KB of tiles
// next to none of the SM's storage is left as L1, so a register that spills
// costs a trip to L2: the walk lives in one warp for that reason.
#include <algorithm>
#include <atomic>

#include "cache_work.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;

template <int D>
struct Pre {
  static constexpr int kTiles = D == 256 ? 1 : 2;
  static constexpr int kRows = 128 * kTiles;        // of a unit
  static constexpr int kSoftWarps = 4 * kTiles;
  static constexpr int kConvWarps = 12 - kSoftWarps;
  static constexpr int kConvRows = 128 / kConvWarps;   // keys of a tile that a warp converts
  static constexpr int kChunks = D / 64;            // 64-column parts
  static constexpr int kKPiece = 128 * 128;         // K: 128 keys x 64 columns, f16
  static constexpr int kKStages = 4;
  static constexpr int kVKeys = D == 256 ? 64 : 128;   // V: kVKeys keys x D columns
  static constexpr int kVParts = 128 / kVKeys;
  static constexpr int kVPiece = kVKeys * D * 2;
  static constexpr int kVStages = D == 64 ? 4 : 2;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kTiles * kQTile;
  static constexpr int kVOff = kKOff + kKStages * kKPiece;
  static constexpr int kMetaOff = kVOff + kVStages * kVPiece;   // [8 tiles][8 groups] ks, log2 vs, 1/vs
  static constexpr int kPowOff = kMetaOff + 8 * 8 * 16;         // [2 pieces][rows] of q
  static constexpr int kRecOff = kPowOff + 2 * kRows * 4;       // [4 pieces] (Piece)
  static constexpr int kBarOff = kRecOff + 4 * 64;
  static constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kKEmpty = kKFull + kKStages,
                       kVFull = kKEmpty + kKStages, kVEmpty = kVFull + kVStages,
                       kSFull = kVEmpty + kVStages, kPFull = kSFull + 2, kODone = kPFull + 2,
                       kDrain = kODone + 2, kRecFull = kDrain + 1, kRecEmpty = kRecFull + 4,
                       kNumBars = kRecEmpty + 4;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kRedOff = (kMiscOff + 32 + 15) / 16 * 16;   // start: sums and the found entry
  static constexpr int kBytes = kRedOff + 16 * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kTS = 0, kTO = 256, kTmemCols = 512;
  // registers a thread: the launch's 4 * 128 among the four warpgroups
  static constexpr int kRegSoft = 176;
  static constexpr int kRegMisc = kTiles == 1 ? 112 : 48;
  static constexpr int kRegConv = kTiles == 1 ? (512 - kRegSoft - kRegMisc) / 2 : 512 - 2 * kRegSoft - kRegMisc;
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

// 16 bytes of global memory, zeros where `on` is false; and four bytes, `other`
// where it is false.  Kept in program order with the other volatile asm, so
// that a load is issued where it stands, a tile ahead of its use: left to the
// compiler the loads of a tile were waited for one by one.
__device__ __forceinline__ void load_16(uint4& x, const void* src, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
      : "l"(src), "r"(static_cast<uint32_t>(on)));
}
__device__ __forceinline__ uint32_t load_4(const void* src, bool on, uint32_t other) {
  uint32_t x;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, %3;\n\t"
      "@p ld.global.nc.u32 %0, [%1];\n\t}"
      : "=r"(x)
      : "l"(src), "r"(static_cast<uint32_t>(on)), "r"(other));
  return x;
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_prefill_kernel(const __grid_constant__ FwdCacheParams p) {
  using L = Pre<D>;
  using W = Walk<L::kRows, 128>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  volatile int* nan_seen = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 8);   // [4 pieces]
  long long* red = reinterpret_cast<long long*>(smem + L::kRedOff);
  longlong2* found = reinterpret_cast<longlong2*>(smem + L::kRedOff + 128);
  float4* meta = reinterpret_cast<float4*>(smem + L::kMetaOff);
  float* q_pow = reinterpret_cast<float*>(smem + L::kPowOff);
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBarOff + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(bar(L::kQFull), L::kConvWarps);
    mbar_init(bar(L::kQEmpty), 1);
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(bar(L::kKFull + s), L::kConvWarps);
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
      mbar_init(bar(L::kRecEmpty + s), 1 + L::kConvWarps + L::kSoftWarps);
      nan_seen[s] = 0;
    }
    mbar_init(bar(L::kDrain), 1);
    *abort = 0;
    fence_barrier_init();
  }
  bool bad = false;
  const long long total = total_steps<L::kRows, 128, kThreads>(p, red, &bad) * p.Hkv;
  if (bad && blockIdx.x == 0) atomicOr(p.seq.err, kErrCache);
  const long long share = (total + p.ctas - 1) / p.ctas;
  const long long lo = blockIdx.x * share, hi = min(total, lo + share);
  if (lo >= hi) return;
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_holder), L::kTmemCols);
    tmem_relinquish();
  }
  find_entry<L::kRows, 128, kThreads>(p, lo / p.Hkv, red, found);
  W at;
  if (warp == 13) at.start(p, found, lo);
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
      long long left = hi - lo;
      for (int np = 0;; ++np) {
        if (np >= 4 && !wait_uniform(bar(L::kRecEmpty + (np & 3)), ((np >> 2) + 1) & 1, abort)) break;
        volatile Piece* w = reinterpret_cast<volatile Piece*>(smem + L::kRecOff + (np & 3) * 64);
        const int s1 = left > 0 ? static_cast<int>(min(static_cast<long long>(at.steps), at.step + left)) : -1;
        if (lane == 0) {
          w->s0 = at.step;
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
              if (end > at.step) all = min(all, t.full);
            }
            w->all = all;
            w->lim = at.lim;
            w->b = at.e / p.row_tiles;
            w->h = at.h;
            w->row0 = row0;
            w->len = at.seq.len;
            w->n = at.seq.n;
            w->whole = at.step == 0 && s1 == at.steps;
          }
        }
        __syncwarp();
        if (elect_one()) mbar_arrive(bar(L::kRecFull + (np & 3)));
        __syncwarp();
        if (s1 < 0) break;
        left -= s1 - at.step;
        if (left > 0) at.next_unit(p);
      }
    } else if (warp == 12) {
      // ---------------------------------------------------------- products
      constexpr uint32_t kIdS = idesc_f16(128, 128, 0, 0, 0);
      constexpr uint32_t kIdO = idesc_f16(128, D, 0, 0, 1);
      const uint64_t q_desc = smem_desc_sw128(sbase + L::kQOff, 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(sbase + L::kKOff, 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(sbase + L::kVOff, L::kVKeys * 128, 1024);
      int kp = 0, vp = 0;                 // pieces of K and V consumed
      int pf[2] = {0, 0};                 // P_FULL phases consumed, by score buffer
      bool ok = true;
      // S = Q K^T of row tile u into score buffer `buf`, from K pieces
      // `first` on; `free`: the pieces' last use
      auto scores = [&](int u, int buf, int first, bool free) -> bool {
        #pragma unroll 1
        for (int c = 0; c < L::kChunks; ++c) {
          const int n = first + c, s = n % L::kKStages;
          if (!wait_uniform(bar(L::kKFull + s), (n / L::kKStages) & 1, abort)) return false;
          tc_fence_after();
          const uint64_t ks = desc_add(k_desc, s * L::kKPiece);
          const uint64_t qs = desc_add(q_desc, u * L::kQTile + c * (128 * 128));
          #pragma unroll
          for (int w = 0; w < 4; ++w)
            mma_ss(tmem + L::kTS + 128 * buf, desc_add(qs, w * 32), desc_add(ks, w * 32), kIdS,
                   (c > 0 || w > 0) ? 1u : 0u);
          if (free) mma_commit(bar(L::kKEmpty + s));
        }
        mma_commit(bar(L::kSFull + buf));
        return true;
      };
      auto values = [&](int u, int buf, int first, bool fresh, bool free) -> bool {
        #pragma unroll 1
        for (int h = 0; h < L::kVParts; ++h) {
          const int n = first + h, s = n % L::kVStages;
          if (!wait_uniform(bar(L::kVFull + s), (n / L::kVStages) & 1, abort)) return false;
          tc_fence_after();
          const uint64_t vs = desc_add(v_desc, s * L::kVPiece);
          #pragma unroll
          for (int w = 0; w < L::kVKeys / 16; ++w)
            mma_ts(tmem + L::kTO + D * u, tmem + L::kTS + 128 * buf + (h * (L::kVKeys / 16) + w) * 8,
                   desc_add(vs, w * 2048), kIdO, (!fresh || h > 0 || w > 0) ? 1u : 0u);
          if (free) mma_commit(bar(L::kVEmpty + s));
        }
        return true;
      };
      int g = 0;   // tiles so far (d = 256: selects the score buffer)
      for (int np = 0; ok; ++np) {
        if (!piece_wait(np)) break;
        // (read from lane 0: the same in every lane, on the uniform datapath)
        struct { int s0, s1, end[2]; } w;
        w.s0 = __shfl_sync(0xffffffffu, piece(np)->s0, 0);
        w.s1 = __shfl_sync(0xffffffffu, piece(np)->s1, 0);
        w.end[0] = __shfl_sync(0xffffffffu, piece(np)->end[0], 0);
        w.end[1] = __shfl_sync(0xffffffffu, piece(np)->end[1], 0);
        piece_done(np);
        if (w.s1 < 0) break;
        ok = wait_uniform(bar(L::kQFull), np & 1, abort);
        if (!ok) break;
        tc_fence_after();
        if constexpr (L::kTiles == 1) {
          ok = scores(0, g & 1, kp, true);
          for (int j = w.s0; ok && j < w.s1; ++j, ++g) {
            if (j + 1 < w.s1) {
              if (!scores(0, (g + 1) & 1, kp + L::kChunks, true)) { ok = false; break; }
            } else {
              mma_commit(bar(L::kQEmpty));
            }
            if (!wait_uniform(bar(L::kPFull + (g & 1)), (g >> 1) & 1, abort)) { ok = false; break; }
            tc_fence_after();
            if (!values(0, g & 1, vp, j == w.s0, true)) { ok = false; break; }
            mma_commit(bar(L::kODone));
            kp += L::kChunks;
            vp += L::kVParts;
          }
        } else {
          const bool a0 = w.s0 < w.end[0], b0 = w.s0 < w.end[1];
          if (a0) ok = scores(0, 0, kp, !b0);
          if (ok && b0) ok = scores(1, 1, kp, true);
          if (w.s1 - w.s0 == 1) mma_commit(bar(L::kQEmpty));
          for (int j = w.s0; ok && j < w.s1; ++j) {
            // tile u takes part in this step (v) and in the next (n)
            const bool v0 = j < w.end[0], v1 = j < w.end[1];
            const bool n0 = j + 1 < w.end[0], n1 = j + 1 < w.end[1];
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (!ok || !(u ? v1 : v0)) continue;
              if (!wait_uniform(bar(L::kPFull + u), pf[u] & 1, abort)) { ok = false; continue; }
              ++pf[u];
              tc_fence_after();
              ok = values(u, u, vp, j == w.s0, u == 1 || !v1);
              if (ok && j + 1 == w.end[u]) mma_commit(bar(L::kODone + u));
              if (ok && (u ? n1 : n0)) ok = scores(u, u, kp + L::kChunks, u == 1 || !n1);
            }
            if (j + 2 == w.s1) mma_commit(bar(L::kQEmpty));
            kp += L::kChunks;
            vp += L::kVParts;
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
    uint4 kr[L::kChunks][kI], vr[L::kChunks][kI];
    int page[kI];
    float ks = 1.f, vs = 1.f;
    int tile = 0, lim = 0, b = 0, h = 0;      // the tile that is loaded next, and its piece
    auto enter = [&](int np) {
      tile = piece(np)->s0;
      lim = piece(np)->lim;
      b = piece(np)->b;
      h = piece(np)->h;
    };
    auto pages_of = [&]() {
      const int* row = p.table + static_cast<long long>(b) * p.width;
      #pragma unroll
      for (int i = 0; i < kI; ++i) {
        const int key = tile * 128 + L::kConvRows * cw + 8 * i;   // (a page holds whole groups of 16)
        page[i] = static_cast<int>(load_4(row + (key >> p.page_log2), key < lim, 0u));
      }
      #pragma unroll
      for (int i = 0; i < kI; ++i)
        if (static_cast<unsigned>(page[i]) >= static_cast<unsigned>(p.pages)) {
          atomicOr(p.seq.err, kErrCache);
          page[i] = 0;
        }
      // the scales of the warp's 16-key groups, one a lane
      int mine = page[0];
      if constexpr (kI > 2) mine = lane == 0 ? page[0] : page[2];
      const long long sc = static_cast<long long>(mine) * p.Hkv + h;
      const bool on = lane < kI / 2 && tile * 128 + L::kConvRows * cw + 16 * lane < lim;
      ks = __uint_as_float(load_4(p.k_scale + sc, on, 0x3f800000u));
      vs = __uint_as_float(load_4(p.v_scale + sc, on, 0x3f800000u));
    };
    // rows past the keys that any row sees are zeros
    auto load = [&](const unsigned char* base, const Strides& st, int c, uint4 (&x)[kI]) {
      const unsigned char* head = base + h * st.h + 64 * c + 16 * c16;
      #pragma unroll
      for (int i = 0; i < kI; ++i) {
        const int key = tile * 128 + L::kConvRows * cw + 8 * i + r8;
        load_16(x[i], head + page[i] * st.b + (key & ((1 << p.page_log2) - 1)) * st.n, key < lim);
      }
    };
    auto put = [&](uint32_t rows, int r, const uint4& x) {
      uint32_t w[8];
      widen4(x.x, w[0], w[1]);
      widen4(x.y, w[2], w[3]);
      widen4(x.z, w[4], w[5]);
      widen4(x.w, w[6], w[7]);
      const uint32_t row = rows + r * 128;
      st_shared_v4(row + (((2 * c16) ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
      st_shared_v4(row + (((2 * c16 + 1) ^ (r & 7)) << 4), w[4], w[5], w[6], w[7]);
    };
    bool ok = piece_wait(0);
    bool more = ok;
    if (ok) {
      enter(0);
      pages_of();
      #pragma unroll
      for (int c = 0; c < L::kChunks; ++c) load(p.k, p.ks, c, kr[c]);
      #pragma unroll
      for (int c = 0; c < L::kChunks; ++c) load(p.v, p.vs, c, vr[c]);
    }
    int kp = 0, vp = 0, g = 0;
    for (int np = 0; ok && more; ++np) {
      // ---- q: rows as f16, once the last scores of the piece before are done
      if (np > 0 && !wait_uniform(bar(L::kQEmpty), (np - 1) & 1, abort)) break;
      // the next piece's flag: no converting warp is there before this one has
      // announced this piece's q, and the results of piece np - 3 are written
      if (cw == 0 && lane == 0) nan_seen[(np + 1) & 3] = 0;
      {
        constexpr int kLanes = D / 8, kPer = 32 / kLanes;        // lanes of a row, rows at a time
        constexpr int kRowsW = L::kRows / L::kConvWarps, kBatch = 4;
        const int rl = lane / kLanes, cl = lane % kLanes;
        const int row0 = piece(np)->row0 + cw * kRowsW + rl, live = piece(np)->n;
        const uint16_t* src = p.q + b * p.qs.b + h * p.seq.G * p.qs.h + 8 * cl;
        #pragma unroll 1
        for (int i0 = 0; i0 < kRowsW; i0 += kPer * kBatch) {
          uint4 x[kBatch];
          #pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int r = row0 + i0 + k * kPer;
            const int i = r / p.seq.G;
            load_16(x[k], src + (r - i * p.seq.G) * p.qs.h + i * p.qs.n, r < p.rows && i < live);
          }
          #pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int rr = cw * kRowsW + i0 + k * kPer + rl;
            uint32_t y[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            float up = 1.f, down = 1.f;
            if (p.bf16) {
              float amax = 0.f;
              #pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float2 f = unpack2<true>(y[c]);
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
              #pragma unroll
              for (int m = kLanes / 2; m > 0; m >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
              row_power(amax, &up, &down);
              #pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float2 f = unpack2<true>(y[c]);
                y[c] = pack2<false>(f.x * down, f.y * down);
              }
            }
            if (cl == 0) q_pow[(np & 1) * L::kRows + rr] = up;
            const int r = rr & 127;
            st_shared_v4(sbase + L::kQOff + (rr >> 7) * L::kQTile + (cl >> 3) * (128 * 128) +
                             r * 128 + (((cl & 7) ^ (r & 7)) << 4),
                         y[0], y[1], y[2], y[3]);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(bar(L::kQFull));
      const int full = piece(np)->all, s1 = piece(np)->s1;
      for (int j = piece(np)->s0; j < s1; ++j, ++g) {
        const float ks_now = ks, vs_now = vs;
        // on to the next tile
        if (j + 1 < s1) {
          ++tile;
        } else {
          piece_done(np);
          ok = piece_wait(np + 1);
          more = ok && piece(np + 1)->s1 >= 0;
          if (more) enter(np + 1);
        }
        if (!ok) break;
        if (more) pages_of();
        #pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          const int s = kp % L::kKStages;
          if (kp >= L::kKStages && ok)
            ok = wait_uniform(bar(L::kKEmpty + s), (kp / L::kKStages + 1) & 1, abort);
          if (ok) {
            if (c == 0 && lane < kI / 2) {
              // when K of tile g is written the scores of tile g - 4 are done,
              // so P V of tile g - 5 is: eight tiles of these live at a time
              const float lv = log2f(vs_now);
              meta[(g & 7) * 8 + (kI / 2) * cw + lane] = make_float4(ks_now, lv, ex2_approx(-lv), 0.f);
            }
            #pragma unroll
            for (int i = 0; i < kI; ++i)
              put(sbase + L::kKOff + s * L::kKPiece, L::kConvRows * cw + 8 * i + r8, kr[c][i]);
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(L::kKFull + s));
          }
          ++kp;
          if (more) load(p.k, p.ks, c, kr[c]);
        }
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
          if (any != 0) nan_seen[np & 3] = 1;
        }
        #pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          #pragma unroll
          for (int i = 0; i < kI; ++i)
            put(sbase + L::kVOff + s * L::kVPiece + c * (L::kVKeys * 128),
                (L::kConvRows * cw + 8 * i + r8) & (L::kVKeys - 1), vr[c][i]);
          if (c + 1 == L::kChunks) {
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(L::kVFull + s));
          }
          if (more) load(p.v, p.vs, c, vr[c]);
        }
      }
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
        const float4* mt = meta + ((g + j - s0) & 7) * 8;
        float top = kNoMax;
        #pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float* x = s + 16 * c;
          const float a = fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmax3(x[6], x[7], x[8]));
          const float b = fmax3(fmax3(x[9], x[10], x[11]), fmax3(x[12], x[13], x[14]), x[15]);
          const float2 sc = *reinterpret_cast<const float2*>(mt + c);
          top = fmaxf(top, fmaf(fmaxf(a, b), row_scale * sc.x, sc.y));
        }
        const bool grow = top > m + kGrow;
        const bool any = __any_sync(0xffffffffu, grow);
        float alpha = 1.f;
        if (any) {
          const float now = fmaxf(m, top);
          alpha = ex2_approx(m - now);
          m = now;
          l *= alpha;
        }
        // the weights over S as f16, 32 columns at a time
        #pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 sc = mt[2 * c + h];
            const float ksr = row_scale * sc.x, sub = sc.y - m;
            const f2 k2 = {ksr, ksr}, m2 = {sub, sub};
            f2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              const f2 arg = ffma2(f2{s[32 * c + 16 * h + 2 * i], s[32 * c + 16 * h + 2 * i + 1]}, k2, m2);
              const f2 pe = {ex2_approx(arg.x), ex2_approx(arg.y)};
              pk[8 * h + i] = pack2<false>(pe.x, pe.y);
              sum[i & 1] = fadd2(sum[i & 1], pe);
            }
            const f2 all = fadd2(sum[0], sum[1]);
            l = fmaf(all.x + all.y, sc.z, l);
          }
          tmem_st16(tS + 16 * c, pk);
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
        // d <= 128: S of this tile was issued after P V of the tile before on
        // the same rows, and its completion tells of that as well
        if (any && j > s0) {
          tc_fence_after();
          #pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_ld_wait();
            reg_fence(o);
            #pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tO + 32 * c, o);
          }
          tmem_st_wait();
        }
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
      const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      const bool nans = nan_seen[np & 3] != 0;
      const int nan_from = max(s0, w->all / 128) * 128, nan_to = min(s1 * 128, sees);
      piece_done(np);
      #pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        #pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
        if (some) {
          tmem_ld32(tO + 32 * c, o);
          tmem_ld_wait();
          reg_fence(o);
        }
        if (nans && in) {
          // NaN codes among the values that this row sees in tiles where the
          // conversion left them out (rare: a loop over those keys)
          for (int key = nan_from; key < nan_to; ++key) {
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
      }
      if (in) {
        if (whole)
          p.lse[(static_cast<long long>(b) * p.H + head) * p.seq.Nq + i] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLogE2;
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

template <int D>
cudaError_t launch(FwdCacheParams& p, int sms, cudaStream_t stream) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kern = cache_prefill_kernel<D>;
  if (!set[dev & 63]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pre<D>::kAlloc);
    if (e != cudaSuccess) return e;
    set[dev & 63] = true;
  }
  p.ctas = sms;
  kern<<<p.ctas, kThreads, Pre<D>::kAlloc, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_cache_merge<D, Pre<D>::kRows, 128>(p, stream);
}

}  // namespace

int cache_prefill_rows(int d) { return d == 256 ? Pre<256>::kRows : Pre<128>::kRows; }

cudaError_t launch_cache_prefill(const Cache& cache, FwdCacheParams& p, int sms,
                                 cudaStream_t stream) {
  switch (cache.d) {
    case 64: return launch<64>(p, sms, stream);
    case 128: return launch<128>(p, sms, stream);
    case 256: return launch<256>(p, sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
