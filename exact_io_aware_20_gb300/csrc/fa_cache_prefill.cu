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
// Roles: warps 0-3 softmax of tile A, 4-7 of tile B (d = 256: idle), 8-11
// conversion and q, 12 issues the products.  512 threads start with 128
// registers each; the softmax groups rise to 192, the converters keep 88 and
// the last group 40 (2 * 192 + 88 + 40 = 4 * 128).
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
  static constexpr int kBarOff = kPowOff + 2 * kRows * 4;
  static constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kKEmpty = kKFull + kKStages,
                       kVFull = kKEmpty + kKStages, kVEmpty = kVFull + kVStages,
                       kSFull = kVEmpty + kVStages, kPFull = kSFull + 2, kODone = kPFull + 2,
                       kDrain = kODone + 2, kNumBars = kDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kRedOff = (kMiscOff + 32 + 15) / 16 * 16;   // start: sums and the found entry
  static constexpr int kBytes = kRedOff + 16 * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kTS = 0, kTO = 256, kTmemCols = 512;
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

// A piece of a unit: its steps [s0, s1) of the share, and for each of its row
// tiles the end of the tile's steps and the keys that all its live rows see.
template <int D>
struct Piece {
  int s0, s1;
  int end[Pre<D>::kTiles], full[Pre<D>::kTiles];
};
template <int D>
__device__ __forceinline__ Piece<D> piece_at(const FwdCacheParams& p,
                                             const Walk<Pre<D>::kRows, 128>& at, long long left) {
  Piece<D> w;
  w.s0 = at.step;
  w.s1 = static_cast<int>(min(static_cast<long long>(at.steps), at.step + left));
  const int row0 = at.e % p.row_tiles * Pre<D>::kRows;
  #pragma unroll
  for (int u = 0; u < Pre<D>::kTiles; ++u) {
    const int r0 = row0 + 128 * u, r1 = min(p.rows, r0 + 128);
    TileLimits t = {0, 0};
    if (r0 < r1) t = tile_limits(p.seq, at.seq, r0, r1);
    w.end[u] = min(w.s1, (t.lim + 127) / 128);
    w.full[u] = t.full;
  }
  return w;
}

// The keys that every live row of a piece's tiles sees.
template <int D>
__device__ __forceinline__ int seen_by_all(const Piece<D>& w) {
  int full = 0x7fffffff;
  #pragma unroll
  for (int u = 0; u < Pre<D>::kTiles; ++u)
    if (w.end[u] > w.s0) full = min(full, w.full[u]);
  return full;
}

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
    mbar_init(bar(L::kQFull), 4);       // one arrival per converting warp
    mbar_init(bar(L::kQEmpty), 1);
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(bar(L::kKFull + s), 4);
      mbar_init(bar(L::kKEmpty + s), 1);
    }
    for (int s = 0; s < L::kVStages; ++s) {
      mbar_init(bar(L::kVFull + s), 4);
      mbar_init(bar(L::kVEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::kSFull + s), 1);
      mbar_init(bar(L::kPFull + s), 4);   // one arrival per softmax warp
      mbar_init(bar(L::kODone + s), 1);
    }
    for (int s = 0; s < 4; ++s) nan_seen[s] = 0;
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
  at.start(p, found, lo);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  long long left = hi - lo;

  if (warp >= 12) {
    fewer_registers<40>();
    if (warp == 12) {
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
      for (int np = 0; ok && left > 0; ++np) {
        const Piece<D> w = piece_at<D>(p, at, left);
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
        left -= w.s1 - w.s0;
        if (left > 0) at.next_unit(p);
      }
      mma_commit(bar(L::kDrain));
      drain_wait(bar(L::kDrain), 0);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ conversion
    fewer_registers<88>();
    const int cw = warp - 8;
    const int r8 = lane >> 2, c16 = lane & 3;   // row of eight, 16-column part of 64
    const W begin = at;
    W ld = begin;                 // of the loads, one piece ahead
    long long ld_left = left;
    int ld_j = at.step, ld_part = 0;   // ld_part: K pieces, then V pieces of a tile
    constexpr int kParts = L::kChunks + L::kVParts;
    auto row_of = [&](const Strides& st, const unsigned char* base, int e, int h, int key) {
      const int b = e / p.row_tiles;
      int page = p.table[static_cast<long long>(b) * p.width + (key >> p.page_log2)];
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) {
        atomicOr(p.seq.err, kErrCache);
        page = 0;
      }
      return base + page * st.b + h * st.h + (key & ((1 << p.page_log2) - 1)) * st.n;
    };
    uint4 nxt[8];
    float nks = 1.f, nvs = 1.f;
    // loads of part ld_part of tile ld_j (rows past the keys that any row
    // sees are zeros), and on to the next part
    auto load = [&]() {
      if (ld_left <= 0) return;
      #pragma unroll
      for (int i = 0; i < 8; ++i) nxt[i] = make_uint4(0u, 0u, 0u, 0u);
      if (ld_part < L::kChunks) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = ld_j * 128 + 32 * cw + 8 * i + r8;
          if (key < ld.lim)
            nxt[i] = *reinterpret_cast<const uint4*>(row_of(p.ks, p.k, ld.e, ld.h, key) +
                                                     64 * ld_part + 16 * c16);
        }
        if (ld_part == 0) {
          // the scales of the warp's two 16-key groups, in lanes 0 and 1
          nks = nvs = 1.f;
          const int key = ld_j * 128 + 32 * cw + 16 * lane;
          if (lane < 2 && key < ld.lim) {
            int page = p.table[static_cast<long long>(ld.e / p.row_tiles) * p.width + (key >> p.page_log2)];
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) page = 0;
            nks = p.k_scale[static_cast<long long>(page) * p.Hkv + ld.h];
            nvs = p.v_scale[static_cast<long long>(page) * p.Hkv + ld.h];
          }
        }
      } else {
        constexpr int kRowsW = L::kVKeys / 4;      // rows of a warp
        #pragma unroll
        for (int i = 0; i < kRowsW / 8; ++i) {
          const int key = ld_j * 128 + (ld_part - L::kChunks) * L::kVKeys + kRowsW * cw + 8 * i + r8;
          if (key < ld.lim) {
            const unsigned char* row = row_of(p.vs, p.v, ld.e, ld.h, key) + 16 * c16;
            #pragma unroll
            for (int c = 0; c < L::kChunks; ++c)
              nxt[i * L::kChunks + c] = *reinterpret_cast<const uint4*>(row + 64 * c);
          }
        }
      }
      if (++ld_part == kParts) {
        ld_part = 0;
        --ld_left;
        if (++ld_j == ld.steps && ld_left > 0) {
          ld.next_unit(p);
          ld_j = 0;
        }
      }
    };
    auto put = [&](uint32_t piece, int rows, int r, int c, const uint4& x) {
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t h[8];
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[2 * i] = widen(w[i] & 0xffffu);
        h[2 * i + 1] = widen(w[i] >> 16);
      }
      const uint32_t row = piece + c * rows * 128 + r * 128;
      st_shared_v4(row + (((2 * c16) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
      st_shared_v4(row + (((2 * c16 + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
    };
    load();
    int kp = 0, vp = 0, g = 0;
    bool ok = true;
    for (int np = 0; ok && left > 0; ++np) {
      const Piece<D> w = piece_at<D>(p, at, left);
      const int b = at.e / p.row_tiles, row0 = at.e % p.row_tiles * L::kRows;
      // ---- q: rows as f16, once the last scores of the unit before are done
      if (np > 0 && !wait_uniform(bar(L::kQEmpty), (np - 1) & 1, abort)) break;
      // the next piece's flag: no converting warp is there before this one has
      // announced this piece's q, and the results of piece np - 3 are written
      if (cw == 0 && lane == 0) nan_seen[(np + 1) & 3] = 0;
      {
        constexpr int kLanes = D / 8, kPer = 32 / kLanes;        // lanes of a row, rows at a time
        constexpr int kRowsW = L::kRows / 4, kBatch = 4;
        const int rl = lane / kLanes, cl = lane % kLanes;
        #pragma unroll 1
        for (int i0 = 0; i0 < kRowsW; i0 += kPer * kBatch) {
          uint4 x[kBatch];
          #pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int r = row0 + cw * kRowsW + i0 + k * kPer + rl;
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (r < p.rows && r / p.seq.G < at.seq.n)
              x[k] = *reinterpret_cast<const uint4*>(
                  p.q + b * p.qs.b + (at.h * p.seq.G + r % p.seq.G) * p.qs.h +
                  (r / p.seq.G) * p.qs.n + 8 * cl);
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
      const int full = seen_by_all<D>(w);
      for (int j = w.s0; ok && j < w.s1; ++j, ++g) {
        #pragma unroll
        for (int part = 0; part < kParts; ++part) {
          const bool key = part < L::kChunks;
          uint4 cur[8];
          #pragma unroll
          for (int i = 0; i < 8; ++i) cur[i] = nxt[i];
          const float ks = nks, vs = nvs;
          load();
          if (key) {
            const int s = kp % L::kKStages;
            if (kp >= L::kKStages && !wait_uniform(bar(L::kKEmpty + s), (kp / L::kKStages + 1) & 1, abort)) {
              ok = false;
              break;
            }
            if (part == 0 && lane < 2) {
              // when K of tile g is written the scores of tile g - 4 are done,
              // so P V of tile g - 5 is: eight tiles of these live at a time
              const float lv = log2f(vs);
              meta[(g & 7) * 8 + 2 * cw + lane] = make_float4(ks, lv, ex2_approx(-lv), 0.f);
            }
            const uint32_t piece = sbase + L::kKOff + s * L::kKPiece;
            #pragma unroll
            for (int i = 0; i < 4; ++i) put(piece, 128, 32 * cw + 8 * i + r8, 0, cur[i]);
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(L::kKFull + s));
            ++kp;
          } else {
            const int s = vp % L::kVStages;
            if (vp >= L::kVStages && !wait_uniform(bar(L::kVEmpty + s), (vp / L::kVStages + 1) & 1, abort)) {
              ok = false;
              break;
            }
            constexpr int kRowsW = L::kVKeys / 4;
            if (j * 128 + 128 > full) {
              // NaN in a place that some row may not see: 0 instead, and the
              // rows that see it are mended when they are written
              uint32_t any = 0;
              #pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint32_t* c = reinterpret_cast<uint32_t*>(&cur[i]);
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t n = nan_bytes(c[k]);
                  any |= n;
                  c[k] &= ~n;
                }
              }
              if (any != 0) nan_seen[np & 3] = 1;
            }
            const uint32_t piece = sbase + L::kVOff + s * L::kVPiece;
            #pragma unroll
            for (int i = 0; i < kRowsW / 8; ++i)
              #pragma unroll
              for (int c = 0; c < L::kChunks; ++c)
                put(piece, L::kVKeys, kRowsW * cw + 8 * i + r8, c, cur[i * L::kChunks + c]);
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(L::kVFull + s));
            ++vp;
          }
        }
      }
      left -= w.s1 - w.s0;
      if (left > 0) at.next_unit(p);
    }
  } else {
    // ------------------------------------------------------------ softmax
    more_registers<192>();
    const int u = warp >> 2;                      // row tile of this warpgroup
    const int r_tile = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + L::kTO + (L::kTiles == 2 ? D * u : 0) + lane_off;
    int cs = 0, od = 0;     // S_FULL phases (d = 256: tiles), O_DONE phases consumed
    int g = 0;              // tiles of the CTA so far
    bool ok = u < L::kTiles;
    for (int np = 0; ok && left > 0; ++np) {
      int s0, s1, end, full, all_see;   // all_see: the keys that every live row of the unit sees
      {
        const Piece<D> w = piece_at<D>(p, at, left);
        s0 = w.s0;
        s1 = w.s1;
        end = (L::kTiles == 2 && u) ? w.end[L::kTiles - 1] : w.end[0];
        full = (L::kTiles == 2 && u) ? w.full[L::kTiles - 1] : w.full[0];
        all_see = seen_by_all<D>(w);
      }
      const int r = at.e % p.row_tiles * L::kRows + 128 * u + r_tile;
      const int sees = r < p.rows ? max(0, row_limit(p.seq, at.seq, r)) : 0;
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
      const int b = at.e / p.row_tiles, i = r / p.seq.G, head = at.h * p.seq.G + r % p.seq.G;
      const bool in = r < p.rows;
      const float sum = (in && i < at.seq.n) ? l : 0.f;
      const bool whole = s0 == 0 && s1 == at.steps;
      const long long slot = 2ll * blockIdx.x + (s0 > 0 ? 0 : 1);
      const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      const bool nans = nan_seen[np & 3] != 0;
      const int nan_from = max(s0, all_see / 128) * 128, nan_to = min(s1 * 128, sees);
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
                p.v + page * p.vs.b + at.h * p.vs.h + (key & ((1 << p.page_log2) - 1)) * p.vs.n + 32 * c);
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
      left -= s1 - s0;
      if (left > 0) at.next_unit(p);
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
