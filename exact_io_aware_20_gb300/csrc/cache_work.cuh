// The work of fa_fwd_cache, shared by its two kernels: lengths read on the
// device, the flat order of the steps and its cut into equal shares, and the
// kernel that joins the pieces of units that lie in several shares.
//
// A unit is a tile of RT query rows of one key/value head of one sequence, a
// step STEP of its keys.  Units follow one another in the order (sequence, row
// tile, head), each with OVER steps ahead of its own that stand for what a
// unit costs besides them (its queries' load, its results); CTA c takes places
// [c * share, (c + 1) * share) of them all, so that every CTA has the same
// work whatever the lengths are (without OVER, CTAs whose share held many
// short units took twice the average's time on a causal prompt).  A CTA's
// first unit may have begun in the share before and its last may go on in the
// next: it writes those as pieces (slot 0: the piece does not begin its unit,
// slot 1: it does), the units inside it as results.
#pragma once

#include "fa_internal.h"
#include "sm103_ptx.cuh"

// 1: for the kernels with the mask of a tree of drafted tokens.  They are
// compiled from the same sources as the others (fa_cache_fwd_tree.cu,
// fa_cache_prefill_tree.cu), which so carry none of it; what differs lies in a
// namespace of its own.
#ifndef FA_CACHE_TREE
#define FA_CACHE_TREE 0
#endif

namespace fa {

// The tcgen05 kernels, for many query rows (fa_cache_prefill.cu): rows of a unit.
int cache_prefill_rows(int d);

#if FA_CACHE_TREE
#define FA_CACHE_NAMESPACE tree
#else
#define FA_CACHE_NAMESPACE plain
#endif
inline namespace FA_CACHE_NAMESPACE {

constexpr bool kTree = FA_CACHE_TREE != 0;

struct SeqParams {
  const int *seq_lens, *new_lens;
  int B, G, Nq, causal;
  long long capacity;   // tokens that a table row can map
  unsigned int* err;
};

struct FwdCacheParams {
  SeqParams seq;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  Strides qs, os;
  const unsigned char *k, *v;
  Strides ks, vs;         // bytes
  const float *k_scale, *v_scale;
  const int* table;
  int width, pages, page_log2;
  int H, Hkv, rows;       // rows = G * Nq of a unit's key/value head
  int row_tiles;
  int bf16;
  float scale_log2;
  float* part_o;          // [CTA][2][RT][D]: O of a piece, not divided by its sum
  float2* part_ml;        // [CTA][2][RT]: its m (see kHead) and sum
  int4* joins;            // [CTA], the many-row kernel's: its unit that goes on behind its share
  int ctas;
  const uint32_t* tree;   // of a tree: [1 or B][Nq][tree_words], bit j of row i: it sees drafted token j
  long long tree_batch;   // words from a sequence's to the next's
  int tree_words;
};

constexpr float kNoMax = -1e30f;    // running maximum before the first key
// Weights are 2^(their log2 - m).  m is set kHead below a row's maximum and moves
// when that grows by more than kGrow: the largest weight is between 2^7 and
// 2^15, inside f16 (to 2^16), and the 25 powers below 1 that f16 has left (its
// steps end at 2^-24) go to the others.  With m at the maximum itself keys of
// less than 2^-25 of it were lost from the products, which over 2^17 keys came
// to 2^-8 of a result.
// Sums and O of parts (warps, softmax groups, pieces; a row's own when m moves) are
// taken times 2^(m - the joined m), which fp32 ends at 2^-126: a part whose maximum
// is 2^-118 of the whole one's or more is never lost, as m may stand 8 higher in it.
constexpr float kHead = 7.f, kGrow = 8.f;   // (log2 units)
// 2^-kHead: row sums are kept without it, their terms' factor 2^-kHead / vs as a
// product (2^-7 over the largest scale, 2^120, is no normal number, and the
// exponential would give 0)
constexpr float kHeadInv = 1.f / 128.f;
constexpr float kLogE2 = 0.6931471805599453f;

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
#if FA_CACHE_TREE
  if (s.len < s.n) {
    *bad = true;
    s.len = s.n = 0;
  }
#endif
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
#if FA_CACHE_TREE
    t.full = s.len - s.n;      // (p.causal is 0)
#endif
  }
  return t;
}
// The keys that row r sees.
__device__ __forceinline__ int row_limit(const SeqParams& p, const Sequence& s, int r) {
  return p.causal ? min(s.len, s.len - s.n + r / p.G + 1) : s.len;
}

// The mask row of token i of sequence b.
__device__ __forceinline__ const uint32_t* tree_row(const FwdCacheParams& p, int b, int i) {
  return p.tree + b * p.tree_batch + static_cast<long long>(i) * p.tree_words;
}
// Whether the row sees `key`, before the drafted tokens (from `base` on) or
// among them; key < the sequence's length.
__device__ __forceinline__ bool tree_sees(const uint32_t* row, int base, int key) {
  return key < base || (row[(key - base) >> 5] >> ((key - base) & 31) & 1);
}
// What the row sees of the 32 keys from key0 on, a bit each; none from `end` on.
__device__ __forceinline__ uint32_t tree_window(const uint32_t* row, int words, int base, int key0, int end) {
  const int k = (key0 - base) >> 5;      // (rounds down: -1 and less stand before the drafted tokens)
  const uint32_t lo = k < 0 ? ~0u : k < words ? row[k] : 0u;
  const uint32_t hi = k + 1 < 0 ? ~0u : k + 1 < words ? row[k + 1] : 0u;
  const uint32_t bits = __funnelshift_r(lo, hi, (key0 - base) & 31);
  const int left = end - key0;
  return left >= 32 ? bits : left <= 0 ? 0u : bits & ((1u << left) - 1u);
}

// Four e4m3 codes -> two f16x2.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

// Bytes that are NaN codes (0x7f, 0xff), as a byte mask.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// The power of two that brings a row with largest magnitude amax to
// [2^TOP, 2^(TOP + 1)) (1 for rows of zeros, NaN or infinities): `down` it, `up`
// its reciprocal.  Both are kept normal numbers, so that a row of the smallest
// magnitudes ends lower, and with TOP = 0 one of the largest an octave higher;
// its bits stay what they are.
template <int TOP>
__device__ __forceinline__ void row_power(float amax, float* up, float* down) {
  const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23), 1 + TOP), min(253 + TOP, 254));
  const bool plain = !(amax > 0.f) || !(amax < __uint_as_float(0x7f800000u));
  *down = plain ? 1.f : __uint_as_float(static_cast<uint32_t>(254 + TOP - e) << 23);   // 2^(127 + TOP - e)
  *up = plain ? 1.f : __uint_as_float(static_cast<uint32_t>(e - TOP) << 23);
}

template <int STEP>
__device__ __forceinline__ int steps_of(int lim) {
  return (lim + STEP - 1) / STEP;
}

// Limits of entry e = b * row_tiles + row tile.
template <int RT>
__device__ __forceinline__ TileLimits limits_of(const FwdCacheParams& p, int e, Sequence* s,
                                                bool* bad) {
  const int b = e / p.row_tiles, rt = e % p.row_tiles;
  *s = sequence_at(p.seq, b, bad);
  return tile_limits(p.seq, *s, rt * RT, min(p.rows, (rt + 1) * RT));
}

// Places that a unit of `lim` keys takes.
template <int STEP, int OVER>
__device__ __forceinline__ int places_of(int lim) {
  return lim > 0 ? OVER + steps_of<STEP>(lim) : 0;
}

// Counts the places of the call, one key/value head counted (the result, the
// same in every thread), and finds the entry in which place `which(count)`
// lies, if that is not negative: found->x the entry, found->y the places
// before it.  All threads of the block; red: two values a warp.
template <int RT, int STEP, int OVER, int THREADS, class Which>
__device__ __forceinline__ long long find_place(const FwdCacheParams& p, long long* red,
                                                longlong2* found, bool* bad, Which which) {
  constexpr int kWarps = THREADS / 32;
  const int entries = p.seq.B * p.row_tiles, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // this thread's entry of the block of entries from e0 on: its places
  auto places_at = [&](int e0) -> long long {
    const int e = e0 + static_cast<int>(threadIdx.x);
    if (e >= entries) return 0;
    Sequence s;
    return places_of<STEP, OVER>(limits_of<RT>(p, e, &s, bad).lim);
  };
  // inclusive sum over the block's threads, and all of them
  auto scan = [&](long long mine, long long* all, long long* space) -> long long {
    #pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, mine, m);
      if (lane >= m) mine += x;
    }
    if (lane == 31) space[warp] = mine;
    __syncthreads();
    *all = 0;
    #pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) mine += space[i];
      *all += space[i];
    }
    return mine;
  };
  long long all, mine = places_at(0);
  long long upto = scan(mine, &all, red), count = all;
  if (entries > THREADS) {
    long long rest = 0, behind;
    for (int e0 = THREADS; e0 < entries; e0 += THREADS) rest += places_at(e0);
    scan(rest, &behind, red + kWarps);
    count += behind;
  }
  const long long at = which(count);
  if (at >= 0) {
    long long before = 0;
    for (int e0 = 0;;) {
      if (mine > 0 && before + upto - mine <= at && at < before + upto) {
        found->x = e0 + static_cast<int>(threadIdx.x);
        found->y = before + upto - mine;
      }
      before += all;
      e0 += THREADS;
      if (e0 >= entries || at < before) break;
      __syncthreads();
      mine = places_at(e0);
      upto = scan(mine, &all, red);
    }
    __syncthreads();
  }
  return count;
}

// A walk over the pieces of a share.
template <int RT, int STEP, int OVER>
struct Walk {
  int e, h;                // entry and key/value head of the unit
  int steps, lim, full;    // its steps and limits
  Sequence seq;
  int place;               // where the share is in it
  long long left;          // places left of the share
  int s0, s1;              // the piece: the unit's steps [s0, s1)
  __device__ __forceinline__ void enter(const FwdCacheParams& p) {
    bool bad = false;
    const TileLimits t = limits_of<RT>(p, e, &seq, &bad);
    lim = t.lim;
    full = t.full;
    steps = steps_of<STEP>(lim);
  }
  // To place lo of all (found: of place lo / Hkv; entry e's Hkv units stand
  // one after another from place found->y * Hkv on), for n places.
  __device__ __forceinline__ void start(const FwdCacheParams& p, const longlong2* found,
                                        long long lo, long long n) {
    e = static_cast<int>(found->x);
    enter(p);
    const long long rest = lo - found->y * p.Hkv;
    h = static_cast<int>(rest / (OVER + steps));
    place = static_cast<int>(rest % (OVER + steps));
    left = n;
  }
  // The next piece that has a step (s0, s1); false behind the last.
  __device__ __forceinline__ bool next(const FwdCacheParams& p) {
    while (left > 0) {
      if (place == OVER + steps) {
        place = 0;
        if (++h == p.Hkv) {
          h = 0;
          const int entries = p.seq.B * p.row_tiles;
          do {
            if (++e >= entries) { left = 0; return false; }
            enter(p);
          } while (steps == 0);
        }
      }
      const int to = static_cast<int>(min(static_cast<long long>(OVER + steps), place + left));
      s0 = max(0, place - OVER);
      s1 = to - OVER;
      left -= to - place;
      place = to;
      if (s1 > s0) return true;
    }
    return false;
  }
};

// Joins the pieces of units that lie in several shares, and writes the units
// that see no key.  Block (c, y) looks for the unit whose steps begin in share
// c and go on behind it; its warps take a row each, or with RECORDS four (there
// are few pieces and many rows): the pieces' weights first, then their O, four
// loads in flight.
//
// RECORDS: the attention kernel has left that unit in p.joins[c] (entry, head,
// last CTA, tokens of the sequence; last CTA < 0: there is none).  With many
// rows a unit is many blocks' work, and each block's own search was most of
// this kernel's time (d = 128, 4 prompts of 2048 tokens: 20 us of the call's
// 130; 10 with the records, 6 with four rows a warp).  With few rows the search
// is over before the attention kernel's end, and a record would be one more
// read behind it.
constexpr int kMergeThreads = 128, kMergeRows = 4, kPairRows = 2;
template <int D, int RT, int STEP, int OVER, bool RECORDS, int ROWS>
__global__ void __launch_bounds__(kMergeThreads)
cache_merge_kernel(const __grid_constant__ FwdCacheParams p) {
  constexpr int kVec = D / 32, kWarps = kMergeThreads / 32;
  constexpr int kRows = ROWS;                          // of a warp at a time
  constexpr int kLanes = 32 / kRows;                   // that share out a row's pieces
  constexpr int kPieces = ROWS > kPairRows ? 1 : 4;    // whose O is in flight at once
  __shared__ long long red[2 * kWarps];
  __shared__ longlong2 found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_first = blockIdx.y * kWarps + warp, row_step = gridDim.y * kWarps;
  bool bad = false;
  const int c0 = blockIdx.x;
  int4 join = make_int4(0, 0, -1, 0);
  if constexpr (RECORDS) {
    grid_dependency_wait();
    join = p.joins[c0];
  } else {
    long long share = 0, end = 0;
    bool joins = false;
    find_place<RT, STEP, OVER, kMergeThreads>(p, red, &found, &bad, [&](long long count) {
      const long long total = count * p.Hkv;
      share = (total + p.ctas - 1) / p.ctas;
      end = (c0 + 1) * share;
      joins = end < total && share > 0;      // (share > 0 wherever a step is)
      return joins ? (end - 1) / p.Hkv : -1ll;
    });
    if (joins) {
      Walk<RT, STEP, OVER> at;
      at.start(p, &found, end - 1, 1);
      const long long first = end - 1 - at.place + OVER, last = first + at.steps - 1;   // its steps
      if (last >= end && first >= end - share && first < end)
        join = make_int4(at.e, at.h, static_cast<int>(last / share), at.seq.n);
    }
    grid_dependency_wait();   // (every CTA: this grid's end is to imply the other's)
  }
  const int c1 = join.z;
  if (c1 > c0) {
    const int b = join.x / p.row_tiles, row0 = (join.x - b * p.row_tiles) * RT;
    const int own = lane / kLanes, pl = lane % kLanes;    // the weights that this lane works out
    for (int first = kRows * row_first; first < RT && row0 + first < p.rows; first += kRows * row_step) {
      const int rr = first + own;
      const bool on = row0 + rr < p.rows;
      float top = kNoMax, sum = 0.f;
      if constexpr (ROWS == kPairRows) {
        // two rows of a block of eight: a lane has every second one's columns
        // 4 (lane / 2) + 64 t, so that two lanes read a sector
        constexpr int kPart = D / 64;
        const int y = lane & 1, col4 = lane >> 1;
        float4 acc[kPart];
        #pragma unroll
        for (int t = 0; t < kPart; ++t) acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0 + pl; on && c <= c1; c += kLanes)
          top = fmaxf(top, p.part_ml[(2ll * c + (c == c0)) * RT + rr].x);
        #pragma unroll
        for (int x = kLanes / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        for (int cb = c0; cb <= c1; cb += kLanes) {
          float2 ml = make_float2(kNoMax, 0.f);
          const int mine = cb + pl;
          if (on && mine <= c1) ml = p.part_ml[(2ll * mine + (mine == c0)) * RT + rr];
          const float w = ex2_approx(ml.x - top);
          float part = ml.y == 0.f ? 0.f : ml.y * w;
          #pragma unroll
          for (int x = kLanes / 2; x > 0; x >>= 1) part += __shfl_xor_sync(0xffffffffu, part, x);
          sum += part;
          // a piece without keys for the row has left its O unwritten
          const uint32_t has = __ballot_sync(0xffffffffu, ml.y != 0.f);
          const int n = min(kLanes, c1 - cb + 1);
          for (int k0 = 0; k0 < n; k0 += kPieces) {
            float4 x[kPieces][kPart];
            float wk[kPieces];
            #pragma unroll
            for (int k = 0; k < kPieces; ++k) {
              const int c = cb + k0 + k, from = kLanes * y + ((k0 + k) & (kLanes - 1));
              wk[k] = __shfl_sync(0xffffffffu, w, from);
              const bool there = k0 + k < n && (has >> from & 1);
              const float4* src = reinterpret_cast<const float4*>(
                  p.part_o + ((2ll * c + (c == c0)) * RT + (first & ~7)) * D) + 8 * col4 + (first & 7) + y;
              #pragma unroll
              for (int t = 0; t < kPart; ++t) {
                x[k][t] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (there) x[k][t] = src[8 * 16 * t];
              }
            }
            #pragma unroll
            for (int k = 0; k < kPieces; ++k)
              #pragma unroll
              for (int t = 0; t < kPart; ++t) {
                acc[t].x = fmaf(x[k][t].x, wk[k], acc[t].x);
                acc[t].y = fmaf(x[k][t].y, wk[k], acc[t].y);
                acc[t].z = fmaf(x[k][t].z, wk[k], acc[t].z);
                acc[t].w = fmaf(x[k][t].w, wk[k], acc[t].w);
              }
          }
        }
        if ((row0 + rr) / p.seq.G >= join.w) sum = 0.f;
        const float total = __shfl_sync(0xffffffffu, sum, kLanes * y), m = __shfl_sync(0xffffffffu, top, kLanes * y);
        const int r = row0 + first + y;
        if (r < p.rows) {
          const int i = r / p.seq.G, head = join.y * p.seq.G + r - i * p.seq.G;
          const float inv = total == 0.f ? 0.f : kHeadInv / total;
          uint2* dst = reinterpret_cast<uint2*>(p.o + b * p.os.b + head * p.os.h + i * p.os.n) + col4;
          #pragma unroll
          for (int t = 0; t < kPart; ++t) {
            uint2 z = make_uint2(0u, 0u);
            if (total != 0.f)
              z = p.bf16 ? make_uint2(pack2<true>(acc[t].x * inv, acc[t].y * inv), pack2<true>(acc[t].z * inv, acc[t].w * inv))
                         : make_uint2(pack2<false>(acc[t].x * inv, acc[t].y * inv), pack2<false>(acc[t].z * inv, acc[t].w * inv));
            dst[16 * t] = z;
          }
          if (col4 == 0)
            p.lse[(static_cast<long long>(b) * p.H + head) * p.seq.Nq + i] =
                total == 0.f ? -INFINITY : (m + kHead + log2f(total)) * kLogE2;
        }
        continue;
      }
      float acc[kRows][kVec];
      #pragma unroll
      for (int k = 0; k < kRows; ++k)
        #pragma unroll
        for (int v = 0; v < kVec; ++v) acc[k][v] = 0.f;
      for (int c = c0 + pl; on && c <= c1; c += kLanes)
        top = fmaxf(top, p.part_ml[(2ll * c + (c == c0)) * RT + rr].x);
      #pragma unroll
      for (int x = kLanes / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      for (int cb = c0; cb <= c1; cb += kLanes) {
        float2 ml = make_float2(kNoMax, 0.f);
        const int mine = cb + pl;
        if (on && mine <= c1) ml = p.part_ml[(2ll * mine + (mine == c0)) * RT + rr];
        const float w = ex2_approx(ml.x - top);
        float part = ml.y == 0.f ? 0.f : ml.y * w;
        #pragma unroll
        for (int x = kLanes / 2; x > 0; x >>= 1) part += __shfl_xor_sync(0xffffffffu, part, x);
        sum += part;
        // a piece without keys for the row has left its O unwritten
        const uint32_t has = __ballot_sync(0xffffffffu, ml.y != 0.f);
        const int n = min(kLanes, c1 - cb + 1);
        for (int k0 = 0; k0 < n; k0 += kPieces) {
          float x[kRows][kPieces][kVec], wk[kRows][kPieces];
          #pragma unroll
          for (int k = 0; k < kPieces; ++k) {
            const int c = cb + k0 + k;
            #pragma unroll
            for (int y = 0; y < kRows; ++y) {
              const int from = kLanes * y + ((k0 + k) & (kLanes - 1));
              wk[y][k] = __shfl_sync(0xffffffffu, w, from);
              #pragma unroll
              for (int v = 0; v < kVec; ++v) x[y][k][v] = 0.f;
              if (k0 + k < n && (has >> from & 1)) {
                const float* src = p.part_o + ((2ll * c + (c == c0)) * RT + first + y) * D + lane * kVec;
                #pragma unroll
                for (int v = 0; v < kVec; v += 2) {
                  const float2 z = *reinterpret_cast<const float2*>(src + v);
                  x[y][k][v] = z.x;
                  x[y][k][v + 1] = z.y;
                }
              }
            }
          }
          #pragma unroll
          for (int k = 0; k < kPieces; ++k)
            #pragma unroll
            for (int y = 0; y < kRows; ++y)
              #pragma unroll
              for (int v = 0; v < kVec; ++v) acc[y][v] = fmaf(x[y][k][v], wk[y][k], acc[y][v]);
        }
      }
      if ((row0 + rr) / p.seq.G >= join.w) sum = 0.f;
      #pragma unroll
      for (int y = 0; y < kRows; ++y) {
        const int r = row0 + first + y;
        const float total = __shfl_sync(0xffffffffu, sum, kLanes * y), m = __shfl_sync(0xffffffffu, top, kLanes * y);
        if (r >= p.rows) break;
        const int i = r / p.seq.G, head = join.y * p.seq.G + r - i * p.seq.G;
        const float inv = total == 0.f ? 0.f : kHeadInv / total;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + b * p.os.b + head * p.os.h + i * p.os.n + lane * kVec);
        #pragma unroll
        for (int v = 0; v < kVec; v += 2)
          dst[v / 2] = total == 0.f ? 0u
                       : p.bf16 ? pack2<true>(acc[y][v] * inv, acc[y][v + 1] * inv)
                                : pack2<false>(acc[y][v] * inv, acc[y][v + 1] * inv);
        if (lane == 0)
          p.lse[(static_cast<long long>(b) * p.H + head) * p.seq.Nq + i] =
              total == 0.f ? -INFINITY : (m + kHead + log2f(total)) * kLogE2;
      }
    }
  }
  for (int e = blockIdx.x; e < p.seq.B * p.row_tiles; e += gridDim.x) {
    Sequence seq;
    if (limits_of<RT>(p, e, &seq, &bad).lim > 0) continue;
    const int row0 = e % p.row_tiles * RT, b = e / p.row_tiles;
    for (int h = 0; h < p.Hkv; ++h)
      for (int rr = row_first; rr < RT && row0 + rr < p.rows; rr += row_step) {
        const int r = row0 + rr, i = r / p.seq.G, head = h * p.seq.G + r % p.seq.G;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + b * p.os.b + head * p.os.h + i * p.os.n + lane * kVec);
        #pragma unroll
        for (int v = 0; v < kVec; v += 2) dst[v / 2] = 0u;
        if (lane == 0) p.lse[(static_cast<long long>(b) * p.H + head) * p.seq.Nq + i] = -INFINITY;
      }
  }
}

// Launches the join behind the attention kernel, as its programmatic
// dependent.  With records, units of one tile of rows (`rows` of them at most, not
// 0), which lie in many pieces, have two rows a warp, of results that lie in
// blocks of eight rows [columns / 4][row][4]: the attention kernel's threads, a
// row each, so write whole lines (a tree's 100 rows, 8 sequences of 8192 tokens,
// d = 128: rows one behind another, four a warp 51 us, one 49, in blocks 47; d =
// 256, 128 rows of 4 x 32768 136.3 -> 134.6; with two tiles, 256 rows, d = 128, 8
// of 8192, one row a warp instead of four 79 -> 82, so not there).
template <int D, int RT, int STEP, int OVER, bool RECORDS>
cudaError_t launch_cache_merge(const FwdCacheParams& p, cudaStream_t stream, int rows = 0) {
  constexpr int kWarps = kMergeThreads / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas), RECORDS ? RT / (kWarps * kMergeRows) : RT > 8 ? RT / 8 : 1, 1);
  auto kern = cache_merge_kernel<D, RT, STEP, OVER, RECORDS, RECORDS ? kMergeRows : 1>;
  if constexpr (RECORDS && kTree) {
    if (rows > 0) {
      kern = cache_merge_kernel<D, RT, STEP, OVER, true, kPairRows>;
      cfg.gridDim.y = static_cast<unsigned>((rows + kWarps * kPairRows - 1) / (kWarps * kPairRows));
    }
  }
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// The launch of the many-row kernels.
cudaError_t launch_cache_prefill(const Cache& cache, FwdCacheParams& p, int sms,
                                 cudaStream_t stream);

}  // namespace tree, plain

}  // namespace fa
