// Attention over the paged 8-bit cache (fa_fwd_cache).
//
// Scores and weights.  For a page with scales ks and vs and codes K8, V8,
//     s = scale * ks * (q . K8),    O = sum_j p_j vs V8_j / sum_j p_j.
// e4m3 codes widen to f16 exactly, so both products run on f16 operands with
// fp32 sums: q as f16 (a bf16 row is first divided by the power of two of its
// largest element, which loses nothing that the product could show), and the
// weights as f16 with the value scale taken into the exponent,
//     p'_j = 2^(s_j log2 e + log2 vs - m),  m = max_j (s_j log2 e + log2 vs) - 7,
// so that they lie in [0, 2^7] whatever the pages' scales are; the row sum adds
// 2^-7 p'_j / vs in fp32.  m is moved only when the maximum grows by more
// than 8 (p' then stays below 2^15, inside f16), so that most tiles need
// one vote and no reduction.
//
// Work.  What bounds it for few query rows is the cache's bytes: the G query
// heads of a key/value head, times the query tokens, form the rows of one
// unit, so a page is read once for all of them.  Sequences have unlike
// lengths that only the device knows: the steps (of 4 warps x kTile keys) of
// all units, laid end to end, are cut into equal shares, one for each
// resident CTA, so every CTA streams the same number of bytes.  A unit that
// lies in several shares leaves normalisation to the merge kernel: each piece
// writes its maximum, sum and unnormalised O, at most two pieces a CTA.
//
// A warp has its own ring of kStages tiles (kTile keys of K and V, 8 KB) in
// shared memory, filled by TMA through the page table, and its own m,
// sum and O; the four warps of a CTA meet only where a unit ends.
// With S^T = K Q^T and O^T = V^T P^T the cache is the A operand (16 keys or 16
// columns a fragment), so 8 query rows fill an MMA: a step of mma.sync
// m16n8k16 costs nothing that shows beside the loads.
//
// Measured (32 heads on 8, d = 128, one token a sequence): four sequences of up
// to 131072 tokens 122 us, 5.9 TB/s (89% of what a copy reaches); eight of 8192
// 33.5 us, 4.0 TB/s: a call's ends (the lengths, the first copies, the join) are
// a third of that, 10 us with one sequence of 1000.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache_work.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
// A unit's cost besides its steps, in steps (1 / 2 / 3 / 4 / 5 / 6: 32 sequences of
// up to 4096 tokens take 41 / 36 / 34 / 34 / 34 / 35 us, 128 of up to 700 41 / 35 /
// 35 / 35 / 35 / 36, 64 of up to 2000 at d = 64 52 / 44 / 44 / 42 / 43 / 46, 16 of up
// to 4000 at d = 256 26 / 24 / 23 / 23 / 22 / 23, 8 of 8192 35 / 34 / 34 / 33 / 33 / 33).
constexpr int kOver = 3;

template <int D>
struct Tile {
  static constexpr int kKeys = 4096 / D;                 // keys of a warp's tile
  static constexpr int kStep = kWarps * kKeys;           // keys of a CTA's step
  static constexpr int kBytes = 4096;                    // of K, and of V
  static constexpr int kPitch = D < 128 ? D : 128;       // bytes of a row in shared memory
  static constexpr int kHalves = D / kPitch;             // 128-column parts, one after another
  static constexpr int kSub = kKeys / 16;                // pages that a tile can touch
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The key of a 16-key fragment that row g (of 8) of the fragment's halves
// stands for.  Chosen so that neither the K loads (8 lanes read rows g, g + 1)
// nor the V loads (8 lanes read the four even or odd rows) meet a bank twice
// under TMA's swizzle of the tile.
template <int D>
__device__ __forceinline__ int key_of(int g) {
  if constexpr (D == 64) return (g & 4) | ((g & 1) << 1) | (((g >> 1) ^ g) & 1);
  else return g ^ ((g & 1) << 2);
}

// Byte offset of 16-byte chunk c of row r in a tile part.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (D == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return r * 128 + ((c ^ (r & 7)) << 4);
}

template <int D, int NT>
struct Smem {
  using T = Tile<D>;
  static constexpr int kRing = kWarps * kStages * 2 * T::kBytes;
  static constexpr int kQOff = kRing;
  static constexpr int kQBytes = D * NT * 16;              // q fragments, f16
  static constexpr int kBufOff = kQOff + kQBytes;          // O of warps while they are joined:
  static constexpr int kBufWarps = NT * D < 256 ? 2 : 1;   // of one where two CTAs would not fit an SM
  static constexpr int kBufBytes = kBufWarps * 8 * NT * D * 4;
  static constexpr int kStatOff = kBufOff + kBufBytes;     // (m, sum) [warp][row]
  static constexpr int kStatBytes = kWarps * 8 * NT * 8;
  static constexpr int kQsOff = kStatOff + kStatBytes;     // [row] power of two taken off q
  static constexpr int kMetaOff = kQsOff + 8 * NT * 4;     // (ks, log2 vs, 2^-7 / vs) [warp][stage][page]
  static constexpr int kMetaBytes = kWarps * kStages * T::kSub * 16;
  static constexpr int kBarOff = kMetaOff + kMetaBytes;
  static constexpr int kMiscOff = kBarOff + kWarps * kStages * 8;
  static constexpr int kAlloc = kMiscOff + 64 + 1024;      // slack to align the base
  static_assert(2 * (kAlloc + 1024) <= 228 * 1024, "two CTAs an SM");
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads)
cache_fwd_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ FwdCacheParams p) {
  using T = Tile<D>;
  using S = Smem<D, NT>;
  constexpr int RT = 8 * NT;                   // rows of a unit
  constexpr int kMT = D / 16;                  // 16-column fragments of O^T
  constexpr int kChunks = D / 64;              // 64-column parts of a row
  constexpr bool kQRegs = kChunks * 8 * NT <= 32;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  long long* red = reinterpret_cast<long long*>(smem + S::kBufOff);
  longlong2* found = reinterpret_cast<longlong2*>(smem + S::kBufOff + 128);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kMiscOff);
  uint2* q_frag = reinterpret_cast<uint2*>(smem + S::kQOff);
  float2* stat = reinterpret_cast<float2*>(smem + S::kStatOff);
  float* q_pow = reinterpret_cast<float*>(smem + S::kQsOff);
  const uint32_t meta = base + S::kMetaOff + warp * kStages * T::kSub * 16;
  const uint32_t ring = base + warp * kStages * 2 * T::kBytes;
  const uint32_t bars = base + S::kBarOff + warp * kStages * 8;

  grid_launch_dependents();   // the merge may be set up; it waits for this grid's end
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(base + S::kBarOff + 8 * i, 1);
    *abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  bool bad = false;
  long long lo = 0, hi = 0;
  find_place<RT, T::kStep, kOver, kThreads>(p, red, found, &bad, [&](long long count) {
    const long long total = count * p.Hkv, share = (total + p.ctas - 1) / p.ctas;
    lo = blockIdx.x * share;
    hi = min(total, lo + share);
    return lo < hi ? lo / p.Hkv : -1ll;
  });
  if (bad && blockIdx.x == 0) atomicOr(p.seq.err, kErrCache);
  if (lo >= hi) return;
  Walk<RT, T::kStep, kOver> at;
  at.start(p, found, lo, hi - lo);
  __syncthreads();   // found is read; its place is the join buffer's

  // ---------------------------------------------------------------- loads
  const int sub_log2 = min(p.page_log2, 31 - __clz(T::kKeys));   // keys of a box
  const int subs = T::kKeys >> sub_log2;                         // boxes (pages) of a tile
  const uint32_t box_bytes = static_cast<uint32_t>(T::kPitch) << sub_log2;
  Walk<RT, T::kStep, kOver> f = at;
  bool f_more = f.next(p);
  int f_step = f_more ? f.s0 : 0;
  int fetched = 0, done = 0;
  int tb_first = 0, tb_steps = 0;      // steps of f's unit that the table registers cover
  int tb_page = 0;
  float tb_ks = 1.f, tb_lv = 0.f;
  // The scales of a tile go to shared memory when the tile is first needed or
  // the registers are loaded anew, not when its copies are issued: the wait
  // for them is then behind the copies of the tiles that follow.
  int scaled = 0;                      // tiles whose scales are there
  int tile_from[kStages];              // the register lane of each stage's tile
  auto scales = [&]() {
    for (; scaled < fetched; ++scaled) {
      const int stage = scaled % kStages;
      int from = tile_from[0];
      #pragma unroll
      for (int i = 1; i < kStages; ++i) from = stage == i ? tile_from[i] : from;
      const float ks = __shfl_sync(0xffffffffu, tb_ks, from + (lane & (subs - 1)));
      const float lv = __shfl_sync(0xffffffffu, tb_lv, from + (lane & (subs - 1)));
      if (lane < subs)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(meta + (stage * T::kSub + lane) * 16),
                     "f"(ks), "f"(lv), "f"(ex2_approx(-lv) * kHeadInv), "f"(0.f) : "memory");
    }
    __syncwarp();
  };
  bool dead = false;                   // a wait gave up: no further loads
  // Issue the warp's next tile, if it has one left in the share.
  auto fetch = [&]() {
    while (f_more && !dead) {
      const int k0 = (f_step * kWarps + warp) * T::kKeys;
      const bool mine = k0 < f.lim;
      if (mine) {
        if (f_step >= tb_first + tb_steps) {
          // the pages and scales of the next 32 / subs steps, one a lane
          scales();
          tb_first = f_step;
          tb_steps = 32 / subs;
          const int key = ((f_step + lane / subs) * kWarps + warp) * T::kKeys +
                          ((lane & (subs - 1)) << sub_log2);
          tb_page = 0;
          tb_ks = 1.f;
          tb_lv = 0.f;
          if (key < f.lim) {
            const int b = f.e / p.row_tiles;
            tb_page = p.table[static_cast<long long>(b) * p.width + (key >> p.page_log2)];
            if (static_cast<unsigned>(tb_page) >= static_cast<unsigned>(p.pages)) {
              atomicOr(p.seq.err, kErrCache);
              tb_page = 0;
            }
            const long long sc = static_cast<long long>(tb_page) * p.Hkv + f.h;
            tb_ks = p.k_scale[sc];
            tb_lv = log2f(p.v_scale[sc]);
          }
        }
        const int stage = fetched % kStages;
        const int from = (f_step - tb_first) * subs;
        const uint32_t bar = bars + 8 * stage;
        const uint32_t dst = ring + stage * 2 * T::kBytes;
        const int boxes = min(subs, (f.lim - k0 + (1 << sub_log2) - 1) >> sub_log2);
        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * T::kHalves * 2 * box_bytes);
        const int row = subs > 1 ? 0 : k0 & ((1 << p.page_log2) - 1);
        #pragma unroll 1
        for (int i = 0; i < boxes; ++i) {
          const int page = __shfl_sync(0xffffffffu, tb_page, from + i);
          if (lane == 0) {
            #pragma unroll
            for (int c = 0; c < T::kHalves; ++c) {
              const uint32_t to = dst + c * T::kKeys * T::kPitch + i * box_bytes;
              tma_load_4d(to, &tm_k, bar, c * 128, row, f.h, page);
              tma_load_4d(to + T::kBytes, &tm_v, bar, c * 128, row, f.h, page);
            }
          }
        }
        #pragma unroll
        for (int i = 0; i < kStages; ++i) tile_from[i] = stage == i ? from : tile_from[i];
        __syncwarp();
        ++fetched;
      }
      if (++f_step == f.s1) {
        f_more = f.next(p);
        f_step = f.s0;
        tb_steps = 0;
        tb_first = 0;
      }
      if (mine) break;
    }
  };
  #pragma unroll 1
  for (int i = 0; i < kStages; ++i) fetch();

  // This lane's places in a tile: of the K rows that it holds (64-column part
  // 0; part 1 is the same with bit 6 turned), of the even and odd V rows
  const uint32_t k_at = chunk_at<D>(key_of<D>(g), t);
  const uint32_t v_at[2] = {
      chunk_at<D>(key_of<D>(2 * t), D == 64 ? g >> 1 : g) + (D == 64 ? (g & 1) * 8 : 0),
      chunk_at<D>(key_of<D>(2 * t + 1), D == 64 ? g >> 1 : g) + (D == 64 ? (g & 1) * 8 : 0)};
  constexpr uint32_t kFrag = 16 * T::kPitch;    // bytes of 16 rows

  // ---------------------------------------------------------------- units
  while (at.next(p)) {
    const int b = at.e / p.row_tiles, row0 = at.e % p.row_tiles * 8 * NT;
    // q of the unit's rows as B fragments of S^T = K Q^T: lane (g, t) of
    // fragment (64-column part c, j) holds row g, columns 64c + 16t + 4j ..+3
    for (int nt = warp; nt < NT; nt += kWarps) {
      const int r = row0 + nt * 8 + g;
      uint4 w[kChunks][2];
      float amax = 0.f;
      #pragma unroll
      for (int c = 0; c < kChunks; ++c) w[c][0] = w[c][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < p.rows && r / p.seq.G < at.seq.n) {
        const uint16_t* src = p.q + b * p.qs.b + (at.h * p.seq.G + r % p.seq.G) * p.qs.h +
                              (r / p.seq.G) * p.qs.n + 16 * t;
        #pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          w[c][0] = *reinterpret_cast<const uint4*>(src + 64 * c);
          w[c][1] = *reinterpret_cast<const uint4*>(src + 64 * c + 8);
        }
      }
      float down = 1.f;
      if (p.bf16) {
        #pragma unroll
        for (int c = 0; c < kChunks; ++c)
          #pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t u[4] = {w[c][i].x, w[c][i].y, w[c][i].z, w[c][i].w};
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = unpack2<true>(u[k]);
              amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float up;
        row_power<0>(amax, &up, &down);
        if (t == 0) q_pow[nt * 8 + g] = up;
      } else if (t == 0) {
        q_pow[nt * 8 + g] = 1.f;
      }
      #pragma unroll
      for (int c = 0; c < kChunks; ++c)
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t u[4] = {w[c][i].x, w[c][i].y, w[c][i].z, w[c][i].w};
          if (p.bf16) {
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = unpack2<true>(u[k]);
              u[k] = pack2<false>(x.x * down, x.y * down);
            }
          }
          q_frag[((c * 4 + 2 * i) * NT + nt) * 32 + lane] = make_uint2(u[0], u[1]);
          q_frag[((c * 4 + 2 * i + 1) * NT + nt) * 32 + lane] = make_uint2(u[2], u[3]);
        }
    }
    __syncthreads();
    uint2 qr[kQRegs ? kChunks * 4 : 1][kQRegs ? NT : 1];
    if constexpr (kQRegs) {
      #pragma unroll
      for (int i = 0; i < kChunks * 4; ++i)
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) qr[i][nt] = q_frag[(i * NT + nt) * 32 + lane];
    }
    float qscale[NT][2], m[NT][2], l[NT][2];
    float acc[kMT][NT][4];
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      #pragma unroll
      for (int c = 0; c < 2; ++c) {
        qscale[nt][c] = q_pow[nt * 8 + 2 * t + c] * p.scale_log2;
        m[nt][c] = kNoMax;
        l[nt][c] = 0.f;
      }
    #pragma unroll
    for (int i = 0; i < kMT; ++i)
      #pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][nt][k] = 0.f;

    for (int step = at.s0; step < at.s1; ++step) {
      const int k0 = (step * kWarps + warp) * T::kKeys;
      if (k0 >= at.lim) continue;
      const int stage = done % kStages;
      if (scaled <= done) scales();
      if (!dead && !wait_uniform(bars + 8 * stage, (done / kStages) & 1, abort)) dead = true;
      if (dead) continue;
      const uint32_t kt = ring + stage * 2 * T::kBytes, vt = kt + T::kBytes;
      // 16 keys, the mt-th of the tile; PARTIAL: some row may not see some of
      // them (a branch of its own, so that the common one stays short)
      auto fragment = [&](auto is_partial, int mt) {
        constexpr bool PARTIAL = decltype(is_partial)::value;
        float sc[4];
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(sc[0]), "=f"(sc[1]), "=f"(sc[2]), "=f"(sc[3])
                     : "r"(meta + (stage * T::kSub + ((mt * 16) >> sub_log2)) * 16));
        // S^T of the 16 keys
        float s[NT][4];
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        #pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const uint32_t from = kt + (c >> 1) * T::kKeys * T::kPitch + mt * kFrag + (k_at ^ ((c & 1) << 6));
          const uint4 x = ld_shared_v4(from);
          const uint4 y = ld_shared_v4(from + kFrag / 2);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
          #pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            widen4(xs[j], a0, a2);
            widen4(ys[j], a1, a3);
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q2 = kQRegs ? qr[kQRegs ? c * 4 + j : 0][kQRegs ? nt : 0]
                                      : q_frag[((c * 4 + j) * NT + nt) * 32 + lane];
              mma(s[nt], a0, a1, a2, a3, q2.x, q2.y);
            }
          }
        }
        bool grow = false;
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f[2] = {qscale[nt][0] * sc[0], qscale[nt][1] * sc[0]};
          #pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[nt][k] = fmaf(s[nt][k], f[k & 1], sc[1]);
            if constexpr (PARTIAL) {
              const int r = row0 + nt * 8 + 2 * t + (k & 1);
              const int key = k0 + mt * 16 + key_of<D>(g) + (k >> 1) * 8;
              if (key >= row_limit(p.seq, at.seq, r)) s[nt][k] = -INFINITY;
            }
          }
          grow |= fmaxf(s[nt][0], s[nt][2]) > m[nt][0] + (kHead + kGrow) ||
                  fmaxf(s[nt][1], s[nt][3]) > m[nt][1] + (kHead + kGrow);
        }
        if (__any_sync(0xffffffffu, grow)) {
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            #pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(s[nt][c], s[nt][c + 2]);
              #pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              const float now = fmaxf(m[nt][c], top - kHead);
              const float f = ex2_approx(m[nt][c] - now);
              m[nt][c] = now;
              l[nt][c] *= f;
              #pragma unroll
              for (int i = 0; i < kMT; ++i) {
                acc[i][nt][c] *= f;
                acc[i][nt][c + 2] *= f;
              }
            }
        }
        // the weights, as B fragments of O^T = V^T P^T
        uint32_t p0[NT], p1[NT];
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
          #pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = ex2_approx(s[nt][k] - m[nt][k & 1]);
          l[nt][0] = fmaf(w[0] + w[2], sc[2], l[nt][0]);
          l[nt][1] = fmaf(w[1] + w[3], sc[2], l[nt][1]);
          p0[nt] = transpose8x8(pack2<false>(w[0], w[1]));
          p1[nt] = transpose8x8(pack2<false>(w[2], w[3]));
        }
        bool nans = false;
        #pragma unroll
        for (int half = 0; half < T::kHalves; ++half) {
          const uint32_t part = vt + half * T::kKeys * T::kPitch + mt * kFrag;
          constexpr int kWords = D == 64 ? 2 : 4;    // 4-column words of a lane
          uint32_t v[4][kWords];
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t from = part + v_at[i & 1] + (i >> 1) * (kFrag / 2);
            if constexpr (D == 64) {
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[i][0]), "=r"(v[i][1]) : "r"(from) : "memory");
            } else {
              const uint4 x = ld_shared_v4(from);
              v[i][0] = x.x;
              v[i][1] = x.y;
              v[i][2] = x.z;
              v[i][3] = x.w;
            }
          }
          if constexpr (PARTIAL) {
            // a NaN in a masked place would turn 0 * NaN into NaN: NaN codes
            // are taken out here and their effect on the rows that see them
            // is added below
            #pragma unroll
            for (int i = 0; i < 4; ++i)
              #pragma unroll
              for (int w = 0; w < kWords; ++w) {
                const uint32_t n = nan_bytes(v[i][w]);
                nans |= n != 0;
                v[i][w] &= ~n;
              }
          }
          #pragma unroll
          for (int w = 0; w < kWords; ++w)
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t sel = u ? 0x7362u : 0x5140u;
              uint32_t a0, a1, a2, a3;
              widen4(__byte_perm(v[0][w], v[1][w], sel), a0, a1);
              widen4(__byte_perm(v[2][w], v[3][w], sel), a2, a3);
              #pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma(acc[half * 8 + 2 * w + u][nt], a0, a1, a2, a3, p0[nt], p1[nt]);
            }
        }
        if constexpr (PARTIAL) {
          if (__any_sync(0xffffffffu, nans)) {
            // how many NaN values each row sees in each column: the product of
            // the NaN places with the places that the rows see
            uint32_t c0[NT], c1[NT];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float w[4];
              #pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = s[nt][k] == -INFINITY ? 0.f : 1.f;
              c0[nt] = transpose8x8(pack2<false>(w[0], w[1]));
              c1[nt] = transpose8x8(pack2<false>(w[2], w[3]));
            }
            #pragma unroll
            for (int im = 0; im < kMT; ++im) {
              // columns of fragment im held by this lane: words of the loads above
              const int half = im / 8, w = im % 8 / 2, u = im & 1;
              const uint32_t part = vt + half * T::kKeys * T::kPitch + mt * kFrag + 4 * w;
              uint32_t n[4];
              #pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t x;
                asm volatile("ld.shared.b32 %0, [%1];"
                             : "=r"(x) : "r"(part + v_at[i & 1] + (i >> 1) * (kFrag / 2)) : "memory");
                n[i] = nan_bytes(x) & 0x38383838u;     // 1.0 where the code is NaN
              }
              const uint32_t sel = u ? 0x7362u : 0x5140u;
              uint32_t a0, a1, a2, a3;
              widen4(__byte_perm(n[0], n[1], sel), a0, a1);
              widen4(__byte_perm(n[2], n[3], sel), a2, a3);
              #pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float hits[4] = {0.f, 0.f, 0.f, 0.f};
                mma(hits, a0, a1, a2, a3, c0[nt], c1[nt]);
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (hits[k] > 0.f) acc[im][nt][k] = __uint_as_float(0x7fffffffu);
              }
            }
          }
        }
      };
      if (k0 + T::kKeys <= at.full) {
        #pragma unroll
        for (int mt = 0; mt < T::kKeys / 16; ++mt) fragment(std::false_type{}, mt);
      } else {
        #pragma unroll 1
        for (int mt = 0; mt < T::kKeys / 16 && k0 + mt * 16 < at.lim; ++mt) fragment(std::true_type{}, mt);
      }
      __syncwarp();
      ++done;
      fetch();
    }

    // -------------------------------------------------------------- join the warps
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      #pragma unroll
      for (int c = 0; c < 2; ++c) {
        #pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
        if (g == 0) stat[warp * 8 * NT + nt * 8 + 2 * t + c] = make_float2(m[nt][c], l[nt][c]);
      }
    __syncthreads();
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      #pragma unroll
      for (int c = 0; c < 2; ++c) {
        float2 st[kWarps];
        float top = kNoMax;
        #pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          st[w] = stat[w * 8 * NT + nt * 8 + 2 * t + c];
          top = fmaxf(top, st[w].x);
        }
        float sum = 0.f;
        #pragma unroll
        for (int w = 0; w < kWarps; ++w) sum = fmaf(st[w].y, ex2_approx(st[w].x - top), sum);
        const float f = ex2_approx(m[nt][c] - top);
        m[nt][c] = top;
        l[nt][c] = sum;
        #pragma unroll
        for (int i = 0; i < kMT; ++i) {
          acc[i][nt][c] *= f;
          acc[i][nt][c + 2] *= f;
        }
      }
    float4* buf = reinterpret_cast<float4*>(smem + S::kBufOff) + lane;
    auto hand_over = [&](int place) {
      #pragma unroll
      for (int i = 0; i < kMT; ++i)
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          buf[((place * kMT + i) * NT + nt) * 32] =
              make_float4(acc[i][nt][0], acc[i][nt][1], acc[i][nt][2], acc[i][nt][3]);
    };
    auto take_over = [&](int place) {
      #pragma unroll
      for (int i = 0; i < kMT; ++i)
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float4 x = buf[((place * kMT + i) * NT + nt) * 32];
          acc[i][nt][0] += x.x;
          acc[i][nt][1] += x.y;
          acc[i][nt][2] += x.z;
          acc[i][nt][3] += x.w;
        }
    };
    if constexpr (S::kBufWarps == 2) {
      #pragma unroll
      for (int round = 2; round > 0; round >>= 1) {
        if (warp >= round && warp < 2 * round) hand_over(warp - round);
        __syncthreads();
        if (warp < round) take_over(warp);
        __syncthreads();
      }
    } else {
      #pragma unroll 1
      for (int from = 1; from < kWarps; ++from) {
        if (warp == from) hand_over(0);
        __syncthreads();
        if (warp == 0) take_over(0);
        __syncthreads();
      }
    }
    if (warp == 0) {
      const bool whole = at.s0 == 0 && at.s1 == at.steps;
      const long long slot = 2ll * blockIdx.x + (at.s0 > 0 ? 0 : 1);
      constexpr int kVec = D == 64 ? 8 : 16;       // consecutive columns of a lane
      #pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int rr = nt * 8 + 2 * t + c, r = row0 + rr;
          if (r < p.rows) {
            const int i = r / p.seq.G, head = at.h * p.seq.G + r % p.seq.G;
            const bool live = i < at.seq.n;
            const float sum = live ? l[nt][c] : 0.f;
            if (whole) {
              // a sum that is not above 0 is a row without keys, or NaN
              const float inv = sum == 0.f ? 0.f : kHeadInv / sum;
              #pragma unroll
              for (int half = 0; half < T::kHalves; ++half) {
                uint16_t* dst = p.o + b * p.os.b + head * p.os.h + i * p.os.n + 128 * half + kVec * g;
                uint32_t w[kVec / 2];
                #pragma unroll
                for (int k = 0; k < kVec / 2; ++k) {
                  const float x = acc[half * 8 + k][nt][c] * inv;
                  const float y = acc[half * 8 + k][nt][2 + c] * inv;
                  w[k] = sum == 0.f ? 0u : p.bf16 ? pack2<true>(x, y) : pack2<false>(x, y);
                }
                #pragma unroll
                for (int k = 0; k < kVec / 8; ++k)
                  reinterpret_cast<uint4*>(dst)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
              }
              if (g == 0)
                p.lse[(static_cast<long long>(b) * p.H + head) * p.seq.Nq + i] =
                    sum == 0.f ? -INFINITY : (m[nt][c] + kHead + log2f(sum)) * kLogE2;
            } else {
              #pragma unroll
              for (int half = 0; half < T::kHalves; ++half) {
                float* dst = p.part_o + (slot * 8 * NT + rr) * D + 128 * half + kVec * g;
                #pragma unroll
                for (int k = 0; k < kVec / 4; ++k)
                  reinterpret_cast<float4*>(dst)[k] =
                      make_float4(acc[half * 8 + 2 * k][nt][c], acc[half * 8 + 2 * k][nt][2 + c],
                                  acc[half * 8 + 2 * k + 1][nt][c], acc[half * 8 + 2 * k + 1][nt][2 + c]);
              }
              if (g == 0) p.part_ml[slot * 8 * NT + rr] = make_float2(m[nt][c], sum);
            }
          }
        }
    }
  }
  if (dead) {
    // the copies still in flight, before their shared memory goes away
    for (int i = done; i < fetched; ++i) drain_wait(bars + 8 * (i % kStages), (i / kStages) & 1);
    if (lane == 0 && *abort == 2) atomicOr(p.seq.err, kErrTimeout);
  }
}

// The rows that a unit of this kernel holds at most.
int most_rows(int d) { return d == 64 ? 32 : d == 128 ? 16 : 8; }

// Rows of a unit's tile: the fewest 8-row fragments that hold all G * Nq rows.
int row_fragments(int rows, int d) {
  int nt = 1;
  while (8 * nt < most_rows(d) && 8 * nt < rows) nt *= 2;
  return nt;
}

template <int D, int NT>
cudaError_t ctas_for(int sms, int* ctas) {
  static std::atomic<int> per_sm[64];   // by device, 0 = not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (per_sm[dev & 63] == 0) {
    auto kern = cache_fwd_kernel<D, NT>;
    constexpr int smem = Smem<D, NT>::kAlloc;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, smem);
    if (e != cudaSuccess) return e;
    per_sm[dev & 63] = std::max(1, std::min(n, 2));
  }
  *ctas = per_sm[dev & 63] * sms;
  return cudaSuccess;
}

template <int D, int NT>
cudaError_t launch(const Cache& cache, FwdCacheParams& p, int sms, cudaStream_t stream) {
  cudaError_t e = ctas_for<D, NT>(sms, &p.ctas);
  if (e != cudaSuccess) return e;
  constexpr int cols = D < 128 ? D : 128;
  const int box_rows = std::min(cache.page, Tile<D>::kKeys);
  CUtensorMap tk, tv;
  if ((e = make_tmap_u8_4d(&tk, cache.k, D, cache.page, cache.Hkv, cache.pages, cache.ks, cols,
                           box_rows)) != cudaSuccess)
    return e;
  if ((e = make_tmap_u8_4d(&tv, cache.v, D, cache.page, cache.Hkv, cache.pages, cache.vs, cols,
                           box_rows)) != cudaSuccess)
    return e;
  cache_fwd_kernel<D, NT><<<p.ctas, kThreads, Smem<D, NT>::kAlloc, stream>>>(tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_cache_merge<D, 8 * NT, Tile<D>::kStep, kOver, false>(p, stream);
}

}  // namespace

namespace {

// Whether the tcgen05 kernel takes the call: at d <= 128 from more rows than two
// units of this file's kernel hold, at d = 256 than one.  Measured (B = 8,
// 8 key/value heads, 8192 tokens), this kernel / the other: d = 64 at 64 rows
// 57 / 63 us, at 128 rows 91 / 66; d = 128 at 32 rows 64 / 74, at 64 rows
// 107 / 76; d = 256 at 8 rows 64 / 70, at 16 rows 103 / 71.
bool many_rows(long long rows, int d) { return rows > (d == 256 ? 1 : 2) * most_rows(d); }

// Rows of a unit, and CTAs at most.
void unit_shape(long long rows, int d, int sms, size_t* unit_rows, size_t* ctas) {
  const bool many = many_rows(rows, d);
  *unit_rows = many ? cache_prefill_rows(d)
                    : 8 * row_fragments(static_cast<int>(std::min(rows, 1ll << 20)), d);
  *ctas = many ? sms : 2ull * sms;
}

}  // namespace

// Two pieces of a unit's rows for each CTA, and a record.
size_t cache_fwd_workspace_bytes(int H, int Hkv, int Nq, int d, int sms) {
  size_t rows, ctas;
  unit_shape(1ll * H / Hkv * Nq, d, sms, &rows, &ctas);
  return 2 * ctas * rows * (d * sizeof(float) + sizeof(float2)) + ctas * sizeof(int4);
}

cudaError_t launch_cache_fwd(const Cache& cache, const CacheFwdCall& c, int sms,
                             cudaStream_t stream) {
  FwdCacheParams p = {};
  p.seq = {c.seq_lens, c.new_lens, c.B, c.H / cache.Hkv, c.Nq, c.causal,
           static_cast<long long>(cache.width) * cache.page, c.err};
  p.q = static_cast<const uint16_t*>(c.q);
  p.o = static_cast<uint16_t*>(c.o);
  p.lse = c.lse;
  p.qs = c.qs;
  p.os = c.os;
  p.k_scale = cache.k_scale;
  p.v_scale = cache.v_scale;
  p.table = cache.table;
  p.width = cache.width;
  p.pages = cache.pages;
  while ((1 << p.page_log2) < cache.page) ++p.page_log2;
  p.H = c.H;
  p.Hkv = cache.Hkv;
  p.rows = p.seq.G * c.Nq;
  p.bf16 = c.bf16;
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.k = cache.k;
  p.v = cache.v;
  p.ks = cache.ks;
  p.vs = cache.vs;
  size_t unit_rows, ctas;
  unit_shape(p.rows, cache.d, sms, &unit_rows, &ctas);
  p.row_tiles = (p.rows + unit_rows - 1) / unit_rows;
  p.part_o = static_cast<float*>(c.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2 * ctas * unit_rows * cache.d);
  p.joins = reinterpret_cast<int4*>(p.part_ml + 2 * ctas * unit_rows);
  if (many_rows(p.rows, cache.d)) return launch_cache_prefill(cache, p, sms, stream);
  const int nt = static_cast<int>(unit_rows / 8);
  switch (cache.d * 16 + nt) {
    case 64 * 16 + 1: return launch<64, 1>(cache, p, sms, stream);
    case 64 * 16 + 2: return launch<64, 2>(cache, p, sms, stream);
    case 64 * 16 + 4: return launch<64, 4>(cache, p, sms, stream);
    case 128 * 16 + 1: return launch<128, 1>(cache, p, sms, stream);
    case 128 * 16 + 2: return launch<128, 2>(cache, p, sms, stream);
    case 256 * 16 + 1: return launch<256, 1>(cache, p, sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
