// Norms of queries and keys for each head with the rotation in the same pass
// (fa_qk_norm_rope), and the backward pass (fa_qk_norm_rope_bwd).
//
// With h = x r, r = (mean x^2 + eps)^-1/2 and w the weight with its offset,
//     y = turn(h w);      u = turn_back(dy) w,   dx = r (u - h mean(u h)),
//     dw = sum over rows of turn_back(dy) h.
// A row is D / 16 threads next to one another, a slot (8 pairs, as in rope.cuh)
// each: its sums are shuffles among them, and every element is read once.
//
// What bounds it: memory (2 x 8192 tokens of 32 + 8 heads, d = 128, bf16:
// forward, 2 bytes read and 2 written an element, 57.3 us, 5.9 TB/s, 86% of what a
// copy reaches; backward, 4 read and 2 written, 86 us, as much), with the
// arithmetic close behind: two lanes of fp32 an instruction (without 62 and 107
// us).  Short calls: five tokens of four sequences forward 3.4 us, backward 6; 4099
// tokens of 32 heads, d = 64, three axes, backward 16.4 us, of which the start, the
// blocks' sums and the kernel that adds them up are a third.
#include <algorithm>

#include "rope.cuh"

namespace fa {
namespace {

constexpr int kFwdThreads = 128, kNormThreads = 256;

struct NormParams {
  // of q and of k
  const uint16_t* x[2];
  const uint16_t* dy[2];     // backward
  uint16_t* out[2];
  const void* weight[2];     // nullptr: ones
  Strides xs[2], dys[2], os[2];
  int heads[2];
  int weights_f32;
  float eps, offset;
  int N;
  long long items;           // B * N * slots
  int groups_q, heads_per;   // forward: q's head groups, heads of a thread
  long long tiles;           // backward: of 256 / slots tokens
  float* partial;            // [block][2][D] sums of the weights' gradients, nullptr: not wanted
  RopeArgs r;
};

// The columns of a slot: two chunks of eight, so that the chunks that the threads
// of a row read at a time lie next to one another (two chunks next to one another
// a thread are half sectors each: 4099 tokens of 32 heads, d = 64, interleaved,
// backward 20.6 us instead of 16.4; four times as many tokens 59 and 40).  Half-split: chunk b is the other half of
// chunk a's pairs, or both do not turn.  Interleaved: four pairs in each.
struct NormSlot {
  int col_a, col_b;
  int pair_a, pair_b;        // the first pair of a chunk (half-split: of both)
  bool turn_a, turn_b;
};
template <int D, bool PAIRS>
__device__ __forceinline__ NormSlot norm_slot(const RopeArgs& r, int slot) {
  NormSlot s;
  if constexpr (PAIRS) {
    s.col_a = 8 * slot;
    s.col_b = D / 2 + 8 * slot;
    s.pair_a = 4 * slot;
    s.pair_b = D / 4 + 4 * slot;
    s.turn_a = s.col_a < 2 * r.pairs;
    s.turn_b = s.col_b < 2 * r.pairs;
  } else {
    const int turning = r.pairs >> 3, still = slot - turning;
    s.turn_a = s.turn_b = still < 0;
    s.col_a = still < 0 ? 8 * slot : 2 * r.pairs + 8 * still;
    s.col_b = still < 0 ? r.pairs + 8 * slot : r.pairs + D / 2 + 8 * still;
    s.pair_a = s.pair_b = 8 * slot;
  }
  return s;
}

// A slot's 16 values: x1 and x2 of its 8 pairs, two pairs at a time for the packed
// arithmetic.  PAIRS: neighbours in memory (also where the slot does not turn),
// otherwise x1 is the first chunk and x2 the second.
struct Vals {
  f2 a[4], b[4];
};
template <bool BF16, bool PAIRS>
__device__ __forceinline__ Vals unpack_vals(const uint4& u, const uint4& v) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  Vals r;
  #pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 lo = unpack2<BF16>(w[PAIRS ? 2 * k : k]), hi = unpack2<BF16>(w[PAIRS ? 2 * k + 1 : 4 + k]);
    r.a[k] = PAIRS ? f2{lo.x, hi.x} : f2{lo.x, lo.y};
    r.b[k] = PAIRS ? f2{lo.y, hi.y} : f2{hi.x, hi.y};
  }
  return r;
}
template <bool BF16, bool PAIRS>
__device__ __forceinline__ void pack_vals(const Vals& r, uint4& u, uint4& v) {
  uint32_t w[8];
  #pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[PAIRS ? 2 * k : k] = PAIRS ? pack2<BF16>(r.a[k].x, r.b[k].x) : pack2<BF16>(r.a[k].x, r.a[k].y);
    w[PAIRS ? 2 * k + 1 : 4 + k] = PAIRS ? pack2<BF16>(r.a[k].y, r.b[k].y) : pack2<BF16>(r.b[k].x, r.b[k].y);
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  v = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void scale_vals(Vals& r, float x) {
  const f2 f = {x, x};
  #pragma unroll
  for (int k = 0; k < 4; ++k) {
    r.a[k] = fmul2(r.a[k], f);
    r.b[k] = fmul2(r.b[k], f);
  }
}

// The slot's weights with their offset.
template <bool BF16, bool PAIRS>
__device__ __forceinline__ Vals load_weights(const NormParams& p, const void* w, const NormSlot& at) {
  Vals r;
  if (w == nullptr) {
    #pragma unroll
    for (int k = 0; k < 4; ++k) r.a[k] = r.b[k] = f2{1.f, 1.f};
    return r;
  }
  if (p.weights_f32) {
    const float* f = static_cast<const float*>(w);
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* x = f + (PAIRS && k >= 2 ? at.col_b + 4 * k - 8 : at.col_a + (PAIRS ? 4 : 2) * k);
      const float* y = f + at.col_b + 2 * k;
      r.a[k] = PAIRS ? f2{x[0], x[2]} : f2{x[0], x[1]};
      r.b[k] = PAIRS ? f2{x[1], x[3]} : f2{y[0], y[1]};
    }
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(w);
    r = unpack_vals<BF16, PAIRS>(*reinterpret_cast<const uint4*>(h + at.col_a),
                                 *reinterpret_cast<const uint4*>(h + at.col_b));
  }
  const f2 off = {p.offset, p.offset};
  #pragma unroll
  for (int k = 0; k < 4; ++k) {
    r.a[k] = fadd2(r.a[k], off);
    r.b[k] = fadd2(r.b[k], off);
  }
  return r;
}

// cos and sin of the slot's pairs (1 and 0 of those that do not turn).
template <bool PAIRS>
__device__ __forceinline__ void load_angles(const RopeArgs& r, const NormSlot& at, int b, int n, int N,
                                            f2 (&c)[4], f2 (&s)[4]) {
  int pos[4];
  load_positions(r, b, n, N, n, pos);
  float x[8], y[8];
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = 1.f;
    y[j] = 0.f;
    if (!(PAIRS && j >= 4 ? at.turn_b : at.turn_a)) continue;
    const int pair = PAIRS && j >= 4 ? at.pair_b + j - 4 : at.pair_a + j, ax = r.axis[pair];
    const int t = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
    turn_cos_sin(static_cast<uint64_t>(static_cast<int64_t>(t)) * r.turn[pair], x[j], y[j]);
    y[j] = r.inverse ? -y[j] : y[j];
  }
  #pragma unroll
  for (int k = 0; k < 4; ++k) {
    c[k] = {x[2 * k], x[2 * k + 1]};
    s[k] = {y[2 * k], y[2 * k + 1]};
  }
}

template <int SLOTS>
__device__ __forceinline__ float row_sum(f2 x) {
  float y = x.x + x.y;
  #pragma unroll
  for (int m = SLOTS / 2; m > 0; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
  return y;
}
template <int SLOTS>
__device__ __forceinline__ float row_squares(const Vals& x) {
  f2 s = {0.f, 0.f};
  #pragma unroll
  for (int k = 0; k < 4; ++k) s = ffma2(x.a[k], x.a[k], ffma2(x.b[k], x.b[k], s));
  return row_sum<SLOTS>(s);
}

// Rows whose squares, or whose mean and eps together, leave fp32 are taken times
// this, and eps times its square.
constexpr float kDown = 8.470329472543003e-22f;   // 2^-70

// r of a row; where its mean square and eps leave fp32, the row and r are of x 2^-70
// (*down is that factor, 1 otherwise).
template <int SLOTS>
__device__ __forceinline__ float row_norm(float eps, Vals& x, float* down) {
  constexpr float kInf = 3.402823466e38f;
  float mean = fmaf(row_squares<SLOTS>(x), 1.f / (16 * SLOTS), eps);
  *down = 1.f;
  if (__any_sync(0xffffffffu, !(mean <= kInf))) {   // (whole rows: no lane of one alone)
    if (!(mean <= kInf)) {
      *down = kDown;
      scale_vals(x, kDown);
      eps *= kDown;
      eps *= kDown;
    }
    mean = fmaf(row_squares<SLOTS>(x), 1.f / (16 * SLOTS), eps);
  }
  return rsqrtf(mean);
}

// A thread has one slot of one token, and up to heads_per heads of q or of k, two
// of them on their way.  (Blocks of 128 threads, six an SM: 57.3 us for the long
// call above; 256 threads, three an SM 59.4, with four heads on their way 59.2,
// two an SM 66.7.)
template <bool BF16, int SLOTS, bool PAIRS>
__global__ void __launch_bounds__(kFwdThreads, 6) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kAhead = 2;
  const long long item = static_cast<long long>(blockIdx.x) * kFwdThreads + threadIdx.x;
  const bool on = item < p.items;       // (the same for a whole row)
  const int slot = static_cast<int>(item % SLOTS);
  const long long tok = on ? item / SLOTS : 0;
  const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok % p.N);
  const int which = static_cast<int>(blockIdx.y) >= p.groups_q;
  const int h0 = (blockIdx.y - (which ? p.groups_q : 0)) * p.heads_per;
  const int heads = min(p.heads[which], h0 + p.heads_per) - h0;
  const NormSlot at = norm_slot<16 * SLOTS, PAIRS>(p.r, slot);
  const long long in_h = p.xs[which].h, out_h = p.os[which].h;
  const uint16_t* src = p.x[which] + b * p.xs[which].b + n * p.xs[which].n + h0 * in_h;
  uint16_t* dst = p.out[which] + b * p.os[which].b + n * p.os[which].n + h0 * out_h;
  uint4 ra[kAhead], rb[kAhead];
  auto load = [&](int u, int h) {       // (the heads one after another)
    ra[u] = rb[u] = make_uint4(0u, 0u, 0u, 0u);
    if (on && h < heads) {
      ra[u] = *reinterpret_cast<const uint4*>(src + at.col_a);
      rb[u] = *reinterpret_cast<const uint4*>(src + at.col_b);
    }
    src += in_h;
  };
  #pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, u);
  // with h = r x: y1 = h1 w1 c - h2 w2 s, y2 = h2 w2 c + h1 w1 s (in this order, so that
  // no product leaves fp32 whose result does not)
  Vals w = load_weights<BF16, PAIRS>(p, p.weight[which], at), ws;
  if (at.turn_a) {       // (where chunk b turns, a does)
    f2 c[4], s[4];
    load_angles<PAIRS>(p.r, at, b, n, p.N, c, s);
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
      ws.a[k] = fmul2(w.a[k], s[k]);
      ws.b[k] = fmul2(w.b[k], f2{-s[k].x, -s[k].y});
      w.a[k] = fmul2(w.a[k], c[k]);
      w.b[k] = fmul2(w.b[k], c[k]);
    }
  }
  for (int h = 0; h < heads; h += kAhead) {
    #pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      Vals x = unpack_vals<BF16, PAIRS>(ra[u], rb[u]);
      load(u, h + u + kAhead);
      float down;
      const float r = row_norm<SLOTS>(p.eps, x, &down);
      scale_vals(x, r);
      #pragma unroll
      for (int k = 0; k < 4; ++k) {
        f2 y = fmul2(x.a[k], w.a[k]), z = fmul2(x.b[k], w.b[k]);
        if (PAIRS && k >= 2 ? at.turn_b : at.turn_a) {
          y = ffma2(x.b[k], ws.b[k], y);
          z = ffma2(x.a[k], ws.a[k], z);
        }
        x.a[k] = y;
        x.b[k] = z;
      }
      if (on && h + u < heads) {
        uint4 a, v;
        pack_vals<BF16, PAIRS>(x, a, v);
        *reinterpret_cast<uint4*>(dst + at.col_a) = a;
        *reinterpret_cast<uint4*>(dst + at.col_b) = v;
      }
      dst += out_h;
    }
  }
}

// 16 bytes to shared memory (zeros where `on` is false).
__device__ __forceinline__ void copy_async_16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The backward pass.  Units (a tile of 256 / SLOTS tokens, one head), q's first,
// tile by tile, are cut into equal shares, a block each; a thread keeps its
// slot's angles while the tile stays, and its sums of the weights' gradients
// until the block goes from q to k or ends: one partial sum a block, which
// norm_sum_kernel adds up in a fixed order.  A thread's next kRing - 1 units are
// on their way to shared memory of its own (no barrier between them; the long
// call above with kRing 2 / 3 / 4 / 6 94 / 85.5 / 92 / 95.5 us, through registers
// one unit ahead 104; three blocks an SM spill, 141, two 4 bytes a thread at most).
constexpr int kRing = 3;
template <bool BF16, int SLOTS, bool PAIRS>
__global__ void __launch_bounds__(kNormThreads, 2) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int kTokens = kNormThreads / SLOTS, D = 16 * SLOTS, kWarps = kNormThreads / 32;
  extern __shared__ __align__(16) uint4 ring[];      // [kRing][x, x, dy, dy][thread]
  __shared__ float red[kWarps][D];
  const int tid = threadIdx.x, slot = tid % SLOTS;
  const NormSlot at = norm_slot<D, PAIRS>(p.r, slot);
  const long long units = p.tiles * (p.heads[0] + p.heads[1]);
  const long long lo = units * blockIdx.x / gridDim.x, hi = units * (blockIdx.x + 1) / gridDim.x;
  const uint32_t mine = smem_u32(ring) + 16 * tid;
  grid_launch_dependents();
  #pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = p.heads[which];
    const long long first = which ? p.tiles * p.heads[0] : 0;
    const long long u0 = max(lo, first) - first, u1 = min(hi, first + p.tiles * H) - first;
    Vals dw;
    #pragma unroll
    for (int k = 0; k < 4; ++k) dw.a[k] = dw.b[k] = f2{0.f, 0.f};
    if (u0 < u1) {
      f2 c[4], s[4];
      // this thread's token of a tile; false where there is none (then the first)
      auto token = [&](int tile, int* b, int* n) -> bool {
        const long long tok = static_cast<long long>(tile) * kTokens + tid / SLOTS;
        const bool on = tok * SLOTS < p.items;
        *b = on ? static_cast<int>(tok / p.N) : 0;
        *n = on ? static_cast<int>(tok % p.N) : 0;
        return on;
      };
      // the unit that is fetched next, and the one that is worked on
      int f_tile = static_cast<int>(u0 / H), f_h = static_cast<int>(u0 % H), f_left = static_cast<int>(u1 - u0);
      int tile = f_tile, h = f_h, left = f_left;
      bool f_on = false;
      const uint16_t *x = nullptr, *dy = nullptr;
      auto enter = [&]() {
        int b, n;
        f_on = token(f_tile, &b, &n);
        x = p.x[which] + b * p.xs[which].b + n * p.xs[which].n + f_h * p.xs[which].h;
        dy = p.dy[which] + b * p.dys[which].b + n * p.dys[which].n + f_h * p.dys[which].h;
      };
      auto fetch = [&](int stage) {
        if (f_left > 0) {
          const uint32_t to = mine + stage * (4 * 16 * kNormThreads);
          copy_async_16(to, x + at.col_a, f_on);
          copy_async_16(to + 16 * kNormThreads, x + at.col_b, f_on);
          copy_async_16(to + 32 * kNormThreads, dy + at.col_a, f_on);
          copy_async_16(to + 48 * kNormThreads, dy + at.col_b, f_on);
          x += p.xs[which].h;
          dy += p.dys[which].h;
          if (++f_h == H) {
            f_h = 0;
            ++f_tile;
            if (f_left > 1) enter();
          }
          --f_left;
        }
        copy_async_commit();
      };
      enter();
      #pragma unroll
      for (int i = 0; i < kRing - 1; ++i) fetch(i);
      const Vals w = load_weights<BF16, PAIRS>(p, p.weight[which], at);
      bool fresh = true, on = false;       // the unit's tile is another than the last one's
      uint16_t* out = nullptr;
      for (int stage = 0; left > 0; --left, stage = (stage + 1) % kRing) {
        if (fresh) {
          int b, n;
          on = token(tile, &b, &n);
          out = p.out[which] + b * p.os[which].b + n * p.os[which].n + h * p.os[which].h;
          if (at.turn_a) load_angles<PAIRS>(p.r, at, b, n, p.N, c, s);
        }
        copy_async_wait<kRing - 2>();
        const uint4* in = ring + stage * (4 * kNormThreads) + tid;
        Vals v = unpack_vals<BF16, PAIRS>(in[0], in[kNormThreads]);
        Vals g = unpack_vals<BF16, PAIRS>(in[2 * kNormThreads], in[3 * kNormThreads]);
        fetch((stage + kRing - 1) % kRing);
        #pragma unroll
        for (int k = 0; k < 4; ++k) {          // (the angles are turned round: p.r.inverse)
          if (PAIRS && k >= 2 ? at.turn_b : at.turn_a) {
            const f2 a = g.a[k], o = g.b[k];
            g.a[k] = ffma2(a, c[k], fmul2(o, f2{-s[k].x, -s[k].y}));
            g.b[k] = ffma2(o, c[k], fmul2(a, s[k]));
          }
        }
        float down;
        const float r = row_norm<SLOTS>(p.eps, v, &down);
        scale_vals(v, r);                                // h
        f2 dot = {0.f, 0.f};
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
          dw.a[k] = ffma2(g.a[k], v.a[k], dw.a[k]);
          dw.b[k] = ffma2(g.b[k], v.b[k], dw.b[k]);
          g.a[k] = fmul2(g.a[k], w.a[k]);                // u
          g.b[k] = fmul2(g.b[k], w.b[k]);
          dot = ffma2(g.a[k], v.a[k], ffma2(g.b[k], v.b[k], dot));
        }
        const float mean = row_sum<SLOTS>(dot) * (-1.f / D), f = r * down;
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
          g.a[k] = ffma2(v.a[k], f2{mean, mean}, g.a[k]);
          g.b[k] = ffma2(v.b[k], f2{mean, mean}, g.b[k]);
        }
        scale_vals(g, f);
        if (on) {
          uint4 a, o;
          pack_vals<BF16, PAIRS>(g, a, o);
          *reinterpret_cast<uint4*>(out + at.col_a) = a;
          *reinterpret_cast<uint4*>(out + at.col_b) = o;
        }
        out += p.os[which].h;
        fresh = ++h == H;
        if (fresh) {
          h = 0;
          ++tile;
        }
      }
    }
    if (p.partial != nullptr && u0 >= u1) {
      if (tid < D) p.partial[(2ll * blockIdx.x + which) * D + tid] = 0.f;
    } else if (p.partial != nullptr) {
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        float a = j & 1 ? dw.a[j / 2].y : dw.a[j / 2].x, o = j & 1 ? dw.b[j / 2].y : dw.b[j / 2].x;
        #pragma unroll
        for (int m = SLOTS; m < 32; m <<= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, m);
          o += __shfl_xor_sync(0xffffffffu, o, m);
        }
        if ((tid & 31) < SLOTS) {
          const int col = PAIRS ? (j < 4 ? at.col_a + 2 * j : at.col_b + 2 * j - 8) : at.col_a + j;
          red[tid >> 5][col] = a;
          red[tid >> 5][PAIRS ? col + 1 : at.col_b + j] = o;
        }
      }
      __syncthreads();
      if (tid < D) {
        float sum = 0.f;
        #pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += red[i][tid];
        p.partial[(2ll * blockIdx.x + which) * D + tid] = sum;
      }
      __syncthreads();
    }
  }
}

// dw[column] = the blocks' partial sums: block (c, which) takes 32 columns, its
// warps every 32nd partial.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float* partial, float* dq, float* dk,
                                                        int blocks, int D) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, which = blockIdx.y;
  grid_dependency_wait();
  float sum = 0.f;
  for (int i = warp; i < blocks; i += 32) sum += partial[(2ll * i + which) * D + col];
  red[warp][lane] = sum;
  __syncthreads();
  sum = red[lane][warp];         // the warp's column of the 32, a partial a lane
  #pragma unroll
  for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  float* to = which ? dk : dq;
  if (lane == 0 && to != nullptr) to[blockIdx.x * 32 + warp] = sum;
}

void fill(const NormCall& c, const RopeArgs& r, NormParams* p) {
  *p = {};
  p->x[0] = static_cast<const uint16_t*>(c.q);
  p->x[1] = static_cast<const uint16_t*>(c.k);
  p->dy[0] = static_cast<const uint16_t*>(c.dq_out);
  p->dy[1] = static_cast<const uint16_t*>(c.dk_out);
  p->out[0] = static_cast<uint16_t*>(c.q_out);
  p->out[1] = static_cast<uint16_t*>(c.k_out);
  p->weight[0] = c.q_weight;
  p->weight[1] = c.k_weight;
  p->xs[0] = c.qs;
  p->xs[1] = c.ks;
  p->dys[0] = c.dqs;
  p->dys[1] = c.dks;
  p->os[0] = c.qos;
  p->os[1] = c.kos;
  p->heads[0] = c.H;
  p->heads[1] = c.Hkv;
  p->weights_f32 = c.weights_f32;
  p->eps = c.eps;
  p->offset = c.offset;
  p->N = c.N;
  p->items = 1ll * c.B * c.N * (c.d / 16);
  p->partial = c.partial;
  p->r = r;
}

// CALL(bf16, slots, pairs) for the call's types.
template <class Call>
cudaError_t by_type(const NormCall& c, const RopeArgs& r, Call call) {
  auto with_slots = [&](auto slots) -> cudaError_t {
    using T = std::true_type;
    using F = std::false_type;
    const bool pairs = r.interleaved != 0;
    if (c.bf16) return pairs ? call(T{}, slots, T{}) : call(T{}, slots, F{});
    return pairs ? call(F{}, slots, T{}) : call(F{}, slots, F{});
  };
  switch (c.d) {
    case 64: return with_slots(std::integral_constant<int, 4>{});
    case 128: return with_slots(std::integral_constant<int, 8>{});
    case 256: return with_slots(std::integral_constant<int, 16>{});
  }
  return cudaErrorInvalidValue;
}

long long bwd_tiles(int B, int N, int d) {
  const int tokens = kNormThreads / (d / 16);
  return (1ll * B * N + tokens - 1) / tokens;
}
int bwd_blocks(int B, int heads, int N, int d, int sms) {
  return static_cast<int>(std::min(2ll * sms, bwd_tiles(B, N, d) * heads));
}

}  // namespace

cudaError_t launch_qk_norm(const NormCall& c, const RopeArgs& r, int sms, cudaStream_t stream) {
  NormParams p;
  fill(c, r, &p);
  // heads of a thread: as in launch_rope
  const int heads = c.H + c.Hkv;
  const long long want = 1024ll * sms;
  const long long groups = std::max(1ll, std::min(std::min<long long>(heads, 4096), want / p.items));
  p.heads_per = std::min(16, static_cast<int>((heads + groups - 1) / groups));
  p.groups_q = (c.H + p.heads_per - 1) / p.heads_per;
  const dim3 grid(static_cast<unsigned>((p.items + kFwdThreads - 1) / kFwdThreads),
                  static_cast<unsigned>(p.groups_q + (c.Hkv + p.heads_per - 1) / p.heads_per), 1);
  return by_type(c, r, [&](auto bf16, auto slots, auto pairs) -> cudaError_t {
    norm_kernel<bf16.value, slots.value, pairs.value><<<grid, kFwdThreads, 0, stream>>>(p);
    return cudaGetLastError();
  });
}

size_t qk_norm_bwd_workspace_bytes(int B, int heads, int N, int d, int sms) {
  return sizeof(float) * 2 * d * bwd_blocks(B, heads, N, d, sms);
}

cudaError_t launch_qk_norm_bwd(const NormCall& c, const RopeArgs& r, int sms, cudaStream_t stream) {
  NormParams p;
  fill(c, r, &p);
  p.tiles = bwd_tiles(c.B, c.N, c.d);
  const int blocks = bwd_blocks(c.B, c.H + c.Hkv, c.N, c.d, sms);
  cudaError_t e = by_type(c, r, [&](auto bf16, auto slots, auto pairs) -> cudaError_t {
    auto kern = norm_bwd_kernel<bf16.value, slots.value, pairs.value>;
    constexpr int smem = kRing * 4 * 16 * kNormThreads;
    const cudaError_t e2 = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e2 != cudaSuccess) return e2;
    kern<<<blocks, kNormThreads, smem, stream>>>(p);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || c.partial == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c.d / 32), 2, 1);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_sum_kernel, static_cast<const float*>(c.partial), c.dq_weight,
                            c.dk_weight, blocks, c.d);
}

}  // namespace fa
