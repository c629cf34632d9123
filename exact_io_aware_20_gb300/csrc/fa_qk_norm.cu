// Norms of queries and keys for each head with the rotation in the same pass
// (fa_qk_norm_rope), and the backward pass (fa_qk_norm_rope_bwd).
//
// With h = x r, r = (mean x^2 + eps)^-1/2 and w the weight with its offset,
//     y = turn(h w);      u = turn_back(dy) w,   dx = r (u - h mean(u h)),
//     dw = sum over rows of turn_back(dy) h.
// A row is D / 16 threads next to one another, a slot (8 pairs, as in rope.cuh)
// each: its sums are shuffles among them, and every element is read once.
#include <algorithm>

#include "rope.cuh"

namespace fa {
namespace {

constexpr int kNormThreads = 256;

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

// A slot's 16 values x1[8], x2[8] as pairs (PAIRS: neighbours, also where the
// slot does not turn) and back.
template <bool BF16, bool PAIRS>
__device__ __forceinline__ void pack_slot(const float (&x1)[8], const float (&x2)[8], uint4& a, uint4& b) {
  uint32_t w[8];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = PAIRS ? pack2<BF16>(x1[i], x2[i]) : pack2<BF16>(x1[2 * i], x1[2 * i + 1]);
    w[4 + i] = PAIRS ? pack2<BF16>(x1[4 + i], x2[4 + i]) : pack2<BF16>(x2[2 * i], x2[2 * i + 1]);
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}

// The slot's weights with their offset, as x1 and x2 above.
template <bool BF16, bool PAIRS>
__device__ __forceinline__ void load_weights(const NormParams& p, const void* w, const Slot& at,
                                             float (&w1)[8], float (&w2)[8]) {
  if (w == nullptr) {
    #pragma unroll
    for (int j = 0; j < 8; ++j) w1[j] = w2[j] = 1.f;
    return;
  }
  if (p.weights_f32) {
    const float* f = static_cast<const float*>(w);
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
      w1[j] = PAIRS ? (j < 4 ? f[at.col_a + 2 * j] : f[at.col_b + 2 * j - 8]) : f[at.col_a + j];
      w2[j] = PAIRS ? (j < 4 ? f[at.col_a + 2 * j + 1] : f[at.col_b + 2 * j - 7]) : f[at.col_b + j];
    }
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(w);
    unpack_slot<BF16>(*reinterpret_cast<const uint4*>(h + at.col_a),
                      *reinterpret_cast<const uint4*>(h + at.col_b), PAIRS, w1, w2);
  }
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    w1[j] += p.offset;
    w2[j] += p.offset;
  }
}

template <int SLOTS>
__device__ __forceinline__ float row_sum(float x) {
  #pragma unroll
  for (int m = SLOTS / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// bf16 rows whose squares leave fp32 are taken times this (eps is nothing to
// them).
constexpr float kDown = 8.470329472543003e-22f;   // 2^-70

template <int SLOTS>
__device__ __forceinline__ float row_squares(const float (&x1)[8], const float (&x2)[8]) {
  float s[2] = {0.f, 0.f};
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[0] = fmaf(x1[j], x1[j], s[0]);
    s[1] = fmaf(x2[j], x2[j], s[1]);
  }
  return row_sum<SLOTS>(s[0] + s[1]);
}

// r of a row; where its squares leave fp32, the row and r are of x 2^-70 (*down
// is that factor, 1 otherwise).
template <int SLOTS>
__device__ __forceinline__ float row_norm(float eps, float (&x1)[8], float (&x2)[8], float* down) {
  float ss = row_squares<SLOTS>(x1, x2);
  *down = 1.f;
  if (__any_sync(0xffffffffu, !(ss < __uint_as_float(0x7f800000u)))) {   // (whole rows: no lane of one alone)
    if (!(ss < __uint_as_float(0x7f800000u))) {
      *down = kDown;
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        x1[j] *= kDown;
        x2[j] *= kDown;
      }
    }
    ss = row_squares<SLOTS>(x1, x2);
  }
  return rsqrtf(fmaf(ss, 1.f / (16 * SLOTS), *down == 1.f ? eps : 0.f));
}

// A thread has one slot of one token, and up to heads_per heads of q or of k.
template <bool BF16, int SLOTS, bool PAIRS>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kAhead = 2;
  const long long item = static_cast<long long>(blockIdx.x) * kNormThreads + threadIdx.x;
  const bool on = item < p.items;       // (the same for a whole row)
  const int slot = static_cast<int>(item % SLOTS);
  const long long tok = on ? item / SLOTS : 0;
  const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok % p.N);
  const int which = static_cast<int>(blockIdx.y) >= p.groups_q;
  const int h0 = (blockIdx.y - (which ? p.groups_q : 0)) * p.heads_per;
  const int h1 = min(p.heads[which], h0 + p.heads_per);
  const Slot at = slot_of(p.r, slot);
  const Strides xs = p.xs[which], os = p.os[which];
  const uint16_t* src = p.x[which] + b * xs.b + n * xs.n;
  uint16_t* dst = p.out[which] + b * os.b + n * os.n;
  uint4 ra[kAhead], rb[kAhead];
  auto load = [&](int u, int h) {
    ra[u] = rb[u] = make_uint4(0u, 0u, 0u, 0u);
    if (on && h < h1) {
      ra[u] = *reinterpret_cast<const uint4*>(src + h * xs.h + at.col_a);
      rb[u] = *reinterpret_cast<const uint4*>(src + h * xs.h + at.col_b);
    }
  };
  #pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, h0 + u);
  // y1 = r (x1 w1 c - x2 w2 s), y2 = r (x2 w2 c + x1 w1 s)
  float c1[8], c2[8], s1[8], s2[8];
  load_weights<BF16, PAIRS>(p, p.weight[which], at, c1, c2);
  if (at.turns) {
    int pos[4];
    float c[8], s[8];
    load_positions(p.r, b, n, p.N, n, pos);
    slot_cos_sin(p.r, slot, pos, c, s);
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
      s1[j] = c1[j] * s[j];
      s2[j] = c2[j] * s[j];
      c1[j] *= c[j];
      c2[j] *= c[j];
    }
  }
  for (int h = h0; h < h1; h += kAhead) {
    #pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float x1[8], x2[8], down;
      unpack_slot<BF16>(ra[u], rb[u], PAIRS, x1, x2);
      load(u, h + u + kAhead);
      const float r = row_norm<SLOTS>(p.eps, x1, x2, &down);
      if (at.turns) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y1 = fmaf(x1[j], c1[j], -(x2[j] * s2[j])), y2 = fmaf(x2[j], c2[j], x1[j] * s1[j]);
          x1[j] = y1 * r;
          x2[j] = y2 * r;
        }
      } else {
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          x1[j] *= c1[j] * r;
          x2[j] *= c2[j] * r;
        }
      }
      if (on && h + u < h1) {
        uint4 a, v;
        pack_slot<BF16, PAIRS>(x1, x2, a, v);
        *reinterpret_cast<uint4*>(dst + (h + u) * os.h + at.col_a) = a;
        *reinterpret_cast<uint4*>(dst + (h + u) * os.h + at.col_b) = v;
      }
    }
  }
}

// The backward pass.  Units (a tile of 256 / SLOTS tokens, one head), q's first,
// tile by tile, are cut into equal shares, a block each; a thread keeps its
// slot's angles while the tile stays, and its sums of the weights' gradients
// until the block goes from q to k or ends: one partial sum a block, which
// norm_sum_kernel adds up in a fixed order.
template <bool BF16, int SLOTS, bool PAIRS>
__global__ void __launch_bounds__(kNormThreads, 2) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int kTokens = kNormThreads / SLOTS, D = 16 * SLOTS, kWarps = kNormThreads / 32;
  __shared__ float red[kWarps][D];
  const int tid = threadIdx.x, slot = tid % SLOTS;
  const Slot at = slot_of(p.r, slot);
  const long long units = p.tiles * (p.heads[0] + p.heads[1]);
  const long long lo = units * blockIdx.x / gridDim.x, hi = units * (blockIdx.x + 1) / gridDim.x;
  grid_launch_dependents();
  #pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = p.heads[which];
    const long long first = which ? p.tiles * p.heads[0] : 0;
    const long long u0 = max(lo, first) - first, u1 = min(hi, first + p.tiles * H) - first;
    float d1[8], d2[8];
    #pragma unroll
    for (int j = 0; j < 8; ++j) d1[j] = d2[j] = 0.f;
    if (u0 < u1) {
      const Strides xs = p.xs[which], dys = p.dys[which], os = p.os[which];
      float w1[8], w2[8], c[8], s[8];
      load_weights<BF16, PAIRS>(p, p.weight[which], at, w1, w2);
      // the unit that is loaded next: its tile and head, and this thread's token
      long long tile = u0 / H;
      int h = static_cast<int>(u0 % H);
      bool on = false;
      const uint16_t *x = nullptr, *dy = nullptr;
      uint16_t* out = nullptr;
      int b = 0, n = 0;
      auto enter = [&]() {
        const long long tok = tile * kTokens + tid / SLOTS;
        on = tok * SLOTS < p.items;
        b = on ? static_cast<int>(tok / p.N) : 0;
        n = on ? static_cast<int>(tok % p.N) : 0;
        x = p.x[which] + b * xs.b + n * xs.n;
        dy = p.dy[which] + b * dys.b + n * dys.n;
        out = p.out[which] + b * os.b + n * os.n;
      };
      uint4 next[4];
      auto load = [&]() {
        #pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = make_uint4(0u, 0u, 0u, 0u);
        if (on) {
          next[0] = *reinterpret_cast<const uint4*>(x + h * xs.h + at.col_a);
          next[1] = *reinterpret_cast<const uint4*>(x + h * xs.h + at.col_b);
          next[2] = *reinterpret_cast<const uint4*>(dy + h * dys.h + at.col_a);
          next[3] = *reinterpret_cast<const uint4*>(dy + h * dys.h + at.col_b);
        }
      };
      enter();
      load();
      bool fresh = true;       // the unit's tile is another than the last one's
      for (long long u = u0; u < u1; ++u) {
        float x1[8], x2[8], g1[8], g2[8];
        unpack_slot<BF16>(next[0], next[1], PAIRS, x1, x2);
        unpack_slot<BF16>(next[2], next[3], PAIRS, g1, g2);
        uint16_t* dst = out + h * os.h;
        const bool live = on;
        if (fresh && at.turns) {
          int pos[4];
          load_positions(p.r, b, n, p.N, n, pos);
          slot_cos_sin(p.r, slot, pos, c, s);
        }
        fresh = ++h == H;
        if (fresh) {
          h = 0;
          ++tile;
          if (u + 1 < u1) enter();
        }
        if (u + 1 < u1) load();
        if (at.turns) turn_pairs(g1, g2, c, s);      // (the angles are turned round: p.r.inverse)
        float down;
        const float r = row_norm<SLOTS>(p.eps, x1, x2, &down);
        float dot[2] = {0.f, 0.f};
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          x1[j] *= r;                                // h
          x2[j] *= r;
          d1[j] = fmaf(g1[j], x1[j], d1[j]);
          d2[j] = fmaf(g2[j], x2[j], d2[j]);
          g1[j] *= w1[j];                            // u
          g2[j] *= w2[j];
          dot[0] = fmaf(g1[j], x1[j], dot[0]);
          dot[1] = fmaf(g2[j], x2[j], dot[1]);
        }
        const float mean = row_sum<SLOTS>(dot[0] + dot[1]) * (1.f / D), f = r * down;
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          g1[j] = fmaf(-x1[j], mean, g1[j]) * f;
          g2[j] = fmaf(-x2[j], mean, g2[j]) * f;
        }
        if (live) {
          uint4 a, v;
          pack_slot<BF16, PAIRS>(g1, g2, a, v);
          *reinterpret_cast<uint4*>(dst + at.col_a) = a;
          *reinterpret_cast<uint4*>(dst + at.col_b) = v;
        }
      }
    }
    if (p.partial != nullptr) {
      #pragma unroll
      for (int j = 0; j < 8; ++j)
        #pragma unroll
        for (int m = SLOTS; m < 32; m <<= 1) {
          d1[j] += __shfl_xor_sync(0xffffffffu, d1[j], m);
          d2[j] += __shfl_xor_sync(0xffffffffu, d2[j], m);
        }
      if ((tid & 31) < SLOTS) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int a = PAIRS ? (j < 4 ? at.col_a + 2 * j : at.col_b + 2 * j - 8) : at.col_a + j;
          red[tid >> 5][a] = d1[j];
          red[tid >> 5][PAIRS ? a + 1 : at.col_b + j] = d2[j];
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
  const int heads = c.H + c.Hkv;
  const long long want = 1024ll * sms;
  const long long groups = std::max(1ll, std::min(std::min<long long>(heads, 4096), want / p.items));
  p.heads_per = std::min(16, static_cast<int>((heads + groups - 1) / groups));
  p.groups_q = (c.H + p.heads_per - 1) / p.heads_per;
  const dim3 grid(static_cast<unsigned>((p.items + kNormThreads - 1) / kNormThreads),
                  static_cast<unsigned>(p.groups_q + (c.Hkv + p.heads_per - 1) / p.heads_per), 1);
  return by_type(c, r, [&](auto bf16, auto slots, auto pairs) -> cudaError_t {
    norm_kernel<bf16.value, slots.value, pairs.value><<<grid, kNormThreads, 0, stream>>>(p);
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
    norm_bwd_kernel<bf16.value, slots.value, pairs.value><<<blocks, kNormThreads, 0, stream>>>(p);
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
