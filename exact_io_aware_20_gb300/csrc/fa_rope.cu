// Rotary positions of q and k (fa_rope): forward, and with the angles turned
// round the backward pass.
//
// What bounds it: memory, 2 bytes read and 2 written an element (2 x 8192
// tokens of 40 heads, d = 128: 55 us, 6.1 TB/s, 91% of what a copy reaches; the
// backward pass over three axes of 4099 tokens of 32 heads, d = 64, 8.2 us; five
// tokens of four sequences 2.5 us).  A thread keeps the cos and sin of one slot
// (8 pairs) of one token and walks over heads, so the angles, which every head
// shares, are worked out once for up to 16 of them; a warp covers whole
// 128-byte lines of consecutive tokens.
#include <algorithm>

#include "rope.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  Strides qs, ks, qos, kos;
  int H, heads;        // q's heads, and q's and k's together
  int heads_per;       // heads of a thread
  int N, slots;
  long long items;     // B * N * slots
  RopeArgs r;
};

template <bool BF16>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  const long long item = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  if (item >= p.items) return;
  const int slot = static_cast<int>(item % p.slots);
  const long long tok = item / p.slots;
  const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok % p.N);
  int pos[4];
  load_positions(p.r, b, n, p.N, n, pos);
  const RopeRows w = {p.q + b * p.qs.b + n * p.qs.n,
                      p.k + b * p.ks.b + n * p.ks.n,
                      p.q_out + b * p.qos.b + n * p.qos.n,
                      p.k_out + b * p.kos.b + n * p.kos.n,
                      p.qs.h, p.ks.h, p.qos.h, p.kos.h, p.H};
  const int h0 = blockIdx.y * p.heads_per;
  rope_heads<BF16, 2>(p.r, w, slot, h0, min(p.heads, h0 + p.heads_per), pos, true);
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, const RopeArgs& r, int sms, cudaStream_t stream) {
  RopeParams p = {};
  p.q = static_cast<const uint16_t*>(c.q);
  p.k = static_cast<const uint16_t*>(c.k);
  p.q_out = static_cast<uint16_t*>(c.q_out);
  p.k_out = static_cast<uint16_t*>(c.k_out);
  p.qs = c.qs;
  p.ks = c.ks;
  p.qos = c.qos;
  p.kos = c.kos;
  p.H = c.H;
  p.heads = c.H + (c.k != nullptr ? c.Hkv : 0);
  p.N = c.N;
  p.slots = c.d / 16;
  p.items = static_cast<long long>(c.B) * c.N * p.slots;
  p.r = r;
  // Heads of a thread: as many as leave about 1024 threads for each SM, so that
  // a long call works its angles out once and a short one is spread over the
  // chip; 16 at most, so that a long call's blocks fill more than one wave of
  // them.  Threads an SM 512 / 1024 / 1536 / 2048: the backward pass above 8.2 /
  // 8.3 / 9.4 / 10.1 us, 512 tokens of 32 + 8 heads 5.0 / 5.8 / 7.9 / 7.9, 4096 of
  // them 19.6 / 17.1 / 17.9 / 18.8; 2 x 8192 of them with 6 / 10 / 20 / 40 heads a
  // thread 56.2 / 55.2 / 54.9 / 60.8.
  const long long want = 1024ll * sms;
  const long long groups =
      std::max(1ll, std::min(std::min<long long>(p.heads, 4096), want / p.items));
  p.heads_per = std::min(16, static_cast<int>((p.heads + groups - 1) / groups));
  const long long blocks = (p.items + kRopeThreads - 1) / kRopeThreads;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((p.heads + p.heads_per - 1) / p.heads_per), 1);
  if (c.bf16) rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(p);
  else rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
