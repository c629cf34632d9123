// C-ABI layer of the rotary positions and the paged 8-bit cache: argument
// validation and dispatch.  See include/fa.h for the contract.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_internal.h"

namespace fa {
namespace {

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// Sizes shared by the entry points (heads: the largest head count).
int check_sizes(int B, int heads, int N, int d, int dtype) {
  if (B < 1 || heads < 1 || N < 1 || B > 65535 || heads > 65535) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (1ll * B * heads > INT_MAX || 1ll * B * heads * N > INT_MAX || 1ll * N * d > INT_MAX)
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// x turns, |x| <= 1/2, in whole 2^-64 turns modulo one turn.
unsigned long long turns_64(double x) {
  const double u = std::rint(std::ldexp(std::fabs(x), 64));     // <= 2^63
  return x < 0.0 ? 0ull - static_cast<unsigned long long>(u) : static_cast<unsigned long long>(u);
}

// The fraction of a turn that one position adds at `freq` radians (whole turns
// add nothing), in 2^-64 turns.  freq / 2 pi is formed as two doubles, the
// product with 1 / 2 pi and what its rounding and that of 1 / 2 pi left, and
// each gives its own whole turns up exactly: good to 2^-64 turns for |freq| <=
// 2^40, |freq| 2^-105 beyond.  (A product in one double is off by 2^-54 of
// freq, which a position of 2^31 makes 2^-15 radians of at freq = 100.)
unsigned long long turn_of(double freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;   // 1 / 2 pi
  const double turns = freq * kHi;
  const double rest = std::fma(freq, kHi, -turns) + freq * kLo;
  return turns_64(turns - std::rint(turns)) + turns_64(rest - std::rint(rest));
}

int rope_args(const fa_rope_spec* spec, const int* positions, int pos_batch, int B, int d,
              RopeArgs* r) {
  *r = RopeArgs{};
  if (positions != nullptr && (!aligned(positions, 4) || (pos_batch != 1 && pos_batch != B)))
    return FA_ERR_INVALID_ARG;
  if (spec == nullptr) return FA_OK;
  if (spec->axes < 1 || spec->axes > FA_ROPE_MAX_AXES || spec->pairs < 8 || spec->pairs % 8 != 0 ||
      2 * spec->pairs > d || (spec->interleaved != 0 && spec->interleaved != 1))
    return FA_ERR_INVALID_ARG;
  r->axes = spec->axes;
  r->pairs = spec->pairs;
  r->interleaved = spec->interleaved;
  r->positions = positions;
  r->pos_batch = pos_batch;
  for (int i = 0; i < spec->pairs; ++i) {
    if (!std::isfinite(spec->freq[i]) || spec->axis[i] >= spec->axes) return FA_ERR_INVALID_ARG;
    r->turn[i] = turn_of(spec->freq[i]);
    r->axis[i] = spec->axis[i];
  }
  return FA_OK;
}

// Byte strides of a cache array (all zero: contiguous).
bool cache_strides(const fa_strides& s, const fa_cache& c, Strides* out) {
  if (s.batch == 0 && s.head == 0 && s.row == 0) {
    *out = contiguous_strides(c.Hkv, c.page_size, c.d);
    return true;
  }
  const long long v[3] = {s.batch, s.head, s.row};
  for (long long x : v)
    if (x < 16 || x % 16 != 0 || x >= (1ll << 39)) return false;
  *out = {s.batch, s.head, s.row};
  return true;
}

int cache_args(const fa_cache* c, Cache* out) {
  if (c == nullptr) return FA_ERR_INVALID_ARG;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table) return FA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || !aligned(c->block_table, 4))
    return FA_ERR_INVALID_ARG;
  if (c->pages < 1 || c->table_width < 1 || c->Hkv < 1 || c->Hkv > 65535) return FA_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 &&
      c->page_size != 256)
    return FA_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED;
  if (1ll * c->table_width * c->page_size > INT_MAX - 65536) return FA_ERR_INVALID_ARG;
  *out = {static_cast<unsigned char*>(c->k), static_cast<unsigned char*>(c->v), c->k_scale,
          c->v_scale, c->block_table, c->pages, c->page_size, c->table_width, c->Hkv, c->d};
  if (!cache_strides(c->k_strides, *c, &out->ks) || !cache_strides(c->v_strides, *c, &out->vs))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// SMs of the current device, cached per device; 0 when it cannot be asked.
int device_sms() {
  static std::atomic<int> sms[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  if (sms[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    sms[dev] = n;
  }
  return sms[dev];
}

}  // namespace
}  // namespace fa

extern "C" int fa_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int H,
                       int Hkv, int N, int d, int dtype, const fa_rope_spec* spec,
                       const int* positions, int pos_batch, int inverse,
                       const fa_strides* strides, fa_stream_t stream) {
  int st = fa::check_sizes(B, H, N, d, dtype);
  if (st != FA_OK) return st;
  if (k != nullptr && (st = fa::check_sizes(B, Hkv, N, d, dtype)) != FA_OK) return st;
  if (!q || !q_out || (k == nullptr) != (k_out == nullptr) || spec == nullptr ||
      (inverse != 0 && inverse != 1))
    return FA_ERR_INVALID_ARG;
  if (!fa::aligned(q, 16) || !fa::aligned(q_out, 16) || !fa::aligned(k, 16) ||
      !fa::aligned(k_out, 16))
    return FA_ERR_INVALID_ARG;
  fa::RopeArgs r;
  if ((st = fa::rope_args(spec, positions, pos_batch, B, d, &r)) != FA_OK) return st;
  r.inverse = inverse;
  fa::RopeCall c = {q, k, q_out, k_out};
  if (strides != nullptr) {
    fa::Strides s[4];
    if (!fa::valid_strides(strides, 1, s) || !fa::valid_strides(strides + 2, 1, s + 2))
      return FA_ERR_INVALID_ARG;
    if (k != nullptr &&
        (!fa::valid_strides(strides + 1, 1, s + 1) || !fa::valid_strides(strides + 3, 1, s + 3)))
      return FA_ERR_INVALID_ARG;
    c.qs = s[0];
    c.ks = s[1];
    c.qos = s[2];
    c.kos = s[3];
  } else {
    c.qs = c.qos = fa::contiguous_strides(H, N, d);
    c.ks = c.kos = fa::contiguous_strides(Hkv, N, d);
  }
  c.B = B;
  c.H = H;
  c.Hkv = Hkv;
  c.N = N;
  c.d = d;
  c.bf16 = dtype == FA_BF16;
  unsigned int* err = nullptr;
  if ((st = fa::check_device(&err)) != FA_OK) return st;
  cudaError_t e = fa::launch_rope(c, r, std::max(1, fa::device_sms()), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fa::cuda_fail(e, "fa_rope launch");
}

extern "C" int fa_cache_append(const fa_cache* cache, const void* q, const void* k, const void* v,
                               void* q_out, int B, int H, int N, int dtype, const int* seq_lens,
                               const int* new_lens, const fa_rope_spec* spec,
                               const int* positions, int pos_batch, const fa_strides* strides,
                               fa_stream_t stream) {
  fa::Cache ca;
  int st = fa::cache_args(cache, &ca);
  if (st != FA_OK) return st;
  if ((st = fa::check_sizes(B, ca.Hkv, N, ca.d, dtype)) != FA_OK) return st;
  if (q != nullptr && (st = fa::check_sizes(B, H, N, ca.d, dtype)) != FA_OK) return st;
  if (!k || !v || !seq_lens || (q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (!fa::aligned(q, 16) || !fa::aligned(q_out, 16) || !fa::aligned(k, 16) ||
      !fa::aligned(v, 16) || !fa::aligned(seq_lens, 4) || !fa::aligned(new_lens, 4))
    return FA_ERR_INVALID_ARG;
  fa::RopeArgs r;
  if ((st = fa::rope_args(spec, positions, pos_batch, B, ca.d, &r)) != FA_OK) return st;
  fa::AppendCall c = {q, k, v, q_out};
  if (strides != nullptr) {
    fa::Strides s[4];
    if (!fa::valid_strides(strides + 1, 2, s + 1)) return FA_ERR_INVALID_ARG;
    if (q != nullptr &&
        (!fa::valid_strides(strides, 1, s) || !fa::valid_strides(strides + 3, 1, s + 3)))
      return FA_ERR_INVALID_ARG;
    c.qs = s[0];
    c.ks = s[1];
    c.vs = s[2];
    c.qos = s[3];
  } else {
    c.qs = c.qos = fa::contiguous_strides(H, N, ca.d);
    c.ks = c.vs = fa::contiguous_strides(ca.Hkv, N, ca.d);
  }
  c.B = B;
  c.H = q != nullptr ? H : 0;
  c.N = N;
  c.bf16 = dtype == FA_BF16;
  c.seq_lens = seq_lens;
  c.new_lens = new_lens;
  if ((st = fa::check_device(&c.err)) != FA_OK) return st;
  cudaError_t e = fa::launch_cache_append(ca, c, r, std::max(1, fa::device_sms()),
                                          reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fa::cuda_fail(e, "fa_cache_append launch");
}

extern "C" size_t fa_fwd_cache_workspace_size(int B, int H, int Hkv, int Nq, int d) {
  if (Hkv < 1 || fa::check_sizes(B, H, Nq, d, FA_BF16) != FA_OK || H % Hkv != 0) return 0;
  return fa::cache_fwd_workspace_bytes(H, Hkv, Nq, d, fa::device_sms());
}

extern "C" size_t fa_fwd_cache_tree_workspace_size(int B, int H, int Hkv, int Nq, int d) {
  if (Hkv < 1 || fa::check_sizes(B, H, Nq, d, FA_BF16) != FA_OK || H % Hkv != 0) return 0;
  return fa::cache_tree_workspace_bytes(H, Hkv, Nq, d, fa::device_sms());
}

namespace fa {
namespace {

// fa_fwd_cache and, with a mask, fa_fwd_cache_tree.
int attend(const void* q, const fa_cache* cache, void* o, float* lse, int B, int H, int Nq,
           int causal, float scale, int dtype, const int* seq_lens, const int* new_lens,
           const unsigned int* tree, int tree_batch, const fa_strides* strides, void* workspace,
           size_t workspace_bytes, fa_stream_t stream) {
  Cache ca;
  int st = cache_args(cache, &ca);
  if (st != FA_OK) return st;
  if ((st = check_sizes(B, H, Nq, ca.d, dtype)) != FA_OK) return st;
  if (H % ca.Hkv != 0 || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARG;
  if (!q || !o || !lse || !seq_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(seq_lens, 4) ||
      !aligned(new_lens, 4))
    return FA_ERR_INVALID_ARG;
  CacheFwdCall c = {q, o, lse};
  if (strides != nullptr) {
    Strides s[2];
    if (!valid_strides(strides, 2, s)) return FA_ERR_INVALID_ARG;
    c.qs = s[0];
    c.os = s[1];
  } else {
    c.qs = c.os = contiguous_strides(H, Nq, ca.d);
  }
  if (!workspace || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  if ((st = check_device(&c.err)) != FA_OK) return st;
  const int sms = device_sms();
  if (workspace_bytes < (tree != nullptr ? cache_tree_workspace_bytes(H, ca.Hkv, Nq, ca.d, sms)
                                         : cache_fwd_workspace_bytes(H, ca.Hkv, Nq, ca.d, sms)))
    return FA_ERR_WORKSPACE;
  c.B = B;
  c.H = H;
  c.Nq = Nq;
  c.causal = causal;
  c.bf16 = dtype == FA_BF16;
  c.scale = scale;
  c.seq_lens = seq_lens;
  c.new_lens = new_lens;
  c.workspace = workspace;
  c.tree = tree;
  c.tree_batch = tree_batch;
  cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = tree != nullptr ? launch_cache_fwd_tree(ca, c, sms, on) : launch_cache_fwd(ca, c, sms, on);
  return e == cudaSuccess ? FA_OK
                          : cuda_fail(e, tree != nullptr ? "fa_fwd_cache_tree launch" : "fa_fwd_cache launch");
}

// Strides of n views, those of `skip` (a bit each) not looked at.
bool views(const fa_strides* strides, int n, unsigned skip, Strides* out) {
  for (int i = 0; i < n; ++i)
    if (!(skip >> i & 1) && !valid_strides(strides + i, 1, out + i)) return false;
  return true;
}

// What the norms' two directions have in common.
int norm_args(NormCall* c, RopeArgs* r, int weights_f32, float eps, float offset, int B, int H,
              int Hkv, int N, int d, int dtype, const fa_rope_spec* spec, const int* positions,
              int pos_batch) {
  int st = check_sizes(B, H, N, d, dtype);
  if (st != FA_OK) return st;
  if (c->k != nullptr && (st = check_sizes(B, Hkv, N, d, dtype)) != FA_OK) return st;
  if (!c->q || !c->q_out || (c->k == nullptr) != (c->k_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (c->k == nullptr && c->k_weight != nullptr) return FA_ERR_INVALID_ARG;
  if (!aligned(c->q, 16) || !aligned(c->k, 16) || !aligned(c->q_out, 16) || !aligned(c->k_out, 16) ||
      !aligned(c->q_weight, 16) || !aligned(c->k_weight, 16))
    return FA_ERR_INVALID_ARG;
  if ((weights_f32 != 0 && weights_f32 != 1) || !std::isfinite(eps) || eps < std::ldexp(1.f, -100) ||
      !std::isfinite(offset))
    return FA_ERR_INVALID_ARG;
  // (without a rotation the positions are not looked at)
  if ((st = rope_args(spec, spec != nullptr ? positions : nullptr, pos_batch, B, d, r)) != FA_OK) return st;
  c->weights_f32 = weights_f32;
  c->eps = eps;
  c->offset = offset;
  c->B = B;
  c->H = H;
  c->Hkv = c->k != nullptr ? Hkv : 0;
  c->N = N;
  c->d = d;
  c->bf16 = dtype == FA_BF16;
  return FA_OK;
}

// Whether n values at a and m at b, which may be missing, have none in common.
bool apart(const int* a, long long n, const int* b, long long m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return b == nullptr || x + n * sizeof(int) <= y || y + m * sizeof(int) <= x;
}

// The lengths and the cache of fa_cache_keep and fa_cache_fork.
int rows_args(const fa_cache* cache, int B, const int* seq_lens, int* out_lens, Cache* ca) {
  const int st = cache_args(cache, ca);
  if (st != FA_OK) return st;
  if (B < 1 || B > 65535 || 1ll * B * ca->width > INT_MAX || !seq_lens || !out_lens ||
      !aligned(seq_lens, 4) || !aligned(out_lens, 4))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" int fa_fwd_cache(const void* q, const fa_cache* cache, void* o, float* lse, int B,
                            int H, int Nq, int causal, float scale, int dtype,
                            const int* seq_lens, const int* new_lens, const fa_strides* strides,
                            void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  return fa::attend(q, cache, o, lse, B, H, Nq, causal, scale, dtype, seq_lens, new_lens, nullptr, 1,
                    strides, workspace, workspace_bytes, stream);
}

extern "C" int fa_fwd_cache_tree(const void* q, const fa_cache* cache, void* o, float* lse, int B,
                                 int H, int Nq, float scale, int dtype, const int* seq_lens,
                                 const int* new_lens, const unsigned int* tree_mask,
                                 int mask_batch, const fa_strides* strides, void* workspace,
                                 size_t workspace_bytes, fa_stream_t stream) {
  if (!tree_mask || !fa::aligned(tree_mask, 4) || (mask_batch != 1 && mask_batch != B))
    return FA_ERR_INVALID_ARG;
  return fa::attend(q, cache, o, lse, B, H, Nq, 0, scale, dtype, seq_lens, new_lens, tree_mask,
                    mask_batch, strides, workspace, workspace_bytes, stream);
}

extern "C" int fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                               const void* q_weight, const void* k_weight, int weights_f32,
                               float eps, float offset, int B, int H, int Hkv, int N, int d,
                               int dtype, const fa_rope_spec* spec, const int* positions,
                               int pos_batch, const fa_strides* strides, fa_stream_t stream) {
  fa::NormCall c = {};
  c.q = q;
  c.k = k;
  c.q_out = q_out;
  c.k_out = k_out;
  c.q_weight = q_weight;
  c.k_weight = k_weight;
  fa::RopeArgs r;
  int st = fa::norm_args(&c, &r, weights_f32, eps, offset, B, H, Hkv, N, d, dtype, spec, positions,
                         pos_batch);
  if (st != FA_OK) return st;
  if (strides != nullptr) {
    fa::Strides s[4];
    if (!fa::views(strides, 4, k == nullptr ? 0xau : 0u, s)) return FA_ERR_INVALID_ARG;
    c.qs = s[0];
    c.ks = s[1];
    c.qos = s[2];
    c.kos = s[3];
  } else {
    c.qs = c.qos = fa::contiguous_strides(H, N, d);
    c.ks = c.kos = fa::contiguous_strides(c.Hkv, N, d);
  }
  unsigned int* err = nullptr;
  if ((st = fa::check_device(&err)) != FA_OK) return st;
  cudaError_t e = fa::launch_qk_norm(c, r, std::max(1, fa::device_sms()), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fa::cuda_fail(e, "fa_qk_norm_rope launch");
}

extern "C" size_t fa_qk_norm_rope_bwd_workspace_size(int B, int H, int Hkv, int N, int d) {
  if (fa::check_sizes(B, H, N, d, FA_BF16) != FA_OK) return 0;
  if (Hkv != 0 && fa::check_sizes(B, Hkv, N, d, FA_BF16) != FA_OK) return 0;
  return fa::qk_norm_bwd_workspace_bytes(B, H + Hkv, N, d, std::max(1, fa::device_sms()));
}

extern "C" int fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q,
                                   const void* k, void* dq, void* dk, const void* q_weight,
                                   const void* k_weight, int weights_f32, float eps, float offset,
                                   float* dq_weight, float* dk_weight, int B, int H, int Hkv,
                                   int N, int d, int dtype, const fa_rope_spec* spec,
                                   const int* positions, int pos_batch, const fa_strides* strides,
                                   void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  fa::NormCall c = {};
  c.q = q;
  c.k = k;
  c.dq_out = dq_out;
  c.dk_out = dk_out;
  c.q_out = dq;
  c.k_out = dk;
  c.q_weight = q_weight;
  c.k_weight = k_weight;
  c.dq_weight = dq_weight;
  c.dk_weight = dk_weight;
  fa::RopeArgs r;
  int st = fa::norm_args(&c, &r, weights_f32, eps, offset, B, H, Hkv, N, d, dtype, spec, positions,
                         pos_batch);
  if (st != FA_OK) return st;
  if (!dq_out || (k == nullptr) != (dk_out == nullptr) || (!q_weight && dq_weight) ||
      (!k_weight && dk_weight))
    return FA_ERR_INVALID_ARG;
  if (!fa::aligned(dq_out, 16) || !fa::aligned(dk_out, 16) || !fa::aligned(dq_weight, 4) ||
      !fa::aligned(dk_weight, 4))
    return FA_ERR_INVALID_ARG;
  r.inverse = 1;
  if (strides != nullptr) {
    fa::Strides s[6];
    if (!fa::views(strides, 6, k == nullptr ? 0x2au : 0u, s)) return FA_ERR_INVALID_ARG;
    c.dqs = s[0];
    c.dks = s[1];
    c.qs = s[2];
    c.ks = s[3];
    c.qos = s[4];
    c.kos = s[5];
  } else {
    c.qs = c.qos = c.dqs = fa::contiguous_strides(H, N, d);
    c.ks = c.kos = c.dks = fa::contiguous_strides(c.Hkv, N, d);
  }
  const bool sums = dq_weight != nullptr || dk_weight != nullptr;
  if (sums && (!workspace || !fa::aligned(workspace, 256))) return FA_ERR_WORKSPACE;
  unsigned int* err = nullptr;
  if ((st = fa::check_device(&err)) != FA_OK) return st;
  const int sms = std::max(1, fa::device_sms());
  if (sums && workspace_bytes < fa::qk_norm_bwd_workspace_bytes(B, H + c.Hkv, N, d, sms))
    return FA_ERR_WORKSPACE;
  c.partial = sums ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e = fa::launch_qk_norm_bwd(c, r, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fa::cuda_fail(e, "fa_qk_norm_rope_bwd launch");
}

extern "C" int fa_cache_keep(const fa_cache* cache, int B, int N, int K, const int* seq_lens,
                             const int* new_lens, const int* keep, const int* keep_lens,
                             int* out_lens, fa_stream_t stream) {
  fa::Cache ca;
  int st = fa::rows_args(cache, B, seq_lens, out_lens, &ca);
  if (st != FA_OK) return st;
  if (N < 1 || K < 1 || K > N || 1ll * B * K > INT_MAX || !keep || !fa::aligned(keep, 4) ||
      !fa::aligned(new_lens, 4) || !fa::aligned(keep_lens, 4))
    return FA_ERR_INVALID_ARG;
  // (a cluster's CTAs read the lengths each on its own: they have to find the same)
  if (!fa::apart(out_lens, B, seq_lens, B) || !fa::apart(out_lens, B, new_lens, B) ||
      !fa::apart(out_lens, B, keep, 1ll * B * K) || !fa::apart(out_lens, B, keep_lens, B))
    return FA_ERR_INVALID_ARG;
  fa::KeepCall c = {B, N, K, seq_lens, new_lens, keep, keep_lens, out_lens};
  if ((st = fa::check_device(&c.err)) != FA_OK) return st;
  cudaError_t e = fa::launch_cache_keep(ca, c, std::max(1, fa::device_sms()), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fa::cuda_fail(e, "fa_cache_keep launch");
}

extern "C" size_t fa_cache_fork_workspace_size(int B, int pages, int table_width) {
  if (B < 1 || B > 65535 || pages < 1 || table_width < 1 || 1ll * B * table_width > INT_MAX) return 0;
  return fa::cache_fork_workspace_bytes(B, pages, table_width);
}

extern "C" int fa_cache_fork(const fa_cache* cache, int* block_table, int* refs, int B,
                             const int* parents, const int* seq_lens, const int* reserve_lens,
                             int* out_lens, void* workspace, size_t workspace_bytes,
                             fa_stream_t stream) {
  fa::Cache ca;
  int st = fa::rows_args(cache, B, seq_lens, out_lens, &ca);
  if (st != FA_OK) return st;
  if (!block_table || !refs || !parents || !fa::aligned(block_table, 4) || !fa::aligned(refs, 4) ||
      !fa::aligned(parents, 4) || !fa::aligned(reserve_lens, 4))
    return FA_ERR_INVALID_ARG;
  const long long entries = 1ll * B * ca.width;
  if (block_table != ca.table && !fa::apart(block_table, entries, ca.table, entries)) return FA_ERR_INVALID_ARG;
  if (!workspace || !fa::aligned(workspace, 256) ||
      workspace_bytes < fa::cache_fork_workspace_bytes(B, ca.pages, ca.width))
    return FA_ERR_WORKSPACE;
  fa::ForkCall c = {B, block_table, refs, parents, seq_lens, reserve_lens, out_lens, workspace};
  if ((st = fa::check_device(&c.err)) != FA_OK) return st;
  cudaError_t e = fa::launch_cache_fork(ca, c, std::max(1, fa::device_sms()), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fa::cuda_fail(e, "fa_cache_fork launch");
}
