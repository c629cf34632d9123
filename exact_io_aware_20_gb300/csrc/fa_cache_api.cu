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

extern "C" int fa_fwd_cache(const void* q, const fa_cache* cache, void* o, float* lse, int B,
                            int H, int Nq, int causal, float scale, int dtype,
                            const int* seq_lens, const int* new_lens, const fa_strides* strides,
                            void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  fa::Cache ca;
  int st = fa::cache_args(cache, &ca);
  if (st != FA_OK) return st;
  if ((st = fa::check_sizes(B, H, Nq, ca.d, dtype)) != FA_OK) return st;
  if (H % ca.Hkv != 0 || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARG;
  if (!q || !o || !lse || !seq_lens) return FA_ERR_INVALID_ARG;
  if (!fa::aligned(q, 16) || !fa::aligned(o, 16) || !fa::aligned(lse, 4) ||
      !fa::aligned(seq_lens, 4) || !fa::aligned(new_lens, 4))
    return FA_ERR_INVALID_ARG;
  fa::CacheFwdCall c = {q, o, lse};
  if (strides != nullptr) {
    fa::Strides s[2];
    if (!fa::valid_strides(strides, 2, s)) return FA_ERR_INVALID_ARG;
    c.qs = s[0];
    c.os = s[1];
  } else {
    c.qs = c.os = fa::contiguous_strides(H, Nq, ca.d);
  }
  if (!workspace || !fa::aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  if ((st = fa::check_device(&c.err)) != FA_OK) return st;
  const int sms = fa::device_sms();
  if (workspace_bytes < fa::cache_fwd_workspace_bytes(H, ca.Hkv, Nq, ca.d, sms))
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
  cudaError_t e = fa::launch_cache_fwd(ca, c, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fa::cuda_fail(e, "fa_fwd_cache launch");
}
