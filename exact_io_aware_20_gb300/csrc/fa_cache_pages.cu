// Pages of the paged 8-bit cache: keeping some of the last tokens of sequences
// (fa_cache_keep), and forking, reordering, ending and beginning sequences over
// shared pages (fa_cache_fork).
#include <algorithm>

#include "cache_codes.cuh"
#include "cache_keep.cuh"
#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void copy_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}

// (a call: the rare case's code stays out of the loop of the other)
__device__ __noinline__ uint4 rescaled_by_any(uint4 v, float ratio) { return rescaled(v, ratio); }

// Sixteen codes of scale `was` for scale `now` >= was.  Powers of two: the ratio
// as f16 (exact: what it brings below f16's range is below e4m3's too, and 0), so
// that two codes are three instructions.
__device__ __forceinline__ uint4 for_scale(const uint4& v, float was, float now) {
  const uint32_t a = __float_as_uint(was), b = __float_as_uint(now);
  const int down = static_cast<int>((b >> 23) - (a >> 23));
  if (((a | b) & 0x807fffffu) != 0 || a < 0x800000u || down < 0) return rescaled_by_any(v, was / now);
  // 2^-down as f16 (to 2^-24; 448 times less than that is below half of e4m3's
  // smallest, 2^-10)
  const uint32_t one = down <= 14 ? static_cast<uint32_t>(15 - down) << 10 : down <= 24 ? 1u << (24 - down) : 0u;
  const uint32_t ratio = one | one << 16;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 p, q;\n\t.reg .b32 x, y;\n\tmov.b32 {p, q}, %0;\n\t"
        "cvt.rn.f16x2.e4m3x2 x, p;\n\tcvt.rn.f16x2.e4m3x2 y, q;\n\t"
        "mul.rn.f16x2 x, x, %1;\n\tmul.rn.f16x2 y, y, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 p, x;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, y;\n\t"
        "mov.b32 %0, {p, q};\n\t}"
        : "+r"(w[i]) : "r"(ratio));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------ keep
//
// Token base + i of a sequence becomes what token base + keep[i] is, and
// keep[i] >= i: sources lie at or behind their places.  A cluster has K or V of
// one head of one sequence and walks over the pages that take tokens, a run of
// them (`rows` tokens a CTA, whole pages) at a time: all its CTAs read the run's
// sources into shared memory, meet, and write.  What a run writes, the runs
// behind it do not read (their sources lie in pages behind it), so that one
// meeting a run is enough, the next run's sources may be on their way while a run
// is written, and the pages' scales need no second copy.
//
// What bounds it: the dependent reads (lengths, numbers, table, codes) of a short
// window (25 drafts of 64 sequences, 8 heads: 5.2 us; of one 4.5) and of each run
// of a long one (half of 2 x 16384 tokens, 8 heads, d = 128, 54 MB: 20 us, 40% of
// what a copy reaches; with every run's reads behind the writes of the one before
// 25 us).  Loops are left rolled: the code runs once or twice a launch, and its
// instructions come from L2 (unrolled by four the drafts took 10.7 us instead of
// 7.4).
struct KeepParams {
  Cache cache;
  int page_log2, slots_log2;       // 16-byte slots of a row
  int N, K;
  int rows;                        // of a CTA's run, a multiple of a page
  int ctas;                        // of a cluster
  const int *seq_lens, *new_lens, *keep, *keep_lens;
  int* out_lens;
  unsigned int* err;
};

constexpr int kKeepThreads = 512;      // at most

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepParams p) {
  extern __shared__ __align__(16) unsigned char keep_smem[];
  uint4* codes = reinterpret_cast<uint4*>(keep_smem);
  // Of two runs by turns: [row] where it comes from (nullptr: it is there already,
  // or there is none) and the scale that it comes with (below 0: there is none; 0 is
  // a page of zeros, whose tokens are rounded for their new page's scale like any);
  // [page] the bits of its scale (-1: no token of it is there), and its number (-1: out
  // of range)
  const unsigned char** from_of =
      reinterpret_cast<const unsigned char**>(keep_smem + (static_cast<size_t>(p.rows) << (p.slots_log2 + 4)));
  float* scale_of = reinterpret_cast<float*>(from_of + 2 * p.rows);
  const int pages = p.rows >> p.page_log2;
  int* top = reinterpret_cast<int*>(scale_of + 2 * p.rows);
  int* page_of = top + 2 * pages;
  int* verdict = page_of + 2 * pages;
  const Cache& ca = p.cache;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int rank = blockIdx.x % p.ctas, unit = blockIdx.x / p.ctas;
  const int b = unit / (2 * ca.Hkv), h = unit / 2 % ca.Hkv;
  const bool key = (unit & 1) == 0;
  const int len = p.seq_lens[b], n = p.new_lens != nullptr ? p.new_lens[b] : p.N;
  const int kept = p.keep_lens != nullptr ? p.keep_lens[b] : p.K;
  const int* keep = p.keep + static_cast<long long>(b) * p.K;
  const bool first_cta = rank == 0 && h == 0 && key && tid == 0;
  const KeepWindow window = keep_window(len, n, kept, p.N, p.K, static_cast<long long>(ca.width) << p.page_log2);
  const int base = window.base, end = window.end;
  const bool valid = window.valid;
  if (!valid || kept == 0) {         // (the whole cluster)
    if (first_cta) {
      p.out_lens[b] = valid ? base : len;
      if (!valid) atomicOr(p.err, kErrCache);
    }
    return;
  }
  // The numbers, a part of them a CTA; what it comes to is known where the cluster
  // meets ahead of the first write.
  bool bad = false;
  #pragma unroll 1
  for (int i = rank * threads + tid; i < kept; i += p.ctas * threads) {
    const int at = keep[i], before = i > 0 ? keep[i - 1] : -1;
    bad |= at >= n || at <= before;
  }
  const Strides st = key ? ca.ks : ca.vs;
  unsigned char* data = (key ? ca.k : ca.v) + h * st.h;
  float* scales = (key ? ca.k_scale : ca.v_scale) + h;
  const int* table = ca.table + static_cast<long long>(b) * ca.width;
  const int page_mask = (1 << p.page_log2) - 1, slots = 1 << p.slots_log2;
  auto page_at = [&](int tok) -> int {
    const int page = table[tok >> p.page_log2];
    if (static_cast<unsigned>(page) < static_cast<unsigned>(ca.pages)) return page;
    atomicOr(p.err, kErrCache);
    return -1;
  };
  // this CTA's first token of run r, and how many
  const int start = base & ~page_mask, run = p.rows * p.ctas, runs = (end - start + run - 1) / run;
  auto first_of = [&](int r) { return start + r * run + rank * p.rows; };
  auto count_of = [&](int r) { return r < runs ? max(0, min(p.rows, end - first_of(r))) : 0; };
  // The records of run r.
  auto records = [&](int r) {
    const int first = first_of(r), count = count_of(r), at = (r & 1) * p.rows, page0 = (r & 1) * pages;
    for (int i = tid; i << p.page_log2 < count; i += threads)
      page_of[page0 + i] = page_at(first + (i << p.page_log2));
    #pragma unroll 1
    for (int i = tid; i < count; i += threads) {
      const int tok = first + i, number = tok < base ? tok - base : keep[tok - base];
      const int from = number < n ? base + number : -1;      // (below 0: out of range)
      const int page = from >= 0 ? page_at(from) : -1;
      // (without its sign: -0, or a NaN's)
      const float scale = page >= 0 ? fabsf(scales[static_cast<long long>(page) * ca.Hkv]) : -1.f;
      from_of[at + i] = from == tok || page < 0 ? nullptr : data + page * st.b + (from & page_mask) * st.n;
      scale_of[at + i] = scale;
      atomicMax(top + page0 + (i >> p.page_log2), __float_as_int(scale));
    }
  };
  // slot x of run r on its way
  auto fetch = [&](int r, int x) {
    const unsigned char* src = from_of[(r & 1) * p.rows + (x >> p.slots_log2)];
    if (src != nullptr) copy_async_16(smem_u32(codes + x), src + 16 * (x & (slots - 1)));
  };
  for (int i = tid; i < 2 * pages; i += threads) top[i] = -1;
  __syncthreads();
  records(0);
  __syncthreads();
  for (int x = tid; x < count_of(0) << p.slots_log2; x += threads) fetch(0, x);
  for (int r = 0; r < runs; ++r) {
    const int first = first_of(r), count = count_of(r) << p.slots_log2, next = count_of(r + 1) << p.slots_log2;
    const int at = (r & 1) * p.rows, page0 = (r & 1) * pages;
    if (next > 0) records(r + 1);
    copy_async_wait();
    if (r == 0) bad = __syncthreads_or(bad);
    if (p.ctas > 1) {
      if (r == 0 && tid == 0) *verdict = bad;
      cluster_sync();
      if (r == 0)
        for (int i = 0; i < p.ctas; ++i) bad |= ld_cluster(mapa_shared(smem_u32(verdict), i)) != 0;
    } else if (r > 0) {
      __syncthreads();
    }
    if (r == 0) {
      if (first_cta) {
        p.out_lens[b] = bad ? len : end;
        if (bad) atomicOr(p.err, kErrCache);
      }
      if (bad) break;      // (the whole cluster)
    }
    #pragma unroll 1
    for (int x = tid; x < max(count, next); x += threads) {      // (a thread's slots are its own)
      if (x < count) {
        const int i = x >> p.slots_log2, page = page_of[page0 + (i >> p.page_log2)];
        const float was = scale_of[at + i], now = __int_as_float(top[page0 + (i >> p.page_log2)]);
        const bool moved = from_of[at + i] != nullptr;
        // (a row that is there already changes where its page's scale grows)
        if (!(was < 0.f) && page >= 0 && (moved || was != now)) {
          uint4* to = reinterpret_cast<uint4*>(data + page * st.b + ((first + i) & page_mask) * st.n +
                                               16 * (x & (slots - 1)));
          uint4 v = moved ? codes[x] : *to;
          if (was != now) v = for_scale(v, was, now);
          *to = v;
        }
      }
      if (x < next) fetch(r + 1, x);
    }
    __syncthreads();
    for (int i = tid; i < pages; i += threads) {      // (the records' places are free for run r + 2)
      const int bits = top[page0 + i];
      if (bits >= 0 && page_of[page0 + i] >= 0)
        scales[static_cast<long long>(page_of[page0 + i]) * ca.Hkv] = __int_as_float(bits);
      top[page0 + i] = -1;
    }
    __syncthreads();
  }
  if (p.ctas > 1) cluster_sync();      // (the others read this CTA's verdict)
}

// ------------------------------------------------------------------ fork
//
// Two kernels.  The first only reads the table and the counts: a block a
// sequence settles its new row (places that take a free page are numbered within
// the row), and blocks of 8192 pages write down which of them are free, a bit
// each.  The second writes: a block finds its sequence's free pages by the
// numbers of those that the sequences before it take, brings the counts up to
// date, and others copy the tokens of a page that is not full.
//
// What bounds it: two kernels' dependent reads (32 sequences 6.7 us, 256 that
// share whole pages only 8.4), and then the copies: 256 samples of 4 prompts, 28 MB
// read and as much written, 18 us; of one prompt, 67 MB written, 25 us.  (A head
// after another, one slot a thread at a time: 11.3 and 24 us.  More blocks or
// slots a thread: the same.)
constexpr int kChunkWords = 256;                 // of 32 pages

struct ForkInfo {
  int len, need;        // tokens, and pages that the sequence holds
  int tail, tail_rank;  // the page whose tokens are copied (-1: none), and which of the row's free pages takes them
};

struct ForkParams {
  Cache cache;
  int page_log2, slots_log2;
  int B, chunks;
  int *table, *refs;
  const int *parents, *seq_lens, *reserve_lens;
  int* out_lens;
  // workspace
  ForkInfo* info;       // [B]
  int* fresh;           // [B] free pages that the row takes
  int* row;             // [B][width] the new row, -1 where it takes a free page
  int* place;           // [B][width] where it takes them
  uint32_t* bits;       // [chunks][kChunkWords] free pages
  int* counts;          // [chunks] how many
  unsigned int* err;
};

// Sum over the block's threads up to and including this one's, and all of them
// (two barriers; space: kThreads / 32 values).
__device__ __forceinline__ int block_scan(int x, int* all, int* space) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  #pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  if (lane == 31) space[warp] = x;
  __syncthreads();
  int sum = 0;
  #pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) x += space[i];
    sum += space[i];
  }
  *all = sum;
  __syncthreads();
  return x;
}

__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int space[kThreads / 32];
  __shared__ int tail[2];
  const Cache& ca = p.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= p.B) {
    const int c = blockIdx.x - p.B;
    const long long word0 = static_cast<long long>(c) * kChunkWords + 32 * warp;
    uint32_t mine = 0;
    #pragma unroll
    for (int k = 0; k < 32; ++k) {
      const long long page = (word0 + k) * 32 + lane;
      const uint32_t free = __ballot_sync(0xffffffffu, page < ca.pages && p.refs[page] == 0);
      if (lane == k) mine = free;
    }
    p.bits[word0 + lane] = mine;
    int all;
    block_scan(__popc(mine), &all, space);
    if (tid == 0) p.counts[c] = all;
    return;
  }
  const int b = blockIdx.x;
  const long long capacity = static_cast<long long>(ca.width) << p.page_log2;
  bool bad = false;
  int parent = p.parents[b];
  if (parent < -1 || parent >= p.B) {
    bad = true;
    parent = -1;
  }
  int len = parent >= 0 ? p.seq_lens[parent] : 0;
  if (len < 0 || len > capacity) {
    bad = true;
    len = 0;
  }
  int reserve = p.reserve_lens != nullptr ? p.reserve_lens[b] : 0;
  if (reserve > capacity) {
    bad = true;
    reserve = static_cast<int>(capacity);
  }
  const int page_mask = (1 << p.page_log2) - 1;
  const int tokens = max(len, reserve);
  const int need = (tokens >> p.page_log2) + ((tokens & page_mask) != 0), full = len >> p.page_log2;
  if (tid == 0) tail[0] = tail[1] = -1;
  bool before = false;       // a sequence ahead of this one has the same parent
  for (int i = tid; i < b; i += kThreads) before |= p.parents[i] == parent;
  const bool first = !__syncthreads_or(before);
  const long long row = static_cast<long long>(b) * ca.width;
  int taken = 0;
  for (int i0 = 0; i0 < need; i0 += kThreads) {
    const int i = i0 + tid;
    int now = -1, old = -1;
    bool fresh = false;
    if (i < need) {
      if (parent >= 0) old = ca.table[static_cast<long long>(parent) * ca.width + i];
      if (static_cast<unsigned>(old) >= static_cast<unsigned>(ca.pages)) old = -1;
      if (i < full) {
        now = old;
        bad |= old < 0;
      } else if (first && old >= 0 && p.refs[old] == 1) {
        now = old;
      } else {
        fresh = true;
        bad |= old < 0 && i == full && (len & page_mask) != 0;
      }
      p.row[row + i] = now;
    }
    int all;
    const int rank = taken + block_scan(fresh, &all, space) - 1;
    if (fresh) {
      p.place[row + rank] = i;
      if (i == full && (len & page_mask) != 0) {
        tail[0] = old >= 0 ? old : ca.pages - 1;      // (out of range: any page that is there, and reported)
        tail[1] = rank;
      }
    }
    taken += all;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    p.info[b] = {len, need, tail[0], tail[1]};
    p.fresh[b] = taken;
    if (bad) atomicOr(p.err, kErrCache);
  }
}

__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int space[kThreads / 32];
  __shared__ int place[kThreads];      // the row's first places that take free pages
  __shared__ int2 hit[kThreads];       // chunks that hold pages of this row: number, free pages before it
  __shared__ int hits, tail;
  const Cache& ca = p.cache;
  const int tid = threadIdx.x, b = blockIdx.y;
  const bool writes = blockIdx.x == 0;        // the row and the counts; the others copy
  const long long row = static_cast<long long>(b) * ca.width;
  grid_dependency_wait();
  // (what most calls need, read at once)
  const ForkInfo info = p.info[b];
  const int fresh = p.fresh[b], count0 = tid < p.chunks ? p.counts[tid] : 0;
  const uint32_t bits0 = p.bits[tid];
  int before = 0, base;
  for (int i = tid; i < b; i += kThreads) before += p.fresh[i];
  if (writes) {
    if (tid < fresh) place[tid] = p.place[row + tid];
    for (int i = tid; i < ca.width; i += kThreads) {
      const int old = ca.table[row + i], now = i < info.need ? p.row[row + i] : -1;
      if (static_cast<unsigned>(old) < static_cast<unsigned>(ca.pages)) atomicAdd(p.refs + old, -1);
      if (now >= 0) atomicAdd(p.refs + now, 1);
      p.table[row + i] = now;
    }
    if (tid == 0) p.out_lens[b] = info.len;
  }
  if (fresh == 0 || (!writes && info.tail < 0)) return;
  if (tid == 0) tail = -1;
  block_scan(before, &base, space);
  // free pages numbered lo .. hi - 1
  const int lo = writes ? base : base + info.tail_rank, hi = writes ? base + fresh : lo + 1;
  int passed = 0;
  for (int c0 = 0; c0 < p.chunks && passed < hi; c0 += kThreads) {
    const int c = c0 + tid, mine = c0 == 0 ? count0 : c < p.chunks ? p.counts[c] : 0;
    if (tid == 0) hits = 0;
    int all;
    const int upto = passed + block_scan(mine, &all, space);
    if (mine > 0 && upto - mine < hi && upto > lo) hit[atomicAdd(&hits, 1)] = make_int2(c, upto - mine);
    __syncthreads();
    for (int k = 0; k < hits; ++k) {
      uint32_t w = hit[k].x == 0 ? bits0 : p.bits[static_cast<long long>(hit[k].x) * kChunkWords + tid];
      int unused;
      int number = hit[k].y + block_scan(__popc(w), &unused, space) - __popc(w);
      for (; w != 0 && number < hi; w &= w - 1, ++number) {
        if (number < lo) continue;
        const int page = (hit[k].x * kChunkWords + tid) * 32 + __ffs(w) - 1, rank = number - base;
        if (writes) {
          p.table[row + (rank < kThreads ? place[rank] : p.place[row + rank])] = page;
          atomicAdd(p.refs + page, 1);
        }
        if (rank == info.tail_rank) tail = page;
      }
    }
    passed += all;
    __syncthreads();
  }
  if (writes) {
    if (passed < hi && tid == 0) atomicOr(p.err, kErrCache);
    return;
  }
  const int src = info.tail, dst = tail;
  if (dst < 0) return;
  // the page's tokens, 16 bytes a thread, kAhead of them on their way
  constexpr int kAhead = 4;
  const int rows = info.len & ((1 << p.page_log2) - 1), slots = 1 << p.slots_log2;
  const int head = rows << p.slots_log2, part = blockIdx.x - 1, parts = gridDim.x - 1;     // slots of a head
  const int total = 2 * ca.Hkv * head, step = parts * kThreads;
  for (int x0 = part * kThreads + tid; x0 < total; x0 += kAhead * step) {
    uint4 v[kAhead];
    unsigned char* to[kAhead];
    #pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int x = x0 + k * step, hk = x / head, in = x - hk * head;
      to[k] = nullptr;
      if (x0 <= total - 1 - k * step) {
        const Strides st = hk & 1 ? ca.vs : ca.ks;
        unsigned char* at = (hk & 1 ? ca.v : ca.k) + (hk >> 1) * st.h + (in >> p.slots_log2) * st.n + 16 * (in & (slots - 1));
        v[k] = *reinterpret_cast<const uint4*>(at + src * st.b);
        to[k] = at + dst * st.b;
      }
    }
    #pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (to[k] != nullptr) *reinterpret_cast<uint4*>(to[k]) = v[k];
  }
  if (part == 0)
    for (int h = tid; h < ca.Hkv; h += kThreads) {
      const long long to = static_cast<long long>(dst) * ca.Hkv + h, from = static_cast<long long>(src) * ca.Hkv + h;
      ca.k_scale[to] = ca.k_scale[from];
      ca.v_scale[to] = ca.v_scale[from];
    }
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

int fork_chunks(int pages) { return (pages - 1) / (32 * kChunkWords) + 1; }      // (pages may be INT_MAX)

size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_cache_keep(const Cache& cache, const KeepCall& c, int sms, cudaStream_t stream) {
  KeepParams p = {};
  p.cache = cache;
  p.page_log2 = log2_of(cache.page);
  p.slots_log2 = log2_of(cache.d / 16);
  p.N = c.N;
  p.K = c.K;
  p.seq_lens = c.seq_lens;
  p.new_lens = c.new_lens;
  p.keep = c.keep;
  p.keep_lens = c.keep_lens;
  p.out_lens = c.out_lens;
  p.err = c.err;
  const long long units = 2ll * c.B * cache.Hkv;
  // CTAs of a cluster: more while there are fewer than SMs.  What a CTA's run may
  // hold and its threads: by how many of them an SM takes (few CTAs' runs are few
  // meetings, and many threads hide their reads; half of 16384 tokens of one head
  // with 256 / 512 threads 18.7 / 14.5 us, 2 x 8 heads 23.2 / 20.9; half of 256
  // tokens of 64 x 8 heads 9.4 / 14.3, half of 1024 of 16 x 8 heads by 512 CTAs of
  // 512 threads / 256 CTAs 13.7 / 8.4).
  constexpr int kRecord = 2 * (sizeof(void*) + sizeof(float)), kMost = 200 * 1024;
  const int span = (c.K - 1 + cache.page - 1) / cache.page + 1;      // pages that K tokens can touch
  p.ctas = 1;
  while (p.ctas < 8 && p.ctas < span && units * p.ctas < sms) p.ctas *= 2;
  const long long blocks = units * p.ctas;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  // (a cluster's CTAs stand in one GPC: with one CTA an SM fewer clusters than SMs / 8
  // run at a time, half of 16384 tokens of 8 heads 23 us instead of 18)
  const int room = 2 * blocks <= sms ? kMost : blocks <= 2ll * sms ? kMost / 2 : kMost / 4;
  const int most = std::max(1, room / (cache.d + kRecord) / cache.page);      // pages of a CTA's run
  const int each = (span + p.ctas - 1) / p.ctas, runs = (each + most - 1) / most;
  p.rows = (each + runs - 1) / runs * cache.page;                             // (even runs)
  int threads = 128;
  while (threads < (blocks <= 2ll * sms ? kKeepThreads : kKeepThreads / 2) && threads < (p.rows << p.slots_log2) / 8)
    threads *= 2;
  const size_t smem =
      static_cast<size_t>(p.rows) * (cache.d + kRecord) + 4 * sizeof(int) * (p.rows / cache.page) + sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(keep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost + 8192);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, keep_kernel, p);
}

size_t cache_fork_workspace_bytes(int B, int pages, int width) {
  const size_t chunks = fork_chunks(pages), entries = static_cast<size_t>(B) * width;
  return padded(B * sizeof(ForkInfo)) + padded(4ull * B) + 2 * padded(4 * entries) +
         padded(4 * kChunkWords * chunks) + padded(4 * chunks);
}

cudaError_t launch_cache_fork(const Cache& cache, const ForkCall& c, int sms, cudaStream_t stream) {
  ForkParams p = {};
  p.cache = cache;
  p.page_log2 = log2_of(cache.page);
  p.slots_log2 = log2_of(cache.d / 16);
  p.B = c.B;
  p.chunks = fork_chunks(cache.pages);
  p.table = c.block_table;
  p.refs = c.refs;
  p.parents = c.parents;
  p.seq_lens = c.seq_lens;
  p.reserve_lens = c.reserve_lens;
  p.out_lens = c.out_lens;
  p.err = c.err;
  unsigned char* ws = static_cast<unsigned char*>(c.workspace);
  auto take = [&](size_t bytes) -> void* {
    void* at = ws;
    ws += padded(bytes);
    return at;
  };
  const size_t entries = static_cast<size_t>(c.B) * cache.width;
  p.info = static_cast<ForkInfo*>(take(c.B * sizeof(ForkInfo)));
  p.fresh = static_cast<int*>(take(4ull * c.B));
  p.row = static_cast<int*>(take(4 * entries));
  p.place = static_cast<int*>(take(4 * entries));
  p.bits = static_cast<uint32_t*>(take(4ull * kChunkWords * p.chunks));
  p.counts = static_cast<int*>(take(4ull * p.chunks));
  fork_plan_kernel<<<c.B + p.chunks, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // blocks of a sequence that copy: about four an SM in all, as many as a page has
  // four slots a thread for
  const long long slots = 2ll * cache.Hkv * cache.page * cache.d / 16;
  const int parts = static_cast<int>(std::max(1ll, std::min<long long>((4 * sms + c.B - 1) / c.B, slots / (4 * kThreads))));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(parts + 1), static_cast<unsigned>(c.B), 1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fork_apply_kernel, p);
}

}  // namespace fa
