// Pages of the paged 8-bit cache: keeping some of the last tokens of sequences
// (fa_cache_keep), and forking, reordering, ending and beginning sequences over
// shared pages (fa_cache_fork).
#include <algorithm>

#include "cache_codes.cuh"
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

// ------------------------------------------------------------------ keep
//
// Token base + i of a sequence becomes what token base + keep[i] is, and
// keep[i] >= i: sources lie at or behind their places.  A cluster has K or V of
// one head of one sequence and walks over the pages that take tokens, a run of
// them (`rows` tokens a CTA, whole pages) at a time: all its CTAs read the run's
// sources into shared memory, meet, and write.  What a run writes, the runs
// behind it do not read (their sources lie in pages behind it), so that one
// meeting a run is enough, and the pages' scales need no second copy.
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

struct KeepRow {
  const unsigned char* src;   // nullptr: the row stays where it is, as it is
  float scale;                // that it comes with; 0: no row
};

__global__ void __launch_bounds__(kThreads) keep_kernel(const __grid_constant__ KeepParams p) {
  extern __shared__ __align__(16) unsigned char keep_smem[];
  uint4* codes = reinterpret_cast<uint4*>(keep_smem);
  KeepRow* row_of = reinterpret_cast<KeepRow*>(keep_smem + (static_cast<size_t>(p.rows) << (p.slots_log2 + 4)));
  int* top = reinterpret_cast<int*>(row_of + p.rows);     // [page of the run] the bits of its scale
  const Cache& ca = p.cache;
  const int tid = threadIdx.x, rank = blockIdx.x % p.ctas, unit = blockIdx.x / p.ctas;
  const int b = unit / (2 * ca.Hkv), h = unit / 2 % ca.Hkv;
  const bool key = (unit & 1) == 0;
  const int len = p.seq_lens[b], n = p.new_lens != nullptr ? p.new_lens[b] : p.N;
  const int kept = p.keep_lens != nullptr ? p.keep_lens[b] : p.K;
  const int* keep = p.keep + static_cast<long long>(b) * p.K;
  bool bad = n < 0 || n > p.N || len < n || len > (static_cast<long long>(ca.width) << p.page_log2) ||
             kept < 0 || kept > p.K;
  if (!bad)
    for (int i = tid; i < kept; i += kThreads) {
      const int at = keep[i];
      bad |= at >= n || at <= (i > 0 ? keep[i - 1] : -1);
    }
  bad = __syncthreads_or(bad);
  const int base = len - n, end = base + kept;
  if (rank == 0 && h == 0 && key && tid == 0) {
    p.out_lens[b] = bad ? len : end;
    if (bad) atomicOr(p.err, kErrCache);
  }
  if (bad || kept == 0) return;      // (the whole cluster)
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
  const int run = p.rows * p.ctas;
  for (int t0 = base & ~page_mask; t0 < end; t0 += run) {
    const int first = t0 + rank * p.rows;                       // this CTA's tokens
    const int count = max(0, min(p.rows, end - first));
    for (int i = tid; i < p.rows >> p.page_log2; i += kThreads) top[i] = 0;
    __syncthreads();
    for (int i = tid; i < count; i += kThreads) {
      const int tok = first + i, from = tok < base ? tok : base + keep[tok - base];
      const int page = page_at(from);
      KeepRow r = {nullptr, 0.f};
      if (page >= 0) {
        r.scale = scales[static_cast<long long>(page) * ca.Hkv];
        if (from != tok) r.src = data + page * st.b + (from & page_mask) * st.n;
        atomicMax(top + (i >> p.page_log2), __float_as_int(r.scale));
      }
      row_of[i] = r;
    }
    __syncthreads();
    // A row that stays is read where its page's scale grows.
    auto wanted = [&](int i, const KeepRow& r) {
      return r.scale != 0.f && (r.src != nullptr || r.scale != __int_as_float(top[i >> p.page_log2]));
    };
    for (int x = tid; x < count << p.slots_log2; x += kThreads) {
      const int i = x >> p.slots_log2, slot = x & (slots - 1);
      const KeepRow r = row_of[i];
      if (!wanted(i, r)) continue;
      const unsigned char* src = r.src;
      if (src == nullptr) src = data + table[(first + i) >> p.page_log2] * st.b + ((first + i) & page_mask) * st.n;
      copy_async_16(smem_u32(codes + x), src + 16 * slot);
    }
    copy_async_wait();
    if (p.ctas > 1) cluster_sync();
    else __syncthreads();
    for (int x = tid; x < count << p.slots_log2; x += kThreads) {   // (what this thread has read)
      const int i = x >> p.slots_log2, slot = x & (slots - 1);
      const KeepRow r = row_of[i];
      if (!wanted(i, r)) continue;
      const int page = page_at(first + i);
      if (page < 0) continue;
      const float now = __int_as_float(top[i >> p.page_log2]);
      uint4 v = codes[x];
      if (r.scale != now) v = rescaled(v, r.scale / now);
      *reinterpret_cast<uint4*>(data + page * st.b + ((first + i) & page_mask) * st.n + 16 * slot) = v;
    }
    for (int i = tid; i < p.rows >> p.page_log2; i += kThreads) {
      if (top[i] == 0) continue;
      const int page = page_at(first + (i << p.page_log2));
      if (page >= 0) scales[static_cast<long long>(page) * ca.Hkv] = __int_as_float(top[i]);
    }
    __syncthreads();       // the rows' records are written anew
  }
}

// ------------------------------------------------------------------ fork
//
// Two kernels.  The first only reads the table and the counts: a block a
// sequence settles its new row (places that take a free page are numbered within
// the row), and blocks of 8192 pages write down which of them are free, a bit
// each.  The second writes: a block finds its sequence's free pages by the
// numbers of those that the sequences before it take, brings the counts up to
// date and copies the tokens of a page that is not full (several blocks a
// sequence).
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
        tail[0] = old;
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
  __shared__ int2 hit[kThreads];       // chunks that hold pages of this row: number, free pages before it
  __shared__ int hits, tail;
  const Cache& ca = p.cache;
  const int tid = threadIdx.x, b = blockIdx.y;
  const bool writes = blockIdx.x == 0;        // the row and the counts; the others copy only
  grid_dependency_wait();
  const ForkInfo info = p.info[b];
  const int fresh = p.fresh[b];
  const long long row = static_cast<long long>(b) * ca.width;
  if (writes) {
    for (int i = tid; i < ca.width; i += kThreads) {
      const int old = ca.table[row + i], now = i < info.need ? p.row[row + i] : -1;
      if (static_cast<unsigned>(old) < static_cast<unsigned>(ca.pages)) atomicAdd(p.refs + old, -1);
      if (now >= 0) atomicAdd(p.refs + now, 1);
      p.table[row + i] = now;
    }
    if (tid == 0) p.out_lens[b] = info.len;
  }
  if (fresh == 0 || (!writes && info.tail < 0)) return;
  int before = 0, base;
  for (int i = tid; i < b; i += kThreads) before += p.fresh[i];
  if (tid == 0) tail = -1;
  block_scan(before, &base, space);
  // free pages numbered lo .. hi - 1
  const int lo = writes ? base : base + info.tail_rank, hi = writes ? base + fresh : lo + 1;
  int passed = 0;
  for (int c0 = 0; c0 < p.chunks && passed < hi; c0 += kThreads) {
    const int c = c0 + tid, mine = c < p.chunks ? p.counts[c] : 0;
    if (tid == 0) hits = 0;
    int all;
    const int upto = passed + block_scan(mine, &all, space);
    if (mine > 0 && upto - mine < hi && upto > lo) hit[atomicAdd(&hits, 1)] = make_int2(c, upto - mine);
    __syncthreads();
    for (int k = 0; k < hits; ++k) {
      uint32_t w = p.bits[static_cast<long long>(hit[k].x) * kChunkWords + tid];
      int unused;
      int number = hit[k].y + block_scan(__popc(w), &unused, space) - __popc(w);
      for (; w != 0 && number < hi; w &= w - 1, ++number) {
        if (number < lo) continue;
        const int page = (hit[k].x * kChunkWords + tid) * 32 + __ffs(w) - 1, rank = number - base;
        if (writes) {
          p.table[row + p.place[row + rank]] = page;
          atomicAdd(p.refs + page, 1);
        }
        if (rank == info.tail_rank) tail = page;
      }
    }
    passed += all;
    __syncthreads();
  }
  if (writes && passed < hi && tid == 0) atomicOr(p.err, kErrCache);
  const int src = info.tail, dst = tail;
  if (src < 0 || dst < 0) return;
  const int rows = info.len & ((1 << p.page_log2) - 1), slots = 1 << p.slots_log2;
  const int head = rows << p.slots_log2;            // 16-byte slots of a head
  for (int hk = 0; hk < 2 * ca.Hkv; ++hk) {
    const Strides st = hk & 1 ? ca.vs : ca.ks;
    unsigned char* data = (hk & 1 ? ca.v : ca.k) + (hk >> 1) * st.h;
    for (int x = blockIdx.x * kThreads + tid; x < head; x += gridDim.x * kThreads) {
      const long long at = (x >> p.slots_log2) * st.n + 16 * (x & (slots - 1));
      *reinterpret_cast<uint4*>(data + dst * st.b + at) = *reinterpret_cast<const uint4*>(data + src * st.b + at);
    }
  }
  if (writes)
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

int fork_chunks(int pages) { return (pages + 32 * kChunkWords - 1) / (32 * kChunkWords); }

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
  const int span = (c.K - 1 + cache.page - 1) / cache.page + 1;      // pages that K tokens can touch
  const int most = std::max(1, 65536 / cache.d / cache.page);        // of a CTA's run
  p.ctas = 1;
  while (p.ctas < 8 && p.ctas < span && units * p.ctas < 2ll * sms) p.ctas *= 2;
  p.rows = std::min(most, (span + p.ctas - 1) / p.ctas) * cache.page;
  const long long blocks = units * p.ctas;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = static_cast<size_t>(p.rows) * (cache.d + sizeof(KeepRow)) + 4 * (p.rows / cache.page);
  cudaError_t e = cudaFuncSetAttribute(keep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       65536 + 65536 / 64 * static_cast<int>(sizeof(KeepRow)) + 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
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
  // blocks a sequence: about two an SM, as many as a page's head has slots for
  const int slots = cache.page * cache.d / 16;
  const int parts = std::max(1, std::min((2 * sms + c.B - 1) / c.B, (slots + kThreads - 1) / kThreads));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(parts), static_cast<unsigned>(c.B), 1);
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
