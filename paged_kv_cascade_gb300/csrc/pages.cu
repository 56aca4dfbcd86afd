// Pages and slots for new tokens, and pages given back, on the device.
//
// With len_b cached tokens and n_b new ones, request b needs
//   need_b = ceil((len_b + n_b) / ps) - ceil(len_b / ps)
// pages; off_b = sum_{a < b} need_a.  The free page of rank r (the r-th set bit
// of the pool's map) goes to the request with off_b <= r < off_b + need_b, at
// table entry ceil(len_b / ps) + r - off_b; token i then has the slot that
// position len_b + i has in that table.  A map instead of a list of free pages
// makes the result independent of the order in which pages came back.
//
// assign is a chain of scans (lengths, map) with a few bytes behind it, so it is
// bound by latency: one cluster of blocks, every one of which scans the lengths
// and counts the map for itself (both small, from L2), with the map's chunks
// shared out over the blocks.  Up to kFewTokens tokens the same launch fills in
// their places; more go to a second launch over all SMs, which begins while the
// first one runs and finds what it needs of a request at its first token.  Both calls
// for 220,453 tokens of 300 requests: 60.7 us with one launch, 31.9 with the second,
// 26.4 with the requests of a block's tokens found while the first one runs, 32-bit
// divisions and a released row's entries loaded together, 19.8 with eight threads to a
// word of the map (a thread gave out up to 32 pages, one after another: 9 us of the
// launch's 17); 64 single tokens: 9.5 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "pkc_device.cuh"
#include "pkc_internal.h"

namespace pkc {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;  // portable
constexpr int kFewTokens = 8192;
constexpr int kMaxChunks = (int)(PKC_PAGES_MAX_PAGES / 32 / kThreads);

__device__ __forceinline__ int sat_add(int a, int b) {  // both >= 0
  return (int)min((unsigned)a + (unsigned)b, (unsigned)INT_MAX);
}

// Exclusive scan of v (>= 0) over the block, sums saturating at INT_MAX; every
// thread learns the total.  All threads call it; `sums` holds kWarps + 1 words.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x = sat_add(x, y);
  }
  __syncthreads();  // sums may still be read from the call before
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int w = lane < kWarps ? sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w = sat_add(w, y);
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  const int prev = __shfl_up_sync(0xffffffffu, x, 1);
  return sat_add(warp ? before : 0, lane ? prev : 0);
}

// Pages of x tokens (x < 2^32; 64-bit divisions are a hundred instructions each).
__device__ __forceinline__ int pages_of(const PagesParams& p, uint32_t x) {
  const uint32_t n = x / (uint32_t)p.page_size;
  return (int)(n + (n * (uint32_t)p.page_size != x));
}

// The set bits of word w of the map that stand for pages.
__device__ __forceinline__ uint32_t free_word(const PagesParams& p, int64_t w, int64_t words) {
  if (w >= words) return 0;
  uint32_t x = __ldcg(p.free_pages + w);
  const int64_t left = p.num_pages - 32 * w;
  return left < 32 ? x & ((1u << left) - 1) : x;
}

// Last b in 0 .. n - 1 with a[b] <= x (a[0] <= x, a does not descend).
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The place of request b's token at position pos.
__device__ __forceinline__ int64_t slot_at(const PagesParams& p, int b, int pos) {
  return (int64_t)__ldcg(p.block_table + (int64_t)b * p.bt_stride + pos / p.page_size) * p.page_size + pos % p.page_size;
}

// kAll: every token's place; else that of each request's first one, which with
// the flag in the status block is all that places_kernel needs.
template <bool kAll>
__global__ void __launch_bounds__(kThreads, 1) assign_pages_kernel(const PagesParams p) {
  extern __shared__ int smem[];
  int* off = smem;                       // [batch + 1] pages needed by the requests before b
  int* start = off + p.batch + 1;        // [batch + 1] new_indptr
  int* lens = start + p.batch + 1;       // [batch] length; ~length: not served for its own sake
  int* chunk_base = lens + p.batch;      // [chunks + 1] free pages before each chunk of the map
  __shared__ int sums[kWarps + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int n_blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31;
  const bool first_block = rank == 0;
  // (A cluster's barrier releases and acquires what its blocks wrote before it.)
  auto sync_all = [&] {
    if (n_blocks > 1) cluster.sync();
    else __syncthreads();
  };
  if (!kAll) grid_launch_dependents();  // places_kernel
  const int64_t words = (p.num_pages + 31) / 32;
  const int per_chunk = kThreads / p.split, chunks = (int)((words + per_chunk - 1) / per_chunk);
  // On their way while the lengths are scanned: the first word to count and the first
  // one of the block's own chunks, where `split` threads share a word's bits.
  const uint32_t bits = p.split == 1 ? ~0u : 15u << 4 * (tid & 7);
  const uint32_t first_word = free_word(p, tid, words);
  const uint32_t own_word = free_word(p, (int64_t)rank * per_chunk + tid / p.split, words);

  // The ranges have to run upwards within 0 .. total, or nobody is served.
  bool wrong = false;
  for (int b = tid; b <= p.batch; b += kThreads) {
    const int t = p.batch ? p.indptr[b] : 0;
    start[b] = t;
    wrong = wrong || t < 0 || t > p.total || (b > 0 && t < p.indptr[b - 1]);
  }
  for (int c = tid; c <= chunks; c += kThreads) chunk_base[c] = 0;
  wrong = __syncthreads_or(wrong);
  if (wrong && first_block && tid == 0) report(p.status, PKC_ERR_PLAN);

  // What each request needs, and the sum of those before it.
  int needed = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int need = 0;
    if (b < p.batch) {
      const int len = p.cache_seqlens[b], n = wrong ? 0 : start[b + 1] - start[b];
      const uint32_t have = (uint32_t)pages_of(p, (uint32_t)max(len, 0)), want = (uint32_t)pages_of(p, (uint32_t)max(len, 0) + (uint32_t)n);
      bool ok = len >= 0 && !wrong;
      if (ok && n > 0) {
        ok = want <= p.bt_stride;
        if (ok && have * (uint32_t)p.page_size != (uint32_t)len) {  // the new tokens begin in a page that is there
          const int page = p.block_table[(int64_t)b * p.bt_stride + have - 1];
          ok = page >= 0 && page < p.num_pages;
        }
      }
      if (!ok && !wrong && (len < 0 || n > 0) && first_block) report(p.status, PKC_ERR_BLOCK_TABLE);
      lens[b] = ok ? len : ~max(len, 0);
      if (ok) need = (int)(want - have);
    }
    int total;
    const int before = block_scan(need, sums, total);
    if (b < p.batch) off[b] = sat_add(needed, before);
    needed = sat_add(needed, total);
  }
  if (tid == 0) off[p.batch] = needed;

  // Free pages before each chunk of words (a warp's 32 words lie in one).
  if (needed > 0) {  // uniform
    for (int64_t w0 = 0; w0 < words; w0 += kThreads) {
      const uint32_t x = w0 == 0 ? first_word : free_word(p, w0 + tid, words);
      const int n = __reduce_add_sync(0xffffffffu, __popc(x));
      if (lane == 0 && n) atomicAdd(chunk_base + (int)((w0 + tid) / per_chunk), n);
    }
    __syncthreads();
    if (tid < 32) {  // exclusive, in place
      int before = 0;
      for (int c0 = 0; c0 <= chunks; c0 += 32) {
        const int c = c0 + lane, n = c < chunks ? chunk_base[c] : 0;
        int x = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, d);
          if (lane >= d) x += y;
        }
        if (c <= chunks) chunk_base[c] = before + x - n;
        before += __shfl_sync(0xffffffffu, x, 31);
      }
    }
  }
  __syncthreads();
  const int n_free = chunk_base[chunks];
  // Requests are served while the pages last; off does not descend, so the
  // first that does not fit ends it for all that need a page.
  int taken = needed;
  if (needed > n_free) {  // uniform
    taken = off[last_not_above(off, p.batch + 1, n_free)];
    if (first_block && tid == 0) report(p.status, PKC_ERR_NO_PAGES);
  }
  auto served = [&](int b) { return lens[b] >= 0 && (off[b + 1] <= taken || off[b + 1] == off[b]); };
  if (n_blocks > 1) sync_all();  // every block has read the map

  // The taken pages to the table, their bits cleared.
  for (int c = rank; c < chunks && taken > 0; c += n_blocks) {
    if (chunk_base[c] >= taken) break;  // uniform
    const int64_t w = (int64_t)c * per_chunk + tid / p.split;
    const uint32_t x = (c == rank ? own_word : free_word(p, w, words)) & bits;
    int total;
    int r = chunk_base[c] + block_scan(__popc(x), sums, total);
    uint32_t gone = 0;
    if (x && r < taken) {
      int b = last_not_above(off, p.batch + 1, r);
      for (uint32_t y = x; y && r < taken; y &= y - 1, ++r) {
        const int bit = __ffs(y) - 1;
        while (off[b + 1] <= r) ++b;
        const int have = pages_of(p, (uint32_t)lens[b]);
        p.block_table[(int64_t)b * p.bt_stride + have + (r - off[b])] = (int)(32 * w) + bit;
        gone |= 1u << bit;
      }
      atomicAnd(p.free_pages + w, ~gone);
    }
  }
  sync_all();  // the table is complete

  // Where the tokens go, and the lengths.
  if (kAll) {
    for (int t = rank * kThreads + tid; t < p.total; t += n_blocks * kThreads) {
      int64_t slot = -1;
      int pos = 0;
      if (!wrong && p.batch && t >= start[0] && t < start[p.batch]) {
        const int b = last_not_above(start, p.batch + 1, t);
        pos = (lens[b] >= 0 ? lens[b] : p.cache_seqlens[b]) + (t - start[b]);
        if (served(b)) slot = slot_at(p, b, pos);
      }
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
  } else {
    for (int b = rank * kThreads + tid; b < p.batch; b += n_blocks * kThreads)
      if (!wrong && start[b + 1] > start[b]) {
        const int len = lens[b] >= 0 ? lens[b] : p.cache_seqlens[b];
        p.slots[start[b]] = served(b) ? slot_at(p, b, len) : -1;
        p.positions[start[b]] = len;
      }
    if (first_block && tid == 0) p.status[PKC_ASSIGN_FLAG] = wrong || p.batch == 0;
  }
  sync_all();  // the lengths have been read: they may be the ones that grow
  if (first_block && p.seqlens_out)
    for (int b = tid; b < p.batch; b += kThreads)
      p.seqlens_out[b] = served(b) ? lens[b] + (start[b + 1] - start[b]) : p.cache_seqlens[b];
}

constexpr int kPlaceThreads = 256;
constexpr int kPlaceTokens = 4;  // a thread's, one after another

// The places of the tokens behind each request's first one.  While the launch
// before runs, a block finds the requests that its tokens belong to.
__global__ void __launch_bounds__(kPlaceThreads) places_kernel(const PagesParams p) {
  constexpr int kBlockTokens = kPlaceThreads * kPlaceTokens;
  __shared__ int counts[2];  // ranges that begin at or before the block's first and last token
  if (threadIdx.x < 2) counts[threadIdx.x] = 0;
  __syncthreads();
  const int64_t block_t0 = (int64_t)blockIdx.x * kBlockTokens;
  int n[2] = {0, 0};
  for (int b = threadIdx.x; b <= p.batch; b += kPlaceThreads) {
    const int at = p.batch ? p.indptr[b] : 0;
    n[0] += at <= block_t0;
    n[1] += at < block_t0 + kBlockTokens;
  }
  for (int i = 0; i < 2; ++i) {
    const int sum = __reduce_add_sync(0xffffffffu, n[i]);
    if (threadIdx.x % 32 == 0 && sum) atomicAdd(counts + i, sum);
  }
  __syncthreads();
  const int b0 = max(counts[0] - 1, 0), near = max(counts[1], b0 + 1) - b0;
  grid_wait_prerequisites();
  const bool wrong = __ldcg(p.status + PKC_ASSIGN_FLAG) != 0;  // (or no requests at all)
  const int64_t t0 = block_t0 + threadIdx.x * kPlaceTokens;
  if (t0 >= p.total) return;
  const int t1 = (int)min((int64_t)p.total, t0 + kPlaceTokens);
  const int begin = wrong ? p.total : p.indptr[0], end = wrong ? p.total : p.indptr[p.batch];
  int b = -1, from = 0, to = 0, len = 0;  // the request of the tokens [from, to)
  int entry = -1, page = 0;               // the table entry at hand
  bool served = false;
  for (int t = (int)t0; t < t1; ++t) {
    if (t < begin || t >= end) {
      p.slots[t] = -1;
      p.positions[t] = 0;
      continue;
    }
    if (b < 0 || t >= to) {
      if (b < 0) b = b0 + last_not_above(p.indptr + b0, near, t);
      else do ++b; while (p.indptr[b + 1] <= t);
      from = p.indptr[b];
      to = p.indptr[b + 1];
      served = __ldcg(p.slots + from) >= 0;
      len = __ldcg(p.positions + from);
      entry = -1;
    }
    if (t == from) continue;
    const int pos = len + (t - from);
    int64_t slot = -1;
    if (served) {
      const int e = pos / p.page_size;
      if (e != entry) page = __ldcg(p.block_table + (int64_t)b * p.bt_stride + e);
      entry = e;
      slot = (int64_t)page * p.page_size + (pos - e * p.page_size);
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

constexpr int kReleaseThreads = 128;
constexpr int kReleaseEntries = 8;  // a thread's, loaded together

// Entries behind the used ones become -1 and their pages' bits are set (a
// commutative update: any order gives the same map).  Blocks: (entries, requests).
__global__ void __launch_bounds__(kReleaseThreads) release_pages_kernel(const PagesParams p) {
  const int b = blockIdx.y, len = p.cache_seqlens[b];
  const int64_t lo = (int64_t)blockIdx.x * (kReleaseThreads * kReleaseEntries) + threadIdx.x;
  if (len < 0) {
    if (lo == 0) report(p.status, PKC_ERR_PLAN);
    return;
  }
  const int64_t used = pages_of(p, (uint32_t)len);
  int32_t* row = p.block_table + (int64_t)b * p.bt_stride;
  int pages[kReleaseEntries];
#pragma unroll
  for (int i = 0; i < kReleaseEntries; ++i) {
    const int64_t j = lo + i * kReleaseThreads;
    pages[i] = j >= used && j < p.bt_stride ? row[j] : -1;
  }
#pragma unroll
  for (int i = 0; i < kReleaseEntries; ++i) {
    const int page = pages[i];
    if (page < 0) continue;
    if (page >= p.num_pages) {
      report(p.status, PKC_ERR_BLOCK_TABLE);
      continue;
    }
    row[lo + i * kReleaseThreads] = -1;
    const uint32_t bit = 1u << (page & 31);
    if (atomicOr(p.free_pages + (page >> 5), bit) & bit) report(p.status, PKC_ERR_BLOCK_TABLE);
  }
}

}  // namespace

int launch_release_pages(const PagesParams& p, void* stream) {
  if (p.batch <= 0) return 0;
  const int64_t per = kReleaseThreads * kReleaseEntries;
  static_assert(PKC_PAGES_MAX_BATCH <= 65535, "grid.y");
  release_pages_kernel<<<dim3((unsigned)((p.bt_stride + per - 1) / per), p.batch), kReleaseThreads, 0, (cudaStream_t)stream>>>(p);
  return (int)cudaGetLastError();
}

template <bool kAll>
static int launch_assign(const PagesParams& p, int blocks, int smem, void* stream) {
  static std::atomic<uint64_t> raised{0};
  constexpr int kMost = 4 * (3 * PKC_PAGES_MAX_BATCH + 2 + kMaxChunks + 1);
  if (const int e = raise_smem_limit((const void*)assign_pages_kernel<kAll>, kMost, raised)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, assign_pages_kernel<kAll>, p);
}

int launch_assign_pages(const PagesParams& p, void* stream) {
  if (p.batch <= 0 && p.total <= 0) return 0;
  PagesParams q = p;
  if (q.batch == 0) q.num_pages = 0;  // rows of no request alone: neither ranges nor map are read (they may be NULL)
  const int64_t words = (q.num_pages + 31) / 32;
  q.split = words <= 65536 ? 8 : 1;  // (the chunks' counts have to fit in shared memory)
  const int chunks = (int)((words + kThreads / q.split - 1) / (kThreads / q.split));
  const int smem = 4 * (3 * p.batch + 2 + chunks + 1);
  const bool all = p.total <= kFewTokens;
  // a block per 4096 tokens or per kThreads words of the map, whichever are more
  const int64_t parts = std::max<int64_t>(all ? ((int64_t)p.total + 4095) / 4096 : 1, (words + kThreads - 1) / kThreads);
  int blocks = 1;
  while (blocks < kMaxCluster && blocks < parts) blocks *= 2;
  if (all) return launch_assign<true>(q, blocks, smem, stream);
  if (const int e = launch_assign<false>(q, blocks, smem, stream)) return e;
  const int per = kPlaceThreads * kPlaceTokens;
  return launch_programmatic(places_kernel, dim3((unsigned)(((int64_t)p.total + per - 1) / per)), dim3(kPlaceThreads), 0,
                             (cudaStream_t)stream, p);
}

}  // namespace pkc
