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
// assign: one launch of one cluster, for all of it is a chain of scans
// (lengths, map) with a few bytes behind it.  Every block scans the lengths and
// counts the map for itself (both small, from L2); the map's chunks and the
// tokens are shared out over the blocks, with a cluster barrier before the map
// changes and one before the tokens read the table.
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

__global__ void __launch_bounds__(kThreads, 1) assign_pages_kernel(const PagesParams p) {
  extern __shared__ int smem[];
  int* off = smem;                       // [batch + 1] pages needed by the requests before b
  int* start = off + p.batch + 1;        // [batch + 1] new_indptr
  int* ends = start + p.batch + 1;       // [batch] length with the new tokens, -1: not served for its own sake
  int* chunk_base = ends + p.batch;      // [chunks + 1] free pages before each chunk of the map
  __shared__ int sums[kWarps + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int n_blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  const bool first_block = rank == 0;

  // The ranges have to run upwards within 0 .. total, or nobody is served.
  bool wrong = false;
  for (int b = tid; b <= p.batch; b += kThreads) {
    const int t = p.batch ? p.indptr[b] : 0;
    start[b] = t;
    wrong = wrong || t < 0 || t > p.total || (b > 0 && t < p.indptr[b - 1]);
  }
  wrong = __syncthreads_or(wrong);
  if (wrong && first_block && tid == 0) report(p.status, PKC_ERR_PLAN);

  // What each request needs, and the sum of those before it.
  int needed = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int need = 0;
    if (b < p.batch) {
      const int len = p.cache_seqlens[b], n = wrong ? 0 : start[b + 1] - start[b];
      const int64_t end = (int64_t)len + n;
      const int64_t have = ((int64_t)len + p.page_size - 1) / p.page_size;
      const int64_t want = (end + p.page_size - 1) / p.page_size;
      bool ok = len >= 0 && !wrong;
      if (ok && n > 0) {
        ok = want <= p.bt_stride;
        if (ok && len % p.page_size != 0) {  // the new tokens begin in a page that is there
          const int page = p.block_table[(int64_t)b * p.bt_stride + have - 1];
          ok = page >= 0 && page < p.num_pages;
        }
      }
      if (!ok && !wrong && (len < 0 || n > 0) && first_block) report(p.status, PKC_ERR_BLOCK_TABLE);
      ends[b] = ok ? (int)end : -1;
      if (ok) need = (int)(want - have);
    }
    int total;
    const int before = block_scan(need, sums, total);
    if (b < p.batch) off[b] = sat_add(needed, before);
    needed = sat_add(needed, total);
  }
  if (tid == 0) off[p.batch] = needed;

  // Free pages before each chunk of kThreads words.
  const int64_t words = (p.num_pages + 31) / 32;
  const int chunks = (int)((words + kThreads - 1) / kThreads);
  int n_free = 0;
  if (needed > 0) {  // uniform
    for (int c = 0; c < chunks; ++c) {
      if (tid == 0) chunk_base[c] = n_free;
      int total;
      block_scan(__popc(free_word(p, (int64_t)c * kThreads + tid, words)), sums, total);
      n_free += total;
    }
  }
  // Requests are served while the pages last; off does not descend, so the
  // first that does not fit ends it for all that need a page.
  __syncthreads();
  int taken = needed;
  if (needed > n_free) {  // uniform
    taken = off[last_not_above(off, p.batch + 1, n_free)];
    if (first_block && tid == 0) report(p.status, PKC_ERR_NO_PAGES);
  }
  cluster.sync();  // every block has read the map

  // The taken pages to the table, their bits cleared.
  for (int c = rank; c < chunks && taken > 0; c += n_blocks) {
    if (chunk_base[c] >= taken) break;  // uniform
    const int64_t w = (int64_t)c * kThreads + tid;
    const uint32_t x = free_word(p, w, words);
    int total;
    int r = chunk_base[c] + block_scan(__popc(x), sums, total);
    uint32_t gone = 0;
    if (x && r < taken) {
      int b = last_not_above(off, p.batch + 1, r);
      for (uint32_t y = x; y && r < taken; y &= y - 1, ++r) {
        const int bit = __ffs(y) - 1;
        while (off[b + 1] <= r) ++b;
        const int have = (int)(((int64_t)p.cache_seqlens[b] + p.page_size - 1) / p.page_size);
        p.block_table[(int64_t)b * p.bt_stride + have + (r - off[b])] = (int)(32 * w) + bit;
        gone |= 1u << bit;
      }
      p.free_pages[w] &= ~gone;
    }
  }
  __threadfence();
  cluster.sync();  // the table is complete

  // Where every token goes, and the lengths.
  for (int t = rank * kThreads + tid; t < p.total; t += n_blocks * kThreads) {
    int64_t slot = -1;
    int pos = 0;
    if (!wrong && p.batch && t >= start[0] && t < start[p.batch]) {
      const int b = last_not_above(start, p.batch + 1, t);
      const int end = ends[b];
      pos = p.cache_seqlens[b] + (t - start[b]);
      if (end >= 0 && (off[b + 1] <= taken || off[b + 1] == off[b]))
        slot = (int64_t)__ldcg(p.block_table + (int64_t)b * p.bt_stride + pos / p.page_size) * p.page_size +
               pos % p.page_size;
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  cluster.sync();  // the lengths have been read: they may be the ones that grow
  if (first_block && p.seqlens_out)
    for (int b = tid; b < p.batch; b += kThreads) {
      const bool served = ends[b] >= 0 && (off[b + 1] <= taken || off[b + 1] == off[b]);
      p.seqlens_out[b] = served ? ends[b] : p.cache_seqlens[b];
    }
}

constexpr int kReleaseThreads = 256;
constexpr int kSegment = 1024;  // table entries of a warp's turn

// A warp per segment of a table row: entries behind the used ones become -1
// and their pages' bits are set (a commutative update: any order gives the
// same map).
__global__ void __launch_bounds__(kReleaseThreads) release_pages_kernel(const PagesParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t segs = (p.bt_stride + kSegment - 1) / kSegment;
  const int64_t units = segs * p.batch, n_warps = (int64_t)gridDim.x * (kReleaseThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kReleaseThreads / 32) + (threadIdx.x >> 5); u < units; u += n_warps) {
    const int64_t b = u / segs, lo = (u - b * segs) * kSegment;
    const int len = p.cache_seqlens[b];
    if (len < 0) {
      if (lane == 0) report(p.status, PKC_ERR_PLAN);
      continue;
    }
    const int64_t used = ((int64_t)len + p.page_size - 1) / p.page_size;
    const int64_t hi = min(p.bt_stride, lo + kSegment);
    int32_t* row = p.block_table + b * p.bt_stride;
    for (int64_t j = max(lo, used) + lane; j < hi; j += 32) {
      const int page = row[j];
      if (page < 0) continue;
      if (page >= p.num_pages) {
        report(p.status, PKC_ERR_BLOCK_TABLE);
        continue;
      }
      row[j] = -1;
      const uint32_t bit = 1u << (page & 31);
      if (atomicOr(p.free_pages + (page >> 5), bit) & bit) report(p.status, PKC_ERR_BLOCK_TABLE);
    }
  }
}

}  // namespace

int launch_release_pages(const PagesParams& p, void* stream) {
  if (p.batch <= 0) return 0;
  const int64_t units = (p.bt_stride + kSegment - 1) / kSegment * p.batch;
  const int64_t want = (units + kReleaseThreads / 32 - 1) / (kReleaseThreads / 32);
  const int64_t most = (int64_t)num_sms() * (2048 / kReleaseThreads);
  release_pages_kernel<<<(unsigned)std::min(want, most), kReleaseThreads, 0, (cudaStream_t)stream>>>(p);
  return (int)cudaGetLastError();
}

int launch_assign_pages(const PagesParams& p, void* stream) {
  if (p.batch <= 0 && p.total <= 0) return 0;
  static std::atomic<uint64_t> raised{0};
  constexpr int kMost = 4 * (3 * PKC_PAGES_MAX_BATCH + 2 + kMaxChunks + 1);
  if (const int e = raise_smem_limit((const void*)assign_pages_kernel, kMost, raised)) return e;
  const int64_t words = (p.num_pages + 31) / 32;
  const int chunks = (int)((words + kThreads - 1) / kThreads);
  // A block per 4096 tokens or per chunk of the map, whichever are more, in
  // one cluster.
  const int64_t parts = std::max<int64_t>(((int64_t)p.total + 4095) / 4096, chunks);
  int blocks = 1;
  while (blocks < kMaxCluster && blocks < parts) blocks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 4 * (size_t)(3 * p.batch + 2 + chunks + 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, assign_pages_kernel, p);
}

}  // namespace pkc
