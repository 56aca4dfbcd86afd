// Eviction from a paged cache: which tokens a request keeps, and the move of
// the kept ones to the front of its pages.
//
// Select.  Per (request, KV head) the kept slots are the first `sinks`, the
// last `recent`, and of those between the m = budget - sinks - recent with
// the largest accumulated weights, the lower slot of equal ones.  A weight's
// bits become an unsigned key in the same order (NaN above infinity, the
// two zeros equal), and the m-th largest key T is found digit by digit from
// the top (11 + 11 + 10 bits): a histogram of the keys that agree with the
// digits found so far, and the bin in which the count from above reaches m.
// One more pass over the keys, in order, gives each kept slot its rank.  The
// weights are read from memory once, into shared memory; a row is worked on
// by a cluster of up to 8 blocks, which add up their histograms through
// distributed shared memory, so that few long rows use the machine too.
// What bounds it is the chain of passes and barriers per row, not HBM.
//
// Compact.  Row j of a (request, head) becomes row keep[j]; keep ascends
// strictly, so keep[j] >= j.  A block moves one slice of one head's K or V
// rows, chunk after chunk of new slots in order, each chunk in registers
// before any of it is written.  The next chunk's rows lie at or behind its
// own first slot, where nothing has been written yet, so its loads are in
// flight while the current chunk is stored.  Bound by HBM: a kept row is
// read once and written once.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "mx4.cuh"

namespace cg = cooperative_groups;

namespace pkc {
namespace {

// ---------------------------------------------------------------------------
// Select
// ---------------------------------------------------------------------------

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr uint32_t kZeroKey = 0x80000000u;  // the key of weight 0

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct SelectShared {
  int warp_sum[kSelWarps];
  int gt[kSelWarps], eq[kSelWarps];
  int cta_gt, cta_eq;
  int bin, rest;
};
static_assert(sizeof(SelectShared) % 16 == 0, "what follows is read 16 bytes at a time");

// Shared memory: SelectShared, one histogram (two, alternating, when several
// blocks share a row: then one cluster barrier per digit is enough), keys.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_sel[];
  SelectShared& S = *reinterpret_cast<SelectShared*>(smem_sel);
  uint32_t* hists = reinterpret_cast<uint32_t*>(smem_sel + sizeof(SelectShared));
  const int n_cta = p.cluster, n_hist = n_cta > 1 ? 2 : 1;
  uint32_t* keys = hists + n_hist * kBins;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)(blockIdx.x % n_cta);
  const int row = (int)(blockIdx.x / n_cta), b = row / p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* keep = p.keep + (int64_t)row * p.budget;
  const float* w = p.weights + (int64_t)row * p.w_stride;
  int len = p.cache_seqlens[b];
  const int at = rank * kSelThreads + tid, all = n_cta * kSelThreads;  // this thread in the row's cluster

  if (len > p.w_stride) {  // (uniform over the cluster, as every early return)
    if (at == 0) report(p.status, PKC_ERR_PLAN);
    len = 0;
  }
  if (len <= p.budget) {
    for (int j = at; j < p.budget; j += all) keep[j] = j < len ? j : -1;
    return;
  }
  const int n = len - p.sinks - p.recent;       // slots to choose from
  const int m = p.budget - p.sinks - p.recent;  // slots to choose, m < n
  for (int j = at; j < p.sinks; j += all) keep[j] = j;
  for (int j = at; j < p.recent; j += all) keep[p.budget - p.recent + j] = len - p.recent + j;
  if (m == 0) return;

  // This block's part of the choice: keys [lo, lo + mine).  In shared memory
  // it is padded to whole groups of 4 with key 0, which no weight has but a
  // negative NaN's bits (order_key gives NaN the largest): never chosen.
  const int per = (n + n_cta - 1) / n_cta;
  const int lo = min(rank * per, n), mine = min(per, n - lo);
  const bool cached = mine <= p.smem_keys;
  const float* src = w + p.sinks + lo;
  const int quads = (mine + 3) >> 2;
  auto quad_at = [&](int q) -> uint4 {  // keys 4 q .. 4 q + 3
    if (cached) return *reinterpret_cast<const uint4*>(keys + 4 * q);
    uint32_t k[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) k[x] = 4 * q + x < mine ? order_key(src[4 * q + x]) : 0u;
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  for (int i = tid; i < n_hist * kBins; i += kSelThreads) hists[i] = 0;
  __syncthreads();

  // First digit, as the keys come in.  Weights that are exactly 0 are often
  // most of a row: each warp counts them apart, so they do not queue up on
  // one bin.
  int zeros = 0;
#pragma unroll 8
  for (int i0 = warp * 32; i0 < 4 * quads; i0 += kSelThreads) {
    const int i = i0 + lane;
    const uint32_t k = i < mine ? order_key(__ldcs(src + i)) : 0u;
    if (cached && i < 4 * quads) keys[i] = k;
    zeros += __popc(__ballot_sync(0xffffffffu, k == kZeroKey));
    if (i < mine && k != kZeroKey) atomicAdd(&hists[k >> 21], 1u);
  }
  if (lane == 0 && zeros) atomicAdd(&hists[kZeroKey >> 21], (uint32_t)zeros);

  uint32_t prefix = 0;  // digits found, in place
  int rest = m;         // to be chosen among the keys that agree with them
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, width = d == 2 ? 10 : 11;
    uint32_t* hist = hists + (n_cta > 1 ? (d & 1) * kBins : 0);
    if (d > 0) {
      const uint32_t want = prefix >> (shift + width), mask = (1u << width) - 1u;
      if (!cached) __syncthreads();
      for (int q = tid; q < quads; q += kSelThreads) {
        const uint4 k4 = quad_at(q);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if ((k[x] >> (shift + width)) == want && k[x] != kZeroKey) atomicAdd(&hist[(k[x] >> shift) & mask], 1u);
      }
      if (lane == 0 && zeros && (kZeroKey >> (shift + width)) == want)
        atomicAdd(&hist[(kZeroKey >> shift) & mask], (uint32_t)zeros);
    }
    if (n_cta > 1) cluster.sync();  // every block's histogram is complete
    else __syncthreads();
    // Counts of this thread's four bins, from the top: thread 0 has the highest.
    const int bin0 = kBins - 4 - 4 * tid;
    uint4 cnt = *reinterpret_cast<const uint4*>(hist + bin0);
    if (n_cta > 1) {
      uint4 c[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        c[x] = make_uint4(0, 0, 0, 0);
        if (x < n_cta && x != rank)
          c[x] = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(hist, x) + bin0);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        cnt.x += c[x].x; cnt.y += c[x].y; cnt.z += c[x].z; cnt.w += c[x].w;
      }
    }
    const int sum = (int)(cnt.x + cnt.y + cnt.z + cnt.w);
    int above = sum;  // inclusive scan over the block
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, above, x);
      if (lane >= x) above += y;
    }
    if (lane == 31) S.warp_sum[warp] = above;
    if (tid == 0) {  // (replaced below, unless the weights change under the kernel)
      S.bin = 0;
      S.rest = rest;
    }
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int x = 0; x < kSelWarps; ++x) before += x < warp ? S.warp_sum[x] : 0;
    above += before - sum;  // keys in higher bins than this thread's
    if (above < rest && rest <= above + sum) {  // exactly one thread
      const int c[4] = {(int)cnt.w, (int)cnt.z, (int)cnt.y, (int)cnt.x};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (above < rest && rest <= above + c[x]) {
          S.bin = bin0 + 3 - x;
          S.rest = rest - above;
        }
        above += c[x];
      }
    }
    // The next digit's histogram: with one, this; with two, the one before,
    // which every block is past at this digit's barrier.
    if (d < 2 && (n_cta == 1 || d == 1))
      for (int i = tid; i < kBins; i += kSelThreads) hists[i] = 0;
    __syncthreads();
    prefix |= (uint32_t)S.bin << shift;
    rest = S.rest;
    __syncthreads();
  }
  // Keys above T = prefix are kept, and the first `rest` of those equal to it.
  // Each warp takes a consecutive part: counts, then ranks.
  const int part = (quads + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;  // in groups of 4
  const int w_lo = min(warp * part, quads), w_hi = min(w_lo + part, quads);
  int gt = 0, eq = 0;
  for (int q = w_lo + lane; q < w_hi; q += 32) {
    const uint4 k = quad_at(q);
    gt += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
    eq += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    S.gt[warp] = gt;
    S.eq[warp] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;  // before this warp's part
  for (int x = 0; x < warp; ++x) {
    gt0 += S.gt[x];
    eq0 += S.eq[x];
  }
  if (n_cta > 1) {
    if (tid == kSelThreads - 1) {
      S.cta_gt = gt0 + gt;
      S.cta_eq = eq0 + eq;
    }
    cluster.sync();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c < rank) {
        const SelectShared* o = cluster.map_shared_rank(&S, c);
        gt0 += o->cta_gt;
        eq0 += o->cta_eq;
      }
    }
  }
  for (int q0 = w_lo; q0 < w_hi; q0 += 32) {
    const int q = q0 + lane;
    const uint4 k4 = q < w_hi ? quad_at(q) : make_uint4(0, 0, 0, 0);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    int g = 0, e = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      g += k[x] > prefix;
      e += q < w_hi && k[x] == prefix;
    }
    int scan = g | (e << 16);  // both counts of at most 128
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, x);
      if (lane >= x) scan += y;
    }
    const int total = __shfl_sync(0xffffffffu, scan, 31);
    int gr = gt0 + (scan & 0xffff) - g, er = eq0 + (scan >> 16) - e;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const bool is_gt = k[x] > prefix, is_eq = q < w_hi && k[x] == prefix;
      const int rank_of = gr + min(er, rest);  // (below m, unless the weights change under the kernel)
      if ((is_gt || (is_eq && er < rest)) && rank_of < m) keep[p.sinks + rank_of] = p.sinks + lo + 4 * q + x;
      gr += is_gt;
      er += is_eq;
    }
    gt0 += total & 0xffff;
    eq0 += total >> 16;
  }
  if (n_cta > 1) cluster.sync();  // no block leaves while another reads its counts
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 2;  // rows per thread and chunk (two chunks in registers)

__device__ __forceinline__ uint4 load_cg(const uint4* p) { return __ldcg(p); }
__device__ __forceinline__ uint32_t load_cg(const uint32_t* p) { return __ldcg(p); }

// Move rows keep[j] -> j, j < n, in units of V (one unit of a row per
// thread): place(slot) is a slot's place, at(place) this thread's unit of it,
// `row` the thread's row within a pass of `rows` rows.  Called by a whole
// block.  A chunk is kMoveRows passes.  While chunk c is stored, the rows of
// chunk c + 1 are on their way, the places of chunk c + 2 and the slots of
// chunk c + 3.
template <typename V, typename Place, typename At>
__device__ __forceinline__ void move_rows(const int32_t* keep, int n, int row, int rows, Place place, At at) {
  const int chunk = rows * kMoveRows;
  V buf[2][kMoveRows];
  int32_t slot[kMoveRows];                  // chunk c + 3's slots (-1 past the end)
  uint32_t from[kMoveRows], to[kMoveRows];  // chunk c + 2's places
  auto load_slots = [&](int c) {
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int j = c + u * rows + row;
      slot[u] = j < n ? keep[j] : -1;
    }
  };
  auto load_places = [&](int c) {
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int j = c + u * rows + row;
      from[u] = to[u] = 0;
      if (slot[u] >= 0) {
        from[u] = place(slot[u]);
        to[u] = place(j);
      }
    }
  };
  auto load = [&](V (&x)[kMoveRows], uint32_t (&dst)[kMoveRows]) {  // (from == to: nothing to move)
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const bool moves = from[u] != to[u];
      dst[u] = moves ? to[u] : kNoToken;
      if (moves) x[u] = load_cg(at(from[u]));
    }
  };
  auto store = [&](const V (&x)[kMoveRows], const uint32_t (&dst)[kMoveRows]) {
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
      if (dst[u] != kNoToken) *at(dst[u]) = x[u];
  };
  uint32_t dst[2][kMoveRows];
  load_slots(0);
  load_places(0);
  load_slots(chunk);
  load(buf[0], dst[0]);
  load_places(chunk);
  load_slots(2 * chunk);
  for (int c = 0; c < n; c += 2 * chunk) {
    load(buf[1], dst[1]);
    load_places(c + 2 * chunk);
    load_slots(c + 3 * chunk);
    __syncthreads();  // chunk c has been read by every thread
    store(buf[0], dst[0]);
    if (c + chunk >= n) break;
    load(buf[0], dst[0]);
    load_places(c + 3 * chunk);
    load_slots(c + 4 * chunk);
    __syncthreads();
    store(buf[1], dst[1]);
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactParams p) {
  const int part = (int)(blockIdx.x % p.parts);
  const int row = (int)(blockIdx.x / p.parts), b = row / p.hkv, h = row % p.hkv;
  const int tid = threadIdx.x;
  const int len = p.cache_seqlens[b], n = p.budget;
  bool bad_page = false;
  if (len > n) {
    const int32_t* keep = p.keep + (int64_t)row * n;
    const int32_t* bt_row = p.block_table + (int64_t)b * p.bt_stride;
    const PageDiv pages{p.page_size, p.page_shift};
    // Every page of the request must be there, and the row of kept slots
    // ascend within its length; else nothing of it moves.
    const int64_t n_pages = ((int64_t)len + p.page_size - 1) / p.page_size;
    bad_page = n_pages > p.bt_stride;
    if (!bad_page)
      for (int64_t i = tid; i < n_pages; i += kMoveThreads) {
        const int32_t id = bt_row[i];
        bad_page = bad_page || id < 0 || id >= p.num_pages;
      }
    bool bad_keep = p.weights && len > p.w_stride;
    for (int j = tid; j < n; j += kMoveThreads) {
      const int32_t k = keep[j];
      bad_keep = bad_keep || k < (j > 0 ? keep[j - 1] + 1 : 0) || k >= len;
    }
    bad_page = __syncthreads_or(bad_page);
    bad_keep = __syncthreads_or(bad_keep);
    if (bad_page || bad_keep) {
      if (tid == 0) report(p.status, bad_page ? PKC_ERR_BLOCK_TABLE : PKC_ERR_PLAN);
    } else {
      // (strictly ascending and >= 0: keep[j] >= j)
      auto token = [&](int slot) {  // a slot's pool index
        int page, x;
        pages.split(slot, page, x);
        return (uint32_t)bt_row[page] * (uint32_t)p.page_size + (uint32_t)x;
      };
      if (part < 2 * p.slices) {  // a slice of K's or V's rows
        const int units = p.row_bytes / 16 / p.slices;  // 16-byte units of a row in the slice
        uint8_t* base = static_cast<uint8_t*>(part & 1 ? p.v_cache : p.k_cache) + (int64_t)h * p.row_bytes +
                        16 * ((part >> 1) * units + tid % units);
        const uint32_t stride = (uint32_t)p.hkv * (uint32_t)p.row_bytes;
        move_rows<uint4>(keep, n, tid / units, kMoveThreads / units, token, [&](uint32_t t) {
          return reinterpret_cast<uint4*>(const_cast<uint8_t*>(at_row(base, t, stride)));
        });
      } else if (part < 2 * p.slices + (p.k_scales ? 2 : 0)) {  // mx4 scales: 4 bytes a row
        uint32_t* base = static_cast<uint32_t*>((part - 2 * p.slices) ? p.v_scales : p.k_scales) + h;
        move_rows<uint32_t>(keep, n, tid, kMoveThreads, token, [&](uint32_t t) { return base + (int64_t)t * p.hkv; });
      } else {  // weights: the kept ones, zeros behind them
        uint32_t* w = reinterpret_cast<uint32_t*>(p.weights) + (int64_t)row * p.w_stride;
        move_rows<uint32_t>(keep, n, tid, kMoveThreads, [](int slot) { return (uint32_t)slot; },
                            [&](uint32_t t) { return w + t; });
        __syncthreads();
        for (int j = n + tid; j < len; j += kMoveThreads) w[j] = 0u;
      }
    }
  }
  // The lengths shrink once every block has read them: by the block that
  // finishes last, which also resets the counter for the next launch.
  int32_t* ctr = p.status + PKC_COMPACT_COUNTER;
  __shared__ int last, any_bad;
  if (bad_page && tid == 0) atomicExch(ctr + 1, 1);
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(ctr, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (tid == 0) {
    any_bad = atomicExch(ctr + 1, 0);
    atomicExch(ctr, 0);
  }
  __syncthreads();
  for (int r = tid; r < p.batch; r += kMoveThreads) {
    const int l = p.cache_seqlens[r];
    if (l <= n) continue;
    bool ok = true;
    if (any_bad) {  // a request with a missing page keeps its length
      const int64_t n_pages = ((int64_t)l + p.page_size - 1) / p.page_size;
      ok = n_pages <= p.bt_stride;
      for (int64_t i = 0; ok && i < n_pages; ++i) {
        const int32_t id = p.block_table[(int64_t)r * p.bt_stride + i];
        ok = id >= 0 && id < p.num_pages;
      }
    }
    if (ok) p.cache_seqlens[r] = n;
  }
}

}  // namespace

int launch_evict_select(const SelectParams& p_in, void* stream) {
  SelectParams p = p_in;
  const int64_t rows = (int64_t)p.batch * p.hkv;
  if (rows <= 0) return 0;
  // Blocks per row: doubled while the machine has room for them and each
  // still has 2048 keys of the longest row.
  p.cluster = 1;
  while (p.cluster < 8 && rows * p.cluster * 2 <= num_sms() && p.w_stride / (2 * p.cluster) >= 2048) p.cluster *= 2;
  const int64_t per = (p.w_stride + p.cluster - 1) / p.cluster;
  p.smem_keys = (int)std::min<int64_t>((per + 3) & ~int64_t(3), 48 * 1024);
  const int smem = (int)sizeof(SelectShared) + 4 * kBins * (p.cluster > 1 ? 2 : 1) + 4 * p.smem_keys;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return (int)e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * p.cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeClusterDimension;
  la[0].val.clusterDim.x = (unsigned)p.cluster;
  la[0].val.clusterDim.y = la[0].val.clusterDim.z = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

int launch_evict_compact(const CompactParams& p_in, void* stream) {
  CompactParams p = p_in;
  const int64_t rows = (int64_t)p.batch * p.hkv;
  if (rows <= 0) return 0;
  // Whole rows per block while that fills the machine (8 blocks per SM);
  // else slices of a row, down to a 32-byte sector.
  p.slices = 1;
  while (p.row_bytes / p.slices > 32 && rows * 2 * p.slices < 8 * (int64_t)num_sms()) p.slices *= 2;
  p.parts = 2 * p.slices + (p.k_scales ? 2 : 0) + (p.weights ? 1 : 0);
  if (rows * p.parts > INT32_MAX) return (int)cudaErrorInvalidValue;
  evict_compact_kernel<<<(unsigned)(rows * p.parts), kMoveThreads, 0, (cudaStream_t)stream>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace pkc
