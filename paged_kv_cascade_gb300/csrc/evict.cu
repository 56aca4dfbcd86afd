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
// The first histogram reads the weights from memory; a second read (L2) sets
// a bit for every key above the bin and lists the keys in it, a percent or
// so, on which the other digits work (they read the weights again if the
// list is too short, as for a row of equal weights).  Then the bits of the
// kept slots are ranked: a thread per 32 of them, one scan.  A row takes
// 512 threads of 40 registers and about 30 KB of shared memory, so three
// blocks share an SM; a cluster of up to 8 blocks works on one row where
// there are few, adding up their histograms through distributed shared
// memory.  What bounds it is the chain of reads and barriers per row, not
// HBM: 29 us for 512 rows of 1024 to 16384 weights (one read of them at the
// copy rate would be 3), 22 us for 8 rows of 131,056 on 64 blocks.
//
// Compact.  Row j of a (request, head) becomes row keep[j]; keep ascends
// strictly, so keep[j] >= j.  A block moves one slice of one head's K or V
// rows, chunk after chunk of new slots in order, each chunk in registers
// before any of it is written.  The next chunk's rows lie at or behind its
// own first slot, where nothing has been written yet, so its loads are in
// flight while the current chunk is stored.  Bound by HBM: a kept row is
// read once and written once, 256 bytes at a random slot: 116 us for 64
// requests cut to 1024 of up to 6144 tokens, 8 heads of bf16 (549 MB, 4.7
// TB/s of a measured copy rate of 6.8).  Two rows a thread and chunk: four
// take 126 us, eight 137, for want of resident blocks.
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
constexpr int kBins = 4 * kSelThreads;  // (of 11 bits: four per thread where a digit's bin is looked for)
static_assert(kBins == 2048, "digits of 11 bits");
constexpr int kBatch = 8;                    // keys a thread has in flight
constexpr int kListed = 1536;                // keys of a digit's bin that a block lists
constexpr int kMostKeys = 1 << 19;           // keys of one block (two bits each in shared memory)
constexpr int kMostHeld = 32 * 1024;         // keys of one block held in shared memory
constexpr uint32_t kZeroKey = 0x80000000u;   // the key of weight 0

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct SelectShared {
  uint32_t hist[2][kBins];     // alternate between digits: one barrier per digit
  uint2 list[kListed];         // (key, index) of the first digit's bin
  int warp_sum[kSelWarps];
  int cta_gt, cta_eq;
  int bin, rest, n_listed;
  int pad[3];
};

// Shared memory: SelectShared, then two bits per key (kept for certain; equal
// to T), then the keys where there are no more rows than SMs: those rows are
// read once, as a block has an SM to itself (8 rows of 131072: 24 -> 22 us),
// while in a batch more blocks per SM are worth more (512 rows: 28 against
// 31 us).
__global__ void __launch_bounds__(kSelThreads, 3) evict_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_sel[];
  SelectShared& S = *reinterpret_cast<SelectShared*>(smem_sel);
  cg::cluster_group cluster = cg::this_cluster();
  const int n_cta = p.cluster, rank = (int)(blockIdx.x % n_cta);
  const int row = (int)(blockIdx.x / n_cta), b = row / p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* keep = p.keep + (int64_t)row * p.budget;
  int len = p.cache_seqlens[b];

  if (len > p.w_stride) {  // (uniform over the cluster, as every early return)
    if (rank == 0 && tid == 0) report(p.status, PKC_ERR_PLAN);
    len = 0;
  }
  if (len <= p.budget) {
    for (int j = rank * kSelThreads + tid; j < p.budget; j += n_cta * kSelThreads) keep[j] = j < len ? j : -1;
    return;
  }
  const int n = len - p.sinks - p.recent;       // slots to choose from
  const int m = p.budget - p.sinks - p.recent;  // slots to choose, m < n
  for (int j = rank * kSelThreads + tid; j < p.sinks; j += n_cta * kSelThreads) keep[j] = j;
  for (int j = rank * kSelThreads + tid; j < p.recent; j += n_cta * kSelThreads)
    keep[p.budget - p.recent + j] = len - p.recent + j;
  if (m == 0) return;

  // This block's part of the choice: keys [lo, lo + mine), 32 to a word.
  const int per = ((n + n_cta - 1) / n_cta + 31) & ~31;
  const int lo = min(rank * per, n), mine = min(per, n - lo);
  const float* src = p.weights + (int64_t)row * p.w_stride + p.sinks + lo;
  const int words = (mine + 31) >> 5;
  uint32_t* sure = reinterpret_cast<uint32_t*>(smem_sel + sizeof(SelectShared));
  uint32_t* equal = sure + words;
  uint32_t* keys = equal + words;  // the keys themselves, where the launch gave them room
  const bool cached = mine <= p.smem_keys;
  for (int i = tid; i < 2 * kBins; i += kSelThreads) (&S.hist[0][0])[i] = 0;
  if (tid == 0) S.n_listed = 0;
  __syncthreads();

  // kBatch keys of this lane, a block's width apart, all loads in flight
  // together (a shared-memory atomic between two loads would hold the second
  // one back); 0, which no weight has, past the end.
  auto load_keys = [&](uint32_t (&k)[kBatch], int i, bool again) {
    if (again && cached) {
#pragma unroll
      for (int x = 0; x < kBatch; ++x) k[x] = i + x * kSelThreads < mine ? keys[i + x * kSelThreads] : 0u;
      return;
    }
    float f[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) f[x] = i + x * kSelThreads < mine ? src[i + x * kSelThreads] : 0.f;
#pragma unroll
    for (int x = 0; x < kBatch; ++x) k[x] = i + x * kSelThreads < mine ? order_key(f[x]) : 0u;
  };

  // First digit.  Weights that are exactly 0 are often most of a row: each
  // warp counts them apart, so they do not queue up on one bin.
  int zeros = 0;
  for (int i0 = warp * 32; i0 < mine; i0 += kBatch * kSelThreads) {
    uint32_t k[kBatch];
    load_keys(k, i0 + lane, false);
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      if (cached && k[x] != 0u) keys[i0 + lane + x * kSelThreads] = k[x];
      zeros += __popc(__ballot_sync(0xffffffffu, k[x] == kZeroKey));
      if (k[x] != 0u && k[x] != kZeroKey) atomicAdd(&S.hist[0][k[x] >> 21], 1u);
    }
  }
  if (lane == 0 && zeros) atomicAdd(&S.hist[0][kZeroKey >> 21], (uint32_t)zeros);

  uint32_t prefix = 0;  // digits found, in place
  int rest = m;         // to be chosen among the keys that agree with them
  bool listed = true;   // the list holds all keys of the first digit's bin
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, width = d == 2 ? 10 : 11;
    uint32_t* hist = S.hist[d & 1];
    const uint32_t want = d == 0 ? 0u : prefix >> (shift + width), mask = (1u << width) - 1u;
    if (d == 1) {  // the second read: bits of the keys above, list of the keys in the bin
      for (int w0 = warp; w0 < words; w0 += kBatch * kSelWarps) {
        uint32_t k[kBatch];
        load_keys(k, 32 * w0 + lane, true);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int wd = w0 + x * kSelWarps;
          const uint32_t top = k[x] >> 21;
          const uint32_t above = __ballot_sync(0xffffffffu, top > want);
          const uint32_t zero = __ballot_sync(0xffffffffu, k[x] == kZeroKey && top == want);
          if (lane == 0 && wd < words) {
            sure[wd] = above;
            equal[wd] = zero;
          }
          if (top == want && k[x] != 0u && k[x] != kZeroKey) {  // (zeros are counted already, and never listed)
            const int at = atomicAdd(&S.n_listed, 1);
            if (at < kListed) S.list[at] = make_uint2(k[x], (uint32_t)(32 * wd + lane));
            atomicAdd(&hist[(k[x] >> shift) & mask], 1u);
          }
        }
      }
      __syncthreads();
      listed = S.n_listed <= kListed;
    } else if (d == 2) {
      if (listed) {
        for (int i = tid; i < S.n_listed; i += kSelThreads) {
          const uint32_t k = S.list[i].x;
          if ((k >> (shift + width)) == want) atomicAdd(&hist[(k >> shift) & mask], 1u);
        }
      } else {
        for (int i = tid; i < mine; i += kSelThreads) {
          const uint32_t k = order_key(src[i]);
          if ((k >> (shift + width)) == want && k != kZeroKey) atomicAdd(&hist[(k >> shift) & mask], 1u);
        }
      }
    }
    if (d > 0 && lane == 0 && zeros && (kZeroKey >> (shift + width)) == want)
      atomicAdd(&hist[(kZeroKey >> shift) & mask], (uint32_t)zeros);
    if (n_cta > 1) cluster.sync();  // every block's histogram is complete
    else __syncthreads();
    // Counts of this thread's four bins, from the top: thread 0 has the highest.
    const int bin0 = kBins - 4 - 4 * tid;
    int cnt[4];
    {
      const uint4 x = *reinterpret_cast<const uint4*>(hist + bin0);
      cnt[0] = x.w; cnt[1] = x.z; cnt[2] = x.y; cnt[3] = x.x;
    }
    if (n_cta > 1) {
#pragma unroll
      for (int c0 = 0; c0 < 8; c0 += 4) {
        uint4 x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] = make_uint4(0, 0, 0, 0);
          if (c0 + c < n_cta && c0 + c != rank)
            x[c] = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(hist, c0 + c) + bin0);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          cnt[0] += x[c].w; cnt[1] += x[c].z; cnt[2] += x[c].y; cnt[3] += x[c].x;
        }
      }
    }
    const int sum = cnt[0] + cnt[1] + cnt[2] + cnt[3];
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
    above -= sum;  // keys in higher bins than this thread's
#pragma unroll
    for (int x = 0; x < kSelWarps; ++x) above += x < warp ? S.warp_sum[x] : 0;
    if (above < rest && rest <= above + sum) {  // exactly one thread
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (above < rest && rest <= above + cnt[x]) {
          S.bin = bin0 + 3 - x;
          S.rest = rest - above;
        }
        above += cnt[x];
      }
    }
    if (d == 1)  // the third digit's histogram is the first's: every block is past it
      for (int i = tid; i < kBins; i += kSelThreads) S.hist[0][i] = 0;
    __syncthreads();
    prefix |= (uint32_t)S.bin << shift;
    rest = S.rest;
  }
  // T = prefix.  Keys above T are kept, and the first `rest` of those equal
  // to it.  The bits so far: `sure` has the keys above the first digit's bin,
  // `equal` that bin's zeros; now the bin's other keys.
  if (listed) {
    if (prefix != kZeroKey) {
      for (int i = tid; i < words; i += kSelThreads) equal[i] = 0u;
      __syncthreads();
    }
    for (int i = tid; i < S.n_listed; i += kSelThreads) {
      const uint2 k = S.list[i];
      if (k.x > prefix) atomicOr(&sure[k.y >> 5], 1u << (k.y & 31));
      else if (k.x == prefix) atomicOr(&equal[k.y >> 5], 1u << (k.y & 31));
    }
  } else {
    for (int wd = warp; wd < words; wd += kSelWarps) {
      const int i = 32 * wd + lane;
      const uint32_t k = i < mine ? order_key(src[i]) : 0u;
      const uint32_t g = __ballot_sync(0xffffffffu, k > prefix), e = __ballot_sync(0xffffffffu, k == prefix && i < mine);
      if (lane == 0) {
        sure[wd] = g;
        equal[wd] = e;
      }
    }
  }
  __syncthreads();
  // Keys above and equal in the blocks before this one.
  int gt0 = 0, eq0 = 0;
  if (n_cta > 1) {
    int g = 0, e = 0;
    for (int i = tid; i < words; i += kSelThreads) {
      g += __popc(sure[i]);
      e += __popc(equal[i]);
    }
    g = __reduce_add_sync(0xffffffffu, g);
    e = __reduce_add_sync(0xffffffffu, e);
    if (tid == 0) S.cta_gt = S.cta_eq = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&S.cta_gt, g);
      atomicAdd(&S.cta_eq, e);
    }
    cluster.sync();
    for (int c = 0; c < rank; ++c) {
      const SelectShared* o = cluster.map_shared_rank(&S, c);
      gt0 += o->cta_gt;
      eq0 += o->cta_eq;
    }
  }
  // Ranks: a thread per word, 512 words at a time.
  for (int w0 = 0; w0 < words; w0 += kSelThreads) {
    const int wd = w0 + tid;
    const uint32_t s = wd < words ? sure[wd] : 0u;
    uint32_t x = wd < words ? equal[wd] : 0u;
    const int both = __popc(s) | (__popc(x) << 16);  // (512 words have at most 2^14 of each)
    int scan = both;
#pragma unroll
    for (int y = 1; y < 32; y <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, scan, y);
      if (lane >= y) scan += z;
    }
    if (lane == 31) S.warp_sum[warp] = scan;
    __syncthreads();
    int before = scan - both, total = 0;
#pragma unroll
    for (int y = 0; y < kSelWarps; ++y) {
      const int z = S.warp_sum[y];
      before += y < warp ? z : 0;
      total += z;
    }
    const int er = eq0 + (before >> 16);
    int pos = gt0 + (before & 0xffff) + min(er, rest);
    const int spare = (int)__popc(x) - max(min(rest - er, (int)__popc(x)), 0);  // equal ones not taken: the last
    for (int y = 0; y < spare; ++y) x ^= 0x80000000u >> __clz(x);
    for (uint32_t all = s | x; all != 0u; all &= all - 1u, ++pos)
      if (pos < m) keep[p.sinks + pos] = p.sinks + lo + 32 * wd + __ffs(all) - 1;  // (always, unless the weights change under the kernel)
    gt0 += total & 0xffff;
    eq0 += total >> 16;
    __syncthreads();  // warp_sum is free
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
  bool bad_request = false;
  if (len > n) {
    bool bad_page = false;
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
    // Of the whole request: weights shorter than it, or a head with too few
    // slots (as the select leaves it for a row too short, or a request that
    // was within the budget then).
    bool unchosen = p.weights && len > p.w_stride;
    for (int i = tid; i < p.hkv; i += kMoveThreads)
      unchosen = unchosen || p.keep[((int64_t)b * p.hkv + i + 1) * n - 1] < 0;
    bool bad_keep = unchosen;
    for (int j = tid; j < n; j += kMoveThreads) {
      const int32_t k = keep[j];
      bad_keep = bad_keep || k < (j > 0 ? keep[j - 1] + 1 : 0) || k >= len;
    }
    bad_page = __syncthreads_or(bad_page);
    bad_keep = __syncthreads_or(bad_keep);
    unchosen = __syncthreads_or(unchosen);
    if (bad_page || bad_keep) {
      if (tid == 0) report(p.status, bad_page ? PKC_ERR_BLOCK_TABLE : PKC_ERR_PLAN);
      bad_request = bad_page || unchosen;
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
  if (bad_request && tid == 0) atomicExch(ctr + 1, 1);
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
    if (any_bad) {  // a request with a missing page, short weights or a head of too few slots keeps its length
      const int64_t n_pages = ((int64_t)l + p.page_size - 1) / p.page_size;
      ok = n_pages <= p.bt_stride && !(p.weights && l > p.w_stride);
      for (int i = 0; ok && i < p.hkv; ++i) ok = p.keep[((int64_t)r * p.hkv + i + 1) * n - 1] >= 0;
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
  // still has 2048 keys of the longest row (or more than its bits hold).
  p.cluster = 1;
  while (p.cluster < 8 && ((rows * p.cluster * 2 <= num_sms() && p.w_stride / (2 * p.cluster) >= 2048) ||
                           p.w_stride / p.cluster > kMostKeys))
    p.cluster *= 2;
  const int64_t per = ((p.w_stride + p.cluster - 1) / p.cluster + 31) & ~int64_t(31);
  if (per > kMostKeys) return (int)cudaErrorInvalidValue;
  p.smem_keys = rows * p.cluster <= num_sms() && per <= kMostHeld ? (int)per : 0;
  const int smem = (int)sizeof(SelectShared) + (int)(per / 32) * 8 + 4 * p.smem_keys;
  // (the most: bits of kMostKeys, or kMostHeld keys and their bits)
  constexpr int kMostSmem = (int)sizeof(SelectShared) + std::max(kMostKeys / 4, kMostHeld * 17 / 4);
  static_assert(kMostSmem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> raised;
  if (const int e = raise_smem_limit(reinterpret_cast<const void*>(evict_select_kernel), kMostSmem, raised)) return e;
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
