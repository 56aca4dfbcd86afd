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
// kept slots are ranked: a thread per 32 of them, one scan.  Two rows
// share an SM (512 threads of 64 registers each); a cluster of up to 8 blocks
// works on one row where there are few, adding up their histograms through
// distributed shared memory.  What bounds it is instructions (about 100 per
// 32 weights and pass, with the fixed part) and the chain of reads and
// barriers per row, not HBM: 22 us for 512 rows of 1024 to 16384 weights (one
// read of them at the copy rate would be 3), 16 us for 8 rows of 131,056 on
// 64 blocks.
//
// Compact.  Row j of a (request, head) becomes row keep[j]; keep ascends
// strictly, so keep[j] >= j.  A block moves one slice of one head's K or V
// rows, chunk after chunk of new slots in order, a chunk read by the whole
// block before any of it is written.  The next chunk's rows lie at or behind
// its own first slot, where nothing has been written yet, so its copies into
// shared memory are in flight while the current chunk is stored.  Bound by
// HBM: a kept row is read once and written once, 256 bytes at a random slot:
// 100 us for 64 requests cut to 1024 of up to 6144 tokens, 8 heads of bf16
// (549 MB, 5.5 TB/s of a measured copy rate of 6.8).  With the chunks in
// registers, of half the size, it took 120 us.  Where there are few rows, a
// cluster works on each: its chunk is the blocks' chunks together, and its
// barrier keeps a chunk's stores behind all of its reads.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

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

// (-0 + 0 is +0; no weight's key is below 2^21)
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0xffffffffu : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

struct SelectShared {
  uint32_t hist[2][kBins];     // alternate between digits, as do their sums:
  int sums[2][kSelWarps];      // of the 128 bins of a warp, warp 0's the highest
  uint2 list[kListed];         // (key, index) of the first digit's bin
  int warp_sum[kSelWarps];
  int cta_gt, cta_eq;
  int bin, rest, in_bin, n_listed;
  int pad[2];
};

// Shared memory: SelectShared, then two bits per key (kept for certain; equal
// to T), then (kHeld) the keys, so that the weights are read once.  Three
// blocks an SM instead of two spill registers and hold no keys (512 rows:
// 24.1 us; two blocks 23.1, with the keys 22.1).
template <bool kHeld>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const SelectParams p) {
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
  uint2* bits = reinterpret_cast<uint2*>(smem_sel + sizeof(SelectShared));  // x: kept for certain, y: equal to T
  uint32_t* held = reinterpret_cast<uint32_t*>(bits + words);
  for (int i = tid; i < 2 * kBins / 4; i += kSelThreads)
    reinterpret_cast<uint4*>(&S.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) S.n_listed = 0;
  __syncthreads();

  // One pass over the keys: use(k, x, i) for steps x of a batch (kBatch keys
  // of a lane, a block's width apart, all loads in flight together -- a
  // shared-memory atomic between two loads would hold the second one back),
  // i the key's index, then flush(k, i of step 0).  k is 0, which no weight
  // has, past the end of the last batch, whose empty steps are left out.
  const auto pass = [&](auto from_held, auto use, auto flush) {
    for (int i0 = warp * 32; i0 < mine; i0 += kBatch * kSelThreads) {
      uint32_t k[kBatch];
      const int i = i0 + lane;
      if (i0 + (kBatch - 1) * kSelThreads + 32 <= mine) {  // (warp-uniform)
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
          k[x] = from_held ? held[i + x * kSelThreads] : __float_as_uint(src[i + x * kSelThreads]);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          if (!from_held) k[x] = order_key(__uint_as_float(k[x]));
          use(k[x], x, i + x * kSelThreads);
        }
      } else {
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          k[x] = 0u;
          if (i + x * kSelThreads < mine)
            k[x] = from_held ? held[i + x * kSelThreads] : __float_as_uint(src[i + x * kSelThreads]);
        }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          if (i0 + x * kSelThreads >= mine) break;  // (warp-uniform)
          if (!from_held) k[x] = i + x * kSelThreads < mine ? order_key(__uint_as_float(k[x])) : 0u;
          use(k[x], x, i + x * kSelThreads);
        }
      }
      flush(k, i);
    }
  };
  const auto no_flush = [](const uint32_t (&)[kBatch], int) {};
  constexpr std::false_type from_memory{};
  constexpr std::bool_constant<kHeld> again{};

  // First digit.  Weights that are exactly 0 are often most of a row: each
  // thread counts them apart, so they do not queue up on one bin.  (What is
  // past the end counts in bin 0, which has no weights and is not reached:
  // there are more than m of them above it.)
  int zeros = 0;
  pass(from_memory, [&](uint32_t k, int, int i) {
    if (kHeld && i < mine) held[i] = k;
    if (k == kZeroKey) ++zeros;
    else atomicAdd(&S.hist[0][k >> 21], 1u);
  }, no_flush);
  zeros = __reduce_add_sync(0xffffffffu, zeros);
  if (lane == 0 && zeros) atomicAdd(&S.hist[0][kZeroKey >> 21], (uint32_t)zeros);

  uint32_t prefix = 0;  // digits found, in place
  int rest = m;         // to be chosen among the keys that agree with them
  bool listed = true;   // the list holds all keys of the first digit's bin
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, width = d == 2 ? 10 : 11;
    uint32_t* hist = S.hist[d & 1];
    const uint32_t want = d == 0 ? 0u : prefix >> (shift + width), mask = (1u << width) - 1u;
    if (d == 1) {  // the second read: bits of the keys above, list of the keys in the bin
      const bool zero_bin = prefix == kZeroKey;  // (zero is the lowest key of its bin)
      // the bin's keys but zeros, which are counted already and never listed
      const uint32_t low = prefix + (zero_bin ? 1u : 0u), last = prefix | ((1u << 21) - 1u), span = last - low;
      uint32_t in = 0;  // steps of the batch whose key is one of them
      pass(again, [&](uint32_t k, int x, int i) {
        const uint32_t above = __ballot_sync(0xffffffffu, k > last);
        const uint32_t zero = zero_bin ? __ballot_sync(0xffffffffu, k == kZeroKey) : 0u;
        if (lane == 0) bits[i >> 5] = make_uint2(above, zero);
        if (k - low <= span) in |= 1u << x;
      }, [&](const uint32_t (&k)[kBatch], int i) {
        if (!__any_sync(0xffffffffu, in != 0u)) return;
        int at = __popc(in);  // places in the list: one atomic per warp and batch
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, at, x);
          if (lane >= x) at += y;
        }
        int first = 0;
        if (lane == 31) first = atomicAdd(&S.n_listed, at);
        at += __shfl_sync(0xffffffffu, first, 31) - __popc(in);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          if ((in >> x) & 1u) {
            if (at < kListed) S.list[at] = make_uint2(k[x], (uint32_t)(i + x * kSelThreads));
            ++at;
            atomicAdd(&hist[(k[x] >> shift) & mask], 1u);
          }
        }
        in = 0;
      });
    } else if (d == 2) {
      if (listed) {
        for (int i = tid; i < S.n_listed; i += kSelThreads) {
          const uint32_t k = S.list[i].x;
          if ((k >> (shift + width)) == want) atomicAdd(&hist[(k >> shift) & mask], 1u);
        }
      } else {
        pass(again, [&](uint32_t k, int, int) {
          if ((k >> (shift + width)) == want && k != kZeroKey) atomicAdd(&hist[(k >> shift) & mask], 1u);
        }, no_flush);
      }
    }
    if (d > 0 && lane == 0 && zeros && (kZeroKey >> (shift + width)) == want)
      atomicAdd(&hist[(kZeroKey >> shift) & mask], (uint32_t)zeros);
    __syncthreads();  // this block's histogram (and, of the second digit, its list) is complete
    if (d == 1) listed = S.n_listed <= kListed;
    {
      const uint4 x = *reinterpret_cast<const uint4*>(hist + kBins - 4 - 4 * tid);
      const int sum = __reduce_add_sync(0xffffffffu, (int)(x.x + x.y + x.z + x.w));
      if (lane == 0) S.sums[d & 1][warp] = sum;
    }
    if (n_cta > 1) cluster.sync();
    else __syncthreads();
    if (warp == 0) {
      // The bin in which the count from above reaches `rest`: first the group
      // of 128 bins, then the bin, counts of all blocks added up.
      int g = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < n_cta && lane < kSelWarps) g += (c == rank ? &S : cluster.map_shared_rank(&S, c))->sums[d & 1][lane];
      int upto = g;
#pragma unroll
      for (int x = 1; x < kSelWarps; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, x);
        if (lane >= x) upto += y;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, upto - g < rest && rest <= upto);
      const int group = here ? __ffs(here) - 1 : 0;
      const int left = rest - __shfl_sync(0xffffffffu, upto - g, group);
      const int bin0 = kBins - 128 * group - 4 - 4 * lane;
      int cnt[4] = {0, 0, 0, 0};  // from the top
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c < n_cta) {
          const uint4 x = *reinterpret_cast<const uint4*>((c == rank ? hist : cluster.map_shared_rank(hist, c)) + bin0);
          cnt[0] += x.w; cnt[1] += x.z; cnt[2] += x.y; cnt[3] += x.x;
        }
      }
      const int sum = cnt[0] + cnt[1] + cnt[2] + cnt[3];
      int above = sum;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, above, x);
        if (lane >= x) above += y;
      }
      above -= sum;  // keys of the group in higher bins than this lane's
      const bool mine_is_it = above < left && left <= above + sum;
      if (mine_is_it) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (above < left && left <= above + cnt[x]) {
            S.bin = bin0 + 3 - x;
            S.rest = left - above;
            S.in_bin = cnt[x];
          }
          above += cnt[x];
        }
      }
      // (always found, unless the weights change under the kernel)
      if (!__any_sync(0xffffffffu, mine_is_it) && lane == 0) {
        S.bin = d == 0 ? kBins - 1 : 0;
        S.rest = rest;
        S.in_bin = 0;
      }
    } else if (d == 1) {  // the third digit's histogram is the first's: every block is past it
      for (int i = tid - 32; i < kBins / 4; i += kSelThreads - 32)
        reinterpret_cast<uint4*>(S.hist[0])[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    prefix |= (uint32_t)S.bin << shift;
    rest = S.rest;
    // All keys with these digits are kept (often there is one): T is just
    // below them.  (Not where zeros are among them: they have no `sure` bit.)
    if (d == 1 && S.in_bin == rest && prefix != kZeroKey) {
      prefix -= 1u;
      rest = 0;
      break;
    }
  }
  // T = prefix.  Keys above T are kept, and the first `rest` of those equal
  // to it.  The bits so far: those of the keys above the first digit's bin,
  // and that bin's zeros; now the bin's other keys.
  if (listed) {
    if (prefix != kZeroKey) {
      for (int i = tid; i < words; i += kSelThreads) bits[i].y = 0u;
      __syncthreads();
    }
    for (int i = tid; i < S.n_listed; i += kSelThreads) {
      const uint2 k = S.list[i];
      if (k.x > prefix) atomicOr(&bits[k.y >> 5].x, 1u << (k.y & 31));
      else if (k.x == prefix) atomicOr(&bits[k.y >> 5].y, 1u << (k.y & 31));
    }
  } else {
    pass(again, [&](uint32_t k, int, int i) {
      const uint32_t g = __ballot_sync(0xffffffffu, k > prefix), e = __ballot_sync(0xffffffffu, k == prefix);
      if (lane == 0) bits[i >> 5] = make_uint2(g, e);
    }, no_flush);
  }
  __syncthreads();
  // Keys above and equal in the blocks before this one.
  int gt0 = 0, eq0 = 0;
  if (n_cta > 1) {
    int g = 0, e = 0;
    for (int i = tid; i < words; i += kSelThreads) {
      g += __popc(bits[i].x);
      e += __popc(bits[i].y);
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
    const uint2 both_bits = wd < words ? bits[wd] : make_uint2(0u, 0u);
    const uint32_t s = both_bits.x;
    uint32_t x = both_bits.y;
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
// Few large chunks: a chunk costs a barrier and the latency of its copies (2
// rows a thread and 3 chunks 109 us, 3 and 2 106, 4 and 2 100).
constexpr int kMoveRows = 4;    // rows per thread and chunk
constexpr int kMoveStages = 2;  // chunks on their way or being stored

struct MoveShared {
  uint4 rows[kMoveStages][kMoveRows][kMoveThreads];
  uint32_t to[kMoveStages][kMoveRows][kMoveThreads];
};

// Move rows keep[j] -> j, j < n, in units of V (one unit of a row per
// thread): place(slot) is a slot's place, at(place) this thread's unit of it,
// `row` the thread's row within a pass of `rows` rows.  Called by a whole
// block.  A chunk is kMoveRows passes of each block of the cluster.  While
// chunk c is stored, the chunks up to c + kMoveStages - 1 are on their way
// into shared memory (each thread's units in places of its own), the places
// of the next one and the slots of the one after it into registers.
template <typename V, typename Place, typename At, typename Sync>
__device__ __forceinline__ void move_rows(MoveShared& S, const int32_t* keep, int n, int row, int rows, int n_cta,
                                          Place place, At at, Sync sync) {
  const int chunk = rows * kMoveRows * n_cta, tid = threadIdx.x;
  int32_t slot[kMoveRows];                  // (-1 past the end)
  uint32_t from[kMoveRows], to[kMoveRows];
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
  auto copy = [&](int stage) {  // (from == to: nothing to move)
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const bool moves = from[u] != to[u];
      S.to[stage][u][tid] = moves ? to[u] : kNoToken;
      if (moves) {
        const uint32_t dst = smem_u32(&S.rows[stage][u][tid]);
        const uint64_t src = reinterpret_cast<uint64_t>(at(from[u]));
        if constexpr (sizeof(V) == 16) cp_async16(dst, src);
        else cp_async4(dst, src, true);
      }
    }
    cp_async_commit();
  };
  load_slots(0);
  load_places(0);
  load_slots(chunk);
#pragma unroll
  for (int s = 0; s < kMoveStages - 1; ++s) {
    copy(s);
    load_places((s + 1) * chunk);
    load_slots((s + 2) * chunk);
  }
  int stage = 0;
  for (int c = 0; c < n; c += chunk) {
    cp_async_wait<kMoveStages - 2>();
    sync();  // chunk c has been read by every thread of the cluster
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const uint32_t t = S.to[stage][u][tid];
      if (t != kNoToken) *at(t) = *reinterpret_cast<const V*>(&S.rows[stage][u][tid]);
    }
    copy(stage ? stage - 1 : kMoveStages - 1);
    load_places(c + kMoveStages * chunk);
    load_slots(c + (kMoveStages + 1) * chunk);
    stage = stage + 1 == kMoveStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

template <bool kCluster>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactParams p) {
  __shared__ MoveShared S;
  const int n_cta = kCluster ? p.cluster : 1, rank = kCluster ? (int)(blockIdx.x % n_cta) : 0;
  const int part = (int)(blockIdx.x / n_cta % p.parts);
  const int row = (int)(blockIdx.x / n_cta / p.parts), b = row / p.hkv, h = row % p.hkv;
  const int tid = threadIdx.x;
  auto sync = [&]() {
    if constexpr (kCluster) cg::this_cluster().sync();
    else __syncthreads();
  };
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
    if (__syncthreads_or(bad_page || bad_keep)) {
      bad_page = __syncthreads_or(bad_page);
      unchosen = __syncthreads_or(unchosen);
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
        const int rows = kMoveThreads / units;
        move_rows<uint4>(S, keep, n, rank * rows * kMoveRows + tid / units, rows, n_cta, token, [&](uint32_t t) {
          return reinterpret_cast<uint4*>(const_cast<uint8_t*>(at_row(base, t, stride)));
        }, sync);
      } else if (part < 2 * p.slices + (p.k_scales ? 2 : 0)) {  // mx4 scales: 4 bytes a row
        uint32_t* base = static_cast<uint32_t*>((part - 2 * p.slices) ? p.v_scales : p.k_scales) + h;
        move_rows<uint32_t>(S, keep, n, rank * kMoveThreads * kMoveRows + tid, kMoveThreads, n_cta, token,
                            [&](uint32_t t) { return base + (int64_t)t * p.hkv; }, sync);
      } else {  // weights: the kept ones, zeros behind them
        uint32_t* w = reinterpret_cast<uint32_t*>(p.weights) + (int64_t)row * p.w_stride;
        move_rows<uint32_t>(S, keep, n, rank * kMoveThreads * kMoveRows + tid, kMoveThreads, n_cta,
                            [](int slot) { return (uint32_t)slot; }, [&](uint32_t t) { return w + t; }, sync);
        sync();
        for (int64_t j = (int64_t)n + rank * kMoveThreads + tid; j < len; j += n_cta * kMoveThreads) w[j] = 0u;
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
  // Keys are held where two blocks still share an SM, or each has one.
  const int64_t base = (int64_t)sizeof(SelectShared) + per / 32 * 8;
  const bool hold = base + 4 * per <= 113 * 1024 || (rows * p.cluster <= num_sms() && per <= kMostHeld);
  const int smem = (int)(base + (hold ? 4 * per : 0));
  // (the most: bits of kMostKeys, or kMostHeld keys and their bits)
  constexpr int kMostSmem = (int)sizeof(SelectShared) + std::max(kMostKeys / 4, kMostHeld * 17 / 4);
  static_assert(kMostSmem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> raised[2];
  const auto kernel = hold ? evict_select_kernel<true> : evict_select_kernel<false>;
  if (const int e = raise_smem_limit(reinterpret_cast<const void*>(kernel), kMostSmem, raised[hold])) return e;
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
  return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

int launch_evict_compact(const CompactParams& p_in, void* stream) {
  CompactParams p = p_in;
  const int64_t rows = (int64_t)p.batch * p.hkv;
  if (rows <= 0) return 0;
  // Whole rows per block while that fills the machine (4 blocks per SM; twice
  // as many half rows there: 100 -> 102 us); else slices of a row, down to a
  // 32-byte sector.
  p.slices = 1;
  while (p.row_bytes / p.slices > 32 && rows * 2 * p.slices < 4 * (int64_t)num_sms()) p.slices *= 2;
  p.parts = 2 * p.slices + (p.k_scales ? 2 : 0) + (p.weights ? 1 : 0);
  if (rows * p.parts > INT32_MAX) return (int)cudaErrorInvalidValue;
  // Few rows of many slots: a cluster of up to 8 blocks shares each one, while
  // every block keeps a chunk of its own (8 heads cut to 16384 of 131072
  // tokens: 94 -> 65 us, one head to 25000: 88 -> 45).
  const int64_t chunk = (int64_t)kMoveRows * kMoveThreads / (p.row_bytes / 16 / p.slices);
  p.cluster = 1;
  while (p.cluster < 8 && rows * p.parts * p.cluster * 2 <= 4 * (int64_t)num_sms() && p.budget >= 2 * p.cluster * chunk)
    p.cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * p.parts * p.cluster));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeClusterDimension;
  la[0].val.clusterDim.x = (unsigned)p.cluster;
  la[0].val.clusterDim.y = la[0].val.clusterDim.z = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, p.cluster > 1 ? evict_compact_kernel<true> : evict_compact_kernel<false>, p);
}

}  // namespace pkc
