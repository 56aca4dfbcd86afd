// Attention states of a chunk of new tokens per request over its paged cache,
// on the 5th-generation tensor cores.
//
// Row i of request b's n rows stands at position p = len - n + i and attends to
// the tokens t < len with t <= p (causal) and t > p - window:
//   s_t = scale q.k_t,  LSE = log sum exp s_t,  O = sum exp(s_t - LSE) v_t.
//
// An item is 256 query rows of one KV head -- the G query heads of 256 / G
// consecutive tokens -- against the KV tiles of 128 tokens in their reach.  Its
// two halves A and B of 128 rows (the MMA's M) share every K and V tile:
//   S_X = Q_X K_j^T              tcgen05.mma, A and B from shared memory
//   P_X = exp2(S_X c - m_ref)    softmax warps, TMEM -> registers -> TMEM, 16 bits
//   O_X += P_X V_j               tcgen05.mma, P_X read from TMEM
// TMEM is one S (128 columns) that the halves use in turn, P_A, P_B (64 columns
// of 16-bit pairs) and O_A, O_B (128).  S is only in use until the softmax warps
// have read it into registers, so the other half's Q K runs while they work, and
// the next S of a half is there when its softmax is done: a half's chain per tile
// is its softmax, the MMAs run beside it.  (With an S per half and P in its
// columns, Q K of tile j + 1 waited for P V of tile j: 3650 cycles a tile.)  P never
// passes through shared memory, whose bandwidth the MMA's operands need.
// m_ref, a row's reference, is its first tile's maximum (fp16: less kLift; items of at
// most 128 rows: that of every tile, below).  It moves (and the row of O is rescaled, in
// TMEM) only when a tile's P would sum to more than kMoveSum: P is formed at once, and
// again where the sum says so, so the other tiles need no maximum at all (64 instructions
// and a chain ahead of the exponentials).  P stays within fp16's largest number, and a
// row's sum is at least about 1.
// P enters the V product in 16 bits: a remainder beside it, as the decode holds one,
// would be twice the product and columns that tensor memory does not have.  What that
// costs is most where one key holds much of a row and its P is not a power of two, so
// items of few rows, where no others average it out, take the maximum of every tile:
// their error against 64 bits is 1.0 to 1.1 times that of a rounded result for five
// tokens over 128k (1.1 to 1.6 with a reference that seldom moves), at 151 -> 157 us for
// a mixed step.  For all items: 1.1 times in place of 1.3 to 1.4, prompts 525 -> 561 us.
//
// Work split.  An item costs its KV tiles and kOver; all items are laid end to
// end (request, KV head, row tile) and cut evenly over the blocks, one per SM.
// So a block gets whole items but for its ends, few rows over a long cache are
// split over the cache, and no order of execution matters.  A block works the
// cut out for itself, from the lengths on the device: the sums over a request's
// items have a closed form.  A piece of a cut item leaves a partial state; the
// block that finishes last among the item's pieces (bits in the status block
// tell) merges them, always in the order of the cache.  Few tokens over two caches
// of 128k (19 pieces an item): 101 us, 79 of them bytes; the merge is 9 of the rest.
//
// Warps: 0-3 softmax of A, 4-7 of B (a row per thread, epilogue and merge too),
// 8 issues Q K, 9 P V, 10 K copies, 11 V copies, 12 scheduler, 13 Q
// copies.  K and V have a ring each (a wait names a phase modulo 2, so whoever
// fills a place has to have seen every phase of it); a tile is one TMA box per page
// and 64 dims (pages that are not a power of two: boxes of their largest
// power-of-two part).  The lanes of a warp issue their boxes one after another,
// some 50 cycles each, so pages of 16 tokens need a warp for K and one for V, and
// smaller boxes are what bounds the kernel (prompts 505 us with pages of 64, 525 of 16,
// 1040 of 20 or 4, whose boxes hold 4 tokens, 3560 to 3670 of 5 or 1).
// All waits are bounded (2 s) and set PKC_ERR_TIMEOUT when they run out.  Keys that
// one item alone reads pass L2 by (evict first: speculated tokens 111 -> 104 us), all
// others stay (prompts 544 us, 596 if they pass by too).
//
// What bounds it.  A long chunk (2047 tokens over 65,001, 32 / 8 heads) takes 1.55 to
// 1.70 ms by board and run, 1.30 to 1.43 PFLOP/s, at the power limit (1390 W, 1.70 GHz; a
// plain product in a loop holds 1.76 PFLOP/s).  Below it the chain of a half's tile does:
// S out of TMEM, 128 exponentials a thread, P back, with the waits, votes and fences
// between them some 2400 cycles, against 1024 of MMA, two halves at a time (tensor
// pipe 57 % busy on prompts, 48 % with a window; exponentials 30 %).  An item's first
// tile and epilogue cost 3.7 us beside that.  The softmax warps have 216 registers
// for 128 scores, and code that holds more spills (a branch over masked columns: a
// window 161 -> 316 us).  Of the 284 bytes that are spilled the scheduler's 40 registers
// cost 244, outside the loops over tiles.  The instruction cache keeps the softmax, the
// epilogue and the scheduler only while they are short, so most steps here took code away.
//
// Values that a row does not attend to meet P = 0, and 0 times an infinity or a
// NaN would be NaN: slots behind the length are zeroed in the V tile, and a row
// whose O is not finite is computed again key by key (slow_rows) where its boundary
// tiles hold such a value, so it reaches exactly the rows that attend to it, at no
// cost where there is none.  So are rows whose scores pass 2^26 (bf16: 2^30), which
// one rounding moves too far.  A key costs such a row 60 to 100 ns (a NaN among
// 2047 new tokens over 65,001: 209 ms); where that takes more than the 2 s that a
// block's other warps wait, the launch ends with the time-out.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "pkc_device.cuh"
#include "pkc_internal.h"

namespace pkc {
namespace {

constexpr int kHalf = 128;               // rows of a half (MMA M)
constexpr int kRows = 2 * kHalf;         // rows of an item
constexpr int kKv = 128;                 // tokens of a KV tile
constexpr int kSub = 16384;              // 128 rows x 64 elements, 128-byte swizzle
constexpr int kTileBytes = 2 * kSub;
constexpr int kStagesK = 2, kStagesV = 3;  // tiles in flight
constexpr int kItems = 4;                // items the scheduler runs ahead
constexpr int kThreads = 512;
constexpr int kQkWarp = 8, kPvWarp = 9, kKWarp = 10, kVWarp = 11, kSchedWarp = 12, kQWarp = 13;
constexpr int kMaxBlocks = 160;
// What an item costs, measured over whole launches (0.32 us a unit): a KV tile where
// both halves have rows 1.58 us, where only one has 1.35 (1.45 where all SMs run such
// tiles, which is as fast as HBM brings them), and 3.7 us for the item itself (first
// tile, epilogue).  With 17 for the item, the blocks that got short items were done 70 us
// before the others (prompts 542 us, 533 with 12; a mixed batch 161, 155).
constexpr int kTileCost = 5, kHalfTileCost = 4, kOver = 12;
constexpr int kMinCost = 16;             // least cost of a block: a short item has one to itself
// Items of at most so many tiles are not cut: a cut costs partial states and a merge
// (prompts 533 us with 16, 523 with 12; a window's items of 11 tiles 162 with 12, 171
// with 8).
constexpr int kShort = 12;
// A row's reference is its maximum less kLift: fp16 has no P below 2^-25, and what it
// drops from O stays in the sum.  With the lift a weight is lost below 2^-31 of the
// largest, so 2^20 of them are at most half a step of fp16.  bf16 has the exponents.
// (fp16, 5 / 6 / 8 / 10 powers of two against none: prompts 533 / 543 / 543 / 586 us
// against 531, window 173 / 173 / 177 / 193 against 170, mixed 150 / 151 / 152 / 205
// against 150: with more, the reference moves more often.)
template <typename T> constexpr float kLift = std::is_same<T, __half>::value ? 6.f : 0.f;
// A tile's sum of P above which its reference moves (no P is above its sum).
template <typename T> constexpr float kMoveSum = std::is_same<T, __half>::value ? 65504.f : 8192.f;

// P = exp2(s c - m_ref) in one rounding: m_ref = max s c - kLift is rounded, P's largest
// is exp2 of that rounding, at most 2^(m_ref / 2^24), and of the lift.  Rows with |m_ref|
// from here on are computed again with the product rounded too (slow_rows).
// Below, that factor is at most 2^4 in fp16 and 2^64 in bf16, which their P hold.
template <typename T> constexpr float kFar = std::is_same<T, __half>::value ? 0x1p26f : 0x1p30f;

struct Item {
  int b;                 // request; -1: no more items
  int kvh, q_row, n_tok; // KV head, first row of q, tokens
  int pos0, len;         // position of the first token, cached tokens
  int t0, t1;            // KV tiles of the piece
  int lo[2], hi[2];      // those of half A, B (lo == hi: none)
  int once;              // 1: no other item reads these keys
  int off;               // 0: rows 0-127 are A's; 128: B's, and A has none
  int c0, c1;            // first and last block with a piece of the item (c0 == c1: whole)
};

struct __align__(8) Barriers {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kStagesK + kStagesV], kv_empty[kStagesK + kStagesV];  // K's places, then V's
  uint64_t s_full[2], s_free, p_full[2];
  uint64_t pv_done[2];   // P read, O up to date
  uint64_t it_full[kItems], it_empty[kItems];
  uint64_t part_done, merge_go;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int merge;
};

constexpr int kKvOffset = 2 * kTileBytes;
constexpr int kItemOffset = kKvOffset + (kStagesK + kStagesV) * kTileBytes;
constexpr int kBarOffset = kItemOffset + kItems * 64;
constexpr int kSmemBytes = kBarOffset + 512;
static_assert(sizeof(Item) <= 64 && sizeof(Barriers) <= 512 && kSmemBytes <= 227 * 1024, "shared memory");

// ---------------------------------------------------------------- schedule

struct Request {
  int r0, n, len;
};

// sum over i < m of floor(max(a + i s, 0) / 128), s = 2^e
PKC_HD inline int64_t sum_floor(int64_t a, int e, int64_t m) {
  if (a < 0) {  // the terms before the first positive a are 0
    const int64_t skip = (-a + (int64_t(1) << e) - 1) >> e;
    a += skip << e;
    m -= skip;
    if (m <= 0) return 0;
  }
  const int64_t whole = m * (a >> 7), r = a & 127;
  if (e >= 7) return whole + ((m * (m - 1) / 2) << (e - 7));
  // floor((r + i s) / 128) = floor((r / s + i) / per), per = 128 / s, and the sum
  // of floor(i / per) over i < n = per u + v is per u (u - 1) / 2 + v u
  const int d = 7 - e;
  int64_t n[2] = {(r >> e) + m, r >> e}, g[2];
  for (int k = 0; k < 2; ++k) {
    const int64_t u = n[k] >> d, v = n[k] - (u << d);
    g[k] = ((u * (u - 1) / 2) << d) + v * u;
  }
  return whole + g[0] - g[1];
}

// Tokens of an item: 2^shift.
PKC_HD inline int item_shift(const ChunkParams& p) { return 8 - p.g_log2; }

PKC_HD inline int n_items(const ChunkParams& p, const Request& q) {
  const int e = item_shift(p);
  return (q.n + (1 << e) - 1) >> e;
}

// KV tiles [lo, hi) in the reach of tokens j0 .. j1 - 1 of a request.
PKC_HD inline void reach(const ChunkParams& p, const Request& q, int j0, int j1, int& lo, int& hi) {
  const int pos = q.len - q.n;
  const int end = p.causal ? pos + j1 : q.len;
  const int64_t begin = p.window ? (int64_t)pos + j0 - p.window + 1 : 0;
  hi = end > 0 ? (int)(((uint32_t)end + kKv - 1) >> 7) : 0;
  lo = begin > 0 ? (int)(begin >> 7) : 0;
  if (lo > hi) lo = hi;
}

// Cost of a KV tile of a request's item i.
PKC_HD inline int tile_cost(const ChunkParams& p, const Request& q, int i) {
  return (q.n - (i << item_shift(p))) << p.g_log2 <= kHalf ? kHalfTileCost : kTileCost;
}

// Cost of the first m items of a request's KV head.
PKC_HD inline int64_t cost_of(const ChunkParams& p, const Request& q, int m) {
  const int e = item_shift(p), nt = n_items(p, q);
  const int64_t pos = (int64_t)q.len - q.n;
  const int64_t all = ((int64_t)q.len + kKv - 1) >> 7;
  // the last item ends at the length and may have rows for A alone
  const int whole = m < nt ? m : nt - 1;
  int64_t tiles = p.causal ? sum_floor(pos + (1 << e) + kKv - 1, e, whole) : whole * all;
  if (p.window) tiles -= sum_floor(pos - p.window + 1, e, whole);
  int64_t sum = (int64_t)m * kOver + tiles * kTileCost;
  if (m == nt) {
    int lo, hi;
    reach(p, q, (nt - 1) << e, q.n, lo, hi);
    sum += (int64_t)(hi - lo) * tile_cost(p, q, nt - 1);
  }
  return sum;
}

// ---------------------------------------------------------------- helpers

// D[tmem] (+)= A[tmem] * B[smem]: A 16-bit, two elements a column.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Registers per thread from here on; the warps of a warpgroup call it together.
template <int kRegs> __device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs> __device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// True in one lane of a warp whose lanes are all here.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one != 0;
}

// Arrive for a warp that is all here: a predicate in place of a branch, which
// costs some 200 cycles in the softmax loop.
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane) {
  __syncwarp();
  asm volatile("{ .reg .pred p; .reg .b64 st; setp.eq.s32 p, %1, 0; @p mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(bar),
               "r"(lane)
               : "memory");
}
// mbar_wait that looks at the clock only where the wait is a long one.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  return mbar_try_wait(bar, parity) || mbar_wait(bar, parity, abort, status);
}

// The n lowest bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// 32 columns (float32, already normalised) to column `col` of output row `row`.
// A thread has a row of its own, so a store is as wide as it gets: 32 bytes, a
// sector, where o allows it.
template <typename T>
__device__ __forceinline__ void store_out(const ChunkParams& p, int64_t row, int col, const float (&o)[32]) {
  if (p.out_dtype == PKC_F32) {
    float* dst = static_cast<float*>(p.o) + row * PKC_HEAD_DIM + col;
#pragma unroll
    for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    return;
  }
  T* dst = static_cast<T*>(p.o) + row * PKC_HEAD_DIM + col;
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = Elem<T>::from_f2(o[2 * i], o[2 * i + 1]);
  if (p.o_wide) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 2 * i), "r"(w[i]), "r"(w[i + 1]),
                   "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<uint4*>(dst + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// Partial states: part_o[slot][column / 4][row][4] and part_ml[slot][row], a row's
// reference and its sum of exp2(s c - reference).  (Not their LSE: where that is far
// from 0 a float32 holds little or nothing of the sum.)
__device__ __forceinline__ float* part_row(const ChunkParams& p, int slot, int chunk, int row) {
  return p.part_o + (((int64_t)slot * 32 + chunk) * kRows + row) * 4;
}
__device__ __forceinline__ float2* part_sum(const ChunkParams& p, int slot, int row) {
  return reinterpret_cast<float2*>(p.part_ml) + slot * kRows + row;
}
__device__ __forceinline__ int slot_of(int c, int c0) { return 2 * c + (c == c0 ? 1 : 0); }

// The row of q, o and lse that row `row` of an item stands for.
__device__ __forceinline__ int64_t out_row(const ChunkParams& p, int q_row, int kvh, int row) {
  return ((int64_t)q_row + (row >> p.g_log2)) * p.hq + (kvh << p.g_log2) + (row & (p.g - 1));
}

// The bits, within a word, of pieces c0 .. c1 (which may lie outside it): slot_of.
__device__ __forceinline__ uint32_t pieces_of(int c0, int c1) {
  const uint32_t first = c0 >= 0 ? 2u << 2 * c0 : 0u;
  return (0x55555555u & low_bits(2 * c1 + 1) & ~low_bits(2 * c0 + 2)) | first;
}
// Set a bit; true for the one that completes `all`, which are cleared again then.
__device__ __forceinline__ bool set_bit(uint32_t* word, int bit, uint32_t all) {
  if (((atomicOr(word, 1u << bit) | 1u << bit) & all) != all) return false;
  atomicAnd(word, ~all);
  return true;
}

// The tokens [lo, hi) that a row at position pos attends to.
__device__ __forceinline__ void tokens_of(const ChunkParams& p, int pos, int len, int& lo, int& hi) {
  hi = p.causal ? min(len, pos + 1) : len;
  lo = p.window ? (int)max((int64_t)0, (int64_t)pos - p.window + 1) : 0;
}

// The page of key t of request b (-1: none there).
__device__ __forceinline__ int page_of_key(const ChunkParams& p, int b, int t, int end) {
  if (t < 0 || t >= end) return -1;  // (t < 0: past 2^31)
  const int pi = t / p.page_size;
  const int page = pi < p.bt_stride ? p.block_table[(int64_t)b * p.bt_stride + pi] : -1;
  return page < p.num_pages ? page : -1;
}

// Rows again (row0 + a bit), by one warp, key by key over the half's tiles
// [t0, t1).  `far`: rows whose scores lie so far out (kFar) that s c - m_ref in one
// rounding is off by too much; here the product is rounded before the maximum is
// taken off, so the largest weight is 1.  `odd`: rows whose O is not finite.  They
// are right as they are unless a value of the tiles that not all of the warp's rows
// attend to (a key outside [all_lo, all_hi)) is not finite itself.  Lanes hold four
// elements each.  slot: the partial states' place, or -1 for an item that is not cut.  (Out of line, with the item's fields by value: nothing
// of it is held in the loops of those who call it.)
template <typename T>
__device__ __noinline__ void slow_rows(const ChunkParams& p, uint32_t far, uint32_t odd, int row0, int b, int kvh, int q_row,
                                       int pos0, int len, int t0, int t1, int all_lo, int all_hi, int slot,
                                       volatile int* abort) {
  const int lane = threadIdx.x & 31;
  const int begin = t0 * kKv, end = (int)min((int64_t)len, (int64_t)t1 * kKv);
  const T* q = static_cast<const T*>(p.q) + 4 * lane;
  // Four elements of key t; a page that is not there is read as zeros (the load goes
  // somewhere all the same, so that eight are on their way together).
  auto load = [&](const void* pool, int page, int t) {
    const int64_t at = (((int64_t)page * p.page_size + t % p.page_size) * p.hkv + kvh) * PKC_HEAD_DIM;
    const uint2 w = *reinterpret_cast<const uint2*>(page < 0 ? q : static_cast<const T*>(pool) + at + 4 * lane);
    return page < 0 ? make_uint2(0, 0) : w;
  };
  if (odd) {
    float sum = 0.f;  // 0 times the values
    for (int64_t t = begin; t < end; t += 32) {
      if (t >= all_lo && t + 32 <= all_hi) {
        t += (all_hi - t - 32) & ~31;
        continue;
      }
      const int pages = page_of_key(p, b, (int)t + lane, end);
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const uint2 w = load(p.v_cache, __shfl_sync(0xffffffffu, pages, i), (int)t + i);
        const float2 x = Elem<T>::to_f2(w.x), y = Elem<T>::to_f2(w.y);
        sum += 0.f * x.x + 0.f * x.y + 0.f * y.x + 0.f * y.y;
      }
    }
    if (__any_sync(0xffffffffu, !(sum == 0.f))) far |= odd;
  }
  // Four rows and eight keys at a time: 32 scores, summed over the lanes so that
  // lane 8 r + i ends with that of row r and key i, and holds row r's maximum and sum.
  constexpr int kAtOnce = 4;
  while (far) {
    int row[kAtOnce], n = 0, first = end, last = begin, lo = 0, hi = 0;
    float2 q0[kAtOnce], q1[kAtOnce];
    float m = neg_inf(), l = 0.f, o[kAtOnce][4] = {};
#pragma unroll
    for (int r = 0; r < kAtOnce; ++r) {
      row[r] = r && !far ? row[r - 1] : row0 + __ffs(far) - 1;  // (the last one again where there are fewer)
      n += far != 0;
      far &= far - 1;
      int a, z;
      tokens_of(p, pos0 + (row[r] >> p.g_log2), len, a, z);
      a = max(a, begin);
      z = min(z, end);
      first = min(first, a);
      last = max(last, z);
      if (lane >> 3 == r) lo = a, hi = z;
      const uint2 w = *reinterpret_cast<const uint2*>(q + out_row(p, q_row, kvh, row[r]) * PKC_HEAD_DIM);
      q0[r] = Elem<T>::to_f2(w.x);
      q1[r] = Elem<T>::to_f2(w.y);
    }
    for (int64_t tb = first; tb < last && !*abort; tb += 32) {
      const int pages = page_of_key(p, b, (int)tb + lane, last);
#pragma unroll 1
      for (int i0 = 0; i0 < 32 && tb + i0 < last; i0 += 8) {
        uint2 vw[8];
        float s[8 * kAtOnce];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int page = __shfl_sync(0xffffffffu, pages, i0 + i);
          const uint2 kw = load(p.k_cache, page, (int)tb + i0 + i);
          vw[i] = load(p.v_cache, page, (int)tb + i0 + i);
          const float2 k0 = Elem<T>::to_f2(kw.x), k1 = Elem<T>::to_f2(kw.y);
#pragma unroll
          for (int r = 0; r < kAtOnce; ++r) s[8 * r + i] = q0[r].x * k0.x + q0[r].y * k0.y + q1[r].x * k1.x + q1[r].y * k1.y;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          const bool up = lane & d;
#pragma unroll
          for (int j = 0; j < d; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? s[j] : s[j + d], d);
            s[j] = (up ? s[j + d] : s[j]) + other;
          }
        }
        const int64_t t = tb + i0 + (lane & 7);
        const bool in = t >= lo && t < hi;
        const float score = in ? __fmul_rn(s[0], p.scale_log2) : neg_inf();
        float now = fmaxf(m, score);
#pragma unroll
        for (int d = 4; d; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
        const float ref = now == neg_inf() ? 0.f : now, w = ex2(m - ref), e = in ? ex2(__fsub_rn(score, ref)) : 0.f;
        float sum = e;
#pragma unroll
        for (int d = 4; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        m = now;
        l = l * w + sum;
        const uint32_t ins = __ballot_sync(0xffffffffu, in);
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
          const float wr = __shfl_sync(0xffffffffu, w, 8 * r);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[r][i] *= wr;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v0 = Elem<T>::to_f2(vw[i].x), v1 = Elem<T>::to_f2(vw[i].y);
#pragma unroll
          for (int r = 0; r < kAtOnce; ++r) {
            const float er = __shfl_sync(0xffffffffu, e, 8 * r + i);
            if (!(ins >> (8 * r + i) & 1)) continue;  // (uniform; the value may be anything)
            o[r][0] += er * v0.x;
            o[r][1] += er * v0.y;
            o[r][2] += er * v1.x;
            o[r][3] += er * v1.y;
          }
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int r = 0; r < kAtOnce; ++r) {
      const float f = __shfl_sync(0xffffffffu, inv, 8 * r);
      if (r >= n) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[r][i] *= f;
      const int64_t out = out_row(p, q_row, kvh, row[r]);
      if (slot >= 0)
        *reinterpret_cast<float4*>(part_row(p, slot, lane, row[r])) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
      else if (p.out_dtype == PKC_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.o) + out * PKC_HEAD_DIM + 4 * lane) =
            make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
      else
        *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + out * PKC_HEAD_DIM + 4 * lane) =
            make_uint2(Elem<T>::from_f2(o[r][0], o[r][1]), Elem<T>::from_f2(o[r][2], o[r][3]));
      if (lane == 8 * r) {
        if (slot >= 0) *part_sum(p, slot, row[r]) = make_float2(m, l);
        else p.lse[out] = l == 0.f ? neg_inf() : (m + lg2(l)) * kLn2;
      }
    }
  }
}

// The merge of an item's partial states by the eight softmax warps: a warp takes
// 32 rows and 32 columns at a time, three states' loads in flight.
template <typename T>
__device__ __forceinline__ void merge_item(const ChunkParams& p, const Item& it, int warp, int lane) {
  const int rows = it.n_tok << p.g_log2, groups = (rows + 31) / 32, n = it.c1 - it.c0 + 1;
#pragma unroll 1
  for (int u = warp; u < 4 * groups; u += 8) {
    const int row = (u >> 2) * 32 + lane, from = min(row, rows - 1), chunk = (u & 3) * 8;
    float m = neg_inf(), l = 0.f, o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 3) {
      float4 x[3][8];
      float2 w[3];
      float now = m;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int slot = slot_of(it.c0 + min(i0 + i, n - 1), it.c0);
        w[i] = __ldcg(part_sum(p, slot, from));
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = __ldcg(reinterpret_cast<const float4*>(part_row(p, slot, chunk + k, from)));
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) now = fmaxf(now, w[i].x);  // (the last one again where there are fewer)
      const float ref = now == neg_inf() ? 0.f : now, f = ex2(m - ref);
      m = now;
      l *= f;
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] *= f;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (i0 + i >= n) break;
        const float e = w[i].y * ex2(w[i].x - ref);
        l += e;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[4 * k] += e * x[i][k].x;
          o[4 * k + 1] += e * x[i][k].y;
          o[4 * k + 2] += e * x[i][k].z;
          o[4 * k + 3] += e * x[i][k].w;
        }
      }
    }
    if (row < rows) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (not m: that of a row whose scores are NaN is -inf too)
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] *= inv;
      const int64_t out = out_row(p, it.q_row, it.kvh, row);
      store_out<T>(p, out, 4 * chunk, o);
      if (chunk == 0) p.lse[out] = l == 0.f ? neg_inf() : (m + lg2(l)) * kLn2;
    }
  }
}

// ---------------------------------------------------------------- kernel

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ChunkParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023) != 0) {  // uniform: no thread has started yet
    if (threadIdx.x == 0) report(p.status, PKC_ERR_UNSUPPORTED);
    return;
  }
  const uint32_t s_q = smem_u32(smem), s_kv = s_q + kKvOffset;
  Barriers* bars = reinterpret_cast<Barriers*>(smem + kBarOffset);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(bars->q_full[x]), 1);
      mbar_init(bar(bars->q_empty[x]), 1);
      mbar_init(bar(bars->s_full[x]), 1);
      mbar_init(bar(bars->p_full[x]), 4);
      mbar_init(bar(bars->pv_done[x]), 1);
    }
    for (int s = 0; s < kStagesK + kStagesV; ++s) {
      mbar_init(bar(bars->kv_full[s]), 1);
      mbar_init(bar(bars->kv_empty[s]), 1);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(bar(bars->it_full[s]), 1);
      mbar_init(bar(bars->it_empty[s]), 13);  // all warps but the scheduler
    }
    mbar_init(bar(bars->s_free), 4);
    mbar_init(bar(bars->part_done), 8);
    mbar_init(bar(bars->merge_go), 1);
    mbar_init(bar(bars->drain), 2);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kKWarp && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // A wait in the loops over tiles.  Where it runs out nobody leaves the loop: the
  // other waits end at once then, what is computed is not used (the status says
  // so), and the warps stay whole without a vote per wait (50 us of 690 on
  // prompts).  Items and copies are not begun on such a wait.
  auto pass = [&](uint64_t& b, uint32_t parity) {
    wait_for(bar(b), parity, abort, p.status);
    __syncwarp();
  };
  // The k-th item of the block, by a whole warp (lane 0 waits and gives the
  // place back); false at the end.
  auto next_item = [&](int k, Item& it) -> bool {
    bool got = true;
    if (lane == 0) got = wait_for(bar(bars->it_full[k % kItems]), (k / kItems) & 1, abort, p.status);
    got = __shfl_sync(0xffffffffu, got, 0);
    __syncwarp();
    if (!got) return false;
    const int* src = reinterpret_cast<const int*>(smem + kItemOffset + (k % kItems) * 64);
    int* dst = reinterpret_cast<int*>(&it);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) dst[i] = src[i];
    arrive_warp(bar(bars->it_empty[k % kItems]), lane);
    return it.b >= 0;
  };

  // 512 threads start with 128 registers each: the softmax warps take 216 and
  // leave the others 40 (65,536 together).  Every role's code lies behind its own
  // setmaxnreg, so the compiler keeps within it.
  if (warp >= kQkWarp) {
    regs_down<40>();
    if (warp == kSchedWarp) {
      // ---------------- scheduler ----------------
      auto load = [&](int b) -> Request {  // an empty request where there is nothing to do
        Request q = {0, 0, 0};
        if (b < p.batch) {
          const int r0 = p.q_indptr[b], r1 = p.q_indptr[b + 1], len = p.cache_seqlens[b];
          if (r0 < 0 || r1 < r0 || r1 > p.total_q || (len < 0 && r1 > r0)) {
            if (blockIdx.x == 0) report(p.status, PKC_ERR_PLAN);
          } else if (r1 > r0) {
            q = {r0, r1 - r0, len};
          }
        }
        return q;
      };
      // The cost of all requests, then those that hold some of the block's share:
      // one loop for both, for its code is long and shares the instruction cache
      // with the softmax.
      int64_t total = 0, s0 = 0, s1 = 0;
      int n_blocks = 1, k = 0;
      bool turn = false;
      const int c = (int)blockIdx.x;
      bool ok = true;
      // The block that holds place x: the last i with i total / n_blocks <= x.
      auto block_of = [&](int64_t x) {
        int n = 0;
#pragma unroll 1
        for (int i = lane; i < kMaxBlocks; i += 32)
          n += __popc(__ballot_sync(0xffffffffu, i < n_blocks && i * total < (x + 1) * n_blocks));
        return n - 1;
      };
      // i total / n_blocks, in divisions of 32 bits (total < 2^54, n_blocks < 2^8)
      auto share_of = [&](int i) {
        const uint32_t a = (uint32_t)(total >> 24), n = (uint32_t)n_blocks;
        const uint64_t rest = ((uint64_t)(a % n) << 24) | (uint32_t)(total & 0xffffff);  // < n 2^24 <= 2^32
        const uint64_t q = ((uint64_t)(a / n) << 24) + (uint32_t)rest / n;
        return (int64_t)(q * i + (uint32_t)rest % n * i / n);
      };
      auto publish = [&](const Item& it) {
        if (lane == 0 && k >= kItems) ok = wait_for(bar(bars->it_empty[k % kItems]), ((k / kItems) & 1) ^ 1, abort, p.status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok && lane == 0) {
          *reinterpret_cast<Item*>(smem + kItemOffset + (k % kItems) * 64) = it;
          mbar_arrive(bar(bars->it_full[k % kItems]));
        }
        ++k;
      };
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        int64_t base = 0;  // cost of the requests before b0
#pragma unroll 1
        for (int b0 = 0; ok && b0 < p.batch && (pass == 0 || base < s1); b0 += 32) {
          const Request mine = load(b0 + lane);
          const int64_t per_head = mine.n ? cost_of(p, mine, n_items(p, mine)) : 0;
          int64_t before = per_head * p.hkv;
#pragma unroll 1
          for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += y;
          }
          const int64_t all = __shfl_sync(0xffffffffu, before, 31);
          before = base + before - per_head * p.hkv;
          base += all;
          if (pass == 0) continue;
          uint32_t todo = __ballot_sync(0xffffffffu, mine.n > 0 && before < s1 && before + per_head * p.hkv > s0);
#pragma unroll 1
          for (; ok && todo; todo &= todo - 1) {
            const int j = __ffs(todo) - 1;
            const Request q = {__shfl_sync(0xffffffffu, mine.r0, j), __shfl_sync(0xffffffffu, mine.n, j),
                               __shfl_sync(0xffffffffu, mine.len, j)};
            const int64_t ph = __shfl_sync(0xffffffffu, per_head, j);
            const int nt = n_items(p, q);
            int h = 0, i = 0;
            int64_t x0 = __shfl_sync(0xffffffffu, before, j);  // where item (h, i) begins
            if (s0 > x0) {
#pragma unroll 1
              for (int step = 1 << 16; step; step >>= 1)
                if (x0 + step * ph <= s0) h += step, x0 += step * ph;
              // the last i whose items before it cost at most s0 - x0
              int hi = nt;
              int64_t at = 0;
#pragma unroll 1
              while (hi - i > 1) {
                const int mid = (i + hi) >> 1;
                const int64_t cost = cost_of(p, q, mid);
                if (cost <= s0 - x0) i = mid, at = cost;
                else hi = mid;
              }
              x0 += at;
            }
#pragma unroll 1
            while (ok && h < p.hkv && x0 < s1) {
              const int j0 = i << item_shift(p), n_tok = min(1 << item_shift(p), q.n - j0);
              Item it;
              it.b = b0 + j; it.kvh = h; it.q_row = q.r0 + j0; it.n_tok = n_tok;
              it.pos0 = q.len - q.n + j0; it.len = q.len;
              const int half = kHalf >> p.g_log2;
              reach(p, q, j0, j0 + min(n_tok, half), it.lo[0], it.hi[0]);
              it.lo[1] = it.hi[1] = it.hi[0];
              if (n_tok > half) reach(p, q, j0 + half, j0 + n_tok, it.lo[1], it.hi[1]);
              const int lo = it.lo[0], hi = it.hi[1];  // (a later token's reach begins and ends no earlier)
              const int cost = tile_cost(p, q, i);
              const int64_t first = x0 + kOver, end = first + (int64_t)(hi - lo) * cost;  // its tiles lie at first .. end - 1
              it.t0 = lo;
              it.t1 = hi;
              it.c0 = it.c1 = c;
              bool ours = end > s0 && end <= s1;  // a short item is whole, its last place's block has it
              if (hi - lo > kShort) {
                // (a block's share is larger than a tile's cost: no piece between is empty)
                const uint32_t from = (uint32_t)max((int64_t)0, s0 - first), to = (uint32_t)max((int64_t)0, min(s1, end) - first);
                it.t0 = lo + (int)(cost == kTileCost ? from / kTileCost : from / kHalfTileCost);
                it.t1 = lo + (int)(cost == kTileCost ? to / kTileCost : to / kHalfTileCost);
                if (first + cost - 1 < s0) it.c0 = block_of(first + cost - 1);
                if (end > s1) it.c1 = block_of(end - 1);
                ours = it.t0 < it.t1;
              }
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                it.lo[x] = max(it.lo[x], it.t0);
                it.hi[x] = max(it.lo[x], min(it.hi[x], it.t1));
              }
              it.once = nt == 1;
              it.off = 0;
              if (n_tok <= half) {  // every second item of few rows goes to B: one's epilogue runs beside the other's tiles
                it.off = turn ? kHalf : 0;
                if (ours) turn = !turn;
                if (it.off) it.lo[1] = it.lo[0], it.hi[1] = it.hi[0], it.lo[0] = it.hi[0] = it.t0;
              }
              if (ours) publish(it);
              x0 = end;
              if (++i == nt) i = 0, ++h;
            }
          }
        }
        if (pass == 0) {
          total = base;
          n_blocks = (int)max((int64_t)1, min((int64_t)gridDim.x, total / kMinCost));
          s0 = s1 = total;
          if (c < n_blocks) {
            s0 = share_of(c);
            s1 = share_of(c + 1);
          }
        }
      }
      if (ok) {
        Item it;
        it.b = -1;
        publish(it);
      }
    } else if (warp == kQWarp) {
      // ---------------- Q copies ----------------
      const uint64_t pol = l2_policy_evict_first();
      int n[2] = {0, 0};
      Item it = {};
      bool ok = true;
      for (int k = 0; ok && next_item(k, it); ++k) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (it.lo[x] == it.hi[x]) continue;
          if (lane == 0) {
            if (n[x] > 0) ok = wait_for(bar(bars->q_empty[x]), (n[x] - 1) & 1, abort, p.status);
            if (ok) {
              const int row = it.q_row + ((x * kHalf - it.off) >> p.g_log2);
              mbar_arrive_expect_tx(bar(bars->q_full[x]), kTileBytes);
              tma_load_3d(s_q + x * kTileBytes, &tm_q, bar(bars->q_full[x]), 0, it.kvh * p.g, row, pol);
              tma_load_3d(s_q + x * kTileBytes + kSub, &tm_q, bar(bars->q_full[x]), 64, it.kvh * p.g, row, pol);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          ++n[x];
        }
      }
      if (*abort && lane == 0) {  // the copies already issued land before the block exits
        volatile int no_abort = 0;
        for (int x = 0; x < 2; ++x)
          if (n[x] > 0) wait_for(bar(bars->q_full[x]), (n[x] - 1) & 1, &no_abort, p.status);
      }
    } else if (warp == kKWarp || warp == kVWarp) {
      // ---------------- K copies, V copies ----------------
      const uint64_t keep = l2_policy_evict_last(), pass_by = l2_policy_evict_first();
      const int bs = p.box_tokens, boxes = 2 * (kKv / bs);  // box c: tokens (c / 2) bs .. of the tile, dims 64 (c % 2) ..
      const int no_page = (int)max((int64_t)1, p.num_pages);   // outside the pool: read as zeros
      const void* tmap = warp == kVWarp ? (const void*)&tm_v : (const void*)&tm_k;
      const int first = warp == kVWarp ? kStagesK : 0, stages = warp == kVWarp ? kStagesV : kStagesK;
      int g = 0;  // tiles so far
      Item it = {};
      bool ok = true;
      for (int k = 0; ok && next_item(k, it); ++k) {
        const int32_t* table = p.block_table + (int64_t)it.b * p.bt_stride;
        // Page of box c of tile t; the lane's first one is loaded a tile ahead.
        auto page_of = [&](int t, int c) -> int {
          const int token = t * kKv + (c >> 1) * bs;
          if (t >= it.t1 || c >= boxes || token >= it.len) return no_page;
          const int pi = token / p.page_size;
          return pi < p.bt_stride ? table[pi] : -1;
        };
        const uint64_t pol = it.once ? pass_by : keep;
        int ahead = page_of(it.t0, lane);
        for (int t = it.t0; t < it.t1; ++t, ++g) {
          const int page = ahead, st = first + g % stages;
          ahead = page_of(t + 1, lane);
          if (lane == 0) {
            if (g >= stages) ok = wait_for(bar(bars->kv_empty[st]), ((g / stages) & 1) ^ 1, abort, p.status);
            if (ok) mbar_arrive_expect_tx(bar(bars->kv_full[st]), kTileBytes);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          __syncwarp();
          for (int c = lane; c < boxes; c += 32) {
            const int r = (c >> 1) * bs;
            int pg = c == lane ? page : page_of(t, c);
            if (t * kKv + r < it.len && (pg < 0 || pg >= p.num_pages)) {
              report(p.status, PKC_ERR_BLOCK_TABLE);
              pg = no_page;
            }
            tma_load_4d(s_kv + st * kTileBytes + (c & 1) * kSub + r * 128, tmap, bar(bars->kv_full[st]), (c & 1) * 64, it.kvh,
                        (t * kKv + r) % p.page_size, pg, pol);
          }
          __syncwarp();
        }
      }
      if (*abort && lane == 0) {
        volatile int no_abort = 0;
        for (int j = max(0, g - stages); j < g; ++j)
          wait_for(bar(bars->kv_full[first + j % stages]), (j / stages) & 1, &no_abort, p.status);
      }
    } else if (warp == kQkWarp || warp == kPvWarp) {
      // ---------------- MMA issue: Q K, P V ----------------
      // The whole warp runs the loop and one elected lane issues: with uniform
      // control flow the descriptors stay in uniform registers.  Both go tile by
      // tile, A before B.
      constexpr uint32_t kBf16 = std::is_same<T, __half>::value ? 0 : 1;
      constexpr uint32_t idesc_qk = idesc_f16(128, 128, kBf16, 0, 0);
      constexpr uint32_t idesc_pv = idesc_f16(128, 128, kBf16, 0, 1);
      const uint64_t desc_q = smem_desc_sw128(s_q, 16, 1024);
      const uint64_t desc_k = smem_desc_sw128(s_kv, 16, 1024), desc_v = smem_desc_sw128(s_kv, kSub, 1024);
      const bool is_pv = warp == kPvWarp;
      const int first = is_pv ? kStagesK : 0, behind = is_pv ? kStagesK + kStagesV : kStagesK;
      int place = first;             // ring place of the next K or V tile, and its phase
      uint32_t phase = 0, s_par = 1;
      uint32_t par = 0;              // phases of q_full or p_full, a bit per half
      Item it = {};
      for (int k = 0; next_item(k, it); ++k) {
        for (int t = it.t0; t < it.t1; ++t) {
          pass(bars->kv_full[place], phase);
          if (const int live = it.len - t * kKv; is_pv && live < kKv) {
            // Slots behind the length may hold anything, even NaN: zero their V.
            const uint32_t vst = s_kv + place * kTileBytes + live * 128;
            for (int c = lane; c < (kKv - live) * 16; c += 32)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vst + ((c >> 3) & 1) * kSub + (c >> 4) * 128 +
                                                                          (c & 7) * 16),
                           "r"(0u)
                           : "memory");
            fence_proxy_async_smem();
            __syncwarp();
          }
          const uint32_t at = (uint32_t)place * (kTileBytes >> 4);
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            const int lo = x ? it.lo[1] : it.lo[0], hi = x ? it.hi[1] : it.hi[0];
            if (t < lo || t >= hi) continue;
            if (!is_pv) {
              // S = Q K^T once the S before has been read
              if (t == lo) {
                pass(bars->q_full[x], (par >> x) & 1);
                par ^= 1u << x;
              }
              pass(bars->s_free, s_par);
              s_par ^= 1;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll 2
                for (int kk = 0; kk < 8; ++kk) {
                  const uint32_t off = (kk >> 2) * (kSub >> 4) + (kk & 3) * 2;
                  tc_mma_f16(tmem, desc_q + x * (kTileBytes >> 4) + off, desc_k + at + off, idesc_qk, kk > 0);
                }
                tc_commit(bar(bars->s_full[x]));
                if (t == hi - 1) tc_commit(bar(bars->q_empty[x]));
              }
            } else {
              // O += P V once P is there (and O of the piece before has been read
              // out: by the warps that made this P)
              pass(bars->p_full[x], (par >> x) & 1);
              par ^= 1u << x;
              tc_fence_after();
              if (elect_one()) {
                const uint32_t more = t > lo ? 1u : 0u;
#pragma unroll 2
                for (int kk = 0; kk < 8; ++kk)
                  tc_mma_f16_ta(tmem + 256 + x * 128, tmem + 128 + x * 64 + kk * 8, desc_v + at + kk * (2048 >> 4), idesc_pv,
                                kk > 0 ? 1u : more);
                tc_commit(bar(bars->pv_done[x]));
              }
            }
            __syncwarp();
          }
          if (elect_one()) tc_commit(bar(bars->kv_empty[place]));
          __syncwarp();
          if (++place == behind) place = first, phase ^= 1;
        }
      }
      // Every MMA issued above completes before TMEM is released.
      if (elect_one()) tc_commit(bar(bars->drain));
      __syncwarp();
      volatile int no_abort = 0;
      wait_for(bar(bars->drain), 0, &no_abort, p.status);
      __syncwarp();
    }
  } else {
    // ---------------- softmax, epilogue, merge: a row per thread ----------------
    regs_up<216>();
    const int x = warp >> 2, quad = warp & 3;
    const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t t_s = t_lane, t_p = t_lane + 128 + x * 64, t_o = t_lane + 256 + x * 128;
    const uint64_t c2 = pk2(p.scale_log2, p.scale_log2);
    uint32_t* ready = reinterpret_cast<uint32_t*>(p.status) + PKC_CHUNK_READY;
    int n_s = 0, n_merge = 0;  // tiles, cut items so far
    Item it = {};
    bool ok = true;
    for (int k = 0; ok && next_item(k, it); ++k) {
      const int row0 = x * kHalf - it.off + quad * 32, row = row0 + lane;  // of the item; the warp's first one
      const int n_rows = it.n_tok << p.g_log2;
      const int pos = it.pos0 + (row >> p.g_log2);
      const bool valid = row >= 0 && row < n_rows;
      int rlo, rhi;
      tokens_of(p, pos, it.len, rlo, rhi);
      const int lo = x ? it.lo[1] : it.lo[0], hi = x ? it.hi[1] : it.hi[0];
      // tiles [full_lo, full_hi) that all the warp's rows attend to whole: the first
      // row's end and the last row's begin decide
      const int hi_min = __shfl_sync(0xffffffffu, rhi, 0), lo_max = __shfl_sync(0xffffffffu, rlo, 31);
      const int full_hi = hi_min >> 7, full_lo = (int)(((uint32_t)lo_max + kKv - 1) >> 7);
      float m_ref = neg_inf();
      bool all_set = false;  // every row of the warp has a reference
      uint64_t l2a = 0ull, l2b = 0ull;
      for (int t = lo; t < hi; ++t, ++n_s) {
        pass(bars->s_full[x], n_s & 1);
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld_32x32b_x32(t_s + 32 * j, v[j]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) reg_fence32(v[j]);
        tc_fence_before();
        arrive_warp(bar(bars->s_free), lane);
        if (t < full_lo || t >= full_hi) {
          const int c_lo = rlo - t * kKv, c_hi = rhi - t * kKv;  // columns the row attends to
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (t * kKv + 32 * j >= lo_max && hi_min - t * kKv >= 32 * j + 32) continue;  // uniform: kept by all rows
            const uint32_t keep = low_bits(c_hi - 32 * j) & ~low_bits(c_lo - 32 * j);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[j][i] = (keep >> i) & 1 ? v[j][i] : 0xff800000u;
          }
        }
        // P V of the half's tile before has read P and brought O up to date.
        if (n_s > 0) pass(bars->pv_done[x], (n_s - 1) & 1);
        tc_fence_after();
        bool move = t == lo || !all_set || n_rows <= kHalf;  // (few rows: every tile's maximum)
#pragma unroll 1
        for (;;) {
          if (move) {
            float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
            for (int i = 0; i < 32; i += 2)
#pragma unroll
              for (int j = 0; j < 4; ++j) mx[j] = max3(mx[j], __uint_as_float(v[j][i]), __uint_as_float(v[j][i + 1]));
            const float now = fmaxf(m_ref, __fmaf_rn(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), p.scale_log2, -kLift<T>));
            const float f = m_ref == neg_inf() ? 0.f : ex2(m_ref - now);
            const uint64_t f2 = pk2(f, f);
            l2a = fmul2(l2a, f2);
            l2b = fmul2(l2b, f2);
            m_ref = now;
            all_set = !__any_sync(0xffffffffu, now == neg_inf());
            if (t > lo && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
              for (int j = 0; j < 8; ++j) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(t_o + 16 * j, o);
                tmem_ld_wait();
                reg_fence16(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st_32x32b_x16(t_o + 16 * j, o);
              }
            }
          }
          const float neg = m_ref == neg_inf() ? 0.f : -m_ref;
          const uint64_t n2 = pk2(neg, neg);
          uint64_t sa = 0ull, sb = 0ull;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t pw[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 a =
                  upk2(ffma2(pk2(__uint_as_float(v[j][2 * i]), __uint_as_float(v[j][2 * i + 1])), c2, n2));
              const float p0 = ex2(a.x), p1 = ex2(a.y);
              if (i & 1) sb = fadd2(sb, pk2(p0, p1));
              else sa = fadd2(sa, pk2(p0, p1));
              pw[i] = Elem<T>::from_f2(p0, p1);
            }
            tmem_st_32x32b_x16(t_p + 16 * j, pw);
          }
          const float2 s2 = upk2(fadd2(sa, sb));
          // (Not twice for a tile: rows that are still above are far out, kFar.)
          move = !move && __any_sync(0xffffffffu, s2.x + s2.y > kMoveSum<T>);
          if (!move) {
            l2a = fadd2(l2a, sa);
            l2b = fadd2(l2b, sb);
            break;
          }
          tmem_st_wait();  // P again, to the same columns: stores are ordered by this alone
        }
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(bar(bars->p_full[x]), lane);
      }

      // The row's state.
      const bool cut = it.c0 != it.c1, mine = hi > lo, rows_here = row0 >= 0 && row0 < n_rows;  // (uniform)
      if (!cut && !mine && !rows_here) continue;
      const int slot = slot_of((int)blockIdx.x, it.c0);
      const int k_lo = max(rlo, it.t0 * kKv), k_hi = min(rhi, it.t1 * kKv);  // tokens of the piece that the row attends to
      const int64_t out = out_row(p, it.q_row, it.kvh, row);
      float l;
      {
        const float2 a = upk2(l2a), b = upk2(l2b);
        l = k_lo < k_hi ? (a.x + a.y) + (b.x + b.y) : 0.f;
      }
      const bool any = mine && l != 0.f;
      const float inv = any ? 1.f / l : 0.f;
      if (mine) pass(bars->pv_done[x], (n_s - 1) & 1);
      tc_fence_after();
      uint64_t finite = 0ull;  // 0 times all of the row's O
      const uint64_t inv2 = pk2(inv, inv);
#pragma unroll 1
      for (int j = 0; j < 4 && rows_here; ++j) {
        uint32_t v[32];
        float o[32];
        __syncwarp();  // the TMEM loads are the whole warp's
        if (mine) {    // uniform over the half
          tmem_ld_32x32b_x32(t_o + 32 * j, v);
          tmem_ld_wait();
          reg_fence32(v);
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint64_t y = any ? fmul2(pk2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), inv2) : 0ull;
          finite = ffma2(y, 0ull, finite);
          const float2 z = upk2(y);
          o[i] = z.x;
          o[i + 1] = z.y;
        }
        if (valid && !cut) store_out<T>(p, out, 32 * j, o);
        if (valid && cut) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(part_row(p, slot, 8 * j + i, row)) =
                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (valid) {
        if (!cut) p.lse[out] = any ? (m_ref + lg2(l)) * kLn2 : neg_inf();
        else *part_sum(p, slot, row) = make_float2(any ? m_ref : neg_inf(), any ? l : 0.f);
      }
      bool odd;
      {
        const float2 z = upk2(finite);
        odd = !(z.x + z.y == 0.f);
      }
      tc_fence_before();  // O has been read out: the next P's arrival says so
      const bool far = mine && m_ref != neg_inf() && !(fabsf(m_ref) < kFar<T>);
      if (const uint32_t todo = __ballot_sync(0xffffffffu, (odd || far) && valid); todo) {
        __syncwarp();  // the rows' stores by their own lanes come before those by all lanes
        const uint32_t f = __ballot_sync(0xffffffffu, far && valid);
        slow_rows<T>(p, f, todo & ~f, row0, it.b, it.kvh, it.q_row, it.pos0, it.len, lo, hi, lo_max, hi_min, cut ? slot : -1, abort);
      }

      if (cut) {
        // The block whose piece is the item's last one to be there merges all: a bit
        // per piece, and one per word of them where an item's pieces fill several.
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars->part_done));
        if (warp == 0) {
          const bool done = wait_for(bar(bars->part_done), n_merge & 1, abort, p.status);
          if (!__all_sync(0xffffffffu, done)) { ok = false; break; }
          if (lane == 0) {
            const int w = slot >> 5, w0 = it.c0 >> 4, w1 = it.c1 >> 4;
            __threadfence();
            bool last = set_bit(ready + w, slot & 31, pieces_of(it.c0 - 16 * w, it.c1 - 16 * w));
            if (last && w0 != w1) {
              __threadfence();
              last = set_bit(ready + kMaxBlocks / 16, slot_of(w, w0), pieces_of(w0, w1));
            }
            __threadfence();
            bars->merge = last;
            mbar_arrive(bar(bars->merge_go));
          }
          __syncwarp();
        }
        const bool go = wait_for(bar(bars->merge_go), n_merge & 1, abort, p.status);
        if (!__all_sync(0xffffffffu, go)) { ok = false; break; }
        ++n_merge;
        if (*(volatile int*)&bars->merge) merge_item<T>(p, it, warp, lane);
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc(tmem, 512);
}

bool make_maps(const ChunkParams& p, int dtype, CUtensorMap& mq, CUtensorMap& mk, CUtensorMap& mv) {
  const uint64_t row = PKC_HEAD_DIM * 2;
  const uint64_t qd[3] = {(uint64_t)PKC_HEAD_DIM, (uint64_t)p.hq, (uint64_t)p.total_q};
  const uint64_t qs[2] = {row, row * p.hq};
  const uint32_t qb[3] = {64u, (uint32_t)p.g, (uint32_t)(kHalf / p.g)};
  // (dim, head, slot, page) of the pool [num_pages][page_size][Hkv][128]
  const uint64_t d[4] = {(uint64_t)PKC_HEAD_DIM, (uint64_t)p.hkv, (uint64_t)p.page_size,
                         (uint64_t)std::max<int64_t>(1, p.num_pages)};
  const uint64_t st[3] = {row, row * p.hkv, row * p.hkv * p.page_size};
  const uint32_t box[4] = {64u, 1u, (uint32_t)p.box_tokens, 1u};
  return encode_tiled_map(&mq, p.q, dtype, 3, qd, qs, qb, true) &&
         encode_tiled_map(&mk, p.k_cache, dtype, 4, d, st, box, true) &&
         encode_tiled_map(&mv, p.v_cache, dtype, 4, d, st, box, true);
}

template <typename T>
int launch_t(const ChunkParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  if (const int e = raise_smem_limit((const void*)chunk_kernel<T>, kSmemBytes, raised)) return e;
  chunk_kernel<T><<<std::min(num_sms(), kMaxBlocks), kThreads, kSmemBytes, st>>>(mq, mk, mv, p);
  return (int)cudaGetLastError();
}

}  // namespace

size_t chunk_partial_bytes() { return (size_t)2 * kMaxBlocks * kRows * (PKC_HEAD_DIM + 2) * 4; }

int launch_paged_chunk(const ChunkParams& params, int dtype, void* stream) {
  ChunkParams p = params;
  p.part_ml = p.part_o + (size_t)2 * kMaxBlocks * kRows * PKC_HEAD_DIM;
  for (p.g_log2 = 0; 1 << p.g_log2 < p.g;) ++p.g_log2;
  p.o_wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
  p.scale_log2 = std::max(p.scale_log2, FLT_MIN);  // a scale of 0 must not meet a masked score's infinity
  for (p.box_tokens = 1; p.box_tokens < kKv && p.page_size % (2 * p.box_tokens) == 0;) p.box_tokens *= 2;
  CUtensorMap mq, mk, mv;
  if (!make_maps(p, dtype, mq, mk, mv)) return -1;
  return dtype == PKC_BF16 ? launch_t<__nv_bfloat16>(p, mq, mk, mv, (cudaStream_t)stream)
                           : launch_t<__half>(p, mq, mk, mv, (cudaStream_t)stream);
}

}  // namespace pkc
