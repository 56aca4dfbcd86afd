// Single-query paged decode over an mx4 (microscaled 4-bit) cache.
//
// The computation of the other paged decodes -- one query per request and
// head against the request's cached tokens, found through the block table,
// split into KV chunks by the host plan, each chunk an attention state --
// with keys k = 2^(s_b - 127) c_b per block b of 32 elements (format:
// mx4.cuh).  A token costs 68 bytes of K and 68 of V per KV head, half of
// the fp8 cache's, so the work per byte is what bounds the kernel: it keeps
// the conversions and the products on their fastest instructions.
//
// Scores.  S^T = K Q^T on m16n8k16 fp16 tiles (16 tokens x 8 query heads),
// the codes converted exactly, two per instruction.  The scales differ by
// token and block, so the four blocks have an accumulator each and
//   s = sum_b 2^(s_b - 127) acc_b
// is formed in float32 (of bf16 queries times 2^-22, see load_q_f16).
//
// Values.  O^T = V^T P^T, the dims on the tile's 16 rows.  The dims are 4
// blocks whose scales differ by token, so the scale goes on the
// probabilities, one power of two per token and block:
//   O_b += (p 2^(e_b - E_b)) c_b
// with E_b the largest scale byte seen so far in block b (O_b is rescaled
// when it grows).  Probabilities are 2^(s - r) with the reference r 11 below
// the largest score when it was set, rounded up, and at most 2^15 (r moves
// when a score exceeds it by more than 15; both hold for scores of any size,
// also where s - 11 is no float32 number).  They enter as an fp16 high part
// and an fp16 remainder, one product each; the products with the power of two
// are exact down to 2^-24.  So a probability enters with 22 bits, and what is
// lost is below 2^-24 of the largest cached |V| of the block of dims.
//
// Work split.  A block is one work item -- a planned chunk (or request)
// x HG KV heads -- of 4 warps; a warp takes every (4 / HG)-th group of 16
// tokens of one KV head and keeps its own ring of cp.async stages, so no
// warp waits for another until the item ends and any page size and head
// count works.  Four blocks (16 warps of 128 registers) per SM; most forms
// spill 4 to 48 bytes a thread to stay within that.
//
// Measured: 125 us for a batch of 256 with 32 / 8 heads over 476,458 tokens
// (523 MB, 4.2 TB/s of a measured copy rate of 6.8); 44 us for two requests
// of 107,000 tokens with 32 / 4 heads (117 MB), where the join, begun early,
// takes 10 us when it runs alone.  Bound by instructions, 356 per 16 tokens
// and head with up to 4 query heads per KV head, 432 with 8: 128 of the 356
// convert or feed the tensor cores, the rest are addresses, scales, softmax.
// Without the copies' bytes the first takes 5 us less, without the V product
// 21.
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "mx4.cuh"

namespace pkc {
namespace {

constexpr int D = PKC_HEAD_DIM;
constexpr int kWarps = 4;
constexpr int kBlocksPerSm = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                     // tokens per warp and step
constexpr int kStages = 4;
constexpr int kCodes = kTile * kMx4RowBytes;  // K (or V) code bytes per stage
constexpr int kScales = kTile * 4;
constexpr int kStage = 2 * (kCodes + kScales);
constexpr int kRing = kStages * kStage;       // per warp
constexpr int kWarpSmem = kRing + 128 + 256;  // + the tile's probability factors and key scales
constexpr float kRefFloor = -0x1.fffffep127f;  // softmax reference before the first token: the lowest number
constexpr float kLift = 11.f;                 // a new reference is this far below the largest score
constexpr float kMost = kLift + 4.f;          // log2 of the largest probability between rescales

struct Item {
  int valid, req, kb, ke, slot, hg;
};

// Shared memory: the warps' rings, the item, then the merge buffer (warps
// that share a KV head): per warp and head 128 values without the blocks'
// scales, the reference, the sum and the four scale bytes.
constexpr int kMergeRow = D + 4;
template <int G> constexpr int smem_bytes() { return kWarps * kWarpSmem + 64 + kWarps * G * kMergeRow * 4; }

// Byte of 16-byte piece c (0..3) of token t's codes within a stage: the
// fragment reads of K (two tokens t, t + 4 per 8 lanes) and V (tokens
// 4 i .. 4 i + 3, two pieces each, per 16 lanes) touch every bank once.
// Token t + 8 is 512 bytes behind token t.
__device__ __forceinline__ uint32_t code_at(int t, int c) {
  return (uint32_t)(((t >> 1) << 7) + (((t ^ (t >> 2)) & 1) << 6) + ((c ^ (((t >> 1) & 1) << 1)) << 4));
}
// Token of tile row r: rows 2 x, 2 x + 1 hold tokens x, x + 4 (of each 8).
__device__ __forceinline__ int token_of(int r) { return (r & 8) + ((r & 7) >> 1) + 4 * (r & 1); }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// kAligned: the page size is a multiple of 16, so a tile (tokens 16 i ..
// 16 i + 15) lies in one page.
template <typename T, int G, bool kAligned>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    paged_decode_mx4_kernel(const __grid_constant__ Mx4DecodeParams mp) {
  // With at most 4 query heads per KV head the tile's other 4 columns take
  // the probabilities' remainders, at no cost.
  constexpr bool kFold = G <= 4;
  constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;
  const DecodeParams& p = mp.d;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tg = lane & 3;
  Item* item_s = reinterpret_cast<Item*>(smem + kWarps * kWarpSmem);
  float* merge = reinterpret_cast<float*>(smem + kWarps * kWarpSmem + 64);
  const uint32_t ring = smem_u32(smem) + warp * kWarpSmem;
  const uint32_t wbuf = ring + kRing, kbuf = wbuf + 128;
  const int HG = mp.hg, wph = kWarps / HG;
  const int hh = warp % HG, cls = warp / HG;
  const PageDiv pages{p.page_size, mp.page_shift};

  grid_launch_dependents();  // the contraction may be scheduled beside this grid
  const int32_t* pl = p.plan;
  const int32_t hw = pl ? pl[lane] : 0;  // word `lane` of the plan's header
  if (pl && !device_plan_header_ok(hw, p.plan_words, p.batch)) {  // uniform over the grid
    if (threadIdx.x == 0) report(p.status, PKC_ERR_PLAN);
    return;
  }
  // Items: tickets of the shared queue (dynamic), this CTA's list of the plan
  // (static), or the request (no plan); fetched by warp 0.
  const bool dyn = pl && p.dynamic;
  int w_begin = 0, n_w = 1;
  if (pl && !dyn) {
    const int32_t* cta_indptr = pl + __shfl_sync(0xffffffffu, hw, PKC_PLAN_OFF_CTA_INDPTR);
    w_begin = cta_indptr[blockIdx.x];
    n_w = cta_indptr[blockIdx.x + 1] - w_begin;
  }
  DecodeQueue queue(p, HG, dyn && warp == 0, hw);
  DecodeItemWindow items;
  int li = 0, n_fetched = 0;
  auto fetch = [&]() {  // warp 0: the next item into shared memory (two slots)
    DecodeItem d{0, 0, 0, -1};
    int hg = (int)blockIdx.y;
    bool have;
    if (dyn) {
      have = queue.take(p, lane, d, hg);
    } else {
      have = li < n_w;
      if (have) d = items.get(p, blockIdx.x, w_begin, n_w, li, lane);
      ++li;
    }
    if (lane == 0) item_s[n_fetched & 1] = Item{have ? 1 : 0, d.req, d.kb, d.ke, d.slot, hg};
    ++n_fetched;
  };
  if (warp == 0) fetch();
  __syncthreads();

  for (int n_done = 0;; ++n_done) {
    const Item it = item_s[n_done & 1];
    if (!it.valid) break;
    const int kvh = it.hg * HG + hh;
    // This warp's tiles: number tile0 + j wph (tokens 16 x that), j < mine.
    const int tile0 = (it.kb >> 4) + cls;
    const int tiles_end = (it.ke + 15) >> 4;
    const int mine = it.kb < it.ke && tiles_end > tile0 ? (tiles_end - tile0 + wph - 1) / wph : 0;
    const int32_t* bt_row = p.block_table + (int64_t)it.req * p.bt_stride;
    // Pool index (page * page_size + slot) of a token, or kNoToken.
    auto pool_token = [&](int t) -> uint32_t {
      int page, slot;
      pages.split(t, page, slot);
      const int32_t pid = bt_row[page];
      if (pid < 0 || pid >= p.num_pages) {
        report(p.status, PKC_ERR_BLOCK_TABLE);
        return kNoToken;
      }
      return (uint32_t)pid * (uint32_t)p.page_size + (uint32_t)slot;
    };
    // Aligned: lane l holds the first token's pool index of tile j0 + l of a
    // window of 32; the next window is loaded 32 tiles ahead.  Otherwise: of
    // token l % 16 of the next tile.
    auto load_window = [&](int j0) -> uint32_t {
      const int j = j0 + lane;
      return j < mine ? pool_token((tile0 + j * wph) * kTile) : kNoToken;
    };
    auto load_tokens = [&](int j) -> uint32_t {
      const int t = (tile0 + j * wph) * kTile + (lane & 15);
      return j < mine && t >= it.kb && t < it.ke ? pool_token(t) : kNoToken;
    };
    uint32_t win = kAligned ? load_window(0) : load_tokens(0);
    uint32_t win_next = kAligned ? load_window(32) : 0u;

    uint32_t qf[4][4], key_mul;
    const float q_undo = load_q_f16<T, G, kFold>(
        static_cast<const T*>(p.q) + ((int64_t)it.req * p.hq + (int64_t)kvh * G) * D, lane, qf, key_mul);
    // factors of this lane's score columns (heads 2 tg, 2 tg + 1), base 2
    const float sc0 = p.scale_log2 * __shfl_sync(0xffffffffu, q_undo, 8 * tg);
    const float sc1 = p.scale_log2 * __shfl_sync(0xffffffffu, q_undo, 8 * tg + 4);
    // O^T: [block][elements i = 0, 1 | 2, 3][element 2 x: heads 2 tg, + 1; element 2 x + 1: the same]
    float o[4][2][4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int x = 0; x < 2; ++x) o[b][x][0] = o[b][x][1] = o[b][x][2] = o[b][x][3] = 0.f;
    float r0 = kRefFloor, r1 = kRefFloor, l0 = 0.f, l1 = 0.f;  // softmax references and sums
    int e_ref = 0;                                             // E_b of block lane % 4

    // Per lane, the pools at this head's bytes of token 0 and (aligned) the
    // lane's offset within a tile: codes at token g, piece tg, scales at token
    // lane % 16.  A tile's addresses follow from its first token by one wide
    // multiply-add and additions of uniform values.
    const uint32_t code_stride = (uint32_t)p.hkv * kMx4RowBytes, scale_stride = (uint32_t)p.hkv * 4;
    const uint64_t k_lane = reinterpret_cast<uint64_t>(p.k_cache) + kvh * kMx4RowBytes + 16 * tg +
                            (kAligned ? (uint64_t)g * code_stride : 0u);
    const uint64_t s_lane = reinterpret_cast<uint64_t>(lane < 16 ? mp.k_scales : mp.v_scales) + kvh * 4 +
                            (kAligned ? (uint64_t)(lane & 15) * scale_stride : 0u);
    const uint64_t v_minus_k = reinterpret_cast<uint64_t>(p.v_cache) - reinterpret_cast<uint64_t>(p.k_cache);
    const uint64_t code_8 = (uint64_t)code_stride * 8;
    uint32_t st_in = ring;  // stage of the next tile to be copied
    // Tokens that are there, of the tiles in flight, the latest in the low
    // bits: one bit per tile (aligned), or 16.
    using Present = std::conditional_t<kAligned, uint32_t, uint64_t>;
    constexpr int kPresentBits = kAligned ? 1 : 16;
    Present present = 0;
    auto issue = [&](int j) {  // copies of tile j (an empty group past the last one)
      present <<= kPresentBits;
      if (j < mine) {
        const uint32_t dst = st_in + code_at(g, tg);
        const uint32_t dst_s = st_in + 2 * kCodes + 4 * lane;  // scales: lanes 0..15 K, 16..31 V, token lane % 16
        if constexpr (kAligned) {
          if ((j & 31) == 0 && j > 0) {
            win = win_next;
            win_next = load_window(j + 32);
          }
          const uint32_t first = __shfl_sync(0xffffffffu, win, j & 31);
          if (first != kNoToken) {
            present |= 1u;
            const uint64_t ka = row_at(k_lane, first, code_stride), kb = ka + code_8;
            cp_async16(dst, ka);
            cp_async16(dst + 512, kb);
            cp_async16(dst + kCodes, ka + v_minus_k);
            cp_async16(dst + kCodes + 512, kb + v_minus_k);
            // scales of slots outside the chunk become 0: whatever they hold
            // must not count among the largest
            const int t = (tile0 + j * wph) * kTile + (lane & 15);
            cp_async4(dst_s, row_at(s_lane, first, scale_stride), t >= it.kb && t < it.ke);
          } else {  // no such page: zeros
            cp_async16(dst, k_lane, false);
            cp_async16(dst + 512, k_lane, false);
            cp_async16(dst + kCodes, k_lane, false);
            cp_async16(dst + kCodes + 512, k_lane, false);
            cp_async4(dst_s, s_lane, false);
          }
        } else {
          const uint32_t ts = win;
          present |= __ballot_sync(0xffffffffu, ts != kNoToken) & 0xffffu;
          const uint32_t ta = __shfl_sync(0xffffffffu, ts, g), tb = __shfl_sync(0xffffffffu, ts, g + 8);
          win = load_tokens(j + 1);
          const bool oka = ta != kNoToken, okb = tb != kNoToken, oks = ts != kNoToken;
          const uint64_t ka = row_at(k_lane, oka ? ta : 0u, code_stride), kb = row_at(k_lane, okb ? tb : 0u, code_stride);
          cp_async16(dst, ka, oka);
          cp_async16(dst + 512, kb, okb);
          cp_async16(dst + kCodes, ka + v_minus_k, oka);
          cp_async16(dst + kCodes + 512, kb + v_minus_k, okb);
          cp_async4(dst_s, row_at(s_lane, oks ? ts : 0u, scale_stride), oks);
        }
      }
      cp_async_commit();
      st_in = st_in == ring + (kStages - 1) * kStage ? ring : st_in + kStage;
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(s);

    // Tiles whose 16 tokens all belong to the chunk: j - whole_lo < n_whole.
    const int whole_lo = (it.kb & 15) && cls == 0 ? 1 : 0;
    const int whole_hi = mine - ((it.ke & 15) && tile0 + (mine - 1) * wph == (it.ke >> 4) ? 1 : 0);
    const uint32_t n_whole = (uint32_t)max(whole_hi - whole_lo, 0);
    const uint32_t byte_sel = (uint32_t)(tg | (4 + tg) << 4);  // byte tg of two words
    uint32_t st = ring;
    for (int j = 0; j < mine; ++j) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // tile j is in shared memory; tile j - 1's stage is free
      issue(j + kStages - 1);
      const uint32_t v_sc = st + 2 * kCodes + kScales;
      // ---- this tile's key scales and probability factors 2^(e - E) ----
      // lane 4 x + b: block b of tokens token_of(2 x), token_of(2 x + 1)
      {
        const uint32_t at = v_sc + 4 * token_of(2 * g);
        const uint32_t ya = lds32(at - kScales), yc = lds32(at - kScales + 16);
        uint32_t y2 = mx4_scale_pair(prmt(ya, yc, byte_sel));
        if constexpr (kBf16) y2 = bmul2(y2, key_mul);
        sts32(kbuf + 16 * token_of(2 * g) + 4 * tg, y2 << 16);
        sts32(kbuf + 16 * token_of(2 * g) + 64 + 4 * tg, y2 & 0xffff0000u);
        const uint32_t wa = lds32(at), wc = lds32(at + 16);
        const int ea = (int)((wa >> (8 * tg)) & 255u), ec = (int)((wc >> (8 * tg)) & 255u);
        int top = max(ea, ec);
        if (__any_sync(0xffffffffu, top > e_ref)) {
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = max(max(top, __shfl_xor_sync(0xffffffffu, top, 16)), e_ref);
          // 2^(E_old - E_new); 0 where it is below the smallest normal
          const float f = __int_as_float(max(127 + e_ref - top, 0) << 23);
          e_ref = top;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float fb = __shfl_sync(0xffffffffu, f, b);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              o[b][x][0] *= fb; o[b][x][1] *= fb; o[b][x][2] *= fb; o[b][x][3] *= fb;
            }
          }
        }
        // (fp16 holds 2^-24; below it the factor is 0)
        const float fa = __int_as_float(max(127 + ea - e_ref, 64) << 23);
        const float fc = __int_as_float(max(127 + ec - e_ref, 64) << 23);
        sts32(wbuf + 4 * lane, Elem<__half>::from_f2(fa, fc));
      }
      __syncwarp();
      // ---- S^T = K Q^T ----
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const int ta = token_of(g);  // this lane's rows: tokens ta, ta + 8
      {
        const uint32_t at = st + code_at(ta, tg);
        const uint4 ka = lds128(at), kb = lds128(at + 512);
        const uint4 fa = lds128(kbuf + 16 * ta), fb = lds128(kbuf + 16 * ta + 128);
        const uint32_t fka[4] = {fa.x, fa.y, fa.z, fa.w}, fkb[4] = {fb.x, fb.y, fb.z, fb.w};
        // words 0, 1: elements 0..3 of blocks (0, 1), (2, 3); words 2, 3: elements 4..7
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a0[4], a1[4], c0[4], c1[4];
          e2m1x8(half ? ka.y : ka.x, a0);
          e2m1x8(half ? ka.w : ka.z, a1);
          e2m1x8(half ? kb.y : kb.x, c0);
          e2m1x8(half ? kb.w : kb.z, c1);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int b = 2 * half + x;
            float acc[4];
            const uint32_t f0[4] = {a0[2 * x], c0[2 * x], a0[2 * x + 1], c0[2 * x + 1]};
            mma16816_f16_new(acc, f0, qf[b][0], qf[b][1]);
            const uint32_t f1[4] = {a1[2 * x], c1[2 * x], a1[2 * x + 1], c1[2 * x + 1]};
            mma16816<__half>(acc, f1, qf[b][2], qf[b][3]);
            s[0] = fmaf(acc[0], __uint_as_float(fka[b]), s[0]);
            s[1] = fmaf(acc[1], __uint_as_float(fka[b]), s[1]);
            s[2] = fmaf(acc[2], __uint_as_float(fkb[b]), s[2]);
            s[3] = fmaf(acc[3], __uint_as_float(fkb[b]), s[3]);
          }
        }
        s[0] *= sc0; s[1] *= sc1; s[2] *= sc0; s[3] *= sc1;
        // tokens outside the chunk, or without a page, take no part
        uint32_t here;  // one bit per token
        if constexpr (kAligned) here = (present & (1u << (kStages - 1))) ? 0xffffu : 0u;
        else here = (uint32_t)(present >> (16 * (kStages - 1))) & 0xffffu;
        if (here != 0xffffu || (uint32_t)(j - whole_lo) >= n_whole) {  // warp-uniform
          const int t_tile = (tile0 + j * wph) * kTile;
          const bool ok_a = ((here >> ta) & 1u) && t_tile + ta >= it.kb && t_tile + ta < it.ke;
          const bool ok_b = ((here >> (ta + 8)) & 1u) && t_tile + ta + 8 >= it.kb && t_tile + ta + 8 < it.ke;
          s[0] = ok_a ? s[0] : neg_inf();
          s[1] = ok_a ? s[1] : neg_inf();
          s[2] = ok_b ? s[2] : neg_inf();
          s[3] = ok_b ? s[3] : neg_inf();
        }
      }
      // ---- online softmax, base 2, lazy reference ----
      float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
      if (__any_sync(0xffffffffu, t0 - r0 > kMost || t1 - r1 > kMost)) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        const float n0 = fmaxf(__fadd_ru(t0, -kLift), r0), n1 = fmaxf(__fadd_ru(t1, -kLift), r1);
        const float c0 = ex2(r0 - n0), c1 = ex2(r1 - n1);
        r0 = n0;
        r1 = n1;
        l0 *= c0;
        l1 *= c1;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            o[b][x][0] *= c0; o[b][x][1] *= c1; o[b][x][2] *= c0; o[b][x][3] *= c1;
          }
      }
      const float p0 = ex2(s[0] - r0), p1 = ex2(s[1] - r1), p2 = ex2(s[2] - r0), p3 = ex2(s[3] - r1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      // high part and remainder, transposed into B fragments (tokens x heads)
      const uint32_t h01 = Elem<__half>::from_f2(p0, p1), h23 = Elem<__half>::from_f2(p2, p3);
      const float2 f01 = Elem<__half>::to_f2(h01), f23 = Elem<__half>::to_f2(h23);
      const uint32_t r01 = Elem<__half>::from_f2(p0 - f01.x, p1 - f01.y);
      const uint32_t r23 = Elem<__half>::from_f2(p2 - f23.x, p3 - f23.y);
      // (kFold: columns 4 .. 7 repeat heads 0 .. 3 and carry the remainders)
      const bool rest = kFold && tg >= 2;
      const uint32_t pa = movm_t(rest ? r01 : h01), pb = movm_t(rest ? r23 : h23);
      const uint32_t ra = kFold ? 0u : movm_t(r01), rb = kFold ? 0u : movm_t(r23);
      const uint4 wlo = lds128(wbuf + 16 * tg), whi = lds128(wbuf + 64 + 16 * tg);
      const uint32_t fl[4] = {wlo.x, wlo.y, wlo.z, wlo.w}, fh[4] = {whi.x, whi.y, whi.z, whi.w};
      // ---- O_b^T += V_b^T (p 2^(e_b - E_b)) ----
      const uint32_t vst = st + kCodes + 8 * (g & 1);
      const uint32_t va = vst + code_at(tg, g >> 1), vb = vst + code_at(tg + 4, g >> 1);
      const uint2 v0 = lds64(va), v1 = lds64(vb), v2 = lds64(va + 512), v3 = lds64(vb + 512);
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // blocks 2 half, 2 half + 1
        const uint32_t x0 = half ? v0.y : v0.x, x1 = half ? v1.y : v1.x;
        const uint32_t x2 = half ? v2.y : v2.x, x3 = half ? v3.y : v3.x;
        // bytes with the codes of one element of two tokens: elements i = 0, 2
        // of both blocks, then i = 1, 3
        uint32_t e02[4], f02[4], e13[4], f13[4];
        e2m1x8((x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u), e02);
        e2m1x8((x2 & 0x0f0f0f0fu) | ((x3 << 4) & 0xf0f0f0f0u), f02);
        e2m1x8(((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u), e13);
        e2m1x8(((x2 >> 4) & 0x0f0f0f0fu) | (x3 & 0xf0f0f0f0u), f13);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int b = 2 * half + x;
          const uint32_t hb0 = hmul2(pa, fl[b]), hb1 = hmul2(pb, fh[b]);
          uint32_t rb0 = 0, rb1 = 0;
          if constexpr (!kFold) {
            rb0 = hmul2(ra, fl[b]);
            rb1 = hmul2(rb, fh[b]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // elements 2 y (rows g), 2 y + 1 (rows g + 8)
            const uint32_t a[4] = {e02[2 * x + y], e13[2 * x + y], f02[2 * x + y], f13[2 * x + y]};
            mma16816<__half>(o[b][y], a, hb0, hb1);
            if constexpr (!kFold) mma16816<__half>(o[b][y], a, rb0, rb1);
          }
        }
      }
      st = st == ring + (kStages - 1) * kStage ? ring : st + kStage;
    }
    cp_async_wait<0>();

    // ---- end of the item ----
    // The next ticket only now: taken at the item's start it hides its look-ups
    // but spoils the longest-first order (GQA batch: 126 -> 139 us).
    if (warp == 0) fetch();
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if constexpr (kFold) {  // high parts (lanes tg < 2) + remainders (tg >= 2): both get the sum
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[b][x][i] += __shfl_xor_sync(0xffffffffu, o[b][x][i], 2);
    }
    // 4 dims of one (item, head): the partial slot, or the final output
    auto write4 = [&](int hq, int dim, float4 v) {
      if (it.slot >= 0) {
        *reinterpret_cast<float4*>(p.part_o + ((int64_t)it.slot * p.hq + hq) * D + dim) = v;
      } else {
        T* dst = static_cast<T*>(p.o_direct) + ((int64_t)it.req * p.hq + hq) * D + dim;
        *reinterpret_cast<uint2*>(dst) = make_uint2(Elem<T>::from_f2(v.x, v.y), Elem<T>::from_f2(v.z, v.w));
      }
    };
    auto write_lse = [&](int hq, float r, float ll) {
      const float lse = ll == 0.f ? neg_inf() : (r + lg2(ll)) * kLn2;
      if (it.slot >= 0) p.part_lse[(int64_t)it.slot * p.hq + hq] = lse;
      else p.lse_direct[(int64_t)it.req * p.hq + hq] = lse;
    };
    uint32_t e4 = (uint32_t)e_ref << (8 * tg);  // the scale bytes E_0 .. E_3
    e4 |= __shfl_xor_sync(0xffffffffu, e4, 1);
    e4 |= __shfl_xor_sync(0xffffffffu, e4, 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // heads 2 tg, 2 tg + 1: dims 32 b + 4 g .. + 3
      const int hd = 2 * tg + e;
      const float r = e ? r1 : r0, l = e ? l1 : l0;
      // The scale comes last: a value is a mean of codes times a power of two,
      // which neither overflows nor loses bits where the result does not.
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN sum gives NaN)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float4 v = make_float4(o[b][0][e], o[b][0][2 + e], o[b][1][e], o[b][1][2 + e]);
        if (wph == 1) {
          const float f = mx4_scale((e4 >> (8 * b)) & 255u);
          v = make_float4(v.x * inv * f, v.y * inv * f, v.z * inv * f, v.w * inv * f);
        }
        if (hd < G) {
          if (wph == 1) write4(kvh * G + hd, 32 * b + 4 * g, v);
          else *reinterpret_cast<float4*>(merge + (warp * G + hd) * kMergeRow + 32 * b + 4 * g) = v;
        }
      }
      if (hd < G && g == 0) {
        if (wph == 1) {
          write_lse(kvh * G + hd, r, l);
        } else {
          merge[(warp * G + hd) * kMergeRow + D] = r;
          merge[(warp * G + hd) * kMergeRow + D + 1] = l;
          merge[(warp * G + hd) * kMergeRow + D + 2] = __uint_as_float(e4);
        }
      }
    }
    __syncthreads();  // the next item is there; the warps' states are written
    if (wph > 1) {
      // Warps of one head: values, reference, sum and scale bytes, merged by a
      // warp per (KV head, query head) row, 4 dims (of block lane / 8) per lane.
      for (int r = warp; r < HG * G; r += kWarps) {
        const int h = r / G, hd = r - h * G;
        float ref = kRefFloor, ll = 0.f;
        int top = 0;  // the largest scale byte
        const auto scale_byte = [&](const float* src) { return (int)((__float_as_uint(src[D + 2]) >> (lane & 24)) & 255u); };
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < wph; ++c) {
          const float* src = merge + ((h + HG * c) * G + hd) * kMergeRow;
          ref = fmaxf(ref, src[D]);
          top = max(top, scale_byte(src));
        }
        for (int c = 0; c < wph; ++c) {
          const float* src = merge + ((h + HG * c) * G + hd) * kMergeRow;
          const float w = ex2(src[D] - ref);
          ll = fmaf(src[D + 1], w, ll);
          const float wv = w * __int_as_float(max(127 + scale_byte(src) - top, 0) << 23);  // (0 below 2^-126)
          const float4 v = *reinterpret_cast<const float4*>(src + 4 * lane);
          acc.x = fmaf(v.x, wv, acc.x); acc.y = fmaf(v.y, wv, acc.y);
          acc.z = fmaf(v.z, wv, acc.z); acc.w = fmaf(v.w, wv, acc.w);
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll, f = mx4_scale((uint32_t)top);
        acc = make_float4(acc.x * inv * f, acc.y * inv * f, acc.z * inv * f, acc.w * inv * f);
        const int hq = (it.hg * HG + h) * G + hd;
        write4(hq, 4 * lane, acc);
        if (lane == 0) write_lse(hq, ref, ll);
      }
      __syncthreads();  // the merge buffer is free
    }
  }
  if (dyn && warp == 0) queue.finish(lane);
}

// The join of split requests: one block per (request, query head) -- more
// rows each if the uploaded plan has more than the host's copy of it -- its kW
// warps taking every kW-th of the request's chunk states, lane i dims 4 i ..
// + 3; then the warps' sums through shared memory.  The n states' weights
// carry a factor 2^-ceil(log2 n), so that a sum of states near float32's
// largest number stays finite, as their mean does.  An empty request's row is
// (0, -inf).
template <typename T, int kW>
__global__ void __launch_bounds__(kW * 32) join_mx4_kernel(const __grid_constant__ Mx4JoinParams p) {
  __shared__ float4 part[kW][32];
  __shared__ float part_l[kW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = (int)(blockIdx.x % (unsigned)p.hq), stride = (int)(gridDim.x / (unsigned)p.hq);
  const int32_t* pl = p.plan;
  // The list and its places are the uploaded plan's, whatever the host's copy
  // says (a plan that is not there is reported by the decode).
  const int rows = device_plan_ok(pl, p.plan_words, p.batch) ? pl[PKC_PLAN_N_SPLIT] + pl[PKC_PLAN_N_EMPTY] : 0;
  const int off_list = pl[PKC_PLAN_OFF_UNIT_LIST], off_req = pl[PKC_PLAN_OFF_UNIT_REQ];
  const int off_n = pl[PKC_PLAN_OFF_UNIT_N_CHUNKS], off_first = pl[PKC_PLAN_OFF_UNIT_PARTIAL_BEGIN];
  bool waited = false;
  for (int row = (int)(blockIdx.x / (unsigned)p.hq); row < rows; row += stride) {
    const int unit = pl[off_list + row];
    const int n = pl[off_n + unit], first = pl[off_first + unit], req = pl[off_req + unit];
    if (!waited) grid_wait_prerequisites();  // the decode grid's states
    waited = true;
    const int64_t base = (int64_t)first * p.hq + hq;  // state c at base + c hq
    // This warp's first kAhead states are on their way while the largest LSE
    // is found (two long requests: 43.6 -> 42.9 us for both kernels; 8: 43.0).
    constexpr int kAhead = 4;
    float4 va[kAhead];
    float la[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int c = warp + k * kW;
      la[k] = neg_inf();
      va[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < n) {
        const int64_t at = base + (int64_t)c * p.hq;
        la[k] = p.part_lse[at];
        va[k] = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * lane);
      }
    }
    float m = neg_inf();
    for (int c = lane; c < n; c += 32) m = fmaxf(m, p.part_lse[base + (int64_t)c * p.hq]);
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float ref = m == neg_inf() ? 0.f : m;
    const int down = n > 1 ? 32 - __clz(n - 1) : 0;
    const float share = __int_as_float((127 - down) << 23);  // 2^-down
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float w = ex2((la[k] - ref) * kLog2e) * share;  // (0 past the end)
      l += w;
      acc.x = fmaf(va[k].x, w, acc.x); acc.y = fmaf(va[k].y, w, acc.y);
      acc.z = fmaf(va[k].z, w, acc.z); acc.w = fmaf(va[k].w, w, acc.w);
    }
#pragma unroll 4
    for (int c = warp + kAhead * kW; c < n; c += kW) {
      const int64_t at = base + (int64_t)c * p.hq;
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * lane);
      const float w = ex2((p.part_lse[at] - ref) * kLog2e) * share;
      l += w;
      acc.x = fmaf(v.x, w, acc.x); acc.y = fmaf(v.y, w, acc.y);
      acc.z = fmaf(v.z, w, acc.z); acc.w = fmaf(v.w, w, acc.w);
    }
    part[warp][lane] = acc;
    if (lane == 0) part_l[warp] = l;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int x = 1; x < kW; ++x) {
        const float4 v = part[x][lane];
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
        l += part_l[x];
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T* dst = static_cast<T*>(p.o) + ((int64_t)req * p.hq + hq) * D + 4 * lane;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(Elem<T>::from_f2(acc.x * inv, acc.y * inv), Elem<T>::from_f2(acc.z * inv, acc.w * inv));
      if (lane == 0) p.lse[(int64_t)req * p.hq + hq] = l == 0.f ? neg_inf() : ref + (lg2(l) + (float)down) * kLn2;
    }
    __syncthreads();  // `part` is free
  }
  if (!waited) grid_wait_prerequisites();  // (at every exit: what follows this grid must not overtake the decode's)
}

template <typename T, int G>
int launch_g(const Mx4DecodeParams& p, dim3 grid, cudaStream_t st) {
  constexpr int smem = smem_bytes<G>();
  static_assert(kBlocksPerSm * (smem + 1024) <= 228 * 1024, "resident blocks");
  const bool aligned = p.d.page_size % kTile == 0;
  auto kernel = aligned ? paged_decode_mx4_kernel<T, G, true> : paged_decode_mx4_kernel<T, G, false>;
  static std::atomic<uint64_t> raised[2];
  if (const int e = raise_smem_limit(reinterpret_cast<const void*>(kernel), smem, raised[aligned])) return e;
  kernel<<<grid, kThreads, smem, st>>>(p);
  return (int)cudaGetLastError();
}

template <typename T>
int launch_t(const Mx4DecodeParams& p, dim3 grid, cudaStream_t st) {
  switch (p.d.hq / p.d.hkv) {
    case 1: return launch_g<T, 1>(p, grid, st);
    case 2: return launch_g<T, 2>(p, grid, st);
    case 4: return launch_g<T, 4>(p, grid, st);
    case 8: return launch_g<T, 8>(p, grid, st);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace

int launch_paged_decode_mx4(const Mx4DecodeParams& p_in, int n_work, int dtype, void* stream) {
  Mx4DecodeParams p = p_in;
  p.d.dynamic = p.d.plan != nullptr && decode_schedule_dynamic() != 0;
  p.d.sched = p.d.status + 16;
  const int hkv = p.d.hkv;
  p.hg = hkv % 4 == 0 ? 4 : hkv % 2 == 0 ? 2 : 1;
  // Fewer heads per block (more warps per head) while the items leave room
  // for more blocks: a small batch's time is that of one warp's tiles.
  const int64_t items = p.d.plan ? n_work : p.d.batch;
  // Two heads also where four would give fewer than two items a block: half
  // the item balances better (GQA batch of 256, 1000 items of four heads: 147
  // -> 136 us), while one head per block costs more merging than it gains
  // where two fill the machine (two long requests: 54 -> 59 us).
  const int64_t slots = kBlocksPerSm * (int64_t)num_sms();
  if (p.hg == 4 && items * (hkv / 4) < 2 * slots) p.hg = 2;
  while (p.hg > 1 && items * (hkv / p.hg) < slots) p.hg /= 2;
  dim3 grid;
  if (p.d.dynamic) {
    const int64_t n = items * (hkv / p.hg);
    grid = dim3((unsigned)(n < 1 ? 1 : n < slots ? n : slots));
  } else {
    grid = dim3((unsigned)(p.d.plan ? p.num_ctas : p.d.batch), (unsigned)(hkv / p.hg));
  }
  cudaStream_t st = (cudaStream_t)stream;
  return dtype == PKC_BF16 ? launch_t<__nv_bfloat16>(p, grid, st) : launch_t<__half>(p, grid, st);
}

int launch_join_mx4(const Mx4JoinParams& p, int n_rows, int n_states, int dtype, void* stream) {
  const int64_t blocks = (int64_t)(n_rows < 1 ? 1 : n_rows) * p.hq;
  if (blocks > INT32_MAX) return (int)cudaErrorInvalidValue;
  // Launched as the decode's programmatic dependent: the blocks start as the
  // decode's end.  Rows of many states (a long request alone on the machine
  // has one per CTA) get 16 warps, so that all its states are in flight at
  // once; rows of a few, 4.
  const dim3 grid((unsigned)blocks);
  cudaStream_t st = (cudaStream_t)stream;
  const bool many = n_states > 16 * (int64_t)n_rows, bf16 = dtype == PKC_BF16;
  if (many)
    return bf16 ? launch_programmatic(join_mx4_kernel<__nv_bfloat16, 16>, grid, dim3(512), 0, st, p)
                : launch_programmatic(join_mx4_kernel<__half, 16>, grid, dim3(512), 0, st, p);
  return bf16 ? launch_programmatic(join_mx4_kernel<__nv_bfloat16, 4>, grid, dim3(128), 0, st, p)
              : launch_programmatic(join_mx4_kernel<__half, 4>, grid, dim3(128), 0, st, p);
}

}  // namespace pkc
