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
// is formed in float32.
//
// Values.  O^T's 128 dims are 4 blocks whose scales differ by token, so the
// scale goes on the probabilities, one power of two per token and block:
//   O_b += (p 2^(e_b - E_b + 11)) c_b
// with E_b the largest scale byte seen so far in block b (O_b is rescaled
// when it grows) and p <= 2^4 (the softmax reference moves when a score
// exceeds it by more).  A probability enters as an fp16 high part in rows
// 0..7 of the tile and its remainder times 2^11 in rows 8..15, both at the
// cost of one product; the product with the power of two is exact down to
// 2^-24, where the largest are 2^11 and more.  So the error is at most 2^-22
// of the weights plus 2^-25 of the largest cached |V| of the block of dims.
//
// Work split.  A block is one work item -- a planned chunk (or request)
// x HG KV heads -- of 4 warps; a warp takes every (4 / HG)-th group of 16
// tokens of one KV head and keeps its own ring of cp.async stages, so no
// warp waits for another until the item ends and any page size and head
// count works.  The accumulators take 64 registers a thread: three blocks
// (12 warps) per SM leave 160; at 16 warps and 128 the kernel spills.
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "mx4.cuh"

namespace pkc {
namespace {

constexpr int D = PKC_HEAD_DIM;
constexpr int kWarps = 4;
constexpr int kBlocksPerSm = 3;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                     // tokens per warp and step
constexpr int kStages = 4;
constexpr int kCodes = kTile * kMx4RowBytes;  // K (or V) code bytes per stage
constexpr int kScales = kTile * 4;
constexpr int kValid = 2 * (kCodes + kScales);  // two words: bit 4 t of word k, token t + 8 k takes part
constexpr int kStage = kValid + 128;
constexpr int kRing = kStages * kStage;       // per warp
constexpr int kWarpSmem = kRing + 128;        // + the tile's probability factors
constexpr float kRefFloor = -3e38f;           // softmax reference before the first token
constexpr float kLazy = 4.f;                  // log2 of the largest probability between rescales

struct Item {
  int valid, req, kb, ke, slot, hg;
};

// Shared memory: the warps' rings, the item, then the merge buffer (warps
// that share a KV head): per warp and head 128 values, the reference and the
// sum.
template <int G> constexpr int smem_bytes() { return kWarps * kWarpSmem + 64 + kWarps * G * (D + 2) * 4; }

// Byte of 16-byte piece c (0..3) of token t's codes within a stage: the
// fragment reads of K (two tokens t, t + 4 per 8 lanes) and V (tokens
// 4 i .. 4 i + 3, two pieces each, per 16 lanes) touch every bank once.
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

template <typename T, int G>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    paged_decode_mx4_kernel(const __grid_constant__ Mx4DecodeParams mp) {
  const DecodeParams& p = mp.d;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tg = lane & 3;
  Item* item_s = reinterpret_cast<Item*>(smem + kWarps * kWarpSmem);
  float* merge = reinterpret_cast<float*>(smem + kWarps * kWarpSmem + 64);
  const uint32_t ring = smem_u32(smem) + warp * kWarpSmem;
  const uint32_t wbuf = ring + kRing;
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
  int li = 0;
  auto fetch = [&]() {  // warp 0: the next item into shared memory
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
    if (lane == 0) *item_s = Item{have ? 1 : 0, d.req, d.kb, d.ke, d.slot, hg};
  };
  if (warp == 0) fetch();
  __syncthreads();

  while (true) {
    const Item it = *item_s;
    if (!it.valid) break;
    const int kvh = it.hg * HG + hh;
    uint32_t qf[4][4];
    const float q_undo = load_q_f16<T, G>(
        static_cast<const T*>(p.q) + ((int64_t)it.req * p.hq + (int64_t)kvh * G) * D, lane, qf);
    // factors of this lane's score columns (heads 2 tg, 2 tg + 1), base 2
    const float sc0 = p.scale_log2 * __shfl_sync(0xffffffffu, q_undo, 8 * tg);
    const float sc1 = p.scale_log2 * __shfl_sync(0xffffffffu, q_undo, 8 * tg + 4);
    float o[4][4][4];  // [block][element i][rows g: high part, rows g + 8: remainder]
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.f;
    float m0 = kRefFloor, m1 = kRefFloor, l0 = 0.f, l1 = 0.f;
    int e_ref = 0;  // E_b of block lane % 4

    const int n_tiles = it.kb < it.ke ? (it.ke - it.kb + kTile - 1) / kTile : 0;
    const int mine = n_tiles > cls ? (n_tiles - cls + wph - 1) / wph : 0;  // this warp's tiles
    const int32_t* bt_row = p.block_table + (int64_t)it.req * p.bt_stride;
    // Lane's tokens of tile j: lane / 4 and lane / 4 + 8.
    auto tile_token = [&](int j) { return it.kb + (cls + j * wph) * kTile; };
    int32_t pid[2] = {0, 0};
    auto load_pages = [&](int j) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        pid[k] = 0;
        if (j >= mine) continue;
        const int t = tile_token(j) + g + 8 * k;
        if (t < it.ke) {
          int page, slot;
          pages.split(t, page, slot);
          pid[k] = bt_row[page];
        }
      }
    };
    auto issue = [&](int j) {  // copies of tile j (an empty group past the last one)
      if (j < mine) {
        const uint32_t st = ring + (j % kStages) * kStage;
        int64_t row[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = tile_token(j) + g + 8 * k;
          int page, slot;
          pages.split(t, page, slot);
          bool ok = t < it.ke;
          if (ok && (pid[k] < 0 || pid[k] >= p.num_pages)) {
            if (tg == 0) report(p.status, PKC_ERR_BLOCK_TABLE);
            ok = false;
          }
          row[k] = ok ? ((int64_t)pid[k] * p.page_size + slot) * p.hkv + kvh : -1;
          const uint32_t takes_part = __ballot_sync(0xffffffffu, ok);
          if (lane == 0) sts32(st + kValid + 4 * k, takes_part);
          const uint32_t dst = st + code_at(g + 8 * k, tg);
          const int64_t at = max(row[k], (int64_t)0) * kMx4RowBytes + 16 * tg;
          cp_async16(dst, static_cast<const uint8_t*>(p.k_cache) + at, ok);
          cp_async16(dst + kCodes, static_cast<const uint8_t*>(p.v_cache) + at, ok);
        }
        // scales: lanes 0..15 K, 16..31 V, token lane % 16
        const int64_t ra = __shfl_sync(0xffffffffu, row[0], 4 * (lane & 7));
        const int64_t rb = __shfl_sync(0xffffffffu, row[1], 4 * (lane & 7));
        const int64_t r = (lane & 8) ? rb : ra;
        const uint8_t* src = static_cast<const uint8_t*>(lane < 16 ? mp.k_scales : mp.v_scales);
        cp_async4(st + 2 * kCodes + (lane >> 4) * kScales + 4 * (lane & 15), src + max(r, (int64_t)0) * 4, r >= 0);
      }
      cp_async_commit();
    };
    load_pages(0);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      issue(s);
      load_pages(s + 1);
    }

    for (int j = 0; j < mine; ++j) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // tile j is in shared memory; tile j - 1's stage is free
      issue(j + kStages - 1);
      load_pages(j + kStages);
      const uint32_t st = ring + (j % kStages) * kStage;
      const uint32_t k_sc = st + 2 * kCodes, v_sc = k_sc + kScales;
      // ---- this tile's probability factors 2^(e - E + 11) ----
      // lane 4 x + b: block b of tokens token_of(2 x), token_of(2 x + 1)
      {
        const int t = token_of(2 * g);
        const uint32_t wa = lds32(v_sc + 4 * t), wc = lds32(v_sc + 4 * t + 16);
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
            for (int i = 0; i < 4; ++i) {
              o[b][i][0] *= fb; o[b][i][1] *= fb; o[b][i][2] *= fb; o[b][i][3] *= fb;
            }
          }
        }
        // fp16 bits of 2^(d + 11), d = e - E: (d + 26) << 10, zero below
        const uint32_t fa = (uint32_t)max(ea - e_ref + 26, 0), fc = (uint32_t)max(ec - e_ref + 26, 0);
        sts32(wbuf + 4 * lane, (fa << 10) | (fc << 26));
      }
      // ---- S^T = K Q^T ----
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int ta = token_of(g), tb = ta + 8;
        const uint4 ka = lds128(st + code_at(ta, tg)), kb = lds128(st + code_at(tb, tg));
        const uint32_t sa = lds32(k_sc + 4 * ta), sb = lds32(k_sc + 4 * tb);
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
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t f0[4] = {a0[2 * x], c0[2 * x], a0[2 * x + 1], c0[2 * x + 1]};
            mma16816<__half>(acc, f0, qf[b][0], qf[b][1]);
            const uint32_t f1[4] = {a1[2 * x], c1[2 * x], a1[2 * x + 1], c1[2 * x + 1]};
            mma16816<__half>(acc, f1, qf[b][2], qf[b][3]);
            // (255: an infinity, NaN on the zero codes it comes with)
            const float fa = __uint_as_float((b < 3 ? sa << (23 - 8 * b) : sa >> 1) & 0x7f800000u);
            const float fb = __uint_as_float((b < 3 ? sb << (23 - 8 * b) : sb >> 1) & 0x7f800000u);
            s[0] = fmaf(acc[0], fa, s[0]);
            s[1] = fmaf(acc[1], fa, s[1]);
            s[2] = fmaf(acc[2], fb, s[2]);
            s[3] = fmaf(acc[3], fb, s[3]);
          }
        }
        const uint2 takes_part = lds64(st + kValid);
        const bool ok_a = (takes_part.x >> (4 * ta)) & 1u, ok_b = (takes_part.y >> (4 * ta)) & 1u;
        s[0] = ok_a ? s[0] * sc0 : neg_inf();
        s[1] = ok_a ? s[1] * sc1 : neg_inf();
        s[2] = ok_b ? s[2] * sc0 : neg_inf();
        s[3] = ok_b ? s[3] * sc1 : neg_inf();
      }
      // ---- online softmax, base 2, lazy reference ----
      float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
      if (__any_sync(0xffffffffu, t0 > m0 + kLazy || t1 > m1 + kLazy)) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        const float n0 = fmaxf(t0, m0), n1 = fmaxf(t1, m1);
        const float c0 = ex2(m0 - n0), c1 = ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= c0;
        l1 *= c1;
        // rows g of O are head g: column g of the scores, held by lanes tg = g / 2
        const float ca = __shfl_sync(0xffffffffu, c0, g >> 1), cb = __shfl_sync(0xffffffffu, c1, g >> 1);
        const float c = (g & 1) ? cb : ca;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[b][i][0] *= c; o[b][i][1] *= c; o[b][i][2] *= c; o[b][i][3] *= c;
          }
      }
      const float p0 = ex2(s[0] - m0), p1 = ex2(s[1] - m1), p2 = ex2(s[2] - m0), p3 = ex2(s[3] - m1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      const uint32_t h01 = Elem<__half>::from_f2(p0, p1), h23 = Elem<__half>::from_f2(p2, p3);
      const float2 f01 = Elem<__half>::to_f2(h01), f23 = Elem<__half>::to_f2(h23);
      const uint32_t r01 = Elem<__half>::from_f2((p0 - f01.x) * 2048.f, (p1 - f01.y) * 2048.f);
      const uint32_t r23 = Elem<__half>::from_f2((p2 - f23.x) * 2048.f, (p3 - f23.y) * 2048.f);
      const uint32_t pa = movm_t(h01), pb = movm_t(r01), pc = movm_t(h23), pd = movm_t(r23);
      __syncwarp();  // the factors are in shared memory
      const uint4 wlo = lds128(wbuf + 16 * tg), whi = lds128(wbuf + 64 + 16 * tg);
      const uint32_t fl[4] = {wlo.x, wlo.y, wlo.z, wlo.w}, fh[4] = {whi.x, whi.y, whi.z, whi.w};
      // ---- O_b += (p 2^(e_b - E_b + 11)) V_b ----
      const uint32_t vst = st + kCodes + 8 * (g & 1);
      const uint2 v0 = lds64(vst + code_at(tg, g >> 1)), v1 = lds64(vst + code_at(tg + 4, g >> 1));
      const uint2 v2 = lds64(vst + code_at(tg + 8, g >> 1)), v3 = lds64(vst + code_at(tg + 12, g >> 1));
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
          const uint32_t a[4] = {hmul2(pa, fl[b]), hmul2(pb, fl[b]), hmul2(pc, fh[b]), hmul2(pd, fh[b])};
          mma16816<__half>(o[b][0], a, e02[2 * x], f02[2 * x]);
          mma16816<__half>(o[b][1], a, e13[2 * x], f13[2 * x]);
          mma16816<__half>(o[b][2], a, e02[2 * x + 1], f02[2 * x + 1]);
          mma16816<__half>(o[b][3], a, e13[2 * x + 1], f13[2 * x + 1]);
        }
      }
    }
    cp_async_wait<0>();

    // ---- end of the item ----
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    // lane's head is g: its reference and sum, from a lane of columns g
    const float ma = __shfl_sync(0xffffffffu, m0, g >> 1), mb = __shfl_sync(0xffffffffu, m1, g >> 1);
    const float la = __shfl_sync(0xffffffffu, l0, g >> 1), lb = __shfl_sync(0xffffffffu, l1, g >> 1);
    const float m = (g & 1) ? mb : ma, l = (g & 1) ? lb : la;
    float val[4][8];  // dims 32 b + 8 tg + 0..7 of head g
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float f = mx4_scale((uint32_t)__shfl_sync(0xffffffffu, e_ref, b));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        val[b][i] = fmaf(o[b][i][2], 0x1p-11f, o[b][i][0]) * 0x1p-11f * f;
        val[b][4 + i] = fmaf(o[b][i][3], 0x1p-11f, o[b][i][1]) * 0x1p-11f * f;
      }
    }
    // 8 dims of one (item, head): the partial slot, or the final output
    auto write8 = [&](int hq, int dim, const float (&v)[8]) {
      if (it.slot >= 0) {
        float4* dst = reinterpret_cast<float4*>(p.part_o + ((int64_t)it.slot * p.hq + hq) * D + dim);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        T* dst = static_cast<T*>(p.o_direct) + ((int64_t)it.req * p.hq + hq) * D + dim;
        *reinterpret_cast<uint4*>(dst) = make_uint4(Elem<T>::from_f2(v[0], v[1]), Elem<T>::from_f2(v[2], v[3]),
                                                    Elem<T>::from_f2(v[4], v[5]), Elem<T>::from_f2(v[6], v[7]));
      }
    };
    auto write_lse = [&](int hq, float mm, float ll) {
      const float lse = ll == 0.f ? neg_inf() : (mm + lg2(ll)) * kLn2;
      if (it.slot >= 0) p.part_lse[(int64_t)it.slot * p.hq + hq] = lse;
      else p.lse_direct[(int64_t)it.req * p.hq + hq] = lse;
    };
    if (wph == 1) {
      if (g < G) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN sum gives NaN)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
#pragma unroll
          for (int i = 0; i < 8; ++i) val[b][i] *= inv;
          write8(kvh * G + g, 32 * b + 8 * tg, val[b]);
        }
        if (tg == 0) write_lse(kvh * G + g, m, l);
      }
      __syncthreads();  // every warp has read the item
      if (warp == 0) fetch();
      __syncthreads();
      continue;
    }
    // Warps of one head: unnormalised values, reference and sum through
    // shared memory, merged by half a warp per (KV head, query head) row.
    if (g < G) {
      float* dst = merge + (warp * G + g) * (D + 2);
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          *reinterpret_cast<float2*>(dst + 32 * b + 8 * tg + i) = make_float2(val[b][i], val[b][i + 1]);
      if (tg == 0) {
        dst[D] = m;
        dst[D + 1] = l;
      }
    }
    __syncthreads();
    if (warp == 0) fetch();
    for (int r = 2 * warp + (lane >> 4); r < HG * G; r += 2 * kWarps) {  // 8 dims per lane
      const int h = r / G, hd = r - h * G, dim = 8 * (lane & 15);
      float mm = kRefFloor, ll = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < wph; ++c) mm = fmaxf(mm, merge[((h + HG * c) * G + hd) * (D + 2) + D]);
      for (int c = 0; c < wph; ++c) {
        const float* src = merge + ((h + HG * c) * G + hd) * (D + 2);
        const float w = ex2(src[D] - mm);
        ll = fmaf(src[D + 1], w, ll);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(src[dim + i], w, acc[i]);
      }
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] *= inv;
      const int hq = (it.hg * HG + h) * G + hd;
      write8(hq, dim, acc);
      if ((lane & 15) == 0) write_lse(hq, mm, ll);
    }
    __syncthreads();  // the merge buffer and the item are free
  }
  if (dyn && warp == 0) queue.finish(lane);
}

template <typename T, int G>
int launch_g(const Mx4DecodeParams& p, dim3 grid, cudaStream_t st) {
  constexpr int smem = smem_bytes<G>();
  static_assert(kBlocksPerSm * (smem + 1024) <= 228 * 1024, "resident blocks");
  // (an attribute of the current device: set on every call, it is cheap)
  const cudaError_t e = cudaFuncSetAttribute(paged_decode_mx4_kernel<T, G>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return (int)e;
  paged_decode_mx4_kernel<T, G><<<grid, kThreads, smem, st>>>(p);
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
  // Fewer heads per block (more warps per head) while the items leave SMs
  // without a block: a small batch's time is that of one warp's tiles.
  const int64_t items = p.d.plan ? n_work : p.d.batch;
  while (p.hg > 1 && items * (hkv / p.hg) < num_sms()) p.hg /= 2;
  dim3 grid;
  if (p.d.dynamic) {
    const int64_t n = items * (hkv / p.hg), most = kBlocksPerSm * (int64_t)num_sms();
    grid = dim3((unsigned)(n < 1 ? 1 : n < most ? n : most));
  } else {
    grid = dim3((unsigned)(p.d.plan ? p.num_ctas : p.d.batch), (unsigned)(hkv / p.hg));
  }
  cudaStream_t st = (cudaStream_t)stream;
  return dtype == PKC_BF16 ? launch_t<__nv_bfloat16>(p, grid, st) : launch_t<__half>(p, grid, st);
}

}  // namespace pkc
