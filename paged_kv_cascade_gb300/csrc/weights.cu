// Accumulated attention weights over a paged cache.
//
// For request b, KV head h and cached token t, given the step's queries and
// their log-sum-exps (of whatever set of keys the step attended to: the
// cache alone, or a cascade's prefix and suffix):
//   w[b, h, t] <- decay w[b, h, t] + sum over h's query heads of
//                 exp(sm_scale q . k_t - lse)
// which is the statistic that evictions go by.  The kernel reads every cached
// key once (256, 128 or 68 bytes per token and KV head) and each weight once,
// writes each weight once, and is bound by HBM.
//
// A warp takes 16 tokens of one KV head at a time: S^T = K Q^T on m16n8k16
// tiles (tokens x query heads), as in the tensor-core decode.  Which element
// stands where in the products' inner dimension is free as long as K and Q
// agree, so each lane loads 16 consecutive bytes of its two tokens' rows
// straight from global memory into the fragment registers -- no shared
// memory, no barrier.  The loads of the next step are issued before the
// current one is used; the page ids of the step after that before those.
//
// No two warps touch the same weight: results do not depend on the order of
// anything.
//
// Measured: bf16 keys, 64 requests, 164,506 tokens of 8 heads: 59 us (348 MB,
// 5.9 TB/s of a measured copy rate of 6.8).  mx4 keys, 256 requests, 476,458
// tokens: 74 us (292 MB, 3.9 TB/s), bound by the conversions' and scales'
// instructions, not by bytes.
#include <cuda_runtime.h>

#include <algorithm>

#include "mx4.cuh"

namespace pkc {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int D = PKC_HEAD_DIM;

template <int KV> struct KeyTraits;
// kPieces: 16-byte pieces of a row per lane; kTiles: tiles of 16 tokens per
// step; kSteps: steps in registers (the one in use and those on their way)
template <> struct KeyTraits<PKC_F16> { static constexpr int kSteps = 2, kPieces = 4, kTiles = 1, kRow = 256; };
template <> struct KeyTraits<PKC_BF16> { static constexpr int kSteps = 2, kPieces = 4, kTiles = 1, kRow = 256; };
template <> struct KeyTraits<PKC_E4M3> { static constexpr int kSteps = 2, kPieces = 2, kTiles = 2, kRow = 128; };
template <> struct KeyTraits<PKC_MX4> { static constexpr int kSteps = 4, kPieces = 1, kTiles = 1, kRow = kMx4RowBytes; };

// One step's loads of a lane: rows g and g + 8 of each tile.
template <int KV> struct Loads {
  static constexpr int P = KeyTraits<KV>::kPieces, U = KeyTraits<KV>::kTiles;
  uint4 k[U][2][P];
  uint32_t scale[U][2];
  float old[U];
  uint32_t ok;  // bit 2 u + i: row i of tile u is there
};

// kAligned: the page size is a multiple of 16, so a tile (tokens 16 i ..
// 16 i + 15) lies in one page.
template <int KV, typename T, int G, bool kAligned>
__global__ void __launch_bounds__(kThreads, 4) weights_kernel(const WeightsParams p) {
  using KT = KeyTraits<KV>;
  constexpr int U = KT::kTiles, P = KT::kPieces, kStep = 16 * U;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tg = lane & 3;
  const int wph = kWarps / p.hg;  // warps per KV head
  const int seg = (int)(blockIdx.x % p.n_seg);
  const int bh = (int)(blockIdx.x / p.n_seg);
  const int n_hg = p.hkv / p.hg;
  const int b = bh / n_hg, kvh = (bh % n_hg) * p.hg + warp % p.hg;

  int len = p.cache_seqlens[b];
  if (len > p.bt_stride * (int64_t)p.page_size) {
    if (seg == 0 && threadIdx.x == 0) report(p.status, PKC_ERR_BLOCK_TABLE);
    len = (int)(p.bt_stride * p.page_size);
  }
  if (len > p.w_stride) {
    if (seg == 0 && threadIdx.x == 0) report(p.status, PKC_ERR_PLAN);
    len = (int)p.w_stride;
  }
  const int64_t t_first = (int64_t)seg * p.seg_tokens + (warp / p.hg) * kStep;
  const int t_end = (int)min((int64_t)len, ((int64_t)seg + 1) * p.seg_tokens);
  if (t_first >= t_end) return;
  const int t_begin = (int)t_first, t_step = wph * kStep;
  const int steps = (t_end - t_begin + t_step - 1) / t_step;

  const int32_t* bt_row = p.block_table + (int64_t)b * p.bt_stride;
  float* w_row = p.weights + ((int64_t)b * p.hkv + kvh) * p.w_stride;
  const PageDiv pages{p.page_size, p.page_shift};
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
  // Aligned: lane l holds the pool index of the first token of the warp's
  // tile l (a segment has at most 32 a warp).  Otherwise: lane l that of
  // token l of the next step's (at most 32).
  auto load_tiles = [&]() -> uint32_t {
    const int t = t_begin + (lane / U) * t_step + 16 * (lane % U);
    return lane < steps * U && t < t_end ? pool_token(t) : kNoToken;
  };
  auto load_tokens = [&](int s) -> uint32_t {
    const int t = t_begin + s * t_step + lane;
    return s < steps && lane < kStep && t < t_end ? pool_token(t) : kNoToken;
  };
  static_assert(kStep <= 32, "a step's tokens are held one per lane");
  uint32_t win = kAligned ? load_tiles() : load_tokens(0);

  const uint8_t* k_lane = static_cast<const uint8_t*>(p.k_cache) + (int64_t)kvh * KT::kRow + 16 * tg;
  const uint8_t* s_lane = static_cast<const uint8_t*>(p.k_scales) + kvh * 4;
  const uint32_t row_stride = (uint32_t)p.hkv * KT::kRow, scale_stride = (uint32_t)p.hkv * 4;
  float* w_lane = w_row + t_begin + 8 * (tg & 1) + g;  // token g + 8 (tg & 1) of a tile: written by lanes tg < 2
  const int t_lane = t_begin + 8 * (tg & 1) + g;
  constexpr int N = KT::kSteps;
  Loads<KV> buf[N];
  auto load = [&](int s, Loads<KV>& x) {
    x.ok = 0;
    if (s >= steps) return;  // (warp-uniform)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t tok[2];
      if constexpr (kAligned) {
        const uint32_t first = __shfl_sync(0xffffffffu, win, s * U + u);
        tok[0] = first + g;
        tok[1] = first + g + 8;
        if (first != kNoToken) x.ok |= 3u << (2 * u);  // (slots behind the last token are read, not used)
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          tok[i] = __shfl_sync(0xffffffffu, win, 16 * u + 8 * i + g);
          if (tok[i] != kNoToken) x.ok |= 1u << (2 * u + i);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if ((x.ok >> (2 * u + i)) & 1u) {
          const uint8_t* src = at_row(k_lane, tok[i], row_stride);
#pragma unroll
          for (int c = 0; c < P; ++c) x.k[u][i][c] = ldg_stream(src + 64 * c);
          if constexpr (KV == PKC_MX4) x.scale[u][i] = *reinterpret_cast<const uint32_t*>(at_row(s_lane, tok[i], scale_stride));
        } else {
#pragma unroll
          for (int c = 0; c < P; ++c) x.k[u][i][c] = make_uint4(0, 0, 0, 0);
          x.scale[u][i] = 0;
        }
      }
      const int at = s * t_step + 16 * u;
      x.old[u] = 0.f;
      if (p.decay != 0.f && tg < 2 && t_lane + at < t_end) x.old[u] = w_lane[at];
    }
    if constexpr (!kAligned) win = load_tokens(s + 1);
  };

  // Query fragments, elements in the order of the lane's key bytes.
  const T* q0 = static_cast<const T*>(p.q) + ((int64_t)b * p.hkv + kvh) * G * D;
  uint32_t qf[4][4];
  float undo = 1.f;
  uint32_t key_mul = 0;
  if constexpr (KV == PKC_MX4) {
    undo = load_q_f16<T, G>(q0, lane, qf, key_mul);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int dim = KV == PKC_E4M3 ? 64 * (c >> 1) + 16 * tg + 8 * (c & 1) : 32 * c + 8 * tg;
      const uint4 v = *reinterpret_cast<const uint4*>(q0 + (g < G ? g : 0) * D + dim);
      qf[c][0] = g < G ? v.x : 0u;
      qf[c][1] = g < G ? v.y : 0u;
      qf[c][2] = g < G ? v.z : 0u;
      qf[c][3] = g < G ? v.w : 0u;
    }
  }
  // This lane's score columns: heads 2 tg, 2 tg + 1.  An empty set's -inf
  // gives weight 0.
  float sc[2], ls[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int h = 2 * tg + e;
    sc[e] = p.scale_log2 * __shfl_sync(0xffffffffu, undo, (4 * h) & 31);
    const float lse = h < G ? p.lse[((int64_t)b * p.hkv + kvh) * G + h] : neg_inf();
    ls[e] = lse == neg_inf() ? -neg_inf() : lse * kLog2e;
  }

#pragma unroll
  for (int i = 0; i < N - 1; ++i) load(i, buf[i]);
  auto step = [&](int s, const Loads<KV>& x) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (KV == PKC_F16 || KV == PKC_BF16) {
        float acc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 ka = x.k[u][0][c], kb = x.k[u][1][c];
          const uint32_t f0[4] = {ka.x, kb.x, ka.y, kb.y}, f1[4] = {ka.z, kb.z, ka.w, kb.w};
          mma16816<T>(acc, f0, qf[c][0], qf[c][1]);
          mma16816<T>(acc2, f1, qf[c][2], qf[c][3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += acc2[i];
      } else if constexpr (KV == PKC_E4M3) {
        float acc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t ka[4] = {x.k[u][0][c].x, x.k[u][0][c].y, x.k[u][0][c].z, x.k[u][0][c].w};
          const uint32_t kb[4] = {x.k[u][1][c].x, x.k[u][1][c].y, x.k[u][1][c].z, x.k[u][1][c].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t f[4] = {e4m3x2_lo(ka[w]), e4m3x2_lo(kb[w]), e4m3x2_hi(ka[w]), e4m3x2_hi(kb[w])};
            mma16816<__half>(w & 1 ? acc2 : acc, f, qf[2 * c + (w >> 1)][2 * (w & 1)],
                             qf[2 * c + (w >> 1)][2 * (w & 1) + 1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += acc2[i];
      } else {
        const uint4 ka = x.k[u][0][0], kb = x.k[u][1][0];
        const uint32_t sa = x.scale[u][0], sb = x.scale[u][1];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a0[4], a1[4], c0[4], c1[4];
          e2m1x8(half ? ka.y : ka.x, a0);
          e2m1x8(half ? ka.w : ka.z, a1);
          e2m1x8(half ? kb.y : kb.x, c0);
          e2m1x8(half ? kb.w : kb.z, c1);
          uint32_t s2a = mx4_scale_pair(half ? sa >> 16 : sa), s2b = mx4_scale_pair(half ? sb >> 16 : sb);
          if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            s2a = bmul2(s2a, key_mul);
            s2b = bmul2(s2b, key_mul);
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int blk = 2 * half + v;
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t f0[4] = {a0[2 * v], c0[2 * v], a0[2 * v + 1], c0[2 * v + 1]};
            const uint32_t f1[4] = {a1[2 * v], c1[2 * v], a1[2 * v + 1], c1[2 * v + 1]};
            mma16816<__half>(part, f0, qf[blk][0], qf[blk][1]);
            mma16816<__half>(part, f1, qf[blk][2], qf[blk][3]);
            const float fa = __uint_as_float(v ? s2a & 0xffff0000u : s2a << 16);
            const float fb = __uint_as_float(v ? s2b & 0xffff0000u : s2b << 16);
            acc[0] = fmaf(part[0], fa, acc[0]);
            acc[1] = fmaf(part[1], fa, acc[1]);
            acc[2] = fmaf(part[2], fb, acc[2]);
            acc[3] = fmaf(part[3], fb, acc[3]);
          }
        }
      }
      // tokens g and g + 8 (a column of no head counts 0, whatever the key holds)
      const bool h0 = 2 * tg < G, h1 = 2 * tg + 1 < G;
      const float xa = (h0 ? ex2(fmaf(acc[0], sc[0], -ls[0])) : 0.f) + (h1 ? ex2(fmaf(acc[1], sc[1], -ls[1])) : 0.f);
      const float xb = (h0 ? ex2(fmaf(acc[2], sc[0], -ls[0])) : 0.f) + (h1 ? ex2(fmaf(acc[3], sc[1], -ls[1])) : 0.f);
      // sums over the row's four lanes: even lanes token g, odd lanes g + 8
      float sum = (tg & 1) ? xb : xa;
      sum += __shfl_xor_sync(0xffffffffu, (tg & 1) ? xa : xb, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int at = s * t_step + 16 * u;
      if (tg < 2 && t_lane + at < t_end && ((x.ok >> (2 * u + tg)) & 1u))
        w_lane[at] = p.decay != 0.f ? fmaf(p.decay, x.old[u], sum) : sum;
    }
  };
  for (int s = 0; s < steps; s += N) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i > 0 && s + i >= steps) break;
      load(s + i + N - 1, buf[(i + N - 1) % N]);
      step(s + i, buf[i]);
    }
  }
}

template <int KV, typename T, int G>
int launch_g(const WeightsParams& p, int64_t blocks, cudaStream_t st) {
  if (p.page_size % 16 == 0) weights_kernel<KV, T, G, true><<<(unsigned)blocks, kThreads, 0, st>>>(p);
  else weights_kernel<KV, T, G, false><<<(unsigned)blocks, kThreads, 0, st>>>(p);
  return (int)cudaGetLastError();
}

template <int KV, typename T>
int launch_t(const WeightsParams& p, int64_t blocks, cudaStream_t st) {
  switch (p.g) {
    case 1: return launch_g<KV, T, 1>(p, blocks, st);
    case 2: return launch_g<KV, T, 2>(p, blocks, st);
    case 4: return launch_g<KV, T, 4>(p, blocks, st);
    case 8: return launch_g<KV, T, 8>(p, blocks, st);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace

int launch_weights(const WeightsParams& p_in, int q_dtype, int kv_dtype, void* stream) {
  WeightsParams p = p_in;
  // The lengths are on the device: segments are laid over the longest request
  // that the table and the weight rows hold, and blocks past a request's end
  // return at once.  256 tokens per warp (512 of the mx4 cache's short rows)
  // amortise a block's start (length -> page id -> key, three loads in a row;
  // mx4 with 256: 74 -> 79 us) and still balance the end (16-bit with 512: 58
  // -> 65 us); segments are halved while there are fewer than four blocks per
  // SM.
  p.hg = p.hkv % 4 == 0 ? 4 : p.hkv % 2 == 0 ? 2 : 1;
  const int64_t most = std::min(p.bt_stride * (int64_t)p.page_size, p.w_stride);
  const int step = 16 * (kv_dtype == PKC_E4M3 ? 2 : 1) * (kWarps / p.hg);
  const int64_t rows = (int64_t)p.batch * (p.hkv / p.hg);
  int64_t seg = (kv_dtype == PKC_MX4 ? 512 : 256) * (kWarps / p.hg);
  while (seg > step && rows * ((most + seg - 1) / seg) < 4 * (int64_t)num_sms()) seg /= 2;
  p.seg_tokens = (int)seg;
  p.n_seg = (int)((most + seg - 1) / seg);
  const int64_t blocks = rows * p.n_seg;
  if (blocks <= 0) return 0;
  if (blocks > INT32_MAX) return (int)cudaErrorInvalidConfiguration;
  cudaStream_t st = (cudaStream_t)stream;
  switch (kv_dtype) {
    case PKC_F16: return launch_t<PKC_F16, __half>(p, blocks, st);
    case PKC_BF16: return launch_t<PKC_BF16, __nv_bfloat16>(p, blocks, st);
    case PKC_E4M3: return launch_t<PKC_E4M3, __half>(p, blocks, st);
    case PKC_MX4:
      return q_dtype == PKC_BF16 ? launch_t<PKC_MX4, __nv_bfloat16>(p, blocks, st)
                                 : launch_t<PKC_MX4, __half>(p, blocks, st);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace pkc
