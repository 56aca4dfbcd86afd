// Rotary positions applied to a step's queries and keys, and its keys and
// values written to their slots of the paged cache.
//
// Pair i of a row at position p turns by a = p f_i:
//   (x, y) -> s (x cos a - y sin a, x sin a + y cos a).
// The angle matters modulo a turn only, so f_i / 2 pi is kept as a 64-bit
// fraction of a turn: p times it, modulo 2^64, is the fraction of a turn that
// the pair has moved, exactly but for the rounding of f_i itself.  Its upper 32
// bits give sine and cosine to float32; far positions lose nothing.
//
// A row is 128 elements, 16 pieces of 8.  Eight lanes take a row: lane l of the
// first R / 16 holds the two pieces with pairs 8 l .. 8 l + 7 (pieces 2 l and 2 l
// + 1 interleaved, l and l + R / 16 in halves), so a pair is never split between
// lanes; the other lanes pass the rest of the row.  A warp does four rows at a
// time and keeps its sines and cosines over all rows of a token.
//
// HBM bounds it: 44,925 tokens of 32 / 8 heads, 1.10 GB, take 169 us (6.54 TB/s).
// Small blocks that end with their tokens: 174 us with blocks of 256 threads that
// loop over tokens, 179 with such of 128.  2718 tokens of 32 / 32 heads into an
// e4m3 cache, 111 MB: 22.3 us against 16.7 of bytes (24.3 with one part a token, 26.5 with
// blocks of 256).  Those are 2040 blocks of 1064 that the SMs hold at 72 registers, two
// waves, in each of them one chain: frequencies, a barrier, slot and position, sines, rows.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pkc_device.cuh"
#include "pkc_internal.h"

namespace pkc {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 2;        // groups of four rows in flight per warp
constexpr int kGroup = 4 * kUnroll;

// f / 2 pi as a 64-bit fraction of a turn.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const double turns = f * 0.15915494309189535;
  return __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

template <typename T, bool kE4m3>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p) {
  __shared__ uint64_t turn[PKC_HEAD_DIM / 2];
  const int rot8 = p.rotary_dim / 16;  // lanes of a row that turn
  for (int i = threadIdx.x; i < p.rotary_dim / 2; i += kThreads) turn[i] = turn_fraction(p.inv_freq[i]);
  __syncthreads();
  const int lane = threadIdx.x & 31, l = lane & 7, r4 = lane >> 3;
  const bool turns = l < rot8;
  // the lane's two pieces, in elements
  const int e0 = turns && !p.interleaved ? 8 * l : 16 * l;
  const int e1 = turns && !p.interleaved ? 8 * (l + rot8) : 16 * l + 8;
  const int rows = p.hq + 2 * p.hkv;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t < p.total) {
    const int64_t slot = p.slots[t];
    const bool cached = slot >= 0 && slot < p.pool_tokens;
    if (slot >= p.pool_tokens && lane == 0) report(p.status, PKC_ERR_BLOCK_TABLE);
    float c[8], s[8];
    if (turns) {
      const uint64_t pos = (uint64_t)(int64_t)p.positions[t];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // a signed fraction of half a turn, in [-1, 1)
        const float x = (float)(int32_t)(uint32_t)((turn[8 * l + i] * pos) >> 32) * 0x1p-31f;
        float sn, cs;
        sincospif(x, &sn, &cs);
        c[i] = cs * p.amplitude;
        s[i] = sn * p.amplitude;
      }
    }
    const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
    const T* k = static_cast<const T*>(p.k_new) + t * p.kv_stride;
    const T* v = static_cast<const T*>(p.v_new) + t * p.kv_stride;
    T* q_out = static_cast<T*>(p.q_out) + t * p.hq * PKC_HEAD_DIM;
    const int last = cached ? rows : p.hq;
    for (int r0 = (int)blockIdx.y * kGroup; r0 < last; r0 += (int)gridDim.y * kGroup) {
      uint4 a[kUnroll], b[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + 4 * u + r4;
        if (r < last) {
          const T* src = (r < p.hq ? q + r * PKC_HEAD_DIM
                                   : r < p.hq + p.hkv ? k + (r - p.hq) * PKC_HEAD_DIM
                                                      : v + (r - p.hq - p.hkv) * PKC_HEAD_DIM);
          a[u] = *reinterpret_cast<const uint4*>(src + e0);
          b[u] = *reinterpret_cast<const uint4*>(src + e1);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + 4 * u + r4;
        if (r >= last) continue;
        const bool is_v = r >= p.hq + p.hkv;
        float x[8], y[8];
        {
          const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = Elem<T>::to_f2(aw[i]), g = Elem<T>::to_f2(bw[i]);
            x[2 * i] = f.x; x[2 * i + 1] = f.y;
            y[2 * i] = g.x; y[2 * i + 1] = g.y;
          }
        }
        if (turns && !is_v) {
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
              x[2 * i] = x0 * c[i] - x1 * s[i];
              x[2 * i + 1] = x0 * s[i] + x1 * c[i];
              y[2 * i] = y0 * c[4 + i] - y1 * s[4 + i];
              y[2 * i + 1] = y0 * s[4 + i] + y1 * c[4 + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x0 = x[i], y0 = y[i];
              x[i] = x0 * c[i] - y0 * s[i];
              y[i] = x0 * s[i] + y0 * c[i];
            }
          }
        }
        if (kE4m3 && r >= p.hq) {
          // The quotient by the scale, rounded as a quotient: a product with a rounded
          // reciprocal is off by its last bit where that decides between two codes.  The
          // reciprocal of a power of two is exact, and saves a fifth (22.3 us, 28.6 with
          // divisions, for the case above; 32.2 where powers of two are divided by too).
          const float m = is_v ? p.v_scale : p.k_scale, inv = is_v ? p.v_inv_scale : p.k_inv_scale;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = p.divide ? __fdiv_rn(x[i], m) : x[i] * inv;
            y[i] = p.divide ? __fdiv_rn(y[i], m) : y[i] * inv;
          }
          uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                         (slot * p.hkv + (r - p.hq - (is_v ? p.hkv : 0))) * PKC_HEAD_DIM;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            w[i] = e4m3x2(x[4 * i], x[4 * i + 1]) | e4m3x2(x[4 * i + 2], x[4 * i + 3]) << 16;
            w[2 + i] = e4m3x2(y[4 * i], y[4 * i + 1]) | e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16;
          }
          *reinterpret_cast<uint2*>(dst + e0) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(dst + e1) = make_uint2(w[2], w[3]);
        } else {
          T* dst = r < p.hq ? q_out + r * PKC_HEAD_DIM
                            : static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
                                  (slot * p.hkv + (r - p.hq - (is_v ? p.hkv : 0))) * PKC_HEAD_DIM;
          *reinterpret_cast<uint4*>(dst + e0) =
              make_uint4(Elem<T>::from_f2(x[0], x[1]), Elem<T>::from_f2(x[2], x[3]), Elem<T>::from_f2(x[4], x[5]),
                         Elem<T>::from_f2(x[6], x[7]));
          *reinterpret_cast<uint4*>(dst + e1) =
              make_uint4(Elem<T>::from_f2(y[0], y[1]), Elem<T>::from_f2(y[2], y[3]), Elem<T>::from_f2(y[4], y[5]),
                         Elem<T>::from_f2(y[6], y[7]));
        }
      }
    }
  }
}

template <typename T, bool kE4m3>
int launch_t(const RopeParams& p, cudaStream_t st) {
  // One warp per token.  Where that leaves the SMs short of blocks, a token's groups of
  // rows are shared out over blocks of their own (each works out the sines again), up to
  // 2048 threads an SM: at 72 registers two waves, not one, but three parts of the 2718
  // tokens above take 22.3 us, two to twelve others 23.8 to 30.2.
  const int64_t parts = ((int64_t)p.hq + 2 * p.hkv + kGroup - 1) / kGroup;
  const int64_t want = ((int64_t)p.total + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)num_sms() * (2048 / kThreads);
  const dim3 grid((unsigned)want, (unsigned)std::max<int64_t>(1, std::min<int64_t>(parts, most / want)));
  rope_append_kernel<T, kE4m3><<<grid, kThreads, 0, st>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_rope_append(const RopeParams& p, int dtype, int kv_dtype, void* stream) {
  if (p.total <= 0) return 0;
  cudaStream_t st = (cudaStream_t)stream;
  if (kv_dtype == PKC_E4M3)
    return dtype == PKC_BF16 ? launch_t<__nv_bfloat16, true>(p, st) : launch_t<__half, true>(p, st);
  return dtype == PKC_BF16 ? launch_t<__nv_bfloat16, false>(p, st) : launch_t<__half, false>(p, st);
}

}  // namespace pkc
