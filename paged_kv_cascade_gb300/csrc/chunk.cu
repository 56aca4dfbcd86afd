// Attention states of a chunk of new tokens per request over its paged cache.
//
// Row i of request b's n rows stands at position p = len - n + i and attends to
// the tokens t < len with t <= p (causal) and t > p - window:
//   s_t = scale q.k_t,  LSE = log sum exp s_t,  O = sum exp(s_t - LSE) v_t.
// One warp per (row, query head), a key at a time, four elements a lane.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkc_device.cuh"
#include "pkc_internal.h"

namespace pkc {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) chunk_kernel(const ChunkParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t row = u / p.hq;
  const int h = (int)(u % p.hq);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.batch; b += kThreads)
      if (p.q_indptr[b] < 0 || p.q_indptr[b + 1] < p.q_indptr[b] || p.q_indptr[b + 1] > p.total_q)
        report(p.status, PKC_ERR_PLAN);
  if (row >= p.total_q) return;
  // the request of the row
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_indptr[mid] <= row) lo = mid; else hi = mid;
  }
  const int b = lo, r0 = p.q_indptr[b], r1 = p.q_indptr[b + 1], len = p.cache_seqlens[b];
  if (row < r0 || row >= r1) return;
  if (r0 < 0 || r1 > p.total_q || len < 0) {
    if (lane == 0) report(p.status, PKC_ERR_PLAN);
    return;
  }
  const int64_t pos = (int64_t)len - (r1 - row);
  const int64_t t1 = p.causal ? min((int64_t)len, pos + 1) : len;
  const int64_t t0 = p.window ? max((int64_t)0, pos - p.window + 1) : 0;
  const int kvh = h / p.g;
  const uint2 qw = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.q) + u * PKC_HEAD_DIM + 4 * lane);
  const float2 q0 = Elem<T>::to_f2(qw.x), q1 = Elem<T>::to_f2(qw.y);
  float m = neg_inf(), l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t pi = t / p.page_size;
    const int page = pi < p.bt_stride ? p.block_table[(int64_t)b * p.bt_stride + pi] : -1;
    uint2 kw = make_uint2(0, 0), vw = make_uint2(0, 0);
    if (page >= 0 && page < p.num_pages) {
      const int64_t at = (((int64_t)page * p.page_size + t % p.page_size) * p.hkv + kvh) * PKC_HEAD_DIM + 4 * lane;
      kw = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.k_cache) + at);
      vw = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.v_cache) + at);
    } else if (lane == 0) {
      report(p.status, PKC_ERR_BLOCK_TABLE);
    }
    const float2 k0 = Elem<T>::to_f2(kw.x), k1 = Elem<T>::to_f2(kw.y);
    float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), ref = mn == neg_inf() ? 0.f : mn;
    const float w = ex2(m - ref), e = ex2(s - ref);
    m = mn;
    l = l * w + e;
    const float2 v0 = Elem<T>::to_f2(vw.x), v1 = Elem<T>::to_f2(vw.y);
    o[0] = o[0] * w + e * v0.x;
    o[1] = o[1] * w + e * v0.y;
    o[2] = o[2] * w + e * v1.x;
    o[3] = o[3] * w + e * v1.y;
  }
  const bool any = t1 > t0;
  const float inv = any ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = any ? o[i] * inv : 0.f;
  if (p.out_dtype == PKC_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + u * PKC_HEAD_DIM + 4 * lane) =
        make_float4(o[0], o[1], o[2], o[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + u * PKC_HEAD_DIM + 4 * lane) =
        make_uint2(Elem<T>::from_f2(o[0], o[1]), Elem<T>::from_f2(o[2], o[3]));
  if (lane == 0) p.lse[u] = any ? (m + lg2(l)) * kLn2 : neg_inf();
}

}  // namespace

size_t chunk_partial_bytes() { return 256; }

int launch_paged_chunk(const ChunkParams& p, int dtype, void* stream) {
  const int64_t blocks = ((int64_t)p.total_q * p.hq + kThreads / 32 - 1) / (kThreads / 32);
  if (dtype == PKC_BF16) chunk_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, (cudaStream_t)stream>>>(p);
  else chunk_kernel<__half><<<(unsigned)blocks, kThreads, 0, (cudaStream_t)stream>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace pkc
