// Quantising append to, and read-back from, an mx4 paged cache (the format:
// mx4.cuh).
//
// Both kernels move one 256-byte row (a token's 128 values of one head, K or
// V) per 16 lanes: lane 4 b + v holds elements 32 b + 8 v .. + 7, so a
// block's shared exponent is a maximum over 4 lanes and the row's 64 code
// bytes are re-ordered with two shuffles.  A row is 256 bytes in and 68 out,
// or the reverse, and about 40 instructions; HBM and the integer pipe are
// about equally busy: 131 us for both kernels over 65,785 ragged tokens of 8
// heads (682 MB, 5.2 TB/s of a measured copy rate of 6.8).  A warp per token
// pays for the token's place once (with a division and a search per row: 340
// us).  A step of one token per request is launch latency, 4 us a kernel.
//
// Quantising (the microscaling rule): a block of largest magnitude amax gets
// the exponent e = max(floor(log2 amax) - 2, -126), so that amax / 2^e lies
// in [4, 8), and its elements become the nearest e2m1 values of x / 2^e
// (ties to the even code, 6 above 6).  The division by a power of two is
// exact in float32.  A block holding an infinity or a NaN gets scale 255
// (NaN) and zero codes.
#include <cuda_runtime.h>

#include "mx4.cuh"

namespace pkc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;           // rows a 16-lane group has in flight
constexpr int kRows = 2 * kUnroll;   // rows of a token that a warp has in flight

// Request of row t of the ragged token list: indptr[b] <= t < indptr[b + 1],
// or -1 (rows that no request owns).
__device__ __forceinline__ int request_of(const int32_t* indptr, int batch, int t) {
  int lo = 0, hi = batch;  // the last b in [0, batch] with indptr[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (indptr[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo < batch && indptr[lo] <= t && t < indptr[lo + 1] ? lo : -1;
}

struct Place {
  int64_t slot;  // page * page_size + slot, -1: not to be touched
  bool bad;      // a page that is not there
};

// Cache slot of row t: position base[b] + (t - indptr[b]) of its request.
__device__ __forceinline__ Place place_of(const Mx4RowsParams& p, int t) {
  const int b = request_of(p.indptr, p.batch, t);
  if (b < 0) return {-1, false};
  const int base = p.base[b];
  const int64_t pos = (int64_t)base + ((int64_t)t - p.indptr[b]);
  int64_t page_idx;
  int slot;
  PageDiv{p.page_size, p.page_shift}.split(pos, page_idx, slot);
  int32_t page = -1;
  if (base >= 0 && pos < INT32_MAX && page_idx < p.bt_stride) page = p.block_table[(int64_t)b * p.bt_stride + page_idx];
  if (page < 0 || page >= p.num_pages) return {-1, true};
  return {(int64_t)page * p.page_size + slot, false};
}

// A warp works on one token, 8 rows at a time: rows r = 0 .. 2 Hkv - 1 are
// the token's K heads, then its V heads; lanes 0..15 and 16..31 take every
// second one.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_mx4_kernel(const Mx4RowsParams p) {
  const int lane16 = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
  const int j = lane16 >> 2, v = lane16 & 3;
  const int rows = 2 * p.hkv, n_warps = (int)gridDim.x * kWarps;
  bool any_bad = false;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < p.total; t += n_warps) {
    const int64_t src0 = t * p.hkv * PKC_HEAD_DIM + 8 * lane16;  // (V's row r is its head r - Hkv)
    const T* k_src = static_cast<const T*>(p.k_rows) + src0;
    const T* v_src = static_cast<const T*>(p.v_rows) + src0 - p.hkv * PKC_HEAD_DIM;
    Place at{-1, false};
    uint8_t *k_dst = nullptr, *v_dst = nullptr, *k_sc = nullptr, *v_sc = nullptr;
    for (int r0 = (int)blockIdx.y * kRows; r0 < rows; r0 += (int)gridDim.y * kRows) {
      uint4 x[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int r = r0 + 2 * i + half;
        x[i] = r < rows ? ldg_stream((r >= p.hkv ? v_src : k_src) + r * PKC_HEAD_DIM) : make_uint4(0, 0, 0, 0);
      }
      if (r0 == (int)blockIdx.y * kRows) {
        at = place_of(p, (int)t);
        any_bad = any_bad || at.bad;
        const int64_t row0 = at.slot * p.hkv;
        k_dst = static_cast<uint8_t*>(p.k_codes) + row0 * kMx4RowBytes + 16 * v + 4 * j;
        v_dst = static_cast<uint8_t*>(p.v_codes) + (row0 - p.hkv) * kMx4RowBytes + 16 * v + 4 * j;
        k_sc = static_cast<uint8_t*>(p.k_scales) + row0 * 4 + j;
        v_sc = static_cast<uint8_t*>(p.v_scales) + (row0 - p.hkv) * 4 + j;
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int r = r0 + 2 * i + half;
        // the largest magnitude, on 16-bit patterns (ordered as integers, NaN
        // above infinity), two at a time
        uint32_t top = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top & 0xffffu, top >> 16);
        const uint32_t e = __float_as_uint(Elem<T>::to_f2(top).x) >> 23;
        const bool nan = e == 255u;
        const uint32_t s = nan ? 255u : (uint32_t)max((int)e - 2, 1);
        const float mul = __uint_as_float(nan ? 0u : (254u - s) << 23);  // 2^(127 - s)
        const float2 f[4] = {Elem<T>::to_f2(x[i].x), Elem<T>::to_f2(x[i].y), Elem<T>::to_f2(x[i].z),
                             Elem<T>::to_f2(x[i].w)};
        const float y[8] = {f[0].x * mul, f[0].y * mul, f[1].x * mul, f[1].y * mul,
                            f[2].x * mul, f[2].y * mul, f[3].x * mul, f[3].y * mul};
        const uint32_t w = nan ? 0u : to_e2m1x8(y);
        // lane 4 b + v holds words (u = 2 v, b) and (u = 2 v + 1, b); lane
        // 4 j + v stores 32-bit word j of 16-byte piece v: words
        // (u = 2 v + j / 2, b = 2 (j % 2)) and (the same u, b + 1)
        const uint32_t wa = __shfl_sync(0xffffffffu, w, 8 * (j & 1) + v, 16);
        const uint32_t wb = __shfl_sync(0xffffffffu, w, 8 * (j & 1) + 4 + v, 16);
        if (at.slot >= 0 && r < rows) {
          const bool is_v = r >= p.hkv;
          *reinterpret_cast<uint32_t*>((is_v ? v_dst : k_dst) + r * kMx4RowBytes) =
              prmt(wa, wb, (j >> 1) ? 0x7632u : 0x5410u);
          if (v == 0) (is_v ? v_sc : k_sc)[r * 4] = (uint8_t)s;
        }
      }
    }
  }
  // The lengths grow once every block has read them: by the block that
  // finishes last, which also resets the counter for the next launch.
  int32_t* ctr = p.status + PKC_APPEND_COUNTER;
  __shared__ int last, bad;
  if (any_bad) {
    report(p.status, PKC_ERR_BLOCK_TABLE);
    atomicExch(ctr + 1, 1);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(ctr, 1) == (int)(gridDim.x * gridDim.y) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (threadIdx.x == 0) {
    bad = atomicExch(ctr + 1, 0);
    atomicExch(ctr, 0);
  }
  __syncthreads();
  // The ranges must run upwards within 0 .. total: were they to overlap, a
  // request could count rows that another one got.
  bool wrong = false;
  for (int b = threadIdx.x; b < p.batch; b += kThreads)
    wrong = wrong || p.indptr[b] < 0 || p.indptr[b + 1] < p.indptr[b] || p.indptr[b + 1] > p.total;
  if (__syncthreads_or(wrong)) {
    if (threadIdx.x == 0) report(p.status, PKC_ERR_PLAN);
    return;
  }
  for (int b = threadIdx.x; b < p.batch; b += kThreads) {
    const int t0 = p.indptr[b], t1 = p.indptr[b + 1], len = p.base[b];
    if (t0 == t1) continue;
    bool ok = true;
    if (bad) {  // some token had no page: which requests have all of theirs?
      for (int64_t pos = len; ok && pos < (int64_t)len + (t1 - t0);) {
        const int64_t page_idx = pos / p.page_size;
        int32_t page = -1;
        if (len >= 0 && page_idx < p.bt_stride) page = p.block_table[(int64_t)b * p.bt_stride + page_idx];
        ok = page >= 0 && page < p.num_pages && (int64_t)len + (t1 - t0) <= INT32_MAX;
        pos = (page_idx + 1) * p.page_size;
      }
    }
    if (ok) p.lengths[b] = len + (t1 - t0);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gather_mx4_kernel(const Mx4RowsParams p) {
  const int lane16 = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
  const int b = lane16 >> 2, v = lane16 & 3;
  const int rows = 2 * p.hkv, n_warps = (int)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < p.total; t += n_warps) {
    const Place at = place_of(p, (int)t);
    if (at.bad && (threadIdx.x & 31) == 0) report(p.status, PKC_ERR_BLOCK_TABLE);
    if (at.slot < 0 && !at.bad) continue;  // (warp-uniform) a row of no request
    const int64_t row0 = max(at.slot, (int64_t)0) * p.hkv;  // (V's row r is its head r - Hkv)
    const uint8_t* k_src = static_cast<const uint8_t*>(p.k_codes) + row0 * kMx4RowBytes + 16 * v + 4 * b;
    const uint8_t* v_src = static_cast<const uint8_t*>(p.v_codes) + (row0 - p.hkv) * kMx4RowBytes + 16 * v + 4 * b;
    const uint8_t* k_sc = static_cast<const uint8_t*>(p.k_scales) + row0 * 4 + b;
    const uint8_t* v_sc = static_cast<const uint8_t*>(p.v_scales) + (row0 - p.hkv) * 4 + b;
    T* k_dst = static_cast<T*>(p.k_out) + t * p.hkv * PKC_HEAD_DIM + 8 * lane16;
    T* v_dst = static_cast<T*>(p.v_out) + (t - 1) * p.hkv * PKC_HEAD_DIM + 8 * lane16;
    for (int r0 = (int)blockIdx.y * kRows; r0 < rows; r0 += (int)gridDim.y * kRows) {
      uint32_t w[kUnroll], sc[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int r = r0 + 2 * i + half;
        const bool is_v = r >= p.hkv;
        w[i] = sc[i] = 0;  // a row without a page reads as zeros
        if (at.slot >= 0 && r < rows) {
          w[i] = *reinterpret_cast<const uint32_t*>((is_v ? v_src : k_src) + r * kMx4RowBytes);
          sc[i] = (is_v ? v_sc : k_sc)[r * 4];
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int r = r0 + 2 * i + half;
        // the inverse of the append's re-ordering: lane 4 b + v takes the
        // words (u = 2 v, b) and (u = 2 v + 1, b)
        const uint32_t wa = __shfl_sync(0xffffffffu, w[i], 4 * (b >> 1) + v, 16);
        const uint32_t wb = __shfl_sync(0xffffffffu, w[i], 4 * (2 + (b >> 1)) + v, 16);
        uint32_t h2[4];
        e2m1x8(prmt(wa, wb, (b & 1) ? 0x7632u : 0x5410u), h2);
        const float s = mx4_scale(sc[i]);
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = Elem<__half>::to_f2(h2[k]);
          out[k] = Elem<T>::from_f2(f.x * s, f.y * s);
        }
        if (r < rows)
          *reinterpret_cast<uint4*>((r >= p.hkv ? v_dst : k_dst) + r * PKC_HEAD_DIM) =
              make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
}

// One warp per token; the 8-row parts of a token go to blocks of their own
// while there are few tokens.
dim3 grid_for(const Mx4RowsParams& p) {
  const int parts = (2 * p.hkv + kRows - 1) / kRows;
  const int64_t want = ((int64_t)p.total + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)num_sms() * (2048 / kThreads);
  if (want * parts <= most && parts <= 65535) return dim3((unsigned)want, (unsigned)parts);
  return dim3((unsigned)(want < most ? want : most), 1);
}

}  // namespace

int launch_append_mx4(const Mx4RowsParams& p, int dtype, void* stream) {
  if (p.total <= 0 || p.batch <= 0) return 0;
  if (dtype == PKC_BF16) append_mx4_kernel<__nv_bfloat16><<<grid_for(p), kThreads, 0, (cudaStream_t)stream>>>(p);
  else append_mx4_kernel<__half><<<grid_for(p), kThreads, 0, (cudaStream_t)stream>>>(p);
  return (int)cudaGetLastError();
}

int launch_gather_mx4(const Mx4RowsParams& p, int dtype, void* stream) {
  if (p.total <= 0 || p.batch <= 0) return 0;
  if (dtype == PKC_BF16) gather_mx4_kernel<__nv_bfloat16><<<grid_for(p), kThreads, 0, (cudaStream_t)stream>>>(p);
  else gather_mx4_kernel<__half><<<grid_for(p), kThreads, 0, (cudaStream_t)stream>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace pkc
