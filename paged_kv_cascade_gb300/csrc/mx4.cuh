// The microscaled 4-bit cache format ("mx4") and the helpers of its kernels.
//
// One head's 128 elements of one token are 4 blocks of 32 with a shared
// power-of-two scale each (the microscaling formats' shared exponent, E8M0):
//   codes  64 bytes: element 32 b + 4 u + i of the row is nibble i of the
//          16-bit little-endian word 4 u + b  (b block 0..3, u 0..7, i 0..3)
//   scales 4 bytes: s_b stands for 2^(s_b - 127); 255: NaN
// A nibble is e2m1: sign, two exponent bits (bias 1), one mantissa bit, the
// values 0 .5 1 1.5 2 3 4 6.  The word order puts the 8 codes that one lane
// feeds to a tensor-core tile into one aligned load, for K (lane = 8
// consecutive elements of every block: 16 bytes at 16 (lane % 4)) and for V
// (4 elements of every block: 8 bytes at 8 (lane / 4)) alike.
#pragma once
#include "pkc_device.cuh"
#include "pkc_internal.h"

namespace pkc {

constexpr int kMx4RowBytes = 64;

// The 8 codes of a word -> 4 fp16 pairs (byte k -> r[k], low nibble first).
// Every e2m1 value is an fp16 value.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Eight values -> a word of e2m1 codes (x[0] in the lowest nibble), to
// nearest, ties to even, saturating at 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t d;
  asm("{\n.reg .b8 a, b, c, d;\ncvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\ncvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\nmov.b32 %0, {a, b, c, d};\n}"
      : "=r"(d)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return d;
}

// The float a scale byte stands for: 2^(s - 127), exactly (2^-127 is a
// denormal), or NaN for 255.
__device__ __forceinline__ float mx4_scale(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fffffffu : s == 0u ? 0x00400000u : s << 23);
}

// The same of two scale bytes (the low 16 bits) as a bf16 pair, exactly: bf16
// has denormals down to 2^-133.
__device__ __forceinline__ uint32_t mx4_scale_pair(uint32_t two) {
  uint32_t d;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.bf16x2.ue8m0x2 %0, l;\n}" : "=r"(d) : "r"(two));
  return d;
}

// a * b, element by element, of bf16 pairs (denormals included).
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Quotient and remainder by the page size (shift >= 0: a power of two).
struct PageDiv {
  int size, shift;
  template <typename I> __device__ __forceinline__ void split(I t, I& page, int& slot) const {
    if (shift >= 0) {
      page = t >> shift;
      slot = (int)(t & (size - 1));
    } else {
      page = t / size;
      slot = (int)(t - page * size);
    }
  }
};

// Pool index (page * page_size + slot) of a token that is not there.
constexpr uint32_t kNoToken = 0xffffffffu;

// base + row * stride in one wide multiply-add.
__device__ __forceinline__ const uint8_t* at_row(const uint8_t* base, uint32_t row, uint32_t stride) {
  uint64_t d;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(d) : "r"(row), "r"(stride), "l"(base));
  return reinterpret_cast<const uint8_t*>(d);
}

// The same as an address (of global memory).
__device__ __forceinline__ uint64_t row_at(uint64_t base, uint32_t row, uint32_t stride) {
  uint64_t d;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(d) : "r"(row), "r"(stride), "l"(base));
  return d;
}

// Asynchronous copies to shared memory, `ok` false: the bytes become zero
// and nothing is read.
__device__ __forceinline__ void cp_async16(uint32_t dst, uint64_t src, bool ok) {
  asm volatile("{\n.reg .pred p;\nsetp.eq.u32 p, %2, 0;\ncp.async.cg.shared.global [%0], [%1], 16, p;\n}" ::"r"(dst),
               "l"(src), "r"((uint32_t)ok) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, uint64_t src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, uint64_t src, bool ok) {
  asm volatile("{\n.reg .pred p;\nsetp.eq.u32 p, %2, 0;\ncp.async.ca.shared.global [%0], [%1], 4, p;\n}" ::"r"(dst),
               "l"(src), "r"((uint32_t)ok) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// d = a * b for one m16n8k16 fp16 tile (no accumulator to clear first).
__device__ __forceinline__ void mma16816_f16_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Query fragments (B operand of m16n8k16, n = query head lane / 4) for
// products with 4-bit keys, whose fragments are fp16: qf[b][k] are elements
// 32 b + 8 (lane % 4) + 2 k, + 1 of head lane / 4 (zero for heads >= G;
// kRepeat, G <= 4: heads 4 .. 7 repeat 0 .. 3).  fp16 queries are used as
// they are.  A bf16 row is scaled by the power of two that brings its largest
// magnitude into [2^14, 2^15): then every element down to 2^-22 of the
// largest is exact in fp16, and the others are off by at most 2^-39 of it, far
// below the float32 sums' rounding.
//
// Its products with codes are below 2^15 * 192 per block, so a sum over the
// blocks under their scales (2^125 at most for finite keys) could pass
// float32's range although q.k does not.  The key scales are therefore first
// multiplied by key_mul (a bf16 pair): 2^-22 keeps every such sum below
// 2^127.6.  It also drops scales below 2^-111; those count for less than 2^-37
// in a score as long as |q| < 2^64.  A warp with a larger query leaves the
// scales whole (1): keys of 2^105 and more, which may then overflow the sums
// of all its heads, give that query scores beyond float32 in any case.
//
// Returns the factor that undoes both.
template <typename T, int G, bool kRepeat = false>
__device__ __forceinline__ float load_q_f16(const T* qrow0, int lane, uint32_t (&qf)[4][4],
                                            uint32_t& key_mul) {
  const int g = kRepeat ? (lane >> 2) & 3 : lane >> 2, tg = lane & 3;
  const T* row = qrow0 + (g < G ? g : 0) * PKC_HEAD_DIM;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + 32 * b + 8 * tg);
    qf[b][0] = g < G ? u.x : 0u;
    qf[b][1] = g < G ? u.y : 0u;
    qf[b][2] = g < G ? u.z : 0u;
    qf[b][3] = g < G ? u.w : 0u;
  }
  key_mul = 0x3f803f80u;  // (1; not used with fp16 queries)
  if constexpr (std::is_same_v<T, __half>) {
    return 1.f;
  } else {
    uint32_t top = 0;  // largest magnitude's bf16 bits, lane's elements
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int k = 0; k < 4; ++k) top = max(top, max(qf[b][k] & 0x7fffu, (qf[b][k] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = (int)(top >> 7);  // biased exponent; 255: not finite, 0: zero or denormal
    const int shift = e == 255 || top == 0u ? 0 : min(14 - (e - 127), 126);
    const float mul = __int_as_float((127 + shift) << 23);
    uint32_t all = top;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) all = max(all, __shfl_xor_sync(0xffffffffu, all, x));
    const int bias = all < (127u + 64u) << 7 ? 22 : 0;
    if (bias) key_mul = 0x34803480u;  // 2^-22
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = Elem<__nv_bfloat16>::to_f2(qf[b][k]);
        qf[b][k] = Elem<__half>::from_f2(f.x * mul, f.y * mul);
      }
    return __int_as_float((127 - shift + bias) << 23);
  }
}

}  // namespace pkc
