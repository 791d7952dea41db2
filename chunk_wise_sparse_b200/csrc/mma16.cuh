// 16x8x16 matrix products on registers (mma.sync) and the operands the 4-bit
// kernels make for them.  A decode step multiplies 16 keys by one to eight
// queries: a sixteenth of the smallest tcgen05 tile's columns would be
// used, and the codes have to pass through registers to be widened.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace hils {

// c += a b for 16x16 a (row) and 16x8 b (column), fp32 sums
__device__ __forceinline__ void mma16816_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same without a sum to start from
__device__ __forceinline__ void mma16816_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// transpose of an 8x8 matrix of 16-bit values spread over the warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// the two bf16 values of a register in fp32
__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// 2^x.  FAST: without the scaling that keeps results below 2^-126 (weights that small are zero here)
template <bool FAST>
__device__ __forceinline__ float pow2(float x) {
  if constexpr (!FAST) return exp2f(x);
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The power of two that puts `top` (>= 0) in [2^14, 2^15), and its inverse,
// within fp32's normal powers: values so scaled fit fp16, and lose at most
// 2^-24 of the largest.
__device__ __forceinline__ void power_scale(float top, float& up, float& down) {
  int e = int(__float_as_uint(top) >> 23);
  e = e < 30 ? 30 : e > 250 ? 250 : e;
  up = __uint_as_float(uint32_t(268 - e) << 23);      // 2^(141 - e)
  down = __uint_as_float(uint32_t(e - 14) << 23);     // 2^(e - 141)
}

// The four codes of a 16-bit unit of x and of one of y (the upper ones if
// `upper`), side by side, as fp16 subnormals: code 0 in bits 0 .. 3 is
// code 2^-24, code 1 left in bits 4 .. 7 is code 2^-20, and codes 2 and 3
// likewise after a byte's move, which costs nothing in the permutation.
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t y, bool upper, uint32_t (&a)[4]) {
  const uint32_t lo = __byte_perm(x, y, upper ? 0x7632 : 0x5410), hi = __byte_perm(x, y, upper ? 0x7733 : 0x5511);
  a[0] = lo & 0x000F000Fu;
  a[1] = lo & 0x00F000F0u;
  a[2] = hi & 0x000F000Fu;
  a[3] = hi & 0x00F000F0u;
}

// The same centred: code - 8 in a[0] and a[2], 16 (code - 8) in a[1] and a[3],
// exactly (1024 + code, or 1024 + 16 code, has the code where it lies).  For
// sums that have to be good to fp32: a sum of codes from 0 cancels against the
// least values, and the matrix unit does not round its sums to nearest.
__device__ __forceinline__ void codes_f16_centred(uint32_t x, uint32_t y, bool upper, uint32_t (&a)[4]) {
  codes_f16(x, y, upper, a);
  const __half2 off[2] = {__floats2half2_rn(-1032.f, -1032.f), __floats2half2_rn(-1152.f, -1152.f)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = a[i] | 0x64006400u;
    const __half2 v = __hadd2(*reinterpret_cast<const __half2*>(&w), off[i & 1]);
    a[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Four codes of two 16-bit units (one in each half of x) as bf16 pairs of
// code - 8: 16 + code has the code in bits 3 .. 6, and 24 less is exact.
__device__ __forceinline__ void codes_bf16_centred(uint32_t x, uint32_t (&a)[4]) {
  a[0] = ((x << 3) & 0x00780078u) | 0x41804180u;
  a[1] = ((x >> 1) & 0x00780078u) | 0x41804180u;
  a[2] = ((x >> 5) & 0x00780078u) | 0x41804180u;
  a[3] = ((x >> 9) & 0x00780078u) | 0x41804180u;
  const __nv_bfloat162 c24 = __floats2bfloat162_rn(24.f, 24.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a[i]), c24);
    a[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace hils
