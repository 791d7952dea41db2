// The 4-bit rows of a quantised chunk page: layout, rounding, unpacking.
//
// A row of d values is split into groups of 32 dims.  Each group keeps a step
// s = fp16((max - min) / 15) and a least value m = fp16(min) and stands, with
// codes 0 .. 15, for m + s * code: 5 bits per value (fp32 arithmetic, the two
// parameters are the only values rounded to fp16; a bf16 parameter would cost
// the least value of an off-centre channel eight times the error).
//
// Block of one (page, kv head): 64 rows of codes (d/2 bytes each), then 64
// rows of (s, m) pairs (4 bytes per group).  In a row of codes the 16-bit unit
// e * (d/32) + g holds dims 32g + 4e .. + 3, the lowest dim in the lowest
// bits: one aligned read of 2 (d/32) bytes gives four dims of EVERY group, so
// that the eight lanes that share a row (or a column of a matrix fragment)
// read the whole row in consecutive pieces while each lane still has the same
// dims of each group and can apply the group's step to a finished partial sum.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace hils {

constexpr int kQGroup = 32;   // dims that share a step and a least value

template <int D> struct QuantPage {
  static constexpr int G = D / kQGroup;                       // groups per row
  static constexpr int ROW = D / 2;                           // code bytes per row
  static constexpr int PROW = G * 4;                          // parameter bytes per row
  static constexpr int64_t BLOCK = int64_t(kChunk) * (ROW + PROW);
  __host__ __device__ static constexpr int code_off(int row) { return row * ROW; }
  __host__ __device__ static constexpr int param_off(int row) { return kChunk * ROW + row * PROW; }
};

// Quantise and store one row held by D / E neighbouring lanes of a warp, lane
// `sub` of the row holding dims sub * E .. + E - 1 in fp32.  Every lane of the
// warp takes part (shuffles); only those with `store` write.  A group with a
// value that is not finite, or whose parameters leave the range of fp16, is
// stored with NaN parameters and reads back as NaN.
template <int D, int E>
__device__ __forceinline__ void quant_store_row(const float (&x)[E], int sub, uint8_t* block, int row, bool store) {
  using P = QuantPage<D>;
  constexpr int GL = kQGroup / E;      // lanes per group
  static_assert(E == 4 || E == 8, "a lane holds one 16-byte vector of fp32 or bf16");
  float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    bad = fmaf(x[e], 0.f, bad);       // NaN once a value is not finite (fminf and fmaxf drop a NaN)
  }
  if (bad != 0.f) hi = INFINITY;      // true for NaN
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  __half2 par = __halves2half2(__float2half_rn((hi - lo) / 15.f), __float2half_rn(lo));
  float s = __low2float(par), m = __high2float(par);
  if (!(fabsf(s) < INFINITY && fabsf(m) < INFINITY)) {
    par = __halves2half2(__ushort_as_half(0x7FFF), __ushort_as_half(0x7FFF));
    s = 0.f;
    m = 0.f;
  }
  const float inv = s > 0.f ? 1.f / s : 0.f;
  // The quotient rounded to nearest by one correction of t * (1/s) (Markstein's
  // theorem: 1/s is correctly rounded), so that a value half way between two
  // codes, common among bf16 values, is seen as such.  A value below the
  // rounded least one, or (with the step rounded down) above the largest, takes
  // the nearest code; s = 0 gives 0, and so does the NaN of a group that is not
  // finite.  Rounding to an integer by adding 1.5 x 2^23 and packing four codes
  // in fp32 (exact below 2^16) keep to the full-rate pipes.
  constexpr float kRound = 12582912.f;
  uint32_t u[E / 4];
#pragma unroll
  for (int w = 0; w < E / 4; ++w) {
    float four = 0.f;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const float t = x[4 * w + i] - m, q0 = t * inv, q1 = fmaf(fmaf(-q0, s, t), inv, q0);
      const float c = (fminf(fmaxf(q1, 0.f), 15.f) + kRound) - kRound;
      four = fmaf(four, 16.f, c);
    }
    u[w] = __float_as_uint(four + 8388608.f) & 0xFFFFu;
  }
  // a lane of an even group and its neighbour of the next group exchange a
  // unit, so that each stores one aligned 32-bit word
  const int g = sub / GL, j = sub % GL;
  const uint32_t give = (E == 8 && !(g & 1)) ? u[E / 4 - 1] : u[0];
  const uint32_t take = __shfl_xor_sync(0xffffffffu, give, GL);
  if (!store) return;
  uint8_t* codes = block + P::code_off(row);
  if (E == 8) {
    const int e = 2 * j + (g & 1);
    const uint32_t w = (g & 1) ? (take | (u[E / 4 - 1] << 16)) : (u[0] | (take << 16));
    *reinterpret_cast<uint32_t*>(codes + 2 * (e * P::G + (g & ~1))) = w;
  } else if (!(g & 1)) {
    *reinterpret_cast<uint32_t*>(codes + 2 * (j * P::G + g)) = u[0] | (take << 16);
  }
  if (j == 0) *reinterpret_cast<__half2*>(block + P::param_off(row) + 4 * g) = par;
}

}  // namespace hils
