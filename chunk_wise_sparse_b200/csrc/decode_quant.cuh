// One decode step over a 4-bit chunk-paged cache: the scoring, top-K and
// combine kernels of decode.cuh around a partial kernel that reads 4-bit pages.
#pragma once
#include "decode.cuh"
#include "quant.cuh"

namespace hils {

// One warp per (row, slot): slots 0 .. K-1 are the row's kept chunks, K + w is
// window chunk own - w.  Each key row is read by D / 8 lanes; an online
// softmax per key group, merged by shuffles.
template <typename T, int D>
__global__ void __launch_bounds__(128)
decode_partial_quant_kernel(const T* __restrict__ q, const uint8_t* __restrict__ kpg, const uint8_t* __restrict__ vpg,
                            const int32_t* __restrict__ table, int64_t n_pages, const int32_t* __restrict__ seqlens,
                            int64_t cap, int Hq, int G, int Hkv, int K, float tau, const int32_t* __restrict__ sel_ids,
                            const float* __restrict__ sel_scores, float* __restrict__ part_u,
                            float* __restrict__ part_o, int64_t n_items, int wm1) {
  constexpr int E = 8, LPK = D / E, KPI = 32 / LPK;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, grp = lane / LPK, sub = lane % LPK, PS = K + wm1 + 1;
  const int64_t item = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (item >= n_items) return;
  const int64_t row = item / PS;
  const int slot = int(item % PS), b = int(row / Hq), h = int(row % Hq) / G;
  const int64_t own = decode_own_chunk(seqlens, b, cap), nc = cap / kChunk;
  int64_t c = -1;
  if (own >= 0) {
    if (slot >= K) {
      c = own - (slot - K);
    } else {
      c = sel_ids[row * K + slot];
      if (c >= 0 && c >= own - wm1) {
        if (lane == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
        c = -1;
      }
    }
  }
  const int64_t off = c >= 0 ? quant_block_offset<D>(table, n_pages, b, h, c, Hkv, nc) : -1;
  if (off < 0) {
    if (lane == 0) part_u[row * PS + slot] = -INFINITY;
    return;
  }
  const int n_keys = slot == K ? int(seqlens[b] - own * kChunk) : kChunk;
  float qv[E];
  const T* qr = q + row * D + sub * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (sizeof(T) == 2) qv[e] = __bfloat162float(qr[e]);
    else qv[e] = qr[e];
  }
  SoftAcc<E> a;
  a.init();
  for (int r = grp; r < kChunk; r += KPI) {
    float k[E], v[E], part = 0.f;
    quant_load_row<D, E>(kpg + off, r, sub, k);
    quant_load_row<D, E>(vpg + off, r, sub, v);
#pragma unroll
    for (int e = 0; e < E; ++e) part = fmaf(qv[e], k[e], part);
    const float z = group_sum<LPK>(part) * tau;
    if (r < n_keys) a.add(z, v);
  }
#pragma unroll
  for (int o = LPK; o < 32; o <<= 1) a.merge_xor(o);
  if (grp != 0) return;
  const float inv = 1.f / a.l;
#pragma unroll
  for (int e = 0; e < E; ++e) part_o[(row * PS + slot) * D + sub * E + e] = a.acc[e] * inv;
  if (sub == 0) part_u[row * PS + slot] = slot >= K ? a.m + logf(a.l) : sel_scores[row * K + slot];
}

}  // namespace hils
