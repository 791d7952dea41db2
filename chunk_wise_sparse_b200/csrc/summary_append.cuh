// Landmark summaries of the chunks that an append completed, for a ragged
// batch: k' = sum p_j k_j, b' = -sum p_j log p_j with p = softmax(tau lq.k_j),
// as in summary.cuh.
//
// A CTA of four warps looks through `unit` packed tokens (as many as a
// sequence has on average, up to a chunk) for last positions of chunks and
// summarises those it finds, one kv head per CTA.  In a decode step that is one
// token per CTA and latency counts: the four warps share a chunk, 16 keys
// each, all loads in flight at once, and merge through shared memory.
#pragma once
#include "append.cuh"
#include "mma16.cuh"

namespace hils {

struct SummaryParams {
  TokenBatch tb;
  const uint8_t* k_pages;
  const int32_t* table;
  int64_t n_pages, nc, unit;    // tokens that one CTA looks through, at most kUnitMost
  const void* lq;
  float *kp, *bp;
  __nv_bfloat16* kmma;
  int Hkv;
  float tau;
};

constexpr int kUnitMost = 256;

// A completed chunk: its place among the summaries of kv head 0, and its page.
struct Done {
  int64_t unit;
  int page;
};

// The chunks whose last token is among the CTA's, into shared memory; returns
// how many.  128 threads; starts and ends in step.
__device__ __forceinline__ int completed_chunks(const SummaryParams& p, int64_t t0, Done* found, int* count) {
  const int tid = threadIdx.x;
  if (tid == 0) *count = 0;
  __syncthreads();
  for (int64_t t = t0 + tid; t < t0 + p.unit && t < p.tb.n_tokens; t += 128) {
    const Place at = find_place(p.tb, t);
    if (at.b >= 0 && at.pos % kChunk == kChunk - 1) {
      const int64_t c = at.pos / kChunk;
      const int page = __ldg(p.table + at.b * p.nc + c);
      if (page < 0 || page >= p.n_pages) record_error(HILS_ERR_DEVICE_BOUNDS);
      else found[atomicAdd(count, 1)] = Done{at.b * p.Hkv * p.nc + c, page};   // in any order: chunks are independent
    }
  }
  __syncthreads();
  return *count;
}

// The chunk's summary row from its sums, by D threads: k' of this thread's dim
// and b'.
template <int D>
__device__ __forceinline__ void write_summary(const SummaryParams& p, int64_t unit, int dim, float kp, float bias) {
  p.kp[unit * D + dim] = kp;
  if (dim == 0) p.bp[unit] = bias;
  if (p.kmma != nullptr) {
    __nv_bfloat16* row = p.kmma + unit * (D + kExt);
    row[dim] = __float2bfloat16_rn(kp);
    if (dim < kExt) {
      // b'/tau as the sum of two bf16 values (see summary_kernel), then zeros
      const float x = bias / p.tau;
      const __nv_bfloat16 hi = __float2bfloat16_rn(x);
      row[D + dim] = dim == 0 ? hi : dim == 1 ? __float2bfloat16_rn(x - __bfloat162float(hi)) : __float2bfloat16_rn(0.f);
    }
  }
}

// Keys in the cache's own type: D / E lanes per key row.  Each warp's 16 keys
// are loaded at once; their logits' maximum comes before any exponential, so
// the sums need no rescaling inside a warp.  A step of 64 sequences of which
// four complete a chunk (8 kv heads of 128 dims): 6.2 us in a graph, of which a
// launch is about 4; a warp per chunk with four rows in flight took 14.4.
template <typename T, int D>
__global__ void __launch_bounds__(128) summary_append_kernel(SummaryParams p) {
  constexpr int E = Vec16<T>::E, LPK = D / E, KPI = 32 / LPK, ITERS = 16 / KPI;
  __shared__ Done found[kUnitMost];
  __shared__ int count;
  __shared__ __align__(16) float part[4][D];      // written in 16-byte pieces
  __shared__ float stat[4][3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane / LPK, sub = lane % LPK;
  const int64_t h = blockIdx.x % p.Hkv;
  if (blockIdx.x == 0) check_batch(p.tb, threadIdx.x, 128);
  const int n = completed_chunks(p, blockIdx.x / p.Hkv * p.unit, found, &count);
  for (int i = 0; i < n; ++i) {
    const int64_t unit = found[i].unit + h * p.nc, page = found[i].page;
    const T* rows = reinterpret_cast<const T*>(p.k_pages) + ((page * p.Hkv + h) * kChunk + warp * 16) * D + sub * E;
    uint4 k[ITERS];
#pragma unroll
    for (int it = 0; it < ITERS; ++it) k[it] = __ldcs(reinterpret_cast<const uint4*>(rows + (it * KPI + grp) * D));
    float lq[E];
    Vec16<T>::load(static_cast<const T*>(p.lq) + unit * D + sub * E, lq);
    float z[ITERS], m = -INFINITY;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      float x[E], d = 0.f;
      widen<T>(k[it], x);
#pragma unroll
      for (int e = 0; e < E; ++e) d = fmaf(lq[e], x[e], d);
      z[it] = group_sum<LPK>(d) * p.tau;
      m = fmaxf(m, z[it]);
    }
#pragma unroll
    for (int o = LPK; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, s = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const float w = expf(z[it] - m);
      float x[E];
      widen<T>(k[it], x);
      l += w;
      s = fmaf(w, z[it], s);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[e], acc[e]);
    }
#pragma unroll
    for (int o = LPK; o < 32; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    }
    if (grp == 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) part[warp][sub * E + e] = acc[e];
      if (sub == 0) { stat[warp][0] = m; stat[warp][1] = l; stat[warp][2] = s; }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float M = fmaxf(fmaxf(stat[0][0], stat[1][0]), fmaxf(stat[2][0], stat[3][0])), L = 0.f, S = 0.f, a = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = expf(stat[w][0] - M);
        L = fmaf(f, stat[w][1], L);
        S = fmaf(f, stat[w][2], S);
        a = fmaf(f, part[w][threadIdx.x], a);
      }
      write_summary<D>(p, unit, threadIdx.x, a / L, M + logf(L) - S / L);
    }
    __syncthreads();
  }
}

// Keys in 4 bits, by matrix products of 16 keys, of the codes where they lie
// (codes_f16) and fp16 operands, as the decode step reads them; the columns that
// one landmark query leaves free carry the precision of fp32.
//   logits: columns 0 and 1 hold the query, scaled by a power of two that puts
//     its largest value in [2^14, 2^15), as a sum of two fp16 values (22 bits;
//     bf16 is exact in one): z_j = tau sum_g [ s_jg acc_jg + m_jg sum_{i in g} q_i ].
//   sum of keys: with x_jg = p_j s_jg 2^k = hi + lo (k puts the largest step in
//     [2^14, 2^15)), the pair (hi, lo) of a key is columns 0 and 1 of its row, and the
//     transpose that makes the row a column operand is one instruction:
//     k' l = 2^-k sum_j x_jg (code_j - 8) + sum_j p_j (m_jg + 8 s_jg).
// Each WARPS warps share a chunk: 4 where chunks are few (a decode step:
// latency), 1 where they fill the GPU (a prompt: fewer instructions, by which
// it is bound).  Measured on 2048 chunks x 16 heads of 64 dims (84 MB): 53 us;
// in fp32 on pairs of values 59 us, a lane per eight dims with an online
// softmax per key 86 us.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(128, D == 64 ? 5 : 3) summary_quant_kernel(SummaryParams p) {
  using P = QuantPage<D>;
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr int NG = P::G, TILES = 4 / WARPS;
  constexpr bool EXACT = sizeof(T) == 2;      // one fp16 value holds a scaled bf16 one
  __shared__ Done found[kUnitMost];
  __shared__ int count;
  __shared__ __align__(16) float part[4][D];      // written in 16-byte pieces
  __shared__ float stat[4][3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int per = WARPS == 4 ? p.Hkv : (p.Hkv + 3) / 4;      // CTAs per unit
  const int64_t h = WARPS == 4 ? blockIdx.x % per : int64_t(blockIdx.x % per) * 4 + warp;
  if (blockIdx.x == 0) check_batch(p.tb, threadIdx.x, 128);
  const int n = completed_chunks(p, blockIdx.x / per * p.unit, found, &count);
  if (h >= p.Hkv || n == 0) return;        // h: WARPS == 1 only, no barrier follows
  const int key0 = WARPS == 4 ? 16 * warp : 0;

  // rows 16 t + 8 r + gid of a chunk: the lane's code words and all parameters
  uint32_t code[TILES][2][NG], par[TILES][2][NG];
  constexpr int QV = EXACT ? 1 : 2;        // 16-byte pieces of eight values
  uint4 lqv[NG][QV];
  auto load = [&](int i) {
    const uint8_t* block = p.k_pages + (found[i].page * int64_t(p.Hkv) + h) * P::BLOCK;
    const T* lqr = static_cast<const T*>(p.lq) + (found[i].unit + h * p.nc) * D + 8 * tig;
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = key0 + 16 * t + 8 * r + gid;
        if constexpr (NG == 4) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(block + P::code_off(key) + 16 * tig));
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(block + P::param_off(key)));
          code[t][r][0] = u.x; code[t][r][1] = u.y; code[t][r][2] = u.z; code[t][r][3] = u.w;
          par[t][r][0] = w.x; par[t][r][1] = w.y; par[t][r][2] = w.z; par[t][r][3] = w.w;
        } else {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(block + P::code_off(key) + 8 * tig));
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(block + P::param_off(key)));
          code[t][r][0] = u.x; code[t][r][1] = u.y;
          par[t][r][0] = w.x; par[t][r][1] = w.y;
        }
      }
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < QV; ++e) lqv[g][e] = __ldg(reinterpret_cast<const uint4*>(lqr + 32 * g) + e);
  };
  load(0);
  for (int i = 0; i < n; ++i) {
    const int64_t unit = found[i].unit + h * p.nc;
    const uint8_t* block = p.k_pages + (found[i].page * int64_t(p.Hkv) + h) * P::BLOCK;
    // ---- the query as a column operand, dims 32 g + 8 tig + {i, i + 4}; its groups' sums
    uint32_t qb[NG][4];
    float lsum[NG], unscale;
    {
      float x[NG][8], top = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (EXACT) {
          Vec16<T>::unpack(lqv[g][0], x[g]);
        } else {
          const uint32_t w[8] = {lqv[g][0].x, lqv[g][0].y, lqv[g][0].z, lqv[g][0].w,
                                 lqv[g][QV - 1].x, lqv[g][QV - 1].y, lqv[g][QV - 1].z, lqv[g][QV - 1].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) x[g][e] = __uint_as_float(w[e]);
        }
        lsum[g] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lsum[g] += x[g][e];
          top = fmaxf(top, fabsf(x[g][e]));
        }
        lsum[g] += __shfl_xor_sync(0xffffffffu, lsum[g], 1);
        lsum[g] += __shfl_xor_sync(0xffffffffu, lsum[g], 2);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float up;
      power_scale(top, up, unscale);
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = e & 1 ? up * 0.0625f : up, a = x[g][e] * f, b = x[g][e + 4] * f;
          const uint32_t hi = pack_f16(a, b);
          qb[g][e] = gid == 0 ? hi : 0u;
          if constexpr (!EXACT) {
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            if (gid == 1) qb[g][e] = pack_f16(a - back.x, b - back.y);
          }
        }
      unscale *= 16777216.f;      // the codes are multiplied as code 2^-24
    }
    // ---- logits in base 2, in the lanes tig == 0.  The other lanes' columns are
    // zero; what they compute from here on stays in them and in columns from 2 on
    float z[TILES][2], m = -INFINITY;
    __half2 step_top = __floats2half2_rn(0.f, 0.f);       // the largest step, in the lower half
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      float acc[NG][4];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t a[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) codes_f16(code[t][r][g / 2], code[t][r][NG / 2 + g / 2], g & 1, a[r]);
        mma16816_f16_first(acc[g], a[0][0], a[1][0], a[0][1], a[1][1], qb[g][0], qb[g][1]);
        mma16816_f16(acc[g], a[0][2], a[1][2], a[0][3], a[1][3], qb[g][2], qb[g][3]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = 0.f, low = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&par[t][r][g]));
          sum = fmaf(sm.x, EXACT ? acc[g][2 * r] : acc[g][2 * r] + acc[g][2 * r + 1], sum);
          low = fmaf(sm.y, lsum[g], low);
          step_top = __hmax2(step_top, *reinterpret_cast<const __half2*>(&par[t][r][g]));
        }
        z[t][r] = fmaf(sum, unscale, low) * (p.tau * kLog2e);
        m = fmaxf(m, z[t][r]);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float x_up, x_down;       // steps are not negative, so their bits compare as they do
    power_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(__low2float(step_top)))), x_up, x_down);
    // ---- weights, and the sum of keys
    float l = 0.f, s = 0.f, low[NG], acc[NG][2][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      low[g] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[g][e / 4][e % 4] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      uint32_t xb[NG][2], vc[2][2][NG / 2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = key0 + 16 * t + 8 * r + 2 * tig + j;
          if constexpr (NG == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(block + P::code_off(key) + 8 * gid));
            vc[r][j][0] = u.x; vc[r][j][1] = u.y;
          } else {
            vc[r][j][0] = __ldg(reinterpret_cast<const uint32_t*>(block + P::code_off(key) + 4 * gid));
          }
        }
        const float w = pow2<true>(z[t][r] - m);
        l += w;
        s = fmaf(w, z[t][r], s);
        const float ws = w * x_up;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&par[t][r][g]));
          low[g] = fmaf(w, fmaf(8.f, sm.x, sm.y), low[g]);
          const float x = ws * sm.x;
          const __half hi = __float2half_rn(x);
          const __half2 pair = __halves2half2(hi, __float2half_rn(x - __half2float(hi)));
          xb[g][r] = movmatrix(*reinterpret_cast<const uint32_t*>(&pair));
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t a[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) codes_f16_centred(vc[r][0][g / 2], vc[r][1][g / 2], g & 1, a[r]);
        mma16816_f16(acc[g][0], a[0][0], a[0][1], a[1][0], a[1][1], xb[g][0], xb[g][1]);
        mma16816_f16(acc[g][1], a[0][2], a[0][3], a[1][2], a[1][3], xb[g][0], xb[g][1]);
      }
    }
    // the next chunk's loads are on their way while this one is summed up
    if (i + 1 < n) load(i + 1);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
      for (int g = 0; g < NG; ++g) low[g] += __shfl_xor_sync(0xffffffffu, low[g], o);
    }
    // lanes tig == 0: dims 32 g + 4 gid + 0 .. 3 (odd ones multiplied as 16 (code - 8))
    float4 v[NG];
    const float f0 = x_down, f1 = x_down * 0.0625f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      v[g] = make_float4(fmaf(acc[g][0][0] + acc[g][0][1], f0, low[g]), fmaf(acc[g][0][2] + acc[g][0][3], f1, low[g]),
                         fmaf(acc[g][1][0] + acc[g][1][1], f0, low[g]), fmaf(acc[g][1][2] + acc[g][1][3], f1, low[g]));
    if constexpr (WARPS == 1) {
      if (tig == 0) {
        const float inv = 1.f / l, bias = (m - s * inv) * (1.f / kLog2e) + logf(l);
        float* out = p.kp + unit * D + 4 * gid;
        __nv_bfloat16* mrow = p.kmma + unit * (D + kExt);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float4 y = make_float4(v[g].x * inv, v[g].y * inv, v[g].z * inv, v[g].w * inv);
          *reinterpret_cast<float4*>(out + 32 * g) = y;
          if (p.kmma != nullptr) *reinterpret_cast<uint2*>(mrow + 32 * g + 4 * gid) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        }
        if (gid == 0) p.bp[unit] = bias;
        if (p.kmma != nullptr) {      // b'/tau as the sum of two bf16 values (see summary_kernel), then zeros
          const float x = bias / p.tau, hi = __bfloat162float(__float2bfloat16_rn(x));
          reinterpret_cast<uint32_t*>(mrow + D)[gid] = gid == 0 ? pack_bf16(hi, x - hi) : 0u;
        }
      }
    } else {
      if (tig == 0) {
#pragma unroll
        for (int g = 0; g < NG; ++g) *reinterpret_cast<float4*>(&part[warp][32 * g + 4 * gid]) = v[g];
      }
      if (lane == 0) { stat[warp][0] = m; stat[warp][1] = l; stat[warp][2] = s; }
      __syncthreads();
      if (threadIdx.x < D) {
        const float M = fmaxf(fmaxf(stat[0][0], stat[1][0]), fmaxf(stat[2][0], stat[3][0]));
        float L = 0.f, S = 0.f, a = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float f = pow2<true>(stat[q][0] - M);
          L = fmaf(f, stat[q][1], L);
          S = fmaf(f, stat[q][2], S);
          a = fmaf(f, part[q][threadIdx.x], a);
        }
        write_summary<D>(p, unit, threadIdx.x, a / L, (M - S / L) * (1.f / kLog2e) + logf(L));
      }
      __syncthreads();
    }
  }
}

}  // namespace hils
