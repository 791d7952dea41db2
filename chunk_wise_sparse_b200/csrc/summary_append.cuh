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
// the sums need no rescaling inside a warp.
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

// d = a b + c on a pair of fp32 values
__device__ __forceinline__ void fma_pair(float2& d, float2 a, float2 b, float2 c) {
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
}

// Keys in 4 bits.  Four lanes per key row, eight rows per step; a lane has
// eight dims of every group, which its two 16-bit units per group hold as
// pairs (i, i + 4).  One pass: logits of a step, the running maximum (rescaled
// only when a step raises it, about three times in eight steps), and the
// weighted sum, all in fp32 on pairs of values (code - 8, exact in bf16, widened by a
// shift).  WARPS warps share a chunk: 4 where chunks are few (a decode step: latency),
// 1 where they fill the GPU (a prompt: fewer instructions).
// Bound by instructions: about three per pair of codes and four for its two
// products.  Measured on 2048 chunks x 16 heads of 64 dims (84 MB): see
// launch_summary_append.
constexpr int kSummaryAhead = 8;      // steps whose loads are in flight

template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(128, D == 64 ? 5 : 3) summary_quant_kernel(SummaryParams p) {
  using P = QuantPage<D>;
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr int NG = P::G, STEPS = 8 / WARPS, AHEAD = STEPS < kSummaryAhead ? STEPS : kSummaryAhead;
  __shared__ Done found[kUnitMost];
  __shared__ int count;
  __shared__ __align__(16) float part[4][D];      // written in 16-byte pieces
  __shared__ float stat[4][3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane >> 2, sub = lane & 3;
  const int per = WARPS == 4 ? p.Hkv : (p.Hkv + 3) / 4;      // CTAs per unit
  const int64_t h = WARPS == 4 ? blockIdx.x % per : int64_t(blockIdx.x % per) * 4 + warp;
  if (blockIdx.x == 0) check_batch(p.tb, threadIdx.x, 128);
  const int n = completed_chunks(p, blockIdx.x / per * p.unit, found, &count);
  if (h >= p.Hkv || n == 0) return;        // h: WARPS == 1 only, no barrier follows
  const int row0 = (WARPS == 4 ? 16 * warp : 0) + row;
  uint32_t code[AHEAD][NG], par[AHEAD][NG];
  auto load = [&](int i, int st, int to) {
    const uint8_t* block = p.k_pages + (found[i].page * int64_t(p.Hkv) + h) * P::BLOCK;
    const int key = row0 + 8 * st;
    if constexpr (NG == 4) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(block + P::code_off(key) + 16 * sub));
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(block + P::param_off(key)));
      code[to][0] = u.x; code[to][1] = u.y; code[to][2] = u.z; code[to][3] = u.w;
      par[to][0] = w.x; par[to][1] = w.y; par[to][2] = w.z; par[to][3] = w.w;
    } else {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(block + P::code_off(key) + 8 * sub));
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(block + P::param_off(key)));
      code[to][0] = u.x; code[to][1] = u.y;
      par[to][0] = w.x; par[to][1] = w.y;
    }
  };
  constexpr int QV = sizeof(T) == 2 ? 1 : 2;      // 16-byte pieces of eight values
  uint4 lqv[NG][QV];
  auto load_lq = [&](int i) {
    const T* lqr = static_cast<const T*>(p.lq) + (found[i].unit + h * p.nc) * D + 8 * sub;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < QV; ++e) lqv[g][e] = __ldg(reinterpret_cast<const uint4*>(lqr + 32 * g) + e);
  };
  load_lq(0);
#pragma unroll
  for (int st = 0; st < AHEAD; ++st) load(0, st, st);
  for (int i = 0; i < n; ++i) {
    const int64_t unit = found[i].unit + h * p.nc;
    float2 lq[NG][4];       // dims 32 g + 8 sub + {i, i + 4}
    float lsum[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float x[8];
      if constexpr (QV == 1) {
        Vec16<T>::unpack(lqv[g][0], x);
      } else {
        const uint32_t w[8] = {lqv[g][0].x, lqv[g][0].y, lqv[g][0].z, lqv[g][0].w,
                               lqv[g][QV - 1].x, lqv[g][QV - 1].y, lqv[g][QV - 1].z, lqv[g][QV - 1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
      }
      lsum[g] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lq[g][e] = make_float2(x[e], x[e + 4]);
        lsum[g] += x[e] + x[e + 4];
      }
    }
    float m = -INFINITY, l = 0.f, s = 0.f, low[NG];
    float2 acc[NG][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      low[g] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[g][e] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      const int at = st % AHEAD;
      float2 x[NG][4];
      float sg[NG], mg[NG], z = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t a[4];
        codes_bf16<true>(__byte_perm(code[at][g / 2], code[at][NG / 2 + g / 2], g & 1 ? 0x7632 : 0x5410), a);
        const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&par[at][g]));
        sg[g] = sm.x;
        mg[g] = fmaf(8.f, sm.x, sm.y);
        float2 d = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[g][e] = make_float2(lo_bf16(a[e]), hi_bf16(a[e]));
          fma_pair(d, lq[g][e], x[g][e], d);
        }
        z = fmaf(sg[g], d.x + d.y, fmaf(mg[g], lsum[g], z));
      }
      if (st + AHEAD < STEPS) load(i, st + AHEAD, at);
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      z *= p.tau * kLog2e;       // logits in base 2 from here on
      float top = z;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (top > m) {         // the same for the whole warp
        const float f = pow2<true>(m - top);      // 0 the first time
        l *= f;
        s *= f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          low[g] *= f;
#pragma unroll
          for (int e = 0; e < 4; ++e) { acc[g][e].x *= f; acc[g][e].y *= f; }
        }
        m = top;
      }
      const float w = pow2<true>(z - m);
      l += w;
      s = fmaf(w, z, s);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float ws = w * sg[g];
        low[g] = fmaf(w, mg[g], low[g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) fma_pair(acc[g][e], make_float2(ws, ws), x[g][e], acc[g][e]);
      }
    }
    // the next chunk's loads are on their way while this one is summed up
    if (i + 1 < n) {
      load_lq(i + 1);
#pragma unroll
      for (int st = 0; st < AHEAD; ++st) load(i + 1, st, st);
    }
    // ---- sums over the eight rows: each lane ends with the NG sums from `own` on
    float v[8 * NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) { v[8 * g + e] = acc[g][e].x; v[8 * g + 4 + e] = acc[g][e].y; }
    int own = 0;
#pragma unroll
    for (int bit = 16, half = 4 * NG; bit >= 4; bit >>= 1, half >>= 1) {
      const bool up = lane & bit;
      own += up ? half : 0;
#pragma unroll
      for (int e = 0; e < half; ++e) {
        const float give = up ? v[e] : v[e + half], keep = up ? v[e + half] : v[e];
        v[e] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
      for (int g = 0; g < NG; ++g) low[g] += __shfl_xor_sync(0xffffffffu, low[g], o);
    }
    const int g_own = own / 8, dim = 32 * g_own + 8 * sub + own % 8;      // NG neighbouring dims of one group
    float add = low[0];
#pragma unroll
    for (int g = 1; g < NG; ++g) add = g_own == g ? low[g] : add;
    if constexpr (WARPS == 1) {
      const float inv = 1.f / l;
#pragma unroll
      for (int e = 0; e < NG; ++e) v[e] = (v[e] + add) * inv;
      float* out = p.kp + unit * D + dim;
      if constexpr (NG == 4) *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
      else *reinterpret_cast<float2*>(out) = make_float2(v[0], v[1]);
      const float bias = (m - s * inv) * (1.f / kLog2e) + logf(l);
      if (lane == 0) p.bp[unit] = bias;
      if (p.kmma != nullptr) {
        __nv_bfloat16* mrow = p.kmma + unit * (D + kExt);
        if constexpr (NG == 4) *reinterpret_cast<uint2*>(mrow + dim) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else *reinterpret_cast<uint32_t*>(mrow + dim) = pack_bf16(v[0], v[1]);
        if (lane < 8) {      // b'/tau as the sum of two bf16 values (see summary_kernel), then zeros
          const float x = bias / p.tau;
          const float hi = __bfloat162float(__float2bfloat16_rn(x));
          reinterpret_cast<uint32_t*>(mrow + D)[lane] = lane == 0 ? pack_bf16(hi, x - hi) : 0u;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < NG; ++e) part[warp][dim + e] = v[e] + add;
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
