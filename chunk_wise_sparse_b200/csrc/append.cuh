// Filling and reading a chunk-paged cache: the append of new keys and values
// with the position rotation applied on the way, the read-back of a 4-bit
// cache, and the landmark summaries of the chunks that an append completes.
//
// All three take the ragged batch of an append: sequence b has the packed
// tokens cu[b] .. cu[b+1]-1, which are its positions seqlens[b] - n_b ..
// seqlens[b] - 1.
#pragma once
#include "quant.cuh"

namespace hils {

struct TokenBatch {
  const int32_t* cu;        // [B+1], or nullptr: `per` tokens of every sequence
  const int32_t* seqlens;   // [B], after the append
  int64_t n_tokens, per, cap;
  int batch;
};

// Where a packed token lives.  b < 0: nowhere (padding behind the last
// sequence, or a batch description that does not fit, which is recorded).
struct Place {
  int64_t b, pos;
};

__device__ __forceinline__ Place place_in(const TokenBatch& tb, int64_t t, int64_t b, int64_t lo, int64_t hi) {
  Place p{-1, 0};
  const int64_t len = __ldg(tb.seqlens + b), start = len - (hi - lo);
  if (lo < 0 || t < lo || t >= hi || start < 0 || len > tb.cap) {
    record_error(HILS_ERR_DEVICE_BOUNDS);
    return p;
  }
  p.b = b;
  p.pos = start + (t - lo);
  return p;
}

// The place of token t, found by one thread.
__device__ __forceinline__ Place find_place(const TokenBatch& tb, int64_t t) {
  if (tb.cu == nullptr) {
    const int64_t b = t / tb.per;
    return place_in(tb, t, b, b * tb.per, (b + 1) * tb.per);
  }
  if (t >= __ldg(tb.cu + tb.batch)) return Place{-1, 0};   // padding
  int64_t lo = 0, hi = tb.batch;       // the last b with cu[b] <= t
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(tb.cu + mid) <= t) lo = mid; else hi = mid;
  }
  return place_in(tb, t, lo, __ldg(tb.cu + lo), __ldg(tb.cu + lo + 1));
}

// One block (or warp) of a launch looks at the whole of cu_tokens: it has to
// ascend from 0 to at most n_tokens.
__device__ __forceinline__ void check_batch(const TokenBatch& tb, int thread, int threads) {
  if (tb.cu == nullptr) return;
  bool bad = thread == 0 && (__ldg(tb.cu) != 0 || __ldg(tb.cu + tb.batch) > tb.n_tokens);
  for (int j = thread; j < tb.batch; j += threads) bad |= __ldg(tb.cu + j) > __ldg(tb.cu + j + 1);
  if (bad) record_error(HILS_ERR_DEVICE_BOUNDS);
}

// Rows [n_tokens, heads] of d elements with any token and head stride (in elements).
struct RowsView {
  void* data;
  int64_t ts, hs;
};

struct AppendParams {
  TokenBatch tb;
  RowsView q, q_out, k, v;      // q.data nullptr: no queries
  void *k_pages, *v_pages;
  const int32_t* table;
  int64_t n_pages, nc;
  const float* rotary;          // [n_pos, rot]: rot/2 cosines, rot/2 sines
  int64_t n_pos;
  int rot, interleaved;
  int Hq, Hkv;
};

// One CTA per token.  A row (one head of q, k or v) is held by D / E lanes, a
// 16-byte vector each; the angles of the lane's dims are loaded once and used
// for all of its rows.  y = x c + x' s' with x' the other element of the
// pair (another lane's in the half-split style, fetched by a shuffle).
template <typename T, int D, bool Q4>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendParams p) {
  constexpr int E = Vec16<T>::E, LPR = D / E, RPP = 256 / LPR;
  const int64_t t = blockIdx.x;
  if (t == 0) check_batch(p.tb, threadIdx.x, 256);
  const Place at = find_place(p.tb, t);
  if (at.b < 0) return;
  if (p.rot > 0 && at.pos >= p.n_pos) {
    if (threadIdx.x == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
    return;
  }
  const int sub = threadIdx.x % LPR, row0 = threadIdx.x / LPR, lane = threadIdx.x & 31;
  const int64_t page = __ldg(p.table + at.b * p.nc + at.pos / kChunk);
  const bool in_pool = page >= 0 && page < p.n_pages;
  if (!in_pool && threadIdx.x == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
  const int in_chunk = int(at.pos % kChunk);
  // the angles of this lane's dims, the sign of the second term in `s`
  const int dim0 = sub * E, half = p.rot / 2;
  const bool turns = dim0 < p.rot;
  float c[E], s[E];
  int partner = lane;
  if (turns) {
    const float* tr = p.rotary + at.pos * p.rot;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = p.interleaved ? (dim0 + e) / 2 : (dim0 + e) % half;
      const bool second = p.interleaved ? (e & 1) : dim0 >= half;
      c[e] = __ldg(tr + i);
      const float sn = __ldg(tr + half + i);
      s[e] = second ? sn : -sn;
    }
    if (!p.interleaved) partner = lane + (dim0 < half ? half / E : -(half / E));
  }
  const int Hq = p.q.data ? p.Hq : 0, total = Hq + 2 * p.Hkv;
  for (int r0 = 0; r0 < total; r0 += RPP) {
    const int r = r0 + row0;
    const bool live = r < total;
    const int kind = r < Hq ? 0 : r < Hq + p.Hkv ? 1 : 2;    // query, key, value
    const int h = kind == 0 ? r : r - Hq - (kind - 1) * p.Hkv;
    const RowsView& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = *reinterpret_cast<const uint4*>(static_cast<const T*>(src.data) + t * src.ts + h * src.hs + dim0);
    float x[E], y[E];
    if constexpr (E == 8) {
      Vec16<T>::unpack(w, x);
    } else {
      x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
    if (p.rot > 0) {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, w.x, partner);
      o.y = __shfl_sync(0xffffffffu, w.y, partner);
      o.z = __shfl_sync(0xffffffffu, w.z, partner);
      o.w = __shfl_sync(0xffffffffu, w.w, partner);
      float z[E];
      if constexpr (E == 8) {
        Vec16<T>::unpack(o, z);
      } else {
        z[0] = __uint_as_float(o.x); z[1] = __uint_as_float(o.y); z[2] = __uint_as_float(o.z); z[3] = __uint_as_float(o.w);
      }
      if (turns && kind < 2) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = fmaf(x[e], c[e], (p.interleaved ? x[e ^ 1] : z[e]) * s[e]);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = y[e];
      }
    }
    if constexpr (Q4) {
      // every lane takes part in the shuffles, the rows of queries without storing
      uint8_t* pool = static_cast<uint8_t*>(kind == 1 ? p.k_pages : p.v_pages);
      const bool store = live && in_pool && kind > 0;
      quant_store_row<D, E>(x, sub, pool + (store ? (page * p.Hkv + h) * QuantPage<D>::BLOCK : 0), in_chunk, store);
      if (kind > 0) continue;
    }
    if (!live) continue;
    T* dst;
    if (kind == 0) {
      dst = static_cast<T*>(p.q_out.data) + t * p.q_out.ts + h * p.q_out.hs;
    } else {
      if (!in_pool) continue;
      dst = static_cast<T*>(kind == 1 ? p.k_pages : p.v_pages) + ((page * p.Hkv + h) * kChunk + in_chunk) * D;
    }
    Vec16<T>::store(dst + dim0, x);
  }
}

struct ReadParams {
  TokenBatch tb;
  RowsView k, v;               // outputs; data nullptr: not wanted
  const uint8_t *k_pages, *v_pages;
  const int32_t* table;
  int64_t n_pages, nc;
  int Hkv;
};

// One CTA per token, D / E lanes per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_read_quant_kernel(ReadParams p) {
  constexpr int E = Vec16<T>::E, LPR = D / E, RPP = 256 / LPR;
  const int64_t t = blockIdx.x;
  if (t == 0) check_batch(p.tb, threadIdx.x, 256);
  const Place at = find_place(p.tb, t);
  if (at.b < 0) return;
  const int64_t page = __ldg(p.table + at.b * p.nc + at.pos / kChunk);
  if (page < 0 || page >= p.n_pages) {
    if (threadIdx.x == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
    return;
  }
  const int sub = threadIdx.x % LPR;
  for (int r = threadIdx.x / LPR; r < 2 * p.Hkv; r += RPP) {
    const bool key = r < p.Hkv;
    const RowsView& dst = key ? p.k : p.v;
    if (dst.data == nullptr) continue;
    const int h = key ? r : r - p.Hkv;
    float x[E];
    quant_load_row<D, E>((key ? p.k_pages : p.v_pages) + (page * p.Hkv + h) * QuantPage<D>::BLOCK, int(at.pos % kChunk),
                         sub, x);
    Vec16<T>::store(static_cast<T*>(dst.data) + t * dst.ts + h * dst.hs + sub * E, x);
  }
}

// A chunk's key rows, in the cache's type or in 4 bits.
template <typename T, int D> struct DenseRows {
  static constexpr int E = Vec16<T>::E;
  static constexpr int64_t BLOCK = int64_t(kChunk) * D * sizeof(T);
  __device__ __forceinline__ static void load(const uint8_t* block, int row, int sub, float (&x)[E]) {
    Vec16<T>::load_stream(reinterpret_cast<const T*>(block) + row * D + sub * E, x);
  }
};
template <typename T, int D> struct QuantRows {
  static constexpr int E = Vec16<T>::E;
  static constexpr int64_t BLOCK = QuantPage<D>::BLOCK;
  __device__ __forceinline__ static void load(const uint8_t* block, int row, int sub, float (&x)[E]) {
    quant_load_row<D, E>(block, row, sub, x);
  }
};

struct SummaryParams {
  TokenBatch tb;
  const uint8_t* k_pages;
  const int32_t* table;
  int64_t n_pages, nc, unit;    // tokens that one warp looks through
  const void* lq;
  float *kp, *bp;
  __nv_bfloat16* kmma;
  int Hkv;
  float tau;
};

// One warp per (`unit` packed tokens, kv head): it summarises each chunk whose
// last position is among its tokens, as summary_kernel does a chunk.
template <typename T, int D, typename Rows>
__global__ void __launch_bounds__(128) summary_append_kernel(SummaryParams p) {
  constexpr int E = Rows::E, LPK = D / E, KPI = 32 / LPK, ITERS = kChunk / KPI;
  const int lane = threadIdx.x & 31, grp = lane / LPK, sub = lane % LPK;
  const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t n_units = (p.tb.n_tokens + p.unit - 1) / p.unit;
  if (w >= n_units * p.Hkv) return;
  const int64_t h = w % p.Hkv, t0 = w / p.Hkv * p.unit;
  const int64_t t1 = t0 + p.unit < p.tb.n_tokens ? t0 + p.unit : p.tb.n_tokens;
  if (w == 0) check_batch(p.tb, lane, 32);
  for (int64_t tt = t0; tt < t1; tt += 32) {
    Place mine{-1, 0};
    if (tt + lane < t1) mine = find_place(p.tb, tt + lane);
    uint32_t todo = __ballot_sync(0xffffffffu, mine.b >= 0 && mine.pos % kChunk == kChunk - 1);
    while (todo) {
      const int from = __ffs(int(todo)) - 1;
      todo &= todo - 1;
      const int64_t b = __shfl_sync(0xffffffffu, mine.b, from), c = __shfl_sync(0xffffffffu, mine.pos, from) / kChunk;
      const int64_t page = __ldg(p.table + b * p.nc + c), bh = b * p.Hkv + h;
      if (page < 0 || page >= p.n_pages) {
        if (lane == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
        continue;
      }
      const uint8_t* block = p.k_pages + (page * p.Hkv + h) * Rows::BLOCK;
      float lq[E];
      Vec16<T>::load(static_cast<const T*>(p.lq) + (bh * p.nc + c) * D + sub * E, lq);
      float m = -INFINITY, l = 0.f, s = 0.f, acc[E];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
      for (int it = 0; it < ITERS; ++it) {
        float k[E];
        Rows::load(block, it * KPI + grp, sub, k);
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) part = fmaf(lq[e], k[e], part);
        const float z = group_sum<LPK>(part) * p.tau;
        const float mn = fmaxf(m, z), a = expf(m - mn), q = expf(z - mn);
        l = l * a + q;
        s = s * a + q * z;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + q * k[e];
        m = mn;
      }
#pragma unroll
      for (int off = LPK; off < 32; off <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m, off), lo = __shfl_xor_sync(0xffffffffu, l, off);
        const float so = __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, mo), a = expf(m - mn), q = expf(mo - mn);
        l = l * a + lo * q;
        s = s * a + so * q;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + __shfl_xor_sync(0xffffffffu, acc[e], off) * q;
        m = mn;
      }
      if (grp != 0) continue;
      const float inv = 1.f / l, bias = m + logf(l) - s * inv;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= inv;
      float* ko = p.kp + (bh * p.nc + c) * D + sub * E;
#pragma unroll
      for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(ko + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
      if (sub == 0) p.bp[bh * p.nc + c] = bias;
      if (p.kmma != nullptr) {
        __nv_bfloat16* row = p.kmma + (bh * p.nc + c) * (D + kExt);
#pragma unroll
        for (int e = 0; e < E; e += 2)
          *reinterpret_cast<__nv_bfloat162*>(row + sub * E + e) = __floats2bfloat162_rn(acc[e], acc[e + 1]);
        if (sub == 0) {
          // b'/tau as the sum of two bf16 values (see summary_kernel)
          const float x = bias / p.tau;
          __nv_bfloat162 hl;
          hl.x = __float2bfloat16_rn(x);
          hl.y = __float2bfloat16_rn(x - __bfloat162float(hl.x));
          *reinterpret_cast<uint4*>(row + D) = make_uint4(*reinterpret_cast<uint32_t*>(&hl), 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(row + D + 8) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
  }
}

}  // namespace hils
