// Filling and reading a chunk-paged cache: the append of new keys and values
// with the position rotation applied on the way, and the read-back of a 4-bit
// cache.
//
// Both, and the summaries of summary_append.cuh, take the ragged batch of an append: sequence b has the packed
// tokens cu[b] .. cu[b+1]-1, which are its positions seqlens[b] - n_b ..
// seqlens[b] - 1.
#pragma once
#include <type_traits>

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

// The place of token t as one of sequence b's, where the last sequence ends at
// `end`.  A sequence that reaches beyond the packed tokens, or whose neighbours'
// tokens do not precede and follow its own, has no places: counted from a wrong
// border its tokens would land on other positions than theirs, over rows that
// the cache already holds.  All loads at once: a decode step waits for them.
__device__ __forceinline__ Place place_in(const TokenBatch& tb, int64_t t, int64_t b, int64_t end) {
  const int64_t len = __ldg(tb.seqlens + b);
  int64_t lo = b * tb.per, hi = lo + tb.per;
  bool bad = false;
  if (tb.cu != nullptr) {
    const int before = __ldg(tb.cu + (b > 0 ? b - 1 : 0)), after = __ldg(tb.cu + (b + 2 < tb.batch ? b + 2 : tb.batch));
    lo = __ldg(tb.cu + b);
    hi = __ldg(tb.cu + b + 1);
    bad = (b == 0 ? lo != 0 : lo < 0) | (before > lo) | (after < hi);
  }
  const int64_t start = len - (hi - lo);
  bad |= (t < lo) | (t >= hi) | (hi > end) | (hi > tb.n_tokens) | (start < 0) | (len > tb.cap);
  if (bad) {
    record_error(HILS_ERR_DEVICE_BOUNDS);
    return Place{-1, 0};
  }
  return Place{b, start + (t - lo)};
}

// The place of token t, found by one thread.
__device__ __forceinline__ Place find_place(const TokenBatch& tb, int64_t t) {
  if (tb.cu == nullptr) return place_in(tb, t, t / tb.per, tb.n_tokens);
  const int end = __ldg(tb.cu + tb.batch);
  if (t >= end) return Place{-1, 0};   // padding
  int64_t lo = 0, hi = tb.batch;       // the last b with cu[b] <= t
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(tb.cu + mid) <= t) lo = mid; else hi = mid;
  }
  return place_in(tb, t, lo, end);
}

// The place of token t (the same for the whole warp): the last b with
// cu[b] <= t by a 32-way search, one load per lane and round, so that a batch
// of up to 32 sequences costs one load latency and one of up to 1024 two.
__device__ __forceinline__ Place find_place_warp(const TokenBatch& tb, int64_t t, int lane) {
  if (tb.cu == nullptr) return place_in(tb, t, t / tb.per, tb.n_tokens);
  const int end = __ldg(tb.cu + tb.batch);
  int lo = 0, len = tb.batch;
  while (len > 1) {
    const int step = (len + 31) / 32, at = lane * step;
    const bool low = at < len && __ldg(tb.cu + lo + at) <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, low));
    const int skip = n > 0 ? (n - 1) * step : 0;
    lo += skip;
    len = len - skip < step ? len - skip : step;
  }
  if (t >= end) return Place{-1, 0};     // padding
  return place_in(tb, t, lo, end);
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
  int shares, per_share;        // warps per token, and steps of KPI rows of each
};

// A 16-byte piece as E fp32 values.
template <typename T>
__device__ __forceinline__ void widen(uint4 w, float (&x)[Vec16<T>::E]) {
  if constexpr (Vec16<T>::E == 8) {
    Vec16<T>::unpack(w, x);
  } else {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
}

// E fp32 values rounded to the type.
template <typename T>
__device__ __forceinline__ uint4 narrow(const float (&x)[Vec16<T>::E]) {
  uint4 w;
  Vec16<T>::store(reinterpret_cast<T*>(&w), x);
  return w;
}

// One warp per (token, share of its rows).  A row (one head of q, k or v) is
// held by LPR = d / E lanes, a 16-byte piece each, KPI = 32 / LPR rows at a
// time; the token's place and the angles of the lane's dims are found once and
// used for all rows of the warp.  y = x c + x' s' with x' the other element of
// the pair (another lane's in the half-split style, fetched by a shuffle).
// The kinds of row are padded to KPI rows each and have a straight loop each.
// For a prompt bound by the latency of its loads: two pieces per lane are loaded
// while two are worked on, at 64 registers and 32 warps per SM.  Measured on a
// 32K prompt of 16 + 2 x 16 heads of 64 dims (407 MB): 79 us, 5.1 TB/s, 78 % of
// a copy's rate; one loop that tells the kinds apart 81 us, four pieces
// without looking ahead 82 us, three ahead 85 us, 51 registers 96 us, one CTA
// per token with the place found by every thread 178 us.  Into 4 bits, 13.9K
// ragged tokens of 32 + 2 x 8 heads of 128 dims (306 MB): about 72 us.
constexpr int kAppendUnroll = 2;
constexpr int kAppendSteps = 32;      // of KPI rows, per warp, where tokens abound

template <typename T, int D, bool Q4>
__global__ void __launch_bounds__(128, 8) kv_append_kernel(AppendParams p) {
  constexpr int E = Vec16<T>::E, LPR = D / E, KPI = 32 / LPR, U = kAppendUnroll;
  const int lane = threadIdx.x & 31, sub = lane % LPR, grp = lane / LPR;
  if (blockIdx.x == 0) check_batch(p.tb, threadIdx.x, 128);
  const int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t t = item / p.shares;
  if (t >= p.tb.n_tokens) return;
  const int nq = p.q.data ? (p.Hq + KPI - 1) / KPI : 0, nk = (p.Hkv + KPI - 1) / KPI;
  const int it0 = int(item % p.shares) * p.per_share;
  const int it1 = it0 + p.per_share < nq + 2 * nk ? it0 + p.per_share : nq + 2 * nk;
  const Place at = find_place_warp(p.tb, t, lane);
  if (at.b < 0) return;
  if (p.rot > 0 && at.pos >= p.n_pos) {
    if (lane == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
    return;
  }
  const int64_t page = __ldg(p.table + at.b * p.nc + at.pos / kChunk);
  const bool in_pool = page >= 0 && page < p.n_pages;
  if (!in_pool && lane == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
  const int in_chunk = int(at.pos % kChunk);
  // the angles of this lane's dims, the sign of the second term in `s`
  const int dim0 = sub * E, half = p.rot / 2;
  const bool turns = dim0 < p.rot;
  float c[E], s[E];
  int partner = lane;
  if (turns) {
    const float* tr = p.rotary + at.pos * p.rot;
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        c[e] = c[e + 1] = __ldg(tr + (dim0 + e) / 2);
        s[e + 1] = __ldg(tr + half + (dim0 + e) / 2);
        s[e] = -s[e + 1];
      }
    } else {
      const bool second = dim0 >= half;
      const int i = second ? dim0 - half : dim0;     // half is a multiple of 8, E at most 8
      partner = second ? lane - half / E : lane + half / E;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(tr + i + e)), sv = __ldg(reinterpret_cast<const float4*>(tr + half + i + e));
        c[e] = cv.x; c[e + 1] = cv.y; c[e + 2] = cv.z; c[e + 3] = cv.w;
        s[e] = second ? sv.x : -sv.x; s[e + 1] = second ? sv.y : -sv.y;
        s[e + 2] = second ? sv.z : -sv.z; s[e + 3] = second ? sv.w : -sv.w;
      }
    }
  }
  // steps a .. b - 1 (of KPI heads each) of one kind of row
  auto segment = [&](auto kind_, const RowsView& in, int heads, int a, int b) {
    constexpr int KIND = decltype(kind_)::value;       // 0 query, 1 key, 2 value
    constexpr bool CODES = Q4 && KIND > 0;
    if (a >= b) return;
    const T* src = static_cast<const T*>(in.data) + t * in.ts + int64_t(a * KPI + grp) * in.hs + dim0;
    const int64_t next = int64_t(KPI) * in.hs;
    // where head a KPI + grp goes, and how far apart the heads of two steps are (bytes)
    uint8_t* dst;
    int64_t dst_next;
    if constexpr (KIND == 0) {
      dst = reinterpret_cast<uint8_t*>(static_cast<T*>(p.q_out.data) + t * p.q_out.ts + int64_t(a * KPI + grp) * p.q_out.hs + dim0);
      dst_next = int64_t(KPI) * p.q_out.hs * int64_t(sizeof(T));
    } else {
      constexpr int64_t BLOCK = CODES ? QuantPage<D>::BLOCK : int64_t(kChunk) * D * int64_t(sizeof(T));
      dst = static_cast<uint8_t*>(KIND == 1 ? p.k_pages : p.v_pages) +
            ((in_pool ? page : 0) * p.Hkv + a * KPI + grp) * BLOCK + (CODES ? 0 : (in_chunk * D + dim0) * int(sizeof(T)));
      dst_next = KPI * BLOCK;
    }
    int left = heads - (a * KPI + grp);      // heads of this lane group from here on, counted in steps of KPI
    uint4 w[U];
    auto load = [&](uint4 (&x)[U], int ahead) {      // of steps `ahead` .. + U - 1 from src on
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u] = make_uint4(0, 0, 0, 0);
        if (ahead + u < b - a && left > (ahead + u) * KPI) x[u] = *reinterpret_cast<const uint4*>(src + (ahead + u) * next);
      }
    };
    load(w, 0);
    for (; a < b; a += U) {
      uint4 ahead[U];
      load(ahead, U);     // of the next round, while this one is worked on
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (a + u >= b) break;
        if (KIND < 2 && p.rot > 0) {
          float x[E], z[E];
          widen<T>(w[u], x);
          if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < E; ++e) z[e] = x[e ^ 1];
          } else {
            uint4 o;
            o.x = __shfl_sync(0xffffffffu, w[u].x, partner);
            o.y = __shfl_sync(0xffffffffu, w[u].y, partner);
            o.z = __shfl_sync(0xffffffffu, w[u].z, partner);
            o.w = __shfl_sync(0xffffffffu, w[u].w, partner);
            widen<T>(o, z);
          }
          if (turns) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = fmaf(x[e], c[e], z[e] * s[e]);
          }
          if constexpr (CODES) quant_store_row<D, E>(x, sub, dst, in_chunk, left > u * KPI && in_pool);
          else if (turns) w[u] = narrow<T>(x);
        } else if constexpr (CODES) {
          float x[E];
          widen<T>(w[u], x);
          quant_store_row<D, E>(x, sub, dst, in_chunk, left > u * KPI && in_pool);
        }
        if constexpr (!CODES)
          if (left > u * KPI && (KIND == 0 || in_pool)) *reinterpret_cast<uint4*>(dst) = w[u];
        dst += dst_next;
      }
      src += U * next;
      left -= U * KPI;
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = ahead[u];
    }
  };
  auto clip = [](int x, int n) { return x < 0 ? 0 : x < n ? x : n; };
  segment(std::integral_constant<int, 0>{}, p.q, p.Hq, clip(it0, nq), clip(it1, nq));
  segment(std::integral_constant<int, 1>{}, p.k, p.Hkv, clip(it0 - nq, nk), clip(it1 - nq, nk));
  segment(std::integral_constant<int, 2>{}, p.v, p.Hkv, clip(it0 - nq - nk, nk), clip(it1 - nq - nk, nk));
}

struct ReadParams {
  TokenBatch tb;
  RowsView k, v;               // outputs; data nullptr: not wanted
  const uint8_t *k_pages, *v_pages;
  const int32_t* table;
  int64_t n_pages, nc;
  int Hkv, shares, per_share;
};

// One warp per (eight packed tokens, share of the heads): four lanes per token
// read d / 8 bytes of codes each, which are eight neighbouring dims of every
// group, and store those as one piece per group.  HBM-bound: 5 d / 8 bytes in,
// d elements out per row; 128K tokens of 8 kv heads of 128 dims (705 MB): 124 us,
// 5.7 TB/s, 87 % of a copy's rate.  A CTA per token with two-byte loads: 221 us.
template <typename T, int D>
__global__ void __launch_bounds__(128) kv_read_quant_kernel(ReadParams p) {
  using P = QuantPage<D>;
  constexpr int NG = P::G, U = 2;
  const int lane = threadIdx.x & 31, tok = lane >> 2, part = lane & 3;
  if (blockIdx.x == 0) check_batch(p.tb, threadIdx.x, 128);
  const int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t t = item / p.shares * 8 + tok;
  if (item / p.shares * 8 >= p.tb.n_tokens) return;
  const int r0 = int(item % p.shares) * p.per_share;
  const int r1 = r0 + p.per_share < 2 * p.Hkv ? r0 + p.per_share : 2 * p.Hkv;
  Place at{-1, 0};
  if (t < p.tb.n_tokens) at = find_place(p.tb, t);
  if (at.b < 0) return;      // no shuffles below
  const int64_t page = __ldg(p.table + at.b * p.nc + at.pos / kChunk);
  if (page < 0 || page >= p.n_pages) {
    record_error(HILS_ERR_DEVICE_BOUNDS);
    return;
  }
  const int row = int(at.pos % kChunk);
  for (int i0 = r0; i0 < r1; i0 += U) {
    uint32_t code[U][NG], par[U][NG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = i0 + u;
      const bool key = r < p.Hkv;
      const uint8_t* pool = key ? p.k_pages : p.v_pages;
      if (r >= r1 || (key ? p.k.data : p.v.data) == nullptr) continue;
      const uint8_t* block = pool + (page * p.Hkv + (key ? r : r - p.Hkv)) * P::BLOCK;
      if constexpr (NG == 4) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(block + P::code_off(row) + 16 * part));
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(block + P::param_off(row)));
        code[u][0] = a.x; code[u][1] = a.y; code[u][2] = a.z; code[u][3] = a.w;
        par[u][0] = b.x; par[u][1] = b.y; par[u][2] = b.z; par[u][3] = b.w;
      } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(block + P::code_off(row) + 8 * part));
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(block + P::param_off(row)));
        code[u][0] = a.x; code[u][1] = a.y;
        par[u][0] = b.x; par[u][1] = b.y;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = i0 + u;
      const bool key = r < p.Hkv;
      const RowsView& dst = key ? p.k : p.v;
      if (r >= r1 || dst.data == nullptr) continue;
      T* out = static_cast<T*>(dst.data) + t * dst.ts + (key ? r : r - p.Hkv) * dst.hs + 8 * part;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        // words are units (2 part, g), (2 part, g + 1), .. , then those of 2 part + 1
        const uint32_t w = __byte_perm(code[u][g / 2], code[u][NG / 2 + g / 2], g & 1 ? 0x7632 : 0x5410);
        const __half2 sm = *reinterpret_cast<const __half2*>(&par[u][g]);
        const float s = __low2float(sm), m = __high2float(sm);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // bf16 128 + code: exact in fp32 after taking the offset off again
          const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
          x[i] = fmaf(s, __uint_as_float(v << 16) - 128.f, m);
          x[i + 4] = fmaf(s, __uint_as_float(v & 0xFFFF0000u) - 128.f, m);
        }
        if constexpr (sizeof(T) == 2) {
          Vec16<T>::store(out + 32 * g, x);
        } else {
          *reinterpret_cast<float4*>(out + 32 * g) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(out + 32 * g + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
    }
  }
}

}  // namespace hils
