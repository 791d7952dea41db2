// One decode step over a 4-bit chunk-paged cache, in three kernels:
//   Q1 scores : s^ of every candidate chunk (bf16: matrix instructions)
//   Q2 top-K  : the K best chunks of every query row, ids ascending
//   Q3 attend : the kept chunks' and the window's attention and their fusion
// The readings (scores, ties, window, fusion) are those of decode.cuh.
// Q2 and Q3 are launched with programmatic stream serialisation.
#pragma once
#include <cooperative_groups.h>

#include "decode.cuh"
#include "mma16.cuh"
#include "quant.cuh"

namespace hils {

// ---------------------------------------------------------------- Q1
// One warp scores 16 chunks against the query heads of a kv head, eight heads
// per matrix instruction (rows: chunks, columns: heads).  The order of the
// dims inside the sum is free, so each lane reads its operand rows in 16-byte
// pieces (row lane/4 and lane/4 + 8, piece 4 c + lane % 4) and the queries in
// the same order: no shared memory, all loads of the 16 rows in flight at
// once.  HBM-bound: (d + 16) x 2 bytes per (kv head, candidate); 8 x 128K with
// 8 kv heads (38 MB): 10.3 us alone and cold, where a thread per candidate with
// the rows staged in shared memory takes 15.8.
template <int D>
__global__ void __launch_bounds__(128)
quant_scores_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kmma,
                    const int32_t* __restrict__ seqlens, int64_t cap, int64_t nc, int Hq, int G, int Hkv, float tau,
                    float* __restrict__ ws_scores, int wm1) {
  constexpr int NV = D / 32, RS = D + kExt;
  pdl_trigger();
  const int bh = blockIdx.y, b = bh / Hkv, h = bh % Hkv;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int64_t own = decode_own_chunk(seqlens, b, cap);
  if (own < 0) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_error(HILS_ERR_DEVICE_BOUNDS);
    return;
  }
  const int64_t n_cand = own - wm1, c0 = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5)) * 16;
  if (c0 >= n_cand) return;
  const int64_t last = n_cand - 1;
  const int64_t ca = c0 + gid < last ? c0 + gid : last, cb = c0 + gid + 8 < last ? c0 + gid + 8 : last;
  const __nv_bfloat16 *ra = kmma + (int64_t(bh) * nc + ca) * RS, *rb = kmma + (int64_t(bh) * nc + cb) * RS;
  uint4 xa[NV], xb[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    xa[i] = __ldg(reinterpret_cast<const uint4*>(ra + 32 * i + 8 * tig));
    xb[i] = __ldg(reinterpret_cast<const uint4*>(rb + 32 * i + 8 * tig));
  }
  // b'/tau as the sum of two bf16 values
  const uint32_t ea = __ldg(reinterpret_cast<const uint32_t*>(ra + D)), eb = __ldg(reinterpret_cast<const uint32_t*>(rb + D));
  const float ba = lo_bf16(ea) + hi_bf16(ea), bb = lo_bf16(eb) + hi_bf16(eb);
  for (int g0 = 0; g0 < G; g0 += 8) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const bool have = g0 + gid < G;
    const __nv_bfloat16* qr = q + (int64_t(b) * Hq + h * G + g0 + gid) * D + 8 * tig;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint4 y = have ? __ldg(reinterpret_cast<const uint4*>(qr + 32 * i)) : make_uint4(0, 0, 0, 0);
      mma16816_bf16(acc, xa[i].x, xb[i].x, xa[i].y, xb[i].y, y.x, y.y);
      mma16816_bf16(acc, xa[i].z, xb[i].z, xa[i].w, xb[i].w, y.z, y.w);
    }
    const int g = g0 + 2 * tig;
    float* out = ws_scores + (int64_t(b) * Hq + h * G + g) * nc;
    if (c0 + gid < n_cand) {
      if (g < G) out[c0 + gid] = tau * (acc[0] + ba);
      if (g + 1 < G) out[nc + c0 + gid] = tau * (acc[1] + ba);
    }
    if (c0 + gid + 8 < n_cand) {
      if (g < G) out[c0 + gid + 8] = tau * (acc[2] + bb);
      if (g + 1 < G) out[nc + c0 + gid + 8] = tau * (acc[3] + bb);
    }
  }
}

// ---------------------------------------------------------------- Q2
// Exclusive prefix sum over the NT threads of a block; also the total.
template <int NT>
__device__ __forceinline__ int block_exclusive_scan(int x, int* warp_tot, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  // the warps' totals, summed by every warp
  const int t = lane < NT / 32 ? warp_tot[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, t);
  return __reduce_add_sync(0xffffffffu, lane < warp ? t : 0) + incl - x;
}

// A kept (head, slot) pair: chunk id (-1: none), page (-1: outside the pool),
// score.
struct __align__(16) Kept {
  int32_t id, page;
  float score;
  int32_t pad;
};

// A score's place in the order; a NaN of either sign comes first, so that the
// output of its row shows it.
__device__ __forceinline__ uint32_t score_key(float s) { return s != s ? 0xFFFFFFFFu : order_key(s); }
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ uint32_t middle_key(uint32_t lo, uint32_t hi, int step) {
  const uint32_t d = hi - lo, mid = lo + (d >> 1) + (d & 1);
  if (step >= 16) return mid;
  const uint32_t k = order_key(0.5f * key_value(lo) + 0.5f * key_value(hi));
  return k > lo && k <= hi ? k : mid;
}
// The largest key t of this warp's v[] (one value per lane and register, 0: no
// value) with at least K of them >= t, or any t with exactly K; 1 if there are
// fewer than K.  Bisection: first of the scores' interval (nine tenths of the
// keys' is exponents of scores near zero), then of the keys'.
template <int R>
__device__ __forceinline__ uint32_t warp_kth_key(const uint32_t (&v)[R], int K) {
  uint32_t lo = 0xFFFFFFFFu, hi = 0u, some = 0;
#pragma unroll
  for (int e = 0; e < R; ++e) {
    if (v[e]) lo = min(lo, v[e]);
    hi = max(hi, v[e]);
    some += v[e] != 0;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (int(__reduce_add_sync(0xffffffffu, some)) < K) return 1u;
  for (int step = 0; lo < hi; ++step) {
    const uint32_t mid = middle_key(lo, hi, step);
    uint32_t x = 0;
#pragma unroll
    for (int e = 0; e < R; ++e) x += v[e] >= mid;
    const int c = int(__reduce_add_sync(0xffffffffu, x));
    if (c >= K) lo = mid; else hi = mid - 1;
    if (c == K) break;
  }
  return lo;
}

// The K largest scores of a row, ties to the lower ids.  Each of the NT threads
// holds a segment of IT keys (IT = 0: re-reads it from L2).  The K-th largest
// maximum of 256 groups bounds the row's K-th score from below, and one warp
// finds it without barriers; the few keys at or above it (about K) are
// gathered and ranked against one another.  Where more than NT reach the
// bound (tied scores), the K-th key of the whole row is found by bisection
// with a block-wide count per step.  A radix select sends all of a row's scores,
// which share their high bits, through atomics on a few shared counters: 11 us
// for 256 rows of 2048 against 6.5; the block-wide bisection alone took 8.4.
// A kept chunk's page is looked up here, by the thread that keeps it.
template <int IT, int NT>
__global__ void __launch_bounds__(NT)
quant_topk_kernel(Late<float> ws_scores, const int32_t* __restrict__ seqlens, int64_t cap, int64_t nc,
                  int Hq, int K, const int32_t* __restrict__ table, int64_t n_pages, Kept* __restrict__ kept,
                  int32_t* __restrict__ ids_out, float* __restrict__ scores_out, int wm1) {
  constexpr int NW = NT / 32;
  __shared__ uint32_t s_part[2][32], s_max[256], s_bound;
  __shared__ uint2 s_found[NT];      // (key, id) at or above the bound
  __shared__ uint32_t s_taken[32];
  __shared__ int warp_tot[32], s_n;
  pdl_wait();      // the scores
  pdl_trigger();
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = row / Hq, own = decode_own_chunk(seqlens, int(b), cap);
  int64_t n = own < 0 ? 0 : own - wm1;   // candidates
  if (n < 0) n = 0;
  const Late<float> sc = ws_scores + int64_t(row) * nc;
  const int64_t at = int64_t(row) * K;
  auto put = [&](int slot, int32_t id, float s) {
    if (ids_out) ids_out[at + slot] = id;
    if (scores_out) scores_out[at + slot] = s;
    int32_t page = -1;
    if (id >= 0) {
      page = __ldg(table + b * nc + id);
      if (page < 0 || page >= n_pages) {
        record_error(HILS_ERR_DEVICE_BOUNDS);
        page = -1;
      }
    }
    kept[at + slot] = Kept{id, page, s, 0};
  };
  if (n <= K) {
    for (int t = tid; t < K; t += NT) put(t, t < n ? t : -1, t < n ? sc[t] : -INFINITY);
    return;
  }
  const int64_t seg = IT > 0 ? ((n + NT - 1) / NT + 3) / 4 * 4 : (n + NT - 1) / NT;
  const int64_t s0 = tid * seg;
  const int64_t cnt = s0 >= n ? 0 : (s0 + seg <= n ? seg : n - s0);
  constexpr int R = IT > 0 ? IT : 1;
  uint32_t key[R];
  if constexpr (IT > 0) {
    const bool vec = (nc & 3) == 0;      // every row of scores starts on a 16-byte boundary
#pragma unroll
    for (int e = 0; e < IT; e += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (vec && e + 4 <= cnt) {
        v = sc.wide<float4>(s0 + e);
      } else {
        if (e < cnt) v.x = sc[s0 + e];
        if (e + 1 < cnt) v.y = sc[s0 + e + 1];
        if (e + 2 < cnt) v.z = sc[s0 + e + 2];
        if (e + 3 < cnt) v.w = sc[s0 + e + 3];
      }
      // key 0, which no score has, marks the places behind the end
      key[e] = e < cnt ? score_key(v.x) : 0u;
      key[e + 1] = e + 1 < cnt ? score_key(v.y) : 0u;
      key[e + 2] = e + 2 < cnt ? score_key(v.z) : 0u;
      key[e + 3] = e + 3 < cnt ? score_key(v.w) : 0u;
    }
  }
  auto key_at = [&](int64_t e) { return score_key(sc[s0 + e]); };
  auto for_keys = [&](auto f) {   // over this thread's keys (and, with IT > 0, zeros behind them)
    if constexpr (IT > 0) {
#pragma unroll
      for (int e = 0; e < IT; ++e) f(e, key[e]);
    } else {
      for (int64_t e = 0; e < cnt; ++e) f(int(e), key_at(e));
    }
  };
  uint32_t top = 0;
  for_keys([&](int, uint32_t k) { top = max(top, k); });
  // maxima of 256 groups: of a thread, or of four neighbours
  uint32_t group = top;
#pragma unroll
  for (int o = 1; o < NT / 256; o <<= 1) group = max(group, __shfl_xor_sync(0xffffffffu, group, o));
  if (tid % (NT / 256) == 0) s_max[tid / (NT / 256)] = group;
  if (tid == 0) s_n = 0;
  __syncthreads();
  if (warp == 0) {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s_max[lane + 32 * e];
    const uint32_t k = warp_kth_key(v, K);
    if (lane == 0) s_bound = k;
  }
  __syncthreads();
  const uint32_t bound = s_bound;
  if (top >= bound) {
    int mine = 0;
    for_keys([&](int, uint32_t k) { mine += k >= bound; });
    int to = atomicAdd(&s_n, mine);
    for_keys([&](int e, uint32_t k) {
      if (k >= bound && to < NT) s_found[to++] = make_uint2(k, uint32_t(s0 + e));
    });
  }
  __syncthreads();
  const int m = s_n;
  if (m <= NT) {
    // rank by (key, lower id first); then, of those kept, by id
    uint2 mine = make_uint2(0u, 0u);
    int rank = K;
    if (tid < m) {
      mine = s_found[tid];
      rank = 0;
#pragma unroll 4
      for (int j = 0; j < m; ++j) {
        const uint2 x = s_found[j];
        rank += x.x > mine.x || (x.x == mine.x && x.y < mine.y);
      }
    }
    const uint32_t kept_bits = __ballot_sync(0xffffffffu, rank < K);
    if (lane == 0) s_taken[warp] = kept_bits;
    __syncthreads();
    if (rank < K) {
      int pos = 0;
#pragma unroll 4
      for (int j = 0; j < m; ++j) pos += ((s_taken[j >> 5] >> (j & 31)) & 1u) && s_found[j].y < mine.y;
      put(pos, int32_t(mine.y), key_value(mine.x));
    }
    return;
  }
  uint32_t lo = bound, hi = 0u;
  {
    uint32_t v = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) v = max(v, s_max[lane + 32 * e]);
    hi = __reduce_max_sync(0xffffffffu, v);
  }
  int flip = 0;
  auto count = [&](uint32_t t) {   // keys >= t of the whole row
    uint32_t x = 0;
    for_keys([&](int, uint32_t k) { x += k >= t; });
    x = __reduce_add_sync(0xffffffffu, x);
    if (lane == 0) s_part[flip][warp] = x;
    __syncthreads();
    x = lane < NW ? s_part[flip][lane] : 0u;
    flip ^= 1;
    return int(__reduce_add_sync(0xffffffffu, x));
  };
  // the largest t with at least K keys >= t, or any t with exactly K
  bool exact = false;
  for (int step = 0; lo < hi; ++step) {
    const uint32_t mid = middle_key(lo, hi, step);
    const int c = count(mid);
    if (c >= K) lo = mid; else hi = mid - 1;
    if (c == K) { exact = true; break; }
  }
  const int ties = exact || lo == 0xFFFFFFFFu ? K : K - count(lo + 1);   // how many keys equal to lo are kept
  // each thread's keys above lo, and equal to it, in chunk order
  int gt = 0, eq = 0;
  for_keys([&](int, uint32_t k) { gt += k > lo; eq += k == lo; });
  int tot;
  int take_eq = eq;
  if (!exact) {
    take_eq = ties - block_exclusive_scan<NT>(eq, warp_tot, tot);
    take_eq = take_eq < 0 ? 0 : (take_eq > eq ? eq : take_eq);
  }
  int pos = block_exclusive_scan<NT>(gt + take_eq, warp_tot, tot);
  for_keys([&](int e, uint32_t k) {
    bool take = k > lo;
    if (k == lo) take = take_eq-- > 0;
    if (take && pos < K) put(pos++, int32_t(s0 + e), key_value(k));
  });
}

// ---------------------------------------------------------------- Q3
// A cluster of CTAs serves the (up to eight) query heads `oct` of one kv head:
// its warps share out the distinct chunks that any of these heads kept, and the
// window's chunks.  A warp stages a chunk's two 4-bit blocks in its own shared
// memory (copies of the next chunk's keys start as soon as the current ones
// are consumed, its values likewise) and attends it for all heads that kept
// it at once:
//   logits (keys x heads): the codes, masked out in place as fp16 subnormals
//     code 2^-24 or code 2^-20 (codes_f16: one and per two codes), times the
//     queries on the tensor cores, exactly, summed in fp32 per group of 32 dims:
//     acc_jg = sum_{i in g} q_i code_ji; then
//     z = tau sum_g [ s_jg acc_jg + m_jg sum_{i in g} q_i ].
//   output (dims x heads): the codes in the same form times W_j s_jg, and m_jg
//     times W_j, one instruction for all groups; w_j = e^(z_j - lse) e^(u - M)
//     carries the fusion weight, and W_j = 2^k w_j in fp16, with k such that the
//     products with the largest step met so far lie below 2^15, and k <= 15, as
//     w_j <= 1 (without it, weights of about 1/64 and steps below 4e-3 leave
//     fp16's normal range, and values of 1e-4 were off by tens of percent).
//     W_j and W_j s_jg are rounded to fp16, by 2^-11 of them each: together a
//     quarter of a bf16 output's half step of 2^-8 for one key, and less for a
//     sum over keys.
// fp32 models: queries, and the weights times s and m, as sums of three bf16
// values (24 bits), so that the products are fp32's.
// Running maximum, sum and outputs stay in registers over a warp's chunks;
// warps merge in shared memory, CTAs through distributed shared memory.
// Bound by latency: three warps per scheduler wait for chains of their own
// (about 1430 instructions per chunk with their fixed latencies and shared
// memory, then the next chunk's copies), and at the end for the warps that have
// one chunk more; the first chunks of all warps arrive together (3.8 us).  37 %
// of issue slots are busy with 64 chunks per kv head, 48 % with 190.  8
// sequences of 128K, 64 chunks per kv head: 19 us of the step's 37.4 (its 41 MB
// would take 6.3).  Two CTAs of six warps per SM, for 168 registers a thread:
// of eight (128 registers, spills) 43 us for the step, seven 39.6, five 40.3,
// four 38.8, three of four 39.3, one of eight 41.5.  Also measured, for the step
// at the time: a warp per (head, slot) on CUDA cores 118 us; four warps per
// chunk instead of one 55 against 45 (each repeats the softmax and the fusion:
// 2900 instructions per chunk); codes widened to bf16 16 + code 47; slots in
// place of the list of distinct chunks 63 against 47.
constexpr int kQdWarps = 6;

// The power of two (its bits) that puts the largest step, given by its bits, in
// [2^14, 2^15), but 2^15 at most: steps from 2^-1 to fp16's largest, of
// exponent 15, have one of their own.
constexpr uint32_t kWeightMost = uint32_t(127 + 15) << 23;
__device__ __forceinline__ uint32_t weight_scale(uint32_t top) {
  uint32_t e = top >> 23;
  e = e < 126 ? 126 : e > 142 ? 142 : e;
  return (268 - e) << 23;      // 2^(141 - e)
}

template <int D> struct QuantAttend {
  static constexpr int BLOCK = int(QuantPage<D>::BLOCK);
  static constexpr int RS = D + 4;                            // floats per merged row: 16-byte stores of four rows apart
  static constexpr int MERGE = 8 * RS * 4 + 8 * 2 * 4;        // per warp: 8 rows, then (maximum, sum) of 8 heads
  static constexpr int STAGE = 2 * BLOCK > MERGE ? 2 * BLOCK : (MERGE + 15) / 16 * 16;
  // a CTA's sums of one head: D values, maximum, sum.  A CTA that finishes some
  // of eight heads in a cluster of CL keeps ceil(8 / CL) rows of CL, 14 at most
  // (CL = 7)
  static constexpr int PART = D + 4, INBOX = 14 * PART;
  static constexpr int LISTS = 8 * kMaxTopK;                  // kept (head, slot) pairs of a cluster, at most
  static constexpr int ITEMS = LISTS + 16;                    // distinct chunks and window chunks
  // staging, the CTAs' sums of the heads this one finishes, scores of the pairs,
  // places of a pair's chunk in the heads' lists, ids of the pairs, then the
  // items' page and pair
  static constexpr int SMEM = kQdWarps * STAGE + INBOX * 4 + LISTS * (4 + 8 + 4) + ITEMS * 8;
};

template <typename T, int D>
__global__ void __launch_bounds__(kQdWarps * 32, 2)
quant_attend_kernel(const T* __restrict__ q, const uint8_t* __restrict__ kpg, const uint8_t* __restrict__ vpg,
                    const int32_t* __restrict__ table, int64_t n_pages, const int32_t* __restrict__ seqlens,
                    int64_t cap, int Hq, int G, int Hkv, int K, float tau, Late<Kept> kept,
                    T* __restrict__ o, int n_oct, int wm1) {
  using A = QuantAttend<D>;
  using P = QuantPage<D>;
  constexpr int NG = P::G, NS = sizeof(T) == 2 ? 1 : 3;
  constexpr float kLog2e = 1.4426950408889634f;
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t qsm[];
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");      // waited for before the CTAs' sums are exchanged
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, tig = lane & 3;
  const uint32_t CL = gridDim.x, rank = blockIdx.x;     // the cluster is the grid's row
  const int oct = blockIdx.y % n_oct, bh = blockIdx.y / n_oct, b = bh / Hkv, h = bh % Hkv;
  const int g0 = oct * 8, GV = G - g0 < 8 ? G - g0 : 8;
  const int64_t row0 = int64_t(b) * Hq + int64_t(h) * G + g0;
  uint8_t* stage = qsm + warp * A::STAGE;
  float* inbox = reinterpret_cast<float*>(qsm + kQdWarps * A::STAGE);
  float* scs = reinterpret_cast<float*>(qsm + kQdWarps * A::STAGE + A::INBOX * 4);     // [GV][K], x log2 e
  uint8_t* spot = reinterpret_cast<uint8_t*>(scs + A::LISTS);                       // [pair][8 heads]: slot, 0xFF: not kept
  uint32_t* ids = reinterpret_cast<uint32_t*>(spot + A::LISTS * 8);                 // [GV][K]
  int2* items = reinterpret_cast<int2*>(ids + A::LISTS);                            // (page, pair; -1 - w: window chunk w)
  __shared__ int s_count[kQdWarps + 1];
  const uint32_t stage_a = uint32_t(__cvta_generic_to_shared(stage));

  // queries as the column operand: head gid, dims 32 g + 8 tig + {i, i + 4} in
  // register i of group g, the order in which two 16-bit units of codes unpack.
  // NS == 1: in fp16, exact: a head's queries are scaled by a power of two that
  // puts the largest in [2^14, 2^15) (one 2^-24 of it is lost in the rounding),
  // and those of odd i by another 2^-4, because their codes stand 2^4 higher
  uint32_t qb[NS][NG][4], qs2[2] = {0u, 0u};
  float qsum[NG][2];       // NS == 3: sum of the group's q, heads 2 tig, 2 tig + 1
  float zscale[2];         // from a logit's sums to the logit x log2 e, heads 2 tig, 2 tig + 1
  {
    const T* qr = q + (row0 + (gid < GV ? gid : 0)) * D + 8 * tig;
    float x[NG][8], top = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if constexpr (NS == 1) {
        Vec16<T>::load(qr + 32 * g, x[g]);
      } else {
        float y[4], z[4];
        Vec16<T>::load(qr + 32 * g, y);
        Vec16<T>::load(qr + 32 * g + 4, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[g][e] = y[e]; x[g][e + 4] = z[e]; }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (gid >= GV) x[g][e] = 0.f;
        top = fmaxf(top, fabsf(x[g][e]));
      }
    }
    float up = 1.f, down = 1.f;
    if constexpr (NS == 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      power_scale(top, up, down);
    }
    zscale[0] = tau * kLog2e * __shfl_sync(0xffffffffu, down, 8 * tig);
    zscale[1] = tau * kLog2e * __shfl_sync(0xffffffffu, down, 8 * tig + 4);
    if constexpr (NS == 1) {     // codes were multiplied as code 2^-24
      zscale[0] *= 16777216.f;
      zscale[1] *= 16777216.f;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[g][e] *= up;
        s += x[g][e];
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if constexpr (NS == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = i & 1 ? 0.0625f : 1.f;
          qb[0][g][i] = pack_f16(x[g][i] * f, x[g][i + 4] * f);
        }
        // the groups' sums x 2^-8, rows 2 tig, 2 tig + 1 in fp16, rows + 8 what that rounds off
        if (g / 2 == tig) {
          const float v = s * (1.f / 256.f), r = v - __half2float(__float2half_rn(v));
          qs2[0] |= pack_f16(v, 0.f) << (16 * (g % 2));
          qs2[1] |= pack_f16(r, 0.f) << (16 * (g % 2));
        }
      } else {
        qsum[g][0] = __shfl_sync(0xffffffffu, s, 8 * tig);
        qsum[g][1] = __shfl_sync(0xffffffffu, s, 8 * tig + 4);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t r = pack_bf16(x[g][i], x[g][i + 4]);
            qb[n][g][i] = r;
            x[g][i] -= lo_bf16(r);
            x[g][i + 4] -= hi_bf16(r);
          }
      }
    }
  }
  const int64_t own = decode_own_chunk(seqlens, b, cap), nc = cap / kChunk;
  const int n_own = own < 0 ? 0 : int(__ldg(seqlens + b) - own * kChunk);   // keys of the own chunk
  const int64_t n_cand = own - wm1 > 0 ? own - wm1 : 0;
  const int n_sel = own < 0 ? 0 : GV * K;
  const int n_win = own < 0 ? 0 : int(own < wm1 ? own + 1 : wm1 + 1);
  constexpr int TH = kQdWarps * 32, PER = (A::LISTS + TH - 1) / TH;      // kept pairs per thread, at most
  // the window's pages do not depend on the selection
  int win_page = -1;
  if (tid < n_win) {
    win_page = __ldg(table + b * nc + own - tid);
    if (win_page < 0 || win_page >= n_pages) {
      record_error(HILS_ERR_DEVICE_BOUNDS);
      win_page = -1;
    }
  }
  pdl_wait();      // the top-K lists
  int4 mine[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int pair = tid + e * TH;
    mine[e] = make_int4(-1, -1, 0, 0);
    if (pair < n_sel) {
      const Kept k = kept[row0 * K + pair];
      mine[e] = make_int4(k.id, k.page, __float_as_int(k.score), 0);
      ids[pair] = uint32_t(mine[e].x);
      scs[pair] = __int_as_float(mine[e].z) * kLog2e;
    }
  }
  __syncthreads();
  // Who else kept the chunk of each (head, slot) pair: a thread per pair, a
  // binary search in every head's ascending list (as unsigned numbers the -1
  // behind the ids is the largest), four heads' searches interleaved.  The first
  // head that kept a chunk owns it: its pair becomes an item.  The window's
  // chunks are the first items.
  int n_items = 0;
  if (n_win > 0) {
    if (warp == 0) {
      const uint32_t have = __ballot_sync(0xffffffffu, win_page >= 0);
      if (win_page >= 0) items[__popc(have & ((1u << lane) - 1u))] = make_int2(win_page, -1 - tid);
      if (lane == 0) s_count[kQdWarps] = __popc(have);
    }
  } else if (tid == 0) {
    s_count[kQdWarps] = 0;
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    if (e * TH >= n_sel && e > 0) break;      // the same for the whole CTA
    const int pair = tid + e * TH;
    const uint32_t c = uint32_t(mine[e].x);
    bool owner = false;
    if (pair < n_sel && mine[e].x >= 0) {
      const int g_own = pair / K;
      uint32_t place[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      owner = int64_t(mine[e].x) < n_cand;
      if (!owner) record_error(HILS_ERR_DEVICE_BOUNDS);
#pragma unroll 1
      for (int f = 0; f < GV; f += 4) {
        const uint32_t* list[4];       // a head behind the last: the last's again
        int at[4] = {0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < 4; ++g) list[g] = ids + (f + g < GV ? f + g : GV - 1) * K;
        // no branches: four loads in flight per step
#pragma unroll 1
        for (int st = 1 << (31 - __clz(K)); st > 0; st >>= 1)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int to = at[g] + st;
            const uint32_t v = list[g][(to < K ? to : K) - 1];
            at[g] = (to <= K) & (v < c) ? to : at[g];
          }
        uint32_t four = 0xFFFFFFFFu;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const bool has = (f + g < GV) & (at[g] < K) & (list[g][at[g] < K ? at[g] : K - 1] == c);
          four ^= has ? uint32_t(0xFF ^ at[g]) << (8 * g) : 0u;
          owner = owner & !(has & (f + g < g_own));
        }
        if (f == 0) place[0] = four; else place[1] = four;
      }
      if (owner) *reinterpret_cast<uint2*>(spot + pair * 8) = make_uint2(place[0], place[1]);
    }
    const bool item = owner && mine[e].y >= 0;
    const uint32_t have = __ballot_sync(0xffffffffu, item);
    if (lane == 0) s_count[warp] = __popc(have);
    __syncthreads();
    if (e == 0) n_items = s_count[kQdWarps];
    int to = n_items + __popc(have & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kQdWarps; ++w) {
      if (w < warp) to += s_count[w];
      n_items += s_count[w];
    }
    if (item) items[to] = make_int2(mine[e].y, pair);
    __syncthreads();
  }

  // item i as this warp attends it
  struct Work {
    uint32_t heads;    // who attends the chunk
    float u[2];        // their fusion scores x log2 e (heads 2 tig, 2 tig + 1; selected chunks)
    int64_t block;
    int keys;
    bool window;
  };
  const int step = int(CL) * kQdWarps;
  auto find = [&](int i) {
    Work w{0u, {0.f, 0.f}, -1, kChunk, false};
    if (i >= n_items) return w;
    const int2 it = items[i];
    w.block = (int64_t(it.x) * Hkv + h) * P::BLOCK;
    float mine = 0.f;
    if (it.y < 0) {
      w.window = true;
      w.keys = it.y == -1 ? n_own : kChunk;
      w.heads = (1u << GV) - 1u;
    } else {
      const int at = spot[it.y * 8 + (lane & 7)];
      w.heads = __ballot_sync(0xffffffffu, at != 0xFF) & 0xFFu;
      if (at != 0xFF) mine = scs[(lane & 7) * K + at];
    }
    w.u[0] = __shfl_sync(0xffffffffu, mine, 2 * tig);
    w.u[1] = __shfl_sync(0xffffffffu, mine, 2 * tig + 1);
    return w;
  };
  // the staged rows of 64 bytes of codes have the 16-byte pieces of rows 2, 3
  // (mod 4) swapped in halves: with the order of keys below, the 8-byte reads
  // of four rows then fall in different banks
  auto copy = [&](const uint8_t* src, uint32_t dst) {
#pragma unroll
    for (int i = 0; i < A::BLOCK / 512; ++i) {
      const int at = lane + 32 * i;
      const int to = D == 128 && i < kChunk * P::ROW / 512 ? at ^ ((at >> 2) & 2) : at;
      cp_async16(dst + uint32_t(to) * 16u, src + at * 16);
    }
  };
  // keys as rows of the products: row r of eight is key r / 2 (r even) or
  // 4 + (r / 2 ^ 1) (r odd), so that the rows 2 tig + j of the four tig, and the
  // rows 2 i, 2 i + 1, lie in different banks
  const int key_row = gid & 1 ? 4 + ((gid >> 1) ^ 1) : gid >> 1;      // of row gid
  const int key_even = tig, key_odd = 4 + (tig ^ 1);                  // of rows 2 tig, 2 tig + 1
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  auto wait_all_but_one = [] { asm volatile("cp.async.wait_group 1;" ::: "memory"); };

  float acc[NG][2][4], least[2] = {0.f, 0.f}, M[2] = {-INFINITY, -INFINITY}, Z[2] = {0.f, 0.f};
  uint32_t w_up = kWeightMost;      // NS == 1: 2^k, by which weights and sums are scaled
#pragma unroll
  for (int i = 0; i < NG * 8; ++i) acc[i / 8][i / 4 % 2][i % 4] = 0.f;

  int item = int(rank) + warp * int(CL);
  Work cur = find(item);
  if (cur.block >= 0) copy(kpg + cur.block, stage_a);
  commit();
  if (cur.block >= 0) copy(vpg + cur.block, stage_a + A::BLOCK);
  commit();
  while (cur.block >= 0) {
    item += step;
    const Work nxt = find(item);
    wait_all_but_one();
    __syncwarp();
    // ---- logits: tile t of 16 keys, rows gid and gid + 8, columns heads 2 tig, 2 tig + 1
    float z[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t cu[2][NG];      // the lane's code words of the two rows: units of 2 tig, then of 2 tig + 1
      float ps[2][NG], pm[2][NG];
      uint32_t la[2];          // NS == 1: least values of groups 2 tig, 2 tig + 1
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = 16 * t + 8 * r + key_row;
        const uint8_t* par = stage + P::param_off(key);
        if constexpr (NG == 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(stage + P::code_off(key) + 16 * (tig ^ (key & 2)));
          cu[r][0] = u.x; cu[r][1] = u.y; cu[r][2] = u.z; cu[r][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(stage + P::code_off(key) + 8 * tig);
          cu[r][0] = u.x; cu[r][1] = u.y;
        }
        if constexpr (NS == 1) {
          const uint2 m = *reinterpret_cast<const uint2*>(par + 8 * (tig % (NG / 2)));
          la[r] = tig < NG / 2 ? __byte_perm(m.x, m.y, 0x7632) : 0u;
        }
        uint32_t pw[NG];
        if constexpr (NG == 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(par);
          pw[0] = u.x; pw[1] = u.y; pw[2] = u.z; pw[3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(par);
          pw[0] = u.x; pw[1] = u.y;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&pw[g]));
          ps[r][g] = sm.x;
          pm[r][g] = sm.y;
        }
      }
      // sum_g m_g sum_{i in g} q_i: fp32 models below, else one instruction,
      // the sums of q split into two fp16 (22 bits)
      if constexpr (NS == 1) mma16816_f16_first(z[t], la[0], la[1], la[0], la[1], qs2[0], qs2[1]);
      else z[t][0] = z[t][1] = z[t][2] = z[t][3] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float c[4];
        uint32_t a[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (NS == 1) codes_f16(cu[r][g / 2], cu[r][NG / 2 + g / 2], g & 1, a[r]);
          else codes_bf16_centred(__byte_perm(cu[r][g / 2], cu[r][NG / 2 + g / 2], g & 1 ? 0x7632 : 0x5410), a[r]);
        }
        if constexpr (NS == 1) {
          mma16816_f16_first(c, a[0][0], a[1][0], a[0][1], a[1][1], qb[0][g][0], qb[0][g][1]);
          mma16816_f16(c, a[0][2], a[1][2], a[0][3], a[1][3], qb[0][g][2], qb[0][g][3]);
        } else {
#pragma unroll
          for (int n = NS - 1; n >= 0; --n) {
            if (n == NS - 1) mma16816_bf16_first(c, a[0][0], a[1][0], a[0][1], a[1][1], qb[n][g][0], qb[n][g][1]);
            else mma16816_bf16(c, a[0][0], a[1][0], a[0][1], a[1][1], qb[n][g][0], qb[n][g][1]);
            mma16816_bf16(c, a[0][2], a[1][2], a[0][3], a[1][3], qb[n][g][2], qb[n][g][3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (NS == 1)     // the least values' sum in the codes' units: 2^8 / 2^24
            z[t][i] = g == 0 ? fmaf(z[t][i], 1.f / 65536.f, ps[i / 2][g] * c[i]) : fmaf(ps[i / 2][g], c[i], z[t][i]);
          else
            z[t][i] = fmaf(ps[i / 2][g], c[i], fmaf(fmaf(8.f, ps[i / 2][g], pm[i / 2][g]), qsum[g][i % 2], z[t][i]));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) z[t][i] *= zscale[i & 1];
    }
    if (cur.keys < kChunk) {       // the own chunk: keys behind the query
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * t + 8 * (i / 2) + key_row >= cur.keys) z[t][i] = -INFINITY;
    }
    __syncwarp();
    if (nxt.block >= 0) copy(kpg + nxt.block, stage_a);
    commit();
    // ---- the chunk's softmax and its place in the fusion
    float coef[2], alpha[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) m = fmaxf(m, fmaxf(z[t][e], z[t][2 + e]));
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        z[t][e] = pow2<NS == 1>(z[t][e] - m);
        z[t][2 + e] = pow2<NS == 1>(z[t][2 + e] - m);
        l += z[t][e] + z[t][2 + e];
      }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
      const bool kept = (cur.heads >> (2 * tig + e)) & 1u;
      const float u = cur.window ? m + log2f(l) : cur.u[e];
      const float mn = !kept ? M[e] : u != u ? u : fmaxf(M[e], u);      // a NaN score is not dropped
      alpha[e] = mn == -INFINITY ? 1.f : exp2f(M[e] - mn);
      const float beta = kept && mn != -INFINITY ? exp2f(u - mn) : 0.f;
      Z[e] = fmaf(Z[e], alpha[e], beta);
      coef[e] = kept ? beta / l : 0.f;
      M[e] = mn;
    }
    wait_all_but_one();
    __syncwarp();
    // ---- output
    const uint8_t* vst = stage + A::BLOCK;
    if (cur.keys < kChunk) {      // the own chunk: parameters behind the sequence may be anything, their weights are 0
      for (int key = cur.keys + lane; key < kChunk; key += 32)
#pragma unroll
        for (int g = 0; g < NG; ++g) *reinterpret_cast<uint32_t*>(stage + A::BLOCK + P::param_off(key) + 4 * g) = 0u;
      __syncwarp();
    }
    if constexpr (NS == 1) {
      // the largest step; a NaN is not the maximum of anything
      const uint4* par = reinterpret_cast<const uint4*>(vst + P::param_off(0));
      __half2 top = __floats2half2_rn(0.f, 0.f);       // in the lower half
#pragma unroll
      for (int i = 0; i < kChunk * P::PROW / 512; ++i) {
        const uint4 u = par[lane + 32 * i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __hmax2(top, *reinterpret_cast<const __half2*>(&w[e]));
      }
      const uint32_t up = weight_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(__low2float(top))));
      if (up < w_up) {      // powers of two: their bits compare as they do, and differ by the bits of the quotient's exponent
        const float f = __uint_as_float(0x3F800000u - (w_up - up));
        alpha[0] *= f;
        alpha[1] *= f;
        w_up = up;
      }
      coef[0] *= __uint_as_float(w_up);
      coef[1] *= __uint_as_float(w_up);
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[g][i / 4][i % 4] *= alpha[i & 1];
      least[0] *= alpha[0];
      least[1] *= alpha[1];
    }
    float lm[4] = {0.f, 0.f, 0.f, 0.f};      // the chunk's least values, one row per group
    const uint32_t kept_mask = (cur.heads >> gid) & 1u ? 0xFFFFFFFFu : 0u;   // of the column this lane feeds
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // the weights with heads as columns: keys of rows 2 tig, 2 tig + 1 and + 8, head gid
      uint32_t wb[2];        // fp16 pairs
      float wf[2][2];        // or fp32
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float w0 = z[t][2 * r] * coef[0], w1 = z[t][2 * r + 1] * coef[1];
        if constexpr (NS == 1) {
          wb[r] = movmatrix(pack_f16(w0, w1));
        } else {
          const uint32_t lo = movmatrix(__byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x5410)) & kept_mask;
          const uint32_t hi = movmatrix(__byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x7632)) & kept_mask;
          wf[r][0] = __uint_as_float(__byte_perm(lo, hi, 0x5410));
          wf[r][1] = __uint_as_float(__byte_perm(lo, hi, 0x7632));
        }
      }
      uint32_t vc[2][2][NG / 2], vp[2][2][NG];    // codes and parameters of the key of row 8 r + 2 tig + j
      uint32_t vl[2][2];                          // parameters of group gid
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = 16 * t + 8 * r + (j ? key_odd : key_even);
          if constexpr (NG == 4) {
            const uint2 u = *reinterpret_cast<const uint2*>(vst + P::code_off(key) + 8 * (gid ^ (2 * (key & 2))));
            vc[r][j][0] = u.x;
            vc[r][j][1] = u.y;
            const uint4 p = *reinterpret_cast<const uint4*>(vst + P::param_off(key));
            vp[r][j][0] = p.x;
            vp[r][j][1] = p.y;
            vp[r][j][2] = p.z;
            vp[r][j][3] = p.w;
          } else {
            vc[r][j][0] = *reinterpret_cast<const uint32_t*>(vst + P::code_off(key) + 4 * gid);
            const uint2 p = *reinterpret_cast<const uint2*>(vst + P::param_off(key));
            vp[r][j][0] = p.x;
            vp[r][j][1] = p.y;
          }
          if constexpr (NS == 1) vl[r][j] = gid < NG ? *reinterpret_cast<const uint32_t*>(vst + P::param_off(key) + 4 * gid) : 0u;
        }
      // least values of group gid as the rows of one product with the weights
      if constexpr (NS == 1)
        mma16816_f16(lm, __byte_perm(vl[0][0], vl[0][1], 0x7632), 0u, __byte_perm(vl[1][0], vl[1][1], 0x7632), 0u, wb[0], wb[1]);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (NS == 1) {
          uint32_t bs[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t s2 = __byte_perm(vp[r][0][g], vp[r][1][g], 0x5410);
            const __half2 ws = __hmul2(*reinterpret_cast<const __half2*>(&wb[r]), *reinterpret_cast<const __half2*>(&s2));
            bs[r] = *reinterpret_cast<const uint32_t*>(&ws) & kept_mask;
          }
          uint32_t a[2][4];       // codes of dims 32 g + 4 gid + i, the two keys of each half side by side
#pragma unroll
          for (int r = 0; r < 2; ++r) codes_f16(vc[r][0][g / 2], vc[r][1][g / 2], g & 1, a[r]);
          mma16816_f16(acc[g][0], a[0][0], a[0][1], a[1][0], a[1][1], bs[0], bs[1]);
          mma16816_f16(acc[g][1], a[0][2], a[0][3], a[1][2], a[1][3], bs[0], bs[1]);
        } else {
          // w s and w (m + 8 s) as sums of three bf16 values, the latter through
          // rows of ones
          float fs[2][2], fm[2][2];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&vp[r][j][g]));
              fs[r][j] = kept_mask ? wf[r][j] * sm.x : 0.f;
              fm[r][j] = kept_mask ? wf[r][j] * fmaf(8.f, sm.x, sm.y) : 0.f;
            }
          uint32_t a[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r)
            codes_bf16_centred(__byte_perm(vc[r][0][g / 2], vc[r][1][g / 2], g & 1 ? 0x7632 : 0x5410), a[r]);
          // fresh sums per tile, added in fp32: the matrix unit's own sums are not rounded to nearest
          float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f}, cm[4] = {0.f, 0.f, 0.f, 0.f};
          constexpr uint32_t one = 0x3F803F80u;
#pragma unroll
          for (int n = 0; n < 3; ++n) {
            const uint32_t s0 = pack_bf16(fs[0][0], fs[0][1]), s1 = pack_bf16(fs[1][0], fs[1][1]);
            const uint32_t m0 = pack_bf16(fm[0][0], fm[0][1]), m1 = pack_bf16(fm[1][0], fm[1][1]);
            mma16816_bf16(c0, a[0][0], a[0][1], a[1][0], a[1][1], s0, s1);
            mma16816_bf16(c1, a[0][2], a[0][3], a[1][2], a[1][3], s0, s1);
            mma16816_bf16(cm, one, one, one, one, m0, m1);
            fs[0][0] -= lo_bf16(s0); fs[0][1] -= hi_bf16(s0); fs[1][0] -= lo_bf16(s1); fs[1][1] -= hi_bf16(s1);
            fm[0][0] -= lo_bf16(m0); fm[0][1] -= hi_bf16(m0); fm[1][0] -= lo_bf16(m1); fm[1][1] -= hi_bf16(m1);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[g][0][i] += c0[i] + cm[i];
            acc[g][1][i] += c1[i] + cm[i];
          }
        }
      }
    }
    // a NaN among the least values is the kept heads' alone (0 x NaN in the other columns)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if ((cur.heads >> (2 * tig + e)) & 1u) least[e] += lm[e];
    __syncwarp();
    if (nxt.block >= 0) copy(vpg + nxt.block, stage_a + A::BLOCK);
    commit();
    cur = nxt;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();

  // ---- the warp's sums to its stage: row per head, then (maximum, sum)
  float* sums = reinterpret_cast<float*>(stage);
  const float w_down = NS == 1 ? __uint_as_float((254u << 23) - w_up) : 1.f;      // 2^-k
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float add = 0.f, f = 1.f, f4 = 1.f;
      if constexpr (NS == 1) {
        add = __shfl_sync(0xffffffffu, least[e], 4 * g + tig) * w_down;
        // the codes were multiplied as code 2^-24, those of rows gid + 8 (odd dims) as code 2^-20
        f = 16777216.f * w_down;
        f4 = 1048576.f * w_down;
      }
      // dims 32 g + 4 gid + 0 .. 3
      *reinterpret_cast<float4*>(sums + (2 * tig + e) * A::RS + 32 * g + 4 * gid) =
          make_float4(fmaf(acc[g][0][e], f, add), fmaf(acc[g][0][2 + e], f4, add), fmaf(acc[g][1][e], f, add),
                      fmaf(acc[g][1][2 + e], f4, add));
    }
  if (gid == 0)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sums[8 * A::RS + 2 * (2 * tig + e)] = M[e];
      sums[8 * A::RS + 2 * (2 * tig + e) + 1] = Z[e];
    }
  __syncthreads();
  // ---- warps to the CTA's sums, straight to the CTA that finishes the head:
  // CTA g % CL of the cluster, which keeps a row per CTA for each of its heads
  constexpr int WS = A::STAGE / 4;
  const float* all = reinterpret_cast<const float*>(qsm);
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");      // every CTA has started
  for (int i = tid; i < GV * D; i += TH) {
    const int g = i / D, t = i % D;
    float mw[kQdWarps], m = -INFINITY, s = 0.f, zz = 0.f;
#pragma unroll
    for (int w = 0; w < kQdWarps; ++w) {
      mw[w] = all[w * WS + 8 * A::RS + 2 * g];
      m = fmaxf(m, mw[w]);
    }
#pragma unroll
    for (int w = 0; w < kQdWarps; ++w) {
      if (mw[w] == -INFINITY) continue;       // attended nothing for this head
      const float f = exp2f(mw[w] - m);
      s = fmaf(f, all[w * WS + g * A::RS + t], s);
      zz = fmaf(f, all[w * WS + 8 * A::RS + 2 * g + 1], zz);
    }
    const uint32_t turn = uint32_t(g) / CL, to = uint32_t(g) - turn * CL;
    float* row = cluster.map_shared_rank(inbox, to) + (turn * CL + rank) * A::PART;
    row[t] = s;
    if (t < 2) row[D + t] = t ? zz : m;
  }
  cluster.sync();
  for (uint32_t g = rank, turn = 0; g < uint32_t(GV); g += CL, ++turn) {
    for (int t = tid; t < D; t += TH) {
      const float* rows = inbox + turn * CL * A::PART;
      float m = -INFINITY, s = 0.f, zz = 0.f;
      for (uint32_t c = 0; c < CL; ++c) m = fmaxf(m, rows[c * A::PART + D]);
      for (uint32_t c = 0; c < CL; ++c) {
        const float mc = rows[c * A::PART + D];
        if (mc == -INFINITY) continue;
        const float f = exp2f(mc - m);
        s = fmaf(f, rows[c * A::PART + t], s);
        zz = fmaf(f, rows[c * A::PART + D + 1], zz);
      }
      const float y = zz != 0.f ? s / zz : 0.f;       // nothing attended: 0
      T* out = o + (row0 + g) * D + t;
      if constexpr (NS == 1) *out = __float2bfloat16_rn(y);
      else *out = y;
    }
  }
}

}  // namespace hils
