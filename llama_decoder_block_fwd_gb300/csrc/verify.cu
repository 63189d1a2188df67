// Verification of drafted tokens against the target's probabilities ("LLaMA-3 8B ...", section 十:
// the next token is a draw from softmax(z / T); rejection sampling keeps that distribution when a
// cheaper model proposes tokens first).  Row j of a sequence holds the target's logits z_j after its
// j-th new token, the draft's logits y_j, and judges token j + 1, which the draft drew:
//   p = softmax(z / T), q = softmax(y / T); accept d while u q(d) < p(d);
//   at the first rejection the new token is argmax_i max(p_i - q_i, 0) / e_i, e_i given exponential
//   draws (the least of independent exponentials e_i / w_i is i with probability w_i / sum w, so
//   this is a draw from the normalised remainder); when every draft is accepted it is
//   argmax_i p_i / e_i of the last row.  Drafts without a distribution have q = 1 at d: accept while
//   u < p(d), remainder p without d.  T <= 0: accept while d is the argmax, new token the argmax.
//
// HBM bound.  Phase 1 (verify_stats_kernel) reads every judged row of z and y once: warps take the
// 1024-logit parts of all rows in turn, a part's loads in flight together, and leave its (max, sum of
// exponentials).  Phase 2 (verify_pick_kernel, a cluster of up to 8 CTAs per sequence) merges the parts,
// finds the first rejection and reads that row of z, y and e for the race.  Where the remainder is a small
// difference of large p and q the race is run again over 1 - q / p from the logits' differences.
// 64 sequences x 2-5 rows x 128256 logits with a draft distribution: 49.3 us, of which phase 1 27 us (200 MB,
// the slowest SM 27 us, the median warp 24), merging and judging 2, the race 10 (99 MB from L2 and HBM, in
// six dependent turns), cluster exchange and result 4, launches the rest; the bytes alone would take 34.  With
// rows of 128257 logits, three of four of which are not 16-byte aligned and are read a logit at a time, 57.3.
// 48 sequences without a draft distribution 32.4 (36.6); T <= 0 23.5.
// One kernel over both phases (items from a counter, races behind the statistics) took 111 us: each item
// paid two barriers, a fence and three dependent atomics with too few loads in flight.
// A part's sums are formed and merged in a fixed order, and the race keeps the largest score and of equals
// the lowest id, so the result does not depend on timing.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>

#include "kernels.h"

namespace llama {
namespace {

constexpr int VF_THREADS = 256;
constexpr int VF_WARPS = VF_THREADS / 32;
constexpr int VF_UNITS = 8;                               // float4 units per lane in a part
constexpr int VF_PART = 32 * VF_UNITS * 4;                // logits per part, one warp's
constexpr int VF_RACE = 4;                                // float4 units of each row in flight per thread
constexpr int VF_RACE_REST = 3;                           // with a draft row beside them
constexpr int VF_STATS_CTAS = 5, VF_PICK_CTAS = 4;        // per SM (registers)
constexpr int VF_ROWS = 32;                               // rows whose merged statistics are kept
constexpr int VF_CLUSTER = 8;

struct VerifyParams {
  const float *z, *y;              // [T, ld], [T, ld_y]; y may be null
  int64_t ld, ld_y, ld_e;
  int T, V, B, parts, greedy;
  float c;                         // log2(e) / T
  const int *cu, *tokens;
  const float *u, *e;              // [T], [B, ld_e]
  int *n_acc, *out;                // [B], [T]
  float2* stat_z;                  // [T, parts] (max, sum), greedy: (max, id)
  float2* stat_y;
  unsigned* status;
};

__device__ __forceinline__ float vf_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// exp((z - m) / T) for z <= m, m finite: two roundings in the exponent and ex2 (2^-22 relative).  A
// masked logit (-inf) has weight 0, and no finite z or T gives a NaN on the way (c > 0).
__device__ __forceinline__ float vf_exp(const VerifyParams& p, float z, float m) { return vf_ex2((z - m) * p.c); }

__device__ __forceinline__ float4 vf_load4(const float* row, int i, int V, bool vec) {
  if (vec && i + 4 <= V) return __ldg(reinterpret_cast<const float4*>(row + i));
  float4 w = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  if (i < V) w.x = __ldg(row + i);
  if (i + 1 < V) w.y = __ldg(row + i + 1);
  if (i + 2 < V) w.z = __ldg(row + i + 2);
  if (i + 3 < V) w.w = __ldg(row + i + 3);
  return w;
}

__device__ __forceinline__ bool vf_aligned(const float* row) { return (reinterpret_cast<uintptr_t>(row) & 15) == 0; }

// The last sequence b whose rows start at or before `row` (cu[0] = 0 <= row), by a whole warp.
__device__ __forceinline__ int sequence_of(const VerifyParams& p, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.B;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < n && __ldg(p.cu + lo + at) <= row);
    const int k = le ? 31 - __clz(le) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Part u of the rows of z, then of y: the address of its row, null where there is nothing to do (rows
// behind the last sequence; in y the last row of a sequence, which judges no draft).
__device__ __forceinline__ const float* part_row(const VerifyParams& p, int u, int total, int rows_used, int& row,
                                                 int& part) {
  row = 0;
  part = 0;
  if (u >= total) return nullptr;
  const int r = u / p.parts;
  part = u - r * p.parts;
  const bool draft = r >= p.T;
  row = draft ? r - p.T : r;
  if (row >= rows_used) return nullptr;
  if (!draft) return p.z + (int64_t)row * p.ld;
  return __ldg(p.cu + sequence_of(p, row) + 1) - 1 == row ? nullptr : p.y + (int64_t)row * p.ld_y;
}

__device__ __forceinline__ void load_part(const VerifyParams& p, const float* src, int part, float4 (&w)[VF_UNITS]) {
  if (!src) return;
  const bool vec = vf_aligned(src);
  const int i0 = part * VF_PART + (threadIdx.x & 31) * 4;
#pragma unroll
  for (int j = 0; j < VF_UNITS; ++j) w[j] = vf_load4(src, i0 + j * 128, p.V, vec);
}

template <bool GREEDY>
__global__ void __launch_bounds__(VF_THREADS, VF_STATS_CTAS) verify_stats_kernel(const __grid_constant__ VerifyParams p) {
  const int lane = threadIdx.x & 31, nw = gridDim.x * VF_WARPS;
  const int total = p.T * p.parts * (p.y ? 2 : 1);
  pdl_trigger();
  const int rows_used = min(p.T, __ldg(p.cu + p.B));
  for (int u = blockIdx.x * VF_WARPS + (threadIdx.x >> 5); u < total; u += nw) {
    int row, part;
    const float* src = part_row(p, u, total, rows_used, row, part);
    float4 w[VF_UNITS];
    load_part(p, src, part, w);
    if (src) {
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < VF_UNITS; ++j) m = fmaxf(m, fmaxf(fmaxf(w[j].x, w[j].y), fmaxf(w[j].z, w[j].w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float second;
      if (GREEDY) {   // the lowest id that holds the maximum
        int id = INT_MAX;
#pragma unroll
        for (int j = VF_UNITS - 1; j >= 0; --j) {
          const int i = part * VF_PART + j * 128 + lane * 4;
          if (w[j].w == m && i + 3 < p.V) id = i + 3;
          if (w[j].z == m && i + 2 < p.V) id = i + 2;
          if (w[j].y == m && i + 1 < p.V) id = i + 1;
          if (w[j].x == m && i < p.V) id = i;
        }
        second = __int_as_float((int)__reduce_min_sync(0xffffffffu, id));
      } else {
        const float mu = m == -INFINITY ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < VF_UNITS; ++j)
          s += (vf_exp(p, w[j].x, mu) + vf_exp(p, w[j].y, mu)) + (vf_exp(p, w[j].z, mu) + vf_exp(p, w[j].w, mu));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        second = s;
      }
      const int64_t at = (int64_t)row * p.parts + part;
      if (lane == 0 && in_extent(at, 1, (int64_t)p.T * p.parts)) {
        float2* stat = u / p.parts >= p.T ? p.stat_y : p.stat_z;
        stat[at] = make_float2(m, second);
      }
    }
  }
}

// A row's (max, 1 / sum) from its parts, by one warp.
__device__ __forceinline__ float2 merge_parts(const VerifyParams& p, const float2* stat) {
  const int lane = threadIdx.x & 31;
  float2 a[4];                     // the first 128 parts (131072 logits) in flight together
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = lane + 32 * j < p.parts ? __ldcg(stat + lane + 32 * j) : make_float2(-INFINITY, 0.f);
  float m = fmaxf(fmaxf(a[0].x, a[1].x), fmaxf(a[2].x, a[3].x));
  for (int i = lane + 128; i < p.parts; i += 32) m = fmaxf(m, __ldcg(stat + i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) s += a[j].y * vf_exp(p, a[j].x, m);   // a masked part has sum 0
  for (int i = lane + 128; i < p.parts; i += 32) {
    const float2 b = __ldcg(stat + i);
    s += b.y * vf_exp(p, b.x, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return make_float2(m, 1.f / s);
}
// A row's argmax from its parts (greedy), by one warp.
__device__ __forceinline__ int merge_argmax(const VerifyParams& p, const float2* stat) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  int id = INT_MAX;
  for (int i = lane; i < p.parts; i += 32) {
    const float2 a = __ldcg(stat + i);
    if (a.x > m) { m = a.x; id = __float_as_int(a.y); }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o);
    const int oi = __shfl_xor_sync(0xffffffffu, id, o);
    if (om > m || (om == m && oi < id)) { m = om; id = oi; }
  }
  return id == INT_MAX ? 0 : id;
}

// ---- the remainder p - q = p (1 - q / p)
// Where the models are close, the difference of two fp32 probabilities is mostly their rounding.  So it is taken
// from the logits there: log2(q / p) = c ((y - z) - (my - mz)) - log2(Sy / Sz), my, mz the rows' maxima and Sy,
// Sz their sums; y - z and my - mz are taken with what their rounding leaves (the models' logits may be a constant
// apart), which makes the difference of the two exact for close models.
constexpr float VF_CLOSE = 0x1p-6f;     // 1 - q / p of a winner below which the models are close
constexpr float VF_PEAK = 0x1p-13f;     // and so they are where its score is less than this of the largest p / e: what
                                        // that token's p - q is off by could be as large
constexpr float VF_SERIES = 0.25f;      // |log2(q / p)| below which 1 - q / p comes from a series

// a - b and what its rounding left out (Knuth's two-sum); NaN in the latter where the difference is not finite
__device__ __forceinline__ float2 two_diff(float a, float b) {
  const float d = __fsub_rn(a, b), v = __fsub_rn(d, a);
  return make_float2(d, __fsub_rn(__fsub_rn(a, __fsub_rn(d, v)), __fadd_rn(b, v)));
}
// c ((y - z) - (my - mz)), shift = two_diff(my, mz)
__device__ __forceinline__ float log2_ratio(const VerifyParams& p, float z, float y, float2 shift) {
  const float2 d = two_diff(y, z);
  return __fmul_rn(__fadd_rn(__fsub_rn(d.x, shift.x), __fsub_rn(d.y, shift.y)), p.c);
}
// 2^t - 1 for |t| < VF_SERIES: the exponential series up to x^6 / 720 leaves 0.18^6 / 5040 = 7e-9 of it
__device__ __forceinline__ float exp2_less_1(float t) {
  const float x = t * 0.693147180559945f;
  float s = fmaf(x, 1.f / 720.f, 1.f / 120.f);
  s = fmaf(x, s, 1.f / 24.f);
  s = fmaf(x, s, 1.f / 6.f);
  s = fmaf(x, s, 0.5f);
  s = fmaf(x, s, 1.f);
  return x * s;
}

// The better of two (score, key), key = 2 id + mark: the larger score, of equals the lower id.
constexpr unsigned kNone = UINT_MAX;
__device__ __forceinline__ void race_max(float& s, unsigned& key, float os, unsigned okey) {
  if (os > s || (os == s && okey < key)) { s = os; key = okey; }
}

// What the race runs over: REST max(p - q, 0); CLOSE the same for models that are close; NO_DRAFT p without the
// draft; ALL p.
enum RaceKind : int { REST, CLOSE, NO_DRAFT, ALL };

// This CTA's share of the vocabulary: a thread's (best score, its lowest id); scores of 0 do not count.  `lr` is
// log2(Sy / Sz) (CLOSE); in REST the winner's key is marked where its p and q are close, and `peak` is the largest
// p / e of the tokens that are judged: all those above the best score, and whatever others, which being below it
// do not count where peak is compared with it.
// p_i / e_i bounds a score from above, so a token whose p_i is below top * e_i, top the CTA's best score so far
// (less 2^-20, more than the quotients' errors), is out of the race: it needs one exponential and no
// division in place of two and one (48 lookups of 128256 logits: 35.7 -> 33.1 us; with a draft distribution
// 55.6 -> 54.1, and 56 when the draft's row was read for the few tokens that pass only, one wait each).
// Which tokens are left out depends on timing, the best of the others does not.  The first units, all
// judged, give the CTA a score to start from.
template <int KIND>
__device__ __forceinline__ void race(const VerifyParams& p, const float* z, const float* y, const float* e, int d,
                                     float2 sz, float2 sy, float lr, int cr, int P, unsigned* top, float& best,
                                     unsigned& key, float& peak) {
  constexpr bool DRAFT = KIND == REST || KIND == CLOSE;
  const bool vz = vf_aligned(z), vy = DRAFT && vf_aligned(y), ve = vf_aligned(e);
  const int units = (p.V + 3) >> 2, step = P * VF_THREADS, first = cr * VF_THREADS + (int)threadIdx.x;
  best = peak = 0.f;
  key = kNone;
  auto weight = [&](float zi, int i) {
    const float w = __fmul_rn(vf_exp(p, zi, sz.x), sz.y);
    return KIND == NO_DRAFT && i == d ? 0.f : w;
  };
  auto score = [&](float w, float zi, float yi, float ei, int i) {
    float r = w;
    if (KIND == CLOSE) {
      const float t = log2_ratio(p, zi, yi, two_diff(sy.x, sz.x)) - lr;
      if (fabsf(t) < VF_SERIES) r = -w * exp2_less_1(t);
      else r = w - vf_exp(p, yi, sy.x) * sy.y;
    } else if (KIND == REST) {   // both products rounded: fused, one of them would leave its rounding where p = q
      r = __fsub_rn(w, __fmul_rn(vf_exp(p, yi, sy.x), sy.y));
    }
    if (KIND == REST) peak = fmaxf(peak, __fdividef(w, ei));   // (0 / 0 is left out)
    const float s = __fdividef(r, ei);
    if (r > 0.f && s > best) {   // ids grow: an equal later one does not count
      best = s;
      key = 2u * (unsigned)i + (KIND == REST && r < w * VF_CLOSE);
    }
  };
  auto publish = [&]() {
    const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(best));
    if ((threadIdx.x & 31) == 0 && m > *(volatile unsigned*)top) atomicMax(top, m);
  };
  constexpr int DEPTH = DRAFT ? VF_RACE_REST : VF_RACE;
  float4 a[DEPTH], n[DEPTH], c[DEPTH];
  auto load = [&](int q0) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {   // past the end: -inf, which has no weight
      const int i = (q0 + j * step) * 4;
      a[j] = vf_load4(z, i, p.V, vz);
      n[j] = vf_load4(e, i, p.V, ve);
      if (DRAFT) c[j] = vf_load4(y, i, p.V, vy);
    }
  };
  {
    const float4 z0 = vf_load4(z, first * 4, p.V, vz), e0 = vf_load4(e, first * 4, p.V, ve);
    float4 y0 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (DRAFT) y0 = vf_load4(y, first * 4, p.V, vy);
    load(first + step);
    const float za[4] = {z0.x, z0.y, z0.z, z0.w}, ea[4] = {e0.x, e0.y, e0.z, e0.w}, ya[4] = {y0.x, y0.y, y0.z, y0.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float w = weight(za[t], first * 4 + t);
      score(w, za[t], ya[t], ea[t], first * 4 + t);
    }
    publish();
  }
  __syncthreads();
  for (int q0 = first + step; q0 - (int)(threadIdx.x & 31) < units; q0 += DEPTH * step) {   // whole warps
    if (q0 != first + step) load(q0);
    float low = __uint_as_float(*(volatile unsigned*)top) * (1.f - 0x1p-20f);
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {
      const int i = (q0 + j * step) * 4;
      const float za[4] = {a[j].x, a[j].y, a[j].z, a[j].w}, ea[4] = {n[j].x, n[j].y, n[j].z, n[j].w};
      float ya[4] = {0.f, 0.f, 0.f, 0.f};
      if (DRAFT) { ya[0] = c[j].x; ya[1] = c[j].y; ya[2] = c[j].z; ya[3] = c[j].w; }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float w = weight(za[t], i + t);
        if (w > 0.f && !(w < low * ea[t])) {   // (a draw of 0 against an infinite score: NaN, and in)
          score(w, za[t], ya[t], ea[t], i + t);
          low = fmaxf(low, best * (1.f - 0x1p-20f));
        }
      }
    }
    publish();
  }
}

// What the CTAs of a cluster tell each other, per turn of the race.
struct PickShared {
  float wbest[VF_WARPS];
  unsigned wkey[VF_WARPS];
  float wpeak[VF_WARPS];
  float best[3][VF_CLUSTER];      // every CTA's best, written by that CTA
  unsigned key[3][VF_CLUSTER];
  float sum[VF_CLUSTER], peak[VF_CLUSTER];
  unsigned top[3];                // the best score so far
};

// The threads' best candidates -> the cluster's; the same for every CTA.  With PEAK the largest `peak` too.
template <bool PEAK>
__device__ __forceinline__ unsigned race_end(PickShared& sh, int turn, int cr, int P, float& best, unsigned key, float& peak) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    race_max(best, key, __shfl_xor_sync(0xffffffffu, best, o), __shfl_xor_sync(0xffffffffu, key, o));
  if (PEAK) peak = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(peak)));
  if ((tid & 31) == 0) {
    sh.wbest[tid >> 5] = best;
    sh.wkey[tid >> 5] = key;
    if (PEAK) sh.wpeak[tid >> 5] = peak;
  }
  __syncthreads();
  if (tid < P) {   // to every CTA of the cluster, which after the barrier reads only its own memory
    best = sh.wbest[0];
    key = sh.wkey[0];
    for (int k = 1; k < VF_WARPS; ++k) race_max(best, key, sh.wbest[k], sh.wkey[k]);
    *cl.map_shared_rank(&sh.best[turn][cr], tid) = best;
    *cl.map_shared_rank(&sh.key[turn][cr], tid) = key;
    if (PEAK) {
      for (int k = 0; k < VF_WARPS; ++k) peak = fmaxf(peak, sh.wpeak[k]);
      *cl.map_shared_rank(&sh.peak[cr], tid) = peak;
    }
  }
  cl.sync();
  best = 0.f;
  key = kNone;
  for (int r = 0; r < P; ++r) {
    race_max(best, key, sh.best[turn][r], sh.key[turn][r]);
    if (PEAK) peak = fmaxf(peak, sh.peak[r]);
  }
  return key;
}

// log2(Sy / Sz) again, for models that are close: Sy / Sz 2^(c (my - mz)) - 1 = sum_i p_i (2^t_i - 1), t_i the
// log2 ratio without the sums.  The terms are as small as the models' differences, and so is what they are off
// by, where the sums as they stand are off by about 2^-23 of 1.  One more pass over the two rows, and a race after
// it, which only a rejection between close models asks for (64 sequences x 128256, every one of them: 95 us
// against 48).
__device__ __forceinline__ float row_ratio(const VerifyParams& p, const float* z, const float* y, float2 sz, float2 sy,
                                           int cr, int P, PickShared& sh) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cl = cg::this_cluster();
  const bool vz = vf_aligned(z), vy = vf_aligned(y);
  const float2 shift = two_diff(sy.x, sz.x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t i = 4 * (cr * VF_THREADS + (int)threadIdx.x); i < p.V; i += 4 * P * VF_THREADS) {
    const float4 z4 = vf_load4(z, (int)i, p.V, vz), y4 = vf_load4(y, (int)i, p.V, vy);
    const float za[4] = {z4.x, z4.y, z4.z, z4.w}, ya[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float w = vf_exp(p, za[k], sz.x) * sz.y, t = log2_ratio(p, za[k], ya[k], shift);
      acc[k] += fabsf(t) < VF_SERIES ? w * exp2_less_1(t) : vf_exp(p, ya[k], sy.x) * sz.y - w;
    }
  }
  float s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sh.wbest[warp] = s;
  __syncthreads();
  if (threadIdx.x < P) {
    s = 0.f;
    for (int k = 0; k < VF_WARPS; ++k) s += sh.wbest[k];
    *cl.map_shared_rank(&sh.sum[cr], threadIdx.x) = s;
  }
  cl.sync();
  s = 0.f;
  for (int r = 0; r < P; ++r) s += sh.sum[r];
  return log1pf(s) * 1.44269504088896f;
}

// What rarely follows the race of a rejected draft (kept out of the way of its registers): the remainder of close
// models with their ratio found again (turn 1), then, where no p exceeds its q, p (turn 2).
__device__ __noinline__ unsigned race_again(const VerifyParams& p, const float* z, const float* y, const float* e,
                                            float2 sz, float2 sy, int cr, int P, PickShared& sh) {
  float best, peak;
  unsigned key = kNone;
  if (y) {
    const float lr = row_ratio(p, z, y, sz, sy, cr, P, sh);
    race<CLOSE>(p, z, y, e, -1, sz, sy, lr, cr, P, sh.top + 1, best, key, peak);
    key = race_end<false>(sh, 1, cr, P, best, key, peak);
  }
  if (key == kNone) {
    race<ALL>(p, z, nullptr, e, -1, sz, sz, 0.f, cr, P, sh.top + 2, best, key, peak);
    key = race_end<false>(sh, 2, cr, P, best, key, peak);
  }
  return key;
}

__global__ void __launch_bounds__(VF_THREADS, VF_PICK_CTAS) verify_pick_kernel(const __grid_constant__ VerifyParams p) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cl = cg::this_cluster();
  const int P = (int)cl.num_blocks(), cr = (int)cl.block_rank(), b = blockIdx.x / P;
  __shared__ int stop_sh, top_sh;
  __shared__ PickShared sh;
  __shared__ float2 sz_sh[VF_ROWS], sy_sh[VF_ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cl.barrier_arrive();      // waited for before another CTA's memory is written: that CTA has started then
  // the caller's inputs may be read before the statistics are there
  const int lo = max(0, __ldg(p.cu + b)), hi = min(p.T, __ldg(p.cu + b + 1));
  if (tid == 0) {
    stop_sh = hi - 1;
    sh.top[0] = sh.top[1] = sh.top[2] = 0;
  }
  __syncthreads();
  int row = lo + warp, d = -1;
  float zd = 0.f, yd = 0.f, u = 0.f;
  auto inputs = [&]() {   // what row `row` judges its draft by
    if (row >= hi - 1) return;   // the last row judges none
    d = __ldg(p.tokens + row + 1);
    if (p.greedy) return;
    u = __ldg(p.u + row);
    if (d < 0 || d >= p.V) return;
    zd = __ldg(p.z + (int64_t)row * p.ld + d);
    if (p.y) yd = __ldg(p.y + (int64_t)row * p.ld_y + d);
  };
  inputs();
  pdl_wait();
  if (hi <= lo) {           // a sequence without rows (the whole cluster leaves)
    cl.barrier_wait();
    if (cr == 0 && tid == 0 && in_extent(b, 1, p.B)) p.n_acc[b] = 0;
    return;
  }
  // ---- the first row whose draft is turned down (the last row if none is)
  for (; row < hi; row += VF_WARPS, inputs()) {
    if (row == hi - 1) {   // its statistics, should it be the one
      if (!p.greedy && row - lo < VF_ROWS) {
        const float2 sz = merge_parts(p, p.stat_z + (int64_t)row * p.parts);
        if (lane == 0) sz_sh[row - lo] = sz;
      }
      break;
    }
    const bool real = d >= 0 && d < p.V;
    bool ok;
    if (p.greedy) {
      ok = merge_argmax(p, p.stat_z + (int64_t)row * p.parts) == d;
    } else {
      const float2 sz = merge_parts(p, p.stat_z + (int64_t)row * p.parts);
      // u q < p with both sides scaled by the larger exponent, so that it does not depend on how small both are
      // (a p below 2^-1074 is 0, as in 64 bits: a logit masked with the type's lowest value)
      const float xz = (zd - sz.x) * p.c;
      float qd = 1.f, scale = 0.f;
      if (p.y) {
        const float2 sy = merge_parts(p, p.stat_y + (int64_t)row * p.parts);
        const float xy = (yd - sy.x) * p.c;
        scale = fmaxf(xz, xy);
        qd = vf_ex2(xy - scale) * sy.y;
        if (lane == 0 && row - lo < VF_ROWS) sy_sh[row - lo] = sy;
      }
      if (lane == 0 && row - lo < VF_ROWS) sz_sh[row - lo] = sz;
      u = (u >= 0.f) ? fminf(u, 0.99999994f) : 0.f;
      ok = xz > -1074.f &&
           (u == 0.f || (double)u * (double)qd < (double)(vf_ex2(xz - scale) * sz.y));   // the left product is exact
    }
    if (lane == 0) {
      if (!real && cr == 0) atomicOr(p.status, STATUS_BAD_TOKEN);
      if (!real || !ok) atomicMin(&stop_sh, row);
    }
  }
  __syncthreads();
  const int stop = stop_sh;
  const bool rejected = stop < hi - 1;
  int token;
  cl.barrier_wait();
  if (p.greedy) {
    if (warp == 0) {
      const int id = merge_argmax(p, p.stat_z + (int64_t)stop * p.parts);
      if (lane == 0) top_sh = id;
    }
    __syncthreads();
    token = top_sh;
  } else {
    const int kept = min(stop - lo, VF_ROWS - 1);
    if (stop - lo >= VF_ROWS) {   // a long sequence: merged again, in the last place
      __syncthreads();
      if (warp == 0) {
        const float2 s = merge_parts(p, p.stat_z + (int64_t)stop * p.parts);
        if (lane == 0) sz_sh[kept] = s;
      }
      if (warp == 1 && p.y && rejected) {
        const float2 s = merge_parts(p, p.stat_y + (int64_t)stop * p.parts);
        if (lane == 0) sy_sh[kept] = s;
      }
      __syncthreads();
    }
    const float* z = p.z + (int64_t)stop * p.ld;
    const float* e = p.e + (int64_t)b * p.ld_e;
    const float2 sz = sz_sh[kept], sy = p.y && rejected ? sy_sh[kept] : sz;
    const int judged = rejected ? __ldg(p.tokens + stop + 1) : -1;
    const float* y = p.y && rejected ? p.y + (int64_t)stop * p.ld_y : nullptr;
    float best, peak;
    unsigned key;
    if (!rejected) race<ALL>(p, z, nullptr, e, -1, sz, sz, 0.f, cr, P, sh.top, best, key, peak);
    else if (y) race<REST>(p, z, y, e, -1, sz, sy, 0.f, cr, P, sh.top, best, key, peak);
    else race<NO_DRAFT>(p, z, nullptr, e, judged, sz, sz, 0.f, cr, P, sh.top, best, key, peak);
    key = race_end<true>(sh, 0, cr, P, best, key, peak);
    if (rejected && (key == kNone || (key & 1) || best < peak * VF_PEAK)) key = race_again(p, z, y, e, sz, sy, cr, P, sh);
    token = key == kNone ? 0 : (int)(key >> 1);
  }
  if (cr != 0) return;
  if (tid == 0 && in_extent(b, 1, p.B)) p.n_acc[b] = stop - lo;
  for (int r = lo + tid; r < hi; r += VF_THREADS)
    if (in_extent(r, 1, p.T)) p.out[r] = r < stop ? __ldg(p.tokens + r + 1) : r == stop ? token : -1;
}

size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
int64_t parts_of(int64_t V) { return (V + VF_PART - 1) / VF_PART; }

}  // namespace

// Parts are counted in 32 bits.
bool verify_supported(int64_t T, int64_t V) { return 2 * T * parts_of(V) <= INT32_MAX / 2; }

size_t verify_ws_bytes(int64_t T, int64_t V) { return 2 * round256((size_t)T * parts_of(V) * sizeof(float2)); }

int launch_verify(const VerifyDesc& d, int num_sms, unsigned* status, cudaStream_t st) {
  VerifyParams p;
  p.z = d.logits; p.y = d.temperature > 0.f ? d.draft_logits : nullptr;
  p.ld = d.ld; p.ld_y = d.draft_ld; p.ld_e = d.noise_ld;
  p.T = (int)d.T; p.V = (int)d.V; p.B = (int)d.B;
  p.parts = (int)parts_of(d.V);
  p.greedy = !(d.temperature > 0.f);
  // kept a positive finite number for every T > 0, infinity included
  p.c = p.greedy ? 1.f : (float)std::min(std::max(1.4426950408889634074 / (double)d.temperature, (double)FLT_MIN),
                                         (double)FLT_MAX);
  p.cu = d.cu_new; p.tokens = d.tokens; p.u = d.u; p.e = d.noise;
  p.n_acc = d.n_accepted; p.out = d.out_tokens;
  p.stat_z = static_cast<float2*>(d.ws);
  p.stat_y = reinterpret_cast<float2*>(static_cast<char*>(d.ws) + round256((size_t)d.T * p.parts * sizeof(float2)));
  p.status = status;
  if (d.T > 0) {
    // Launched plainly, and that has to stay: the pick kernel reads the caller's inputs before its dependency wait,
    // and they are complete only because this launch has waited for all that came before it.
    const int64_t total = d.T * p.parts * (p.y ? 2 : 1);
    const unsigned grid = (unsigned)std::min<int64_t>((total + VF_WARPS - 1) / VF_WARPS, VF_STATS_CTAS * num_sms);
    if (p.greedy) verify_stats_kernel<true><<<grid, VF_THREADS, 0, st>>>(p);
    else verify_stats_kernel<false><<<grid, VF_THREADS, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -1;
  }
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  // as many CTAs per sequence as are resident together, up to a cluster; an eighth of the room is left to
  // how clusters fall on the GPCs (64 x 128256, three CTAs per SM: clusters of 7 in all the room took a
  // second wave, 70 us; clusters of 6, 57.6 us; of 8 at four per SM, 55.3 us)
  int P = 1;
  if (!p.greedy) P = (int)std::min<int64_t>(VF_CLUSTER, std::max<int64_t>(1, VF_PICK_CTAS * num_sms * 7 / 8 / d.B));
  cfg.gridDim = dim3((unsigned)(d.B * P));
  cfg.blockDim = dim3(VF_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)P;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_pick_kernel, p) == cudaSuccess ? 0 : -1;
}

LLAMA_DEFINE_BOUNDS_READER(verify)

}  // namespace llama
