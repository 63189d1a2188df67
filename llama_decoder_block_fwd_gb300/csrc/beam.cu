// Beam search over the paged cache: choosing the next beams, and making the cache follow them ("LLaMA-3 8B ...",
// section 十 takes the next token from softmax(z); a beam's score is the sum of its tokens' log-probabilities).
//
// select: score(w, i) = scores[w] + z_wi - log sum_j exp(z_wj); the n_out largest over beams w and tokens i, ties
//   to the lower beam, then the lower token.
// reorder: row w of the block table becomes row parents[w]; of the new beams that share an open (not full) last page all
//   but the first get a copy of its rows.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "kernels.h"

namespace llama {
namespace {

constexpr size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

// ---------------------------------------------------------------------------------------- select
// HBM bound for many rows, latency for few.  The rows' batches of BS_BATCH logits, one row after the other, are cut into
// equal ranges, one per CTA (rows that need not be read left out).  A producer warp streams a range's batches into a ring in
// shared memory (bulk copies), 256 threads take them.  Each warp sums the exponentials of its 640 logits of a batch from
// their own maximum; these sums do not depend on where the rows are cut, so equal rows give equal scores.  What beats the
// n_out-th best of a row's piece so far waits in shared memory, and now and then the n_out best are taken anew.  The second
// kernel joins a request's lists and sums.
// 48 requests of 8 beams x 128256, a seventh of them finished (167 MB), 16 kept: 44.4 us, the first kernel 40.2 cold, 4.0 TB/s.
// Each further request costs 0.63 us (6.5 TB/s); the rest, some 18 us, are the ranges' starts, the pieces' first batches, whose
// candidates are many, their ends, and the join.  (Registers loaded ahead instead of the ring 52 us, 4 CTAs per SM 46-60.)  One request
// of 4 beams x 32000: 10.5 us, two launches and their chains.
constexpr int BS_THREADS = 256;
constexpr int BS_WARPS = BS_THREADS / 32;
constexpr int BS_PER = 20;                              // logits of a thread in a batch
constexpr int BS_BATCH = BS_THREADS * BS_PER;
constexpr int BS_STAGES = 3;
constexpr int BS_MAX_K = (int)kBeamMaxOut;
__host__ __device__ constexpr int bs_slack(int K) { return K > 16 ? K : 16; }   // candidates that may wait for the next cut
constexpr int BS_CTAS_PER_SM = 3;
constexpr int BS_MAX_PIECES = 12;                       // of a row, on average: what the join has to look through
constexpr int BS_SCAN = 1 << 14;                        // rows up to which every CTA counts those that have to be read
__host__ __device__ constexpr int bs_room(int K) { return bs_slack(K) + (K > 16 ? K : 16) * BS_PER; }
__host__ __device__ constexpr int bs_smem(int K, bool vec) { return (vec ? BS_STAGES * BS_BATCH * 4 : 0) + (bs_room(K) + 2 * K) * 8; }

struct RowPieces { int slot, n; };   // a row's lists are slot, slot + 1, ..

struct SelectParams {
  const float* z;
  int64_t ld;
  int B, W, V, K, nb;     // nb: batches of a row
  const float* scores;
  const int* finished;
  int pad;
  int *parents, *tokens;
  float* out;
  uint64_t* keys;      // [B W + CTAs, K] the best tokens of a piece, best first (0: none)
  RowPieces* pieces;   // [B W]
  float2* stat;        // [B W, nb, warps] maximum and sum of exp(z - maximum)
  int64_t n_lists;
  unsigned* status;
};

// Logits as integers that order as they do, the lower token above at equal ones: larger is better, 0 is no candidate.
__device__ __forceinline__ uint64_t cand_key(float z, int i) {
  const uint32_t u = __float_as_uint(z + 0.f);          // -0 counts as 0
  const uint32_t ord = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return z > -INFINITY ? ((uint64_t)ord << 32) | (uint32_t)~i : 0;
}
__device__ __forceinline__ float key_logit(uint64_t k) {
  const uint32_t ord = (uint32_t)(k >> 32);
  return __uint_as_float((ord & 0x80000000u) ? ord & 0x7FFFFFFFu : ~ord);
}
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// exp(x - m) with the difference formed first, so that large logits keep their digits.  Off by 2.23 * 2^-24 of the distance (a
// difference, a product and log2(e), each rounded) and 2^-22 (the instruction): with distances whose mean under the softmax is at most
// ln V, two of these and some 25 additions in a row, a sum is off by 2^-18 of itself at most, for 163840 logits.
__device__ __forceinline__ float exp_from(float x, float m) { return exp2_fast((x - m) * 1.4426950408889634f); }
__device__ __forceinline__ void join_sums(float& m, float& s, float m2, float s2) {
  const float mx = fmaxf(m, m2);
  if (mx > -INFINITY) s = s * exp_from(m, mx) + s2 * exp_from(m2, mx);
  m = mx;
}
// Two at a time (one instruction each).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%1, %2};\n\tmov.b64 v, {%3, %4};\n\tadd.rn.f32x2 %0, u, v;\n\t}" : "=l"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%1, %2};\n\tmov.b64 v, {%3, %4};\n\tmul.rn.f32x2 %0, u, v;\n\t}" : "=l"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 exp_from2(float a, float b, float m) {
  const float2 t = mul2(add2(make_float2(a, b), make_float2(-m, -m)), make_float2(1.4426950408889634f, 1.4426950408889634f));
  return make_float2(exp2_fast(t.x), exp2_fast(t.y));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The n-th largest of a warp's values (equal ones counted each; -inf counts).
__device__ __forceinline__ float warp_nth(float v, int n) {
  const int lane = threadIdx.x & 31;
  float t = v;
  for (int i = 1;; ++i) {
    float mx;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(mx) : "f"(t));
    if (i == n) return mx;
    if (lane == __ffs(__ballot_sync(0xffffffffu, t == mx)) - 1) t = -INFINITY;
  }
}

__device__ __forceinline__ bool row_live(const SelectParams& p, int row) {
  const int done = p.finished ? __ldg(p.finished + row) : 0;
  return __ldg(p.scores + row) > -INFINITY && !done;
}
// a / b for 0 <= a, 0 < b: a 64-bit division costs some hundred instructions, and few calls need one.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// T batches in n ranges, as equal as can be and all over alike: where every row gets a whole number, no range ends inside one.
// (With the longer ones all in front 8 requests of 4 rows take 17.5 us, not 15.5.)
struct Ranges {
  int64_t T;
  int n;
  __device__ __forceinline__ int64_t first(int i) const { return quotient(i * T, n); }
  __device__ __forceinline__ int with(int64_t x) const {   // the range that holds batch x
    int i = (int)min((int64_t)n - 1, quotient(x * n, T));
    while (i + 1 < n && first(i + 1) <= x) ++i;
    while (i > 0 && first(i) > x) --i;
    return i;
  }
};
// The pieces of a CTA's range: batches [b0, b1) of a row, the row's place among those that are read.
struct RowWalk { int row, b; int64_t place, left; };
__device__ __forceinline__ bool next_row_piece(const SelectParams& p, RowWalk& s, bool all, int& row, int& b0, int& b1, int64_t& place) {
  if (s.left <= 0) return false;
  if (!all)
    while (!row_live(p, s.row)) {
      if (++s.row >= p.B * p.W) return false;
    }
  row = s.row++;
  place = s.place++;
  b0 = s.b;
  b1 = (int)min((int64_t)p.nb, b0 + s.left);
  s.left -= b1 - b0;
  s.b = 0;
  return true;
}

// VEC: rows start on 16 bytes and come by bulk copies; else each thread loads its own.
template <bool VEC>
__global__ void __launch_bounds__(BS_THREADS + 32, BS_CTAS_PER_SM) beam_part_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint8_t bs_smem_raw[];
  float* ring = reinterpret_cast<float*>(bs_smem_raw);
  const int K = p.K, room = bs_room(K);
  uint64_t* list = reinterpret_cast<uint64_t*>(bs_smem_raw + (VEC ? BS_STAGES * BS_BATCH * 4 : 0));   // candidates that wait
  uint64_t *best = list + room, *other = best + K;                                                     // the best of before
  __shared__ uint64_t full[BS_STAGES], pushed[BS_STAGES];   // a batch has landed; every warp has read it and pushed its candidates
  __shared__ int n_sh, cnt[BS_STAGES], votes[3], wsum[BS_WARPS + 1], start;
  __shared__ volatile int abort_sh;
  __shared__ float red[BS_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rows = p.B * p.W;
  if (tid == 0) {
    for (int i = 0; i < BS_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&pushed[i], BS_WARPS);
      cnt[i] = 0;
    }
    votes[0] = votes[1] = votes[2] = 0;
    abort_sh = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  // the range: of the rows that have to be read, or, of very many, of all (and the others are passed over)
  const bool all = rows > BS_SCAN;
  const int per = all ? 0 : (rows + BS_THREADS + 31) / (BS_THREADS + 32), r0 = min(rows, tid * per), r1 = min(rows, r0 + per);
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += row_live(p, r);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
  int live = 0, first = upto - mine;
  for (int w = 0; w <= BS_WARPS; ++w) {
    if (w < warp) first += wsum[w];
    live += wsum[w];
  }
  if (all) live = rows;
  const int64_t T = (int64_t)live * p.nb;
  // no more ranges than batches, so that each of them has some
  int ranges = (int)min((int64_t)gridDim.x, T);
  // Rows in whole numbers of ranges where that makes a range no more than a batch and a half longer: a range with two pieces has
  // two starts and two ends.  (64 rows of 26 batches 20.9 -> 17.2 us, 400 of 7 23.1 -> 21.7; 256 of 7, a batch and three quarters
  // a CTA more, would go from 19.1 to 20.9.)
  if (live > 0 && live <= ranges) {
    const int whole = ranges - ranges % live;
    if (2 * (ranges - whole) * T <= (int64_t)3 * ranges * whole) ranges = whole;
  }
  if ((int)blockIdx.x >= ranges) return;
  const Ranges cuts{T, ranges};
  const int64_t x0 = cuts.first(blockIdx.x), x1 = cuts.first(blockIdx.x + 1);
  const int place0 = (int)quotient(x0, p.nb);
  if (!all && first <= place0 && place0 < first + mine) {
    int r = r0, k = first;
    for (;; ++r)
      if (row_live(p, r) && k++ == place0) break;
    start = r;
  }
  __syncthreads();
  RowWalk walk{all ? place0 : start, (int)(x0 - (int64_t)place0 * p.nb), place0, x1 - x0};
  int row, b0, b1;
  int64_t place;
  if (warp == BS_WARPS) {   // ------------------------------------------------ producer
    if (VEC && lane == 0) {
      int j = 0;
      bool ok = true;
      while (ok && next_row_piece(p, walk, all, row, b0, b1, place)) {
        if (all && !row_live(p, row)) continue;
        const float* z = p.z + (int64_t)row * p.ld;
        for (int b = b0; b < b1; ++b, ++j) {
          const int st = j % BS_STAGES, e = b * BS_BATCH;
          ok = j < BS_STAGES || mbar_wait(&pushed[st], (j / BS_STAGES - 1) & 1, &abort_sh, p.status);
          if (!ok) break;
          uint32_t bytes = (min(e + BS_BATCH, p.V) - e) / 4 * 16;   // whole vectors; up to three logits behind them are read directly
          if (!in_extent((int64_t)row * p.ld + e, min(BS_BATCH, p.V - e), (int64_t)(rows - 1) * p.ld + p.V)) bytes = 0;
          mbar_arrive_expect_tx(&full[st], bytes);
          if (bytes)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(ring + st * BS_BATCH)), "l"(reinterpret_cast<uint64_t>(z + e)), "r"(bytes), "r"(smem_u32(&full[st]))
                         : "memory");
        }
      }
      int no_abort = 0;   // a CTA that gives up does not leave while its copies are on their way
      for (int k = max(0, j - BS_STAGES); k < j; ++k) mbar_wait(&full[k % BS_STAGES], (k / BS_STAGES) & 1, &no_abort, p.status);
    }
    return;
  }
  // The takers' warps meet at one_gave_up alone: false from meet, and from what calls it, ends all of them.  A warp of which a
  // lane's wait ran out goes there with give_up.
  auto meet = []() -> bool { return !one_gave_up<1, BS_THREADS>(false); };
  auto give_up = []() -> bool { one_gave_up<1, BS_THREADS>(true); return false; };
  int n_votes = 0;
  // The takers for which v holds.  Count i is votes[i % 3]; the next one's is cleared by the time that everyone is here.
  auto count = [&](bool v, int& c) -> bool {
    const int i = n_votes++ % 3;
    const unsigned mask = __ballot_sync(0xffffffffu, v);
    if (tid == 0) votes[(i + 1) % 3] = 0;
    if (lane == 0 && mask) atomicAdd(&votes[i], __popc(mask));
    if (!meet()) return false;
    c = votes[i];
    return true;
  };
  int j = 0;   // batches of this CTA so far
  while (next_row_piece(p, walk, all, row, b0, b1, place)) {
    if (all && !row_live(p, row)) continue;
    const float* z = p.z + (int64_t)row * p.ld;
    // token k of this thread in batch b
    auto token = [&](int b, int k) { return b * BS_BATCH + (VEC ? (k / 4) * BS_THREADS * 4 + tid * 4 + k % 4 : k * BS_THREADS + tid); };
    auto load = [&](int b, float (&x)[BS_PER]) {   // from global memory
#pragma unroll
      for (int k = 0; k < BS_PER; ++k) x[k] = token(b, k) < p.V ? __ldg(z + token(b, k)) : -INFINITY;
    };
    uint64_t floor = 0;        // the piece's K-th best so far: what does not beat it is no candidate
    float bar = -INFINITY;     // its logit; a later equal one has the higher token, so only larger ones count
    int n = 0, have = 0;       // candidates that wait, best ones of before (none or K)
    float x[BS_PER], four[BS_PER / 4];   // a batch's logits, the largest of each four
    // batch b, the CTA's j-th: its logits into x, its sums to memory; *top gets this thread's largest
    auto take = [&](int b, float* top) -> bool {
      const int st = j % BS_STAGES;
      if (!VEC) {
        load(b, x);
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (j / BS_STAGES) & 1, &abort_sh, p.status))) return give_up();
        const float4* v = reinterpret_cast<const float4*>(ring + st * BS_BATCH) + tid;
#pragma unroll
        for (int k = 0; k < BS_PER; k += 4) {
          const float4 w = v[k / 4 * BS_THREADS];
          x[k] = w.x; x[k + 1] = w.y; x[k + 2] = w.z; x[k + 3] = w.w;
        }
        if ((b + 1) * BS_BATCH > p.V) {   // the last one: nothing behind the row's end, and the logits behind the last whole vector
#pragma unroll
          for (int k = 0; k < BS_PER; ++k) {
            const int i = token(b, k);
            if (i >= p.V) x[k] = -INFINITY;
            else if (i >= (p.V & ~3)) x[k] = __ldg(z + i);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < BS_PER; k += 4) four[k / 4] = fmaxf(max3(x[k], x[k + 1], x[k + 2]), x[k + 3]);
      float t = four[0];
#pragma unroll
      for (int k = 1; k < BS_PER / 4; ++k) t = fmaxf(t, four[k]);
      *top = t;
      float m;
      asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(t));
      float sum = 0.f;
      if (m > -INFINITY) {
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int k = 0; k < BS_PER; k += 2) acc[k / 2 % 2] = add2(acc[k / 2 % 2], exp_from2(x[k], x[k + 1], m));
        sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      const int64_t at = ((int64_t)row * p.nb + b) * BS_WARPS + warp;
      if (lane == 0 && in_extent(at, 1, (int64_t)rows * p.nb * BS_WARPS)) p.stat[at] = make_float2(m, sum);
      return true;
    };
    // How many of the best and of those that wait are above a key.
    auto above = [&](uint64_t key) {
      int rank = 0;
      for (int c = 0; c < have; ++c) rank += best[c] > key;
      for (int c = 0; c < n; ++c) rank += list[c] > key;
      return rank;
    };
    // the K best anew, in order; K candidates without a bar are enough for one
    auto cut = [&]() -> bool {
      if (n > bs_slack(K) || (have + n >= K && !floor)) {
        for (int i = tid; i < have + n; i += BS_THREADS) {
          const uint64_t key = i < have ? best[i] : list[i - have];
          const int rank = above(key);
          if (rank < K) other[rank] = key;
        }
        if (!meet()) return false;
        uint64_t* t = best;   // (there are K: bs_slack is no less)
        best = other;
        other = t;
        have = K;
        n = 0;
        floor = best[K - 1];
        bar = key_logit(floor);
      }
      return true;
    };
    // A logit of batch b again, for the few that are looked at twice.
    auto again = [&](int b, int k) { return token(b, k) < p.V ? __ldg(z + token(b, k)) : -INFINITY; };
    // No room for what is above the bar in batch b (one warp's logits, equal ones, rising rows): a higher bar that the
    // bests of K threads reach, by bisection on the keys, which differ.  At least K logits reach it, and at most BS_PER of
    // each of those threads.
    auto squeeze = [&](int b) -> bool {
      uint64_t mine = 0, lo = 1, hi = ~0ull;
      int c;
#pragma unroll 1
      for (int k = 0; k < BS_PER; ++k) {
        const float v = again(b, k);
        const uint64_t key = v > bar ? cand_key(v, token(b, k)) : 0;
        mine = key > mine ? key : mine;
      }
      if (!count(mine >= lo, c)) return false;
      if (c > K)
        while (hi - lo > 1) {
          const uint64_t mid = lo + (hi - lo) / 2;
          if (!count(mine >= mid, c)) return false;
          if (c >= K) {
            lo = mid;
            if (c == K) break;
          } else {
            hi = mid;
          }
        }
      if (tid == 0) n_sh = n;
      if (!meet()) return false;
      if (mine >= lo)
#pragma unroll 1
        for (int k = 0; k < BS_PER; ++k) {
          const float v = again(b, k);
          const uint64_t key = v > bar ? cand_key(v, token(b, k)) : 0;
          if (key >= lo) {
            const int at = atomicAdd(&n_sh, 1);
            if (at < room) list[at] = key;
          }
        }
      if (!meet()) return false;
      n = min(n_sh, room);
      return true;
    };
    // What counts(logit) says of batch b, the CTA's j-th, to the list: the fours that have some are looked at again where
    // they lie (a loop, since a kernel this short pays for the code that it runs through once).
    auto push = [&](int b, auto counts) {
      int* counter = &cnt[j % BS_STAGES];
      unsigned fours = 0;
#pragma unroll
      for (int g = 0; g < BS_PER / 4; ++g) fours |= counts(four[g]) ? 1u << g : 0u;
      const bool whole = VEC && (b + 1) * BS_BATCH <= p.V;
#pragma unroll 1
      for (; fours; fours &= fours - 1) {
        const int k = 4 * (__ffs(fours) - 1);
        float4 v;
        if (whole) v = reinterpret_cast<const float4*>(ring + j % BS_STAGES * BS_BATCH)[k / 4 * BS_THREADS + tid];
        else v = make_float4(again(b, k), again(b, k + 1), again(b, k + 2), again(b, k + 3));
        const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (counts(w[c])) {
            const int at = n + atomicAdd(counter, 1);
            if (at < room) list[at] = cand_key(w[c], token(b, k + c));
          }
      }
    };
    {  // the first batch: in each warp the bests of at least ceil(K / 8) threads reach its own n-th, so at least K logits
       // reach the least of these
      float top;
      if (!take(b0, &top)) return;
      const float w = warp_nth(top, (K + BS_WARPS - 1) / BS_WARPS);
      if (lane == 0) red[warp] = w;
      if (!meet()) return;
      if (tid == 0) cnt[(j + BS_STAGES - 1) % BS_STAGES] = 0;
      float least = red[0];
#pragma unroll
      for (int i = 1; i < BS_WARPS; ++i) least = fminf(least, red[i]);
      if (top >= least) push(b0, [&](float v) { return v >= least && v > -INFINITY; });
      if (!meet()) return;
      if (lane == 0) mbar_arrive(&pushed[j % BS_STAGES]);
      const int c = cnt[j % BS_STAGES];
      if (c <= room) n = c;
      else if (!squeeze(b0)) return;
      if (!cut()) return;
      ++j;
    }
    // The others push what beats the bar and go on; the list is looked at when the next batch has been summed up, so that the
    // warps need not wait for one another.  The CTA's batch i counts in cnt[i % BS_STAGES].
    auto settle = [&](int i, int b) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(&pushed[i % BS_STAGES], (i / BS_STAGES) & 1, &abort_sh, p.status))) return give_up();
      const int c = cnt[i % BS_STAGES];
      if (tid == 0) cnt[(i + BS_STAGES - 1) % BS_STAGES] = 0;      // batch i - 1's, which everyone has read
      if (n + c <= room) n += c;
      else if (!squeeze(b)) return false;
      return cut();
    };
    for (int b = b0 + 1; b < b1; ++b, ++j) {
      float top;
      if (!take(b, &top)) return;
      if (b > b0 + 1 && !settle(j - 1, b - 1)) return;
      if (top > bar) push(b, [&](float v) { return v > bar; });
      __syncwarp();
      if (lane == 0) mbar_arrive(&pushed[j % BS_STAGES]);
    }
    if (b1 > b0 + 1 && !settle(j - 1, b1 - 1)) return;
    // the piece's list in order
    const int64_t slot = place + blockIdx.x;
    const bool in = in_extent(slot, 1, p.n_lists);
    for (int i = tid; i < have + n; i += BS_THREADS) {
      const uint64_t key = i < have ? best[i] : list[i - have];
      const int rank = above(key);
      if (rank < K && in) p.keys[slot * K + rank] = key;
    }
    for (int i = have + n + tid; i < K; i += BS_THREADS)
      if (in) p.keys[slot * K + i] = 0;
    if (b0 == 0 && tid == 0) {   // the row's first piece says how many there are
      const int last = cuts.with((place + 1) * p.nb - 1);
      if (in_extent(row, 1, rows)) p.pieces[row] = RowPieces{(int)slot, last - (int)blockIdx.x + 1};
    }
  }
  meet();
}

// Joins a request's rows: each piece's list is in order, so a candidate below the n_out-th best of the lists' heads is none
// of the n_out best; the others are ranked against each other.  One CTA per request, a chain of loads and block barriers: 10.8 us
// cold for 48 requests of 8 beams and 16 kept.  The candidates that the bar leaves are ranked each against all: for 32 beams and 64
// kept a bar from 64 entries instead of four times n_out left 3000 of them (324 us in all against 85).
constexpr int BM_MOST = BS_MAX_K * BS_MAX_K;   // candidates at most: the bar leaves n_out of n_out lists, or of fewer all
constexpr int BM_LISTS = (int)kBeamMaxW + BS_CTAS_PER_SM * 256;   // of a request, at most (256: kMaxSms)
constexpr int BM_LEAD = 64;
constexpr int BM_LOADS = 8;   // of a lane at a time
constexpr int BM_SMEM = BM_MOST * (int)(2 * sizeof(int64_t) + sizeof(int)) + BM_LISTS * (int)(sizeof(int64_t) + sizeof(uint16_t) + 1);

// Doubles as integers that order as they do.
__device__ __forceinline__ int64_t ordered(double s) {
  const int64_t v = __double_as_longlong(s + 0.0);
  return v < 0 ? v ^ 0x7FFFFFFFFFFFFFFFll : v;
}
__device__ __forceinline__ double from_ordered(int64_t v) { return __longlong_as_double(v < 0 ? v ^ 0x7FFFFFFFFFFFFFFFll : v); }
constexpr int64_t BM_NONE = INT64_MIN;

// log s to 2^-25 for s >= 1, where a double logarithm would cost a few microseconds of this card's 64-bit units: the exponent
// times log 2, and the fp32 logarithm of what lies in [0.75, 1.5).
__device__ __forceinline__ double log_sum(float s) {
  int e = (int)(__float_as_uint(s) >> 23) - 127;
  float f = __uint_as_float((__float_as_uint(s) & 0x7FFFFFu) | 0x3F800000u);
  if (f >= 1.5f) { f *= 0.5f; ++e; }
  return (double)e * 0.6931471805599453094 + (double)logf(f);
}

__global__ void __launch_bounds__(BS_THREADS) beam_merge_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ int64_t score[];                     // [BM_MOST], their keys, each list's best, their rows, each list's row
  uint64_t* key_sh = reinterpret_cast<uint64_t*>(score + BM_MOST);
  int64_t* head_of = reinterpret_cast<int64_t*>(key_sh + BM_MOST);   // the score of a list's best
  int* place = reinterpret_cast<int*>(head_of + BM_LISTS);
  uint16_t* good = reinterpret_cast<uint16_t*>(place + BM_MOST);     // lists whose best reaches the bar
  uint8_t* row_of = reinterpret_cast<uint8_t*>(good + BM_LISTS);
  // a row's candidates score (logit - top) + offset, offset its beam's score less the log of its sum of exp(z - top)
  __shared__ double offset[kBeamMaxW], top[kBeamMaxW];
  __shared__ int64_t bar_sh;
  __shared__ int kind[kBeamMaxW], first[kBeamMaxW + 1], slot0[kBeamMaxW], n_sh[2], n_good, bar_at;   // first: list of each row, of the request's
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, K = p.K;
  // kind: 0 no candidates, 1 logits, 2 finished  (the caller's arrays were complete before the first kernel, which triggered past
  // its own wait)
  if (tid < p.W) {
    const int row = b * p.W + tid;
    const float base = p.scores[row];
    const int done = p.finished ? p.finished[row] : 0;
    kind[tid] = !(base > -INFINITY) ? 0 : done ? 2 : 1;
    offset[tid] = base;
    top[tid] = 0.0;
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  RowPieces pieces{0, 0};
  if (tid < p.W && kind[tid] == 1) pieces = p.pieces[b * p.W + tid];   // on its way while the sums are formed
  for (int w = tid >> 5; w < p.W; w += BS_WARPS) {   // a warp per row
    if (kind[w] != 1) continue;
    const float2* st = p.stat + (int64_t)(b * p.W + w) * p.nb * BS_WARPS;
    const int n = p.nb * BS_WARPS;
    float m = -INFINITY, s = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 32 * BM_LOADS) {
      float2 v[BM_LOADS];
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < BM_LOADS; ++k) {
        const int i = i0 + k * 32 + lane;
        v[k] = i < n ? st[i] : make_float2(-INFINITY, 0.f);
        top = fmaxf(top, v[k].x);
      }
      float mx;
      asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(mx) : "f"(top));
      if (mx == -INFINITY) continue;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < BM_LOADS; ++k) sum += v[k].y * exp_from(v[k].x, mx);
      join_sums(m, s, mx, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && s > 0.f) {   // (a row of -inf has no keys)
      offset[w] -= log_sum(s);
      top[w] = m;
    }
  }
  if (tid < 32) {
    // (a first kernel that gave up may have left some unwritten: whatever lies there, no list is looked for where none is)
    const bool there = pieces.slot >= 0 && pieces.n >= 0 && (int64_t)pieces.slot + pieces.n <= p.n_lists;
    const int n = lane >= p.W ? 0 : kind[lane] == 1 ? (there ? pieces.n : 0) : kind[lane] == 2;
    if (lane < p.W) slot0[lane] = pieces.slot;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    first[lane + 1] = __shfl_sync(0xffffffffu, x, 31) <= BM_LISTS ? x : 0;
    if (lane == 0) { first[0] = 0; n_sh[0] = n_sh[1] = n_good = 0; bar_sh = BM_NONE; bar_at = INT_MAX; }
  }
  __syncthreads();
  const int lists = first[p.W];
  for (int w = 0; w < p.W; ++w)
    for (int l = first[w] + tid; l < first[w + 1]; l += BS_THREADS) row_of[l] = (uint8_t)w;
  auto key_of = [&](int l, int k, int w) -> uint64_t {   // entry k of list l, of row w
    return kind[w] == 1 ? p.keys[(int64_t)(slot0[w] + l - first[w]) * K + k] : k == 0 ? cand_key(0.f, p.pad) : 0;
  };
  __syncthreads();
  // First the lists' leading entries, some four times n_out in all: their n_out-th best is a bar.  Then what reaches it, of all
  // entries.  (One loop for both: a kernel this short pays for the code that it runs through once.)
  const int lead = lists ? min(K, max((K + lists - 1) / lists, max(BM_LEAD, 4 * K) / lists)) : 0;   // of each list
  const int64_t out = (int64_t)b * K;
  const bool in = in_extent(out, K, (int64_t)p.B * K);
  int n = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t bar = bar_sh;
    const int at_bar = bar_at, of_each = pass ? K : lead;
    const uint64_t bar_key = at_bar == INT_MAX ? 0 : key_sh[at_bar];
    const int bar_row = at_bar == INT_MAX ? 0 : place[at_bar];
    __syncthreads();   // (the bar is read before the candidates are written again)
    const bool many = pass && lists * K > BS_THREADS;   // then only lists whose best reaches the bar are walked through
    if (many) {
      for (int l = tid; l < lists; l += BS_THREADS)
        if (head_of[l] >= bar) good[atomicAdd(&n_good, 1)] = (uint16_t)l;
      __syncthreads();
    }
    const int total = (many ? n_good : lists) * of_each;
#pragma unroll 1
    for (int i = tid; i < total; i += BS_THREADS) {
      const int at = i / of_each, k = i - at * of_each, l = many ? good[at] : at, w = row_of[l];
      if (pass && head_of[l] < bar) continue;
      const uint64_t key = key_of(l, k, w);
      const double s = key ? ((double)key_logit(key) - top[w]) + offset[w] : -INFINITY;
      const int64_t o = s > -INFINITY ? ordered(s) : BM_NONE;
      if (!pass && k == 0) head_of[l] = o;
      if (o == BM_NONE) continue;
      // equal scores: the lower beam; within a beam the logits decide, whatever the score's size leaves of them
      if (o > bar || at_bar == INT_MAX || (o == bar && (w < bar_row || (w == bar_row && key >= bar_key)))) {
        const int at = atomicAdd(&n_sh[pass], 1);
        if (at < BM_MOST) { score[at] = o; key_sh[at] = key; place[at] = w; }
      }
    }
    __syncthreads();
    n = min(n_sh[pass], BM_MOST);
#pragma unroll 1
    for (int i = tid; i < n; i += BS_THREADS) {
      const int64_t s = score[i];
      const uint64_t key = key_sh[i];
      const int w = place[i];
      int rank = 0, same = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const int64_t o = score[j];
        rank += o > s;
        same += o == s;
      }
      if (same > 1)
        for (int j = 0; j < n; ++j)
          if (score[j] == s) rank += place[j] < w || (place[j] == w && key_sh[j] > key);
      if (pass == 0) {
        if (rank == K - 1) { bar_sh = s; bar_at = i; }
      } else if (rank < K && in) {
        p.parents[out + rank] = w;
        p.tokens[out + rank] = key_token(key);
        p.out[out + rank] = (float)from_ordered(s);
      }
    }
    __syncthreads();
  }
  for (int i = n + tid; i < K; i += BS_THREADS)
    if (in) { p.parents[out + i] = -1; p.tokens[out + i] = -1; p.out[out + i] = -INFINITY; }
}

// CTAs of the first kernel, at most
int64_t select_grid(int64_t rows, int64_t nb, int64_t ctas) {
  return std::max<int64_t>(1, std::min({ctas, rows * nb, rows * (int64_t)BS_MAX_PIECES}));
}

// --------------------------------------------------------------------------------------- reorder
constexpr int BR_THREADS = 256;
constexpr int BR_MAX_W = (int)kBeamMaxW;
constexpr int BR_MAX_POOLS = kBeamMaxPools;
constexpr int BR_CTAS_PER_SM = 3;
constexpr int BR_CTA_VECS = 4096;    // 16-byte vectors that a CTA copies, where there are enough CTAs
constexpr int BR_BULK_MIN = 512;     // of a CTA's range from which its long runs go by bulk copies
constexpr int BR_LONG = 256;         // vectors of a long run, at least
constexpr int BR_CHUNK = 1024;       // vectors of a bulk copy
constexpr int BR_SLOTS = 3;          // chunks in shared memory,
constexpr int BR_LAG = 1;            // of which so many more are on their way in when one goes out

struct BeamPool {
  char* base;
  int64_t layer_bytes, page_bytes;   // n_pages pages; parts * 128 * row_bytes
  int parts, row_bytes, runs;        // runs = n_layers * parts pieces of a page's copy
};

struct BeamCopy { int src, rows, beam, column; };   // the open page, its rows, the new beam's table entry
struct BeamFound { int copies, dead; int64_t vecs; };   // of a request; vecs: 16-byte vectors that its copies take

struct ReorderParams {
  const int *parents, *n_cached, *table, *free_pages;
  int *n_cached_out, *table_out, *freed, *counts;
  int B, W, n_free, n_pages;
  int64_t max_pages, freed_room;
  BeamFound* found;   // [B]
  BeamCopy* copies;   // [B, W]
  int* dead;          // [B, W max_pages]
  BeamPool pool[BR_MAX_POOLS];
  int n_pools;
  unsigned* status;
};

// 16-byte vectors of `rows` rows of a page in one run of a pool, and in all of it.
__device__ __forceinline__ int run_vecs(const BeamPool& q, int rows) { return (rows * q.row_bytes + 15) / 16; }

// One request per CTA: its new table rows, the copies its new beams need, and its dead pages in order.  A thread takes one
// entry of the table, (column, beam) in that order; the latency of three dependent loads is what it costs, 6.8 us cold.
__global__ void __launch_bounds__(BR_THREADS) beam_plan_kernel(const __grid_constant__ ReorderParams p, int beams_pow2) {
  __shared__ int n[BR_MAX_W], par[BR_MAX_W], tile[BR_THREADS], wsum[BR_THREADS / 32];
  __shared__ int n_copy_sh;
  __shared__ int64_t vecs_sh;
  const int b = blockIdx.x, W = p.W, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t P = p.max_pages;
  pdl_wait();
  pdl_trigger();
  const int* old = p.table + (int64_t)b * W * P;
  int* out = p.table_out + (int64_t)b * W * P;
  bool bad = false;
  if (tid < BR_MAX_W) {
    int c = 0, q = -1;
    if (tid < W) {
      c = p.n_cached[b * W + tid];
      q = p.parents[b * W + tid];
      if (c < 0 || c > P * 128) { bad = true; c = 0; }
      if (q < -1 || q >= W) { bad = true; q = -1; }
    }
    n[tid] = c;
    par[tid] = q;
  }
  __syncthreads();
  unsigned kept = 0;
  int most = 0;
  for (int w = 0; w < W; ++w) {
    if (par[w] >= 0) kept |= 1u << par[w];
    most = max(most, (n[w] + 127) / 128);
  }
  if (warp == 0) {
    // open pages that an earlier new beam already ends in
    const int q = par[lane], mine = q >= 0 ? n[q] : 0;   // positions of the new beam
    const bool open = mine % 128 != 0;
    int page = open ? old[(int64_t)q * P + mine / 128] : 0;
    bool copy = false;
    for (int w = 0; w < W; ++w) {
      const int other = __shfl_sync(0xffffffffu, page, w);
      const bool o2 = __shfl_sync(0xffffffffu, (int)open, w);
      if (open && o2 && w < lane && other == page) copy = true;
    }
    if (open && (page < 0 || page >= p.n_pages)) { bad = true; page = -1; }
    const unsigned copies = __ballot_sync(0xffffffffu, copy);
    int64_t vecs = 0;
    if (copy) {
      BeamCopy c;
      c.src = page;
      c.rows = mine % 128;
      c.beam = lane;
      c.column = mine / 128;
      for (int k = 0; k < p.n_pools; ++k) vecs += (int64_t)p.pool[k].runs * run_vecs(p.pool[k], c.rows);
      const int64_t at = (int64_t)b * W + __popc(copies & ((1u << lane) - 1));
      if (in_extent(at, 1, (int64_t)p.B * W)) p.copies[at] = c;
    }
    if (lane < W && in_extent(b * W + lane, 1, (int64_t)p.B * W)) p.n_cached_out[b * W + lane] = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) vecs += __shfl_xor_sync(0xffffffffu, vecs, o);
    if (lane == 0) { n_copy_sh = __popc(copies); vecs_sh = vecs; }
  }
  const int w = tid % beams_pow2, cols = BR_THREADS / beams_pow2, col0 = tid - w;   // entries of this column: tile[col0 ..]
  int n_dead = 0;
  for (int j0 = 0; j0 < most; j0 += cols) {
    const int j = j0 + tid / beams_pow2;
    const bool held = w < W && j * 128 < n[w];
    const int page = held ? old[w * P + j] : -1;
    tile[tid] = page;
    __syncthreads();       // (behind it the column may be overwritten: the new rows may be written in place)
    bool dead = held;
    if (held && (page < 0 || page >= p.n_pages)) { bad = true; dead = false; }
    if (dead && ((kept >> w) & 1)) dead = false;
    for (int v = 0; dead && v < W; ++v)   // held by a beam that is kept, or listed for a lower one
      if (v != w && tile[col0 + v] == page && (v < w || ((kept >> v) & 1))) dead = false;
    if (w < W && par[w] >= 0 && j * 128 < n[par[w]] && in_extent((int64_t)(b * W + w) * P + j, 1, (int64_t)p.B * W * P))
      out[w * P + j] = tile[col0 + par[w]];
    const unsigned mask = __ballot_sync(0xffffffffu, dead);
    if (lane == 0) wsum[warp] = __popc(mask);
    __syncthreads();
    int at = n_dead + __popc(mask & ((1u << lane) - 1));
    for (int v = 0; v < BR_THREADS / 32; ++v) {
      if (v < warp) at += wsum[v];
      n_dead += wsum[v];
    }
    if (dead && in_extent((int64_t)b * W * P + at, 1, (int64_t)p.B * W * P)) p.dead[(int64_t)b * W * P + at] = page;
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0 && in_extent(b, 1, p.B)) p.found[b] = BeamFound{n_copy_sh, n_dead, vecs_sh};
  if (bad) atomicOr(p.status, STATUS_BAD_PLAN);
}

// Where copy i of request b goes: a dead page of its own, then a free one; -1 if there is none or the source is none.
__device__ __forceinline__ int copy_target(const ReorderParams& p, int b, int i, int n_dead, int first_taken, int src) {
  int dst = -1;
  if (i < n_dead) dst = p.dead[(int64_t)b * p.W * p.max_pages + i];
  else if (first_taken + i - n_dead < p.n_free) dst = p.free_pages[first_taken + i - n_dead];
  return src >= 0 && dst >= 0 && dst < p.n_pages ? dst : -1;
}

// The 16 bytes at `at` of a run of `bytes`, w where they are whole, else word by word.
__device__ __forceinline__ void store_vec(const char* src, char* to, int at, int bytes, const uint4& w) {
  if (at + 16 <= bytes) *reinterpret_cast<uint4*>(to + at) = w;
  else
    for (; at < bytes; at += 4) *reinterpret_cast<uint32_t*>(to + at) = *reinterpret_cast<const uint32_t*>(src + at);
}

// Long runs by bulk copies through a ring in shared memory, all of it one thread's: chunk i comes into slot i % BR_SLOTS and goes
// out when BR_LAG later ones have been asked for.
struct BulkCopies {
  char* ring;
  uint64_t* full;
  struct Out { char* to; uint32_t bytes; } *out;
  volatile int* abort;
  unsigned* status;
  int in = 0, gone = 0;
  __device__ __forceinline__ bool store_next() {
    const int st = gone % BR_SLOTS;
    if (!mbar_wait(&full[st], (gone / BR_SLOTS) & 1, abort, status)) return false;
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(
                     reinterpret_cast<uint64_t>(out[st].to)), "r"(smem_u32(ring + st * BR_CHUNK * 16)), "r"(out[st].bytes)
                 : "memory");
    ++gone;
    return true;
  }
  __device__ __forceinline__ bool copy(const char* src, char* to, uint32_t bytes) {
    const int st = in % BR_SLOTS;
    // slot st's last chunk went out with group in - BR_SLOTS, and in - 1 - BR_LAG is the latest
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(BR_SLOTS - 1 - BR_LAG) : "memory");
    out[st] = Out{to, bytes};
    mbar_arrive_expect_tx(&full[st], bytes);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(ring + st * BR_CHUNK * 16)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(&full[st]))
                 : "memory");
    ++in;
    return in <= BR_LAG || store_next();
  }
  __device__ __forceinline__ void finish() {
    bool ok = true;
    while (ok && gone < in) ok = store_next();
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    int no_abort = 0;   // (a CTA that gives up does not leave while its copies are on their way)
    for (int k = max(0, in - BR_SLOTS); k < in; ++k) mbar_wait(&full[k % BR_SLOTS], (k / BR_SLOTS) & 1, &no_abort, status);
  }
};

// Bound by HBM for many copies, by the latency of a few dependent loads for few.  Every CTA sums up the requests' pages
// taken, pages left over and vectors to copy; entries and freed pages are dealt out by request, and the vectors of
// all copies, one after the other, are cut into equal ranges, one per CTA, where one thread drives bulk copies for the long runs
// (rows) while the other warps move the short ones (scales).  16 requests of 8 beams, eight layers of 8-bit pages of 8 heads x
// 128 (149 MB read and written): 27.6 us with the plan, 22 at a copy's rate; through registers, four loads in flight per thread,
// 34 (the next four on their way before these are stored 36, chunks in turn instead of ranges 32-49); chunks of 4 to 12 KB 28-32,
// four CTAs 29; two CTAs with a slot more 26.6, but 13.6 instead of 12.3 for 16 requests of 4 beams over four bf16 layers
// (9.8 at a copy's rate).  One request of 4 beams over two bf16 layers of 2 heads x 64: 6.5 us.
__global__ void __launch_bounds__(BR_THREADS, BR_CTAS_PER_SM) beam_copy_kernel(const __grid_constant__ ReorderParams p) {
  extern __shared__ int64_t v0[];   // [B + 1] first vector of each request; then [2][B + 1]: first page taken, first page freed
  int* t0 = reinterpret_cast<int*>(v0 + p.B + 1);
  int* f0 = t0 + p.B + 1;
  __shared__ int64_t wsum[3][BR_THREADS / 32];
  __shared__ uint64_t full[BR_SLOTS];
  __shared__ BulkCopies::Out out[BR_SLOTS];
  __shared__ volatile int abort_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < BR_SLOTS; ++i) mbar_init(&full[i], 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  pdl_wait();
  const int per = (p.B + BR_THREADS - 1) / BR_THREADS;
  const int s0 = min(p.B, tid * per), s1 = min(p.B, s0 + per);
  int64_t sum[3] = {0, 0, 0};
  for (int b = s0; b < s1; ++b) {
    const BeamFound v = p.found[b];
    sum[0] += v.vecs;
    sum[1] += max(0, v.copies - v.dead);
    sum[2] += max(0, v.dead - v.copies);
  }
  int64_t at[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int64_t x = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[k][warp] = x;
    at[k] = x - sum[k];
  }
  __syncthreads();
  int64_t all[3] = {0, 0, 0};
  for (int w = 0; w < BR_THREADS / 32; ++w)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (w < warp) at[k] += wsum[k][w];
      all[k] += wsum[k][w];
    }
  for (int b = s0; b < s1; ++b) {
    const BeamFound v = p.found[b];
    v0[b] = at[0];
    t0[b] = (int)min(at[1], (int64_t)INT_MAX);
    f0[b] = (int)min(at[2], (int64_t)INT_MAX);
    at[0] += v.vecs;
    at[1] += max(0, v.copies - v.dead);
    at[2] += max(0, v.dead - v.copies);
  }
  if (tid == 0) {
    v0[p.B] = all[0];
    if (blockIdx.x == 0 && in_extent(0, 2, 2)) {
      p.counts[0] = (int)min(all[1], (int64_t)INT_MAX);
      p.counts[1] = (int)min(all[2], (int64_t)INT_MAX);
      if (all[1] > p.n_free || all[2] > p.freed_room) atomicOr(p.status, STATUS_BAD_PLAN);
    }
  }
  __syncthreads();
  // this CTA's range of vectors
  int64_t x = (int64_t)blockIdx.x * all[0] / gridDim.x;
  const int64_t x1 = (int64_t)(blockIdx.x + 1) * all[0] / gridDim.x;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {   // the last request whose first vector is not behind x
    const int mid = (lo + hi) >> 1;
    if (v0[mid] <= x) lo = mid; else hi = mid;
  }
  // part(q, src, to, nv, bytes, from, n): vectors [from, n) of a copy's runs of nv vectors, `bytes` bytes, in pool q
  auto walk = [&](auto part) {
    int64_t first = v0[lo];   // of copy i's vectors in pool k
    for (int b = lo, i = 0; x < x1;) {
      const BeamFound f = p.found[b];
      if (i == f.copies) { ++b; i = 0; continue; }
      const BeamCopy c = p.copies[(int64_t)b * p.W + i];
      const int dst = copy_target(p, b, i, f.dead, t0[b], c.src);
      for (int k = 0; k < p.n_pools && x < x1; ++k) {
        const BeamPool& q = p.pool[k];
        const int nv = run_vecs(q, c.rows), bytes = c.rows * q.row_bytes;
        const int64_t total = (int64_t)q.runs * nv;
        if (x < first + total) {
          const int v_from = (int)(x - first), v_to = (int)min(total, x1 - first);
          // (a layer holds both pages whole; the last row that is written lies in the last run)
          if (dst >= 0 && in_extent((int64_t)dst * q.page_bytes, q.page_bytes, q.layer_bytes) &&
              in_extent((int64_t)(q.parts - 1) * 128 * q.row_bytes, bytes, q.page_bytes))
            part(q, q.base + (int64_t)c.src * q.page_bytes, q.base + (int64_t)dst * q.page_bytes, nv, bytes, v_from, v_to);
          x = first + v_to;
        }
        first += total;
      }
      ++i;
    }
  };
  const bool bulk = x1 - x >= BR_BULK_MIN;   // then warp 0 has the long runs and the others the rest
  if (bulk && warp == 0) {
    if (lane == 0) {
      BulkCopies copier{reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(f0 + p.B + 1) + 127) & ~uintptr_t(127)), full, out, &abort_sh, p.status};
      bool ok = true;
      walk([&](const BeamPool& q, const char* src, char* to, int nv, int bytes, int v, int v_to) {
        if (nv < BR_LONG) return;
        int run = v / nv, r0 = v - run * nv, layer = run / q.parts, part = run - layer * q.parts;
        while (ok && v < v_to) {
          const int64_t o = layer * q.layer_bytes + (int64_t)part * 128 * q.row_bytes;
          const int r1 = min(min(nv, r0 + BR_CHUNK), r0 + v_to - v), whole = min(r1, bytes / 16);
          if (whole > r0) ok = copier.copy(src + o + (int64_t)r0 * 16, to + o + (int64_t)r0 * 16, (whole - r0) * 16);
          if (whole < r1) store_vec(src + o, to + o, whole * 16, bytes, make_uint4(0, 0, 0, 0));   // the words behind the last whole vector
          v += r1 - r0;
          r0 = r1;
          if (r0 == nv) {
            r0 = 0;
            if (++part == q.parts) { part = 0; ++layer; }
          }
        }
      });
      copier.finish();
    }
  } else {
    const int t = bulk ? tid - 32 : tid, n = bulk ? BR_THREADS - 32 : BR_THREADS;
    walk([&](const BeamPool& q, const char* src, char* to, int nv, int bytes, int v_from, int v_to) {
      if (bulk && nv >= BR_LONG) return;
      for (int v = v_from + t; v < v_to; v += n) {
        const int run = v / nv, layer = run / q.parts, part = run - layer * q.parts, r = (v - run * nv) * 16;
        const int64_t o = layer * q.layer_bytes + (int64_t)part * 128 * q.row_bytes;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r + 16 <= bytes) w = *reinterpret_cast<const uint4*>(src + o + r);
        store_vec(src + o, to + o, r, bytes, w);
      }
    });
  }
  // entries of the copies, and the dead pages left over
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const BeamFound v = p.found[b];
    if (tid < v.copies) {
      const BeamCopy c = p.copies[(int64_t)b * p.W + tid];
      const int dst = copy_target(p, b, tid, v.dead, t0[b], c.src);
      if (c.src >= 0 && dst < 0) atomicOr(p.status, STATUS_BAD_PLAN);
      const int64_t e = ((int64_t)b * p.W + c.beam) * p.max_pages + c.column;
      if (in_extent(e, 1, (int64_t)p.B * p.W * p.max_pages)) p.table_out[e] = dst;
    }
    for (int i = tid; i < v.dead - v.copies; i += BR_THREADS)
      if ((int64_t)f0[b] + i < p.freed_room && in_extent(f0[b], 1, p.freed_room)) p.freed[f0[b] + i] = p.dead[(int64_t)b * p.W * p.max_pages + v.copies + i];
  }
}

}  // namespace

bool beam_select_supported(int64_t B, int64_t W) { return W <= kBeamMaxW && B < ((int64_t)1 << 22) && B * W < ((int64_t)1 << 22); }
constexpr int kMaxSms = 256;   // sizes the workspace, so that it does not depend on the device
static_assert(BM_LISTS >= (int)kBeamMaxW + BS_CTAS_PER_SM * kMaxSms, "a request's lists");
struct SelectWs { size_t pieces, stat, total; int64_t lists; };
SelectWs select_ws(int64_t rows, int64_t V) {
  const int64_t nb = (V + BS_BATCH - 1) / BS_BATCH;
  SelectWs w;
  w.lists = rows + select_grid(rows, nb, BS_CTAS_PER_SM * kMaxSms);
  w.pieces = round256((size_t)w.lists * BS_MAX_K * sizeof(uint64_t));
  w.stat = w.pieces + round256((size_t)rows * sizeof(RowPieces));
  w.total = w.stat + round256((size_t)rows * nb * BS_WARPS * sizeof(float2));
  return w;
}
size_t beam_select_ws_bytes(int64_t B, int64_t W, int64_t V) { return select_ws(B * W, V).total; }

int launch_beam_select(const BeamSelectDesc& d, int num_sms, unsigned* status, cudaStream_t st) {
  SelectParams p;
  const SelectWs ws = select_ws(d.B * d.W, d.V);
  p.z = d.logits; p.ld = d.ld;
  p.B = (int)d.B; p.W = (int)d.W; p.V = (int)d.V; p.K = (int)d.n_out;
  p.nb = (int)((d.V + BS_BATCH - 1) / BS_BATCH);
  p.scores = d.scores; p.finished = d.finished; p.pad = d.pad_token;
  p.parents = d.parents; p.tokens = d.tokens; p.out = d.out_scores;
  p.keys = static_cast<uint64_t*>(d.ws);
  p.pieces = reinterpret_cast<RowPieces*>(static_cast<char*>(d.ws) + ws.pieces);
  p.stat = reinterpret_cast<float2*>(static_cast<char*>(d.ws) + ws.stat);
  p.n_lists = ws.lists;
  p.status = status;
  const bool vec = ((reinterpret_cast<uintptr_t>(d.logits) | (uintptr_t)(d.ld * 4)) & 15) == 0;
  const int smem = bs_smem(p.K, vec), fit = std::min(BS_CTAS_PER_SM, 233472 / (smem + 2048));   // (2 KB: static and the system's)
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return -1;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BM_SMEM) != cudaSuccess ||
        cudaFuncSetAttribute(beam_part_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bs_smem(BS_MAX_K, true)) != cudaSuccess ||
        cudaFuncSetAttribute(beam_part_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bs_smem(BS_MAX_K, false)) != cudaSuccess)
      return -1;
    attr_set[dev] = true;
  }
  const unsigned grid = (unsigned)select_grid(d.B * d.W, p.nb, fit * std::min(num_sms, kMaxSms));
  const dim3 threads(BS_THREADS + 32);
  if ((vec ? launch_after(beam_part_kernel<true>, dim3(grid), threads, smem, st, p)
           : launch_after(beam_part_kernel<false>, dim3(grid), threads, smem, st, p)) != cudaSuccess)
    return -1;
  return launch_after(beam_merge_kernel, dim3((unsigned)d.B), dim3(BS_THREADS), BM_SMEM, st, p) == cudaSuccess ? 0 : -1;
}

size_t beam_reorder_ws_bytes(int64_t B, int64_t W, int64_t max_pages) {
  return round256((size_t)B * sizeof(BeamFound)) + round256((size_t)(B * W) * sizeof(BeamCopy)) +
         round256((size_t)(B * W) * max_pages * sizeof(int));
}

int launch_beam_reorder(const BeamReorderDesc& d, int num_sms, unsigned* status, cudaStream_t st) {
  ReorderParams p;
  memset(&p, 0, sizeof(p));
  p.parents = d.parents; p.n_cached = d.n_cached; p.table = d.table; p.free_pages = d.free_pages;
  p.n_cached_out = d.n_cached_out; p.table_out = d.table_out; p.freed = d.freed; p.counts = d.counts;
  p.B = (int)d.B; p.W = (int)d.W; p.n_free = (int)d.n_free; p.n_pages = (int)d.n_pages;
  p.max_pages = d.max_pages; p.freed_room = d.freed_room;
  char* ws = static_cast<char*>(d.ws);
  p.found = reinterpret_cast<BeamFound*>(ws);
  ws += round256((size_t)d.B * sizeof(BeamFound));
  p.copies = reinterpret_cast<BeamCopy*>(ws);
  ws += round256((size_t)(d.B * d.W) * sizeof(BeamCopy));
  p.dead = reinterpret_cast<int*>(ws);
  p.n_pools = d.n_pools;
  int64_t vecs = 0;
  for (int k = 0; k < d.n_pools; ++k) {
    BeamPool& q = p.pool[k];
    q.base = static_cast<char*>(d.pools[k].base);
    q.parts = (int)d.pools[k].parts;
    q.row_bytes = (int)d.pools[k].row_bytes;
    q.runs = (int)(d.pools[k].n_layers * d.pools[k].parts);
    q.page_bytes = d.pools[k].parts * 128 * d.pools[k].row_bytes;
    q.layer_bytes = d.n_pages * q.page_bytes;
    vecs += q.runs * (int64_t)q.row_bytes * 8;
  }
  p.status = status;
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return -1;
  auto smem = [](int64_t B) { return (int)((B + 1) * (sizeof(int64_t) + 2 * sizeof(int)) + 128 + BR_SLOTS * BR_CHUNK * 16); };
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(beam_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem(kPlanMaxSeqs)) != cudaSuccess)
      return -1;
    attr_set[dev] = true;
  }
  if (d.B > 0) {
    int pow2 = 1;
    while (pow2 < d.W) pow2 *= 2;
    if (launch_after(beam_plan_kernel, dim3((unsigned)d.B), dim3(BR_THREADS), 0, st, p, pow2) != cudaSuccess) return -1;
  }
  // CTAs for a few thousand vectors each, were every beam but one of each request to copy a whole page
  const int64_t work = std::max<int64_t>(d.B, (d.B * (d.W - 1) * vecs + BR_CTA_VECS - 1) / BR_CTA_VECS);
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(BR_CTAS_PER_SM * num_sms, work));
  return launch_after(beam_copy_kernel, dim3(grid), dim3(BR_THREADS), smem(d.B), st, p) == cudaSuccess ? 0 : -1;
}

LLAMA_DEFINE_BOUNDS_READER(beam)

}  // namespace llama
