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
// HBM bound for many rows, latency for few.  A CTA reads one part of a row once, a batch of BS_BATCH logits in registers at
// a time, the next on its way.  Each thread keeps a running maximum and sum of exponentials; what beats the part's
// n_out-th best so far goes to a list in shared memory, which is cut back to the n_out best when it has grown.  All rows
// of a call are cut and summed alike, so equal rows give equal sums.  The second kernel joins a request's parts.
constexpr int BS_THREADS = 256;
constexpr int BS_WARPS = BS_THREADS / 32;
constexpr int BS_PER = 16;                              // logits of a thread in a batch
constexpr int BS_BATCH = BS_THREADS * BS_PER;
constexpr int BS_MAX_K = (int)kBeamMaxOut;
constexpr int BS_KEPT = 2 * BS_MAX_K + 64;              // entries that the list may have between batches
constexpr int BS_LIST = BS_KEPT + 2 * BS_MAX_K * BS_PER;
constexpr int BS_CTAS_PER_SM = 4;
constexpr int BS_MAX_PARTS = 32;

struct SelectParams {
  const float* z;
  int64_t ld;
  int B, W, V, K;
  int parts, part_len;
  const float* scores;
  const int* finished;
  int pad;
  int *parents, *tokens;
  float* out;
  uint64_t* keys;   // [B W, parts, K] the best tokens of a part, best first (0: none)
  float2* stat;     // [B W, parts] maximum and sum of exp(z - maximum)
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

__device__ __forceinline__ void join_sums(float& m, float& s, float m2, float s2) {
  const float mx = fmaxf(m, m2);
  if (mx > -INFINITY) s = s * __expf(m - mx) + s2 * __expf(m2 - mx);
  m = mx;
}

// VEC: rows start on 16 bytes, a thread's logits come four at a time.
template <bool VEC>
__global__ void __launch_bounds__(BS_THREADS, BS_CTAS_PER_SM) beam_part_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint64_t list[2][BS_LIST];
  __shared__ int n_sh, more_sh;
  __shared__ float red[2][BS_WARPS];
  const int row = blockIdx.x / p.parts, part = blockIdx.x % p.parts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  if ((p.finished && __ldg(p.finished + row)) || !(__ldg(p.scores + row) > -INFINITY)) return;   // nothing to read
  const float* z = p.z + (int64_t)row * p.ld;
  const int e0 = part * p.part_len, e1 = min(p.V, e0 + p.part_len), K = p.K;
  // element k of this thread in the batch that starts at e
  auto place = [&](int e, int k) { return VEC ? e + (k / 4) * BS_THREADS * 4 + tid * 4 + k % 4 : e + k * BS_THREADS + tid; };
  auto load = [&](int e, float (&x)[BS_PER]) {
#pragma unroll
    for (int k = 0; k < BS_PER; k += VEC ? 4 : 1) {
      const int i = place(e, k);
      if (VEC && i + 3 < e1) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(z + i));
        x[k] = v.x; x[k + 1] = v.y; x[k + 2] = v.z; x[k + 3] = v.w;
      } else {
#pragma unroll
        for (int c = 0; c < (VEC ? 4 : 1); ++c) x[k + c] = i + c < e1 ? __ldcs(z + i + c) : -INFINITY;
      }
    }
  };
  if (tid == 0) { n_sh = 0; more_sh = 0; }
  float m = -INFINITY, s = 0.f;
  uint64_t floor = 0;        // the part's K-th best so far: what does not beat it is no candidate
  int cur = 0, n = 0;        // the list in use and its length
  float x[BS_PER], next[BS_PER];
  load(e0, x);
  __syncthreads();
  for (int e = e0; e < e1; e += BS_BATCH) {
    if (e + BS_BATCH < e1) load(e + BS_BATCH, next);
    float top = x[0];
#pragma unroll
    for (int k = 1; k < BS_PER; ++k) top = fmaxf(top, x[k]);
    if (top > -INFINITY) {
      if (top > m) {
        s *= __expf(m - top);
        m = top;
      }
      float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < BS_PER; ++k) a[k % 4] += __expf(x[k] - m);
      s += (a[0] + a[1]) + (a[2] + a[3]);
    }
    // a later logit equal to the floor's has the higher token, so only larger ones count
    const float bar = floor ? key_logit(floor) : -INFINITY;
    if (__syncthreads_or(top > bar)) {
      int mine = 0;
      uint64_t best = 0;
#pragma unroll
      for (int k = 0; k < BS_PER; ++k) mine += x[k] > bar;
      if (mine) {
        atomicAdd(&more_sh, mine);
#pragma unroll
        for (int k = 0; k < BS_PER; ++k)
          if (x[k] > bar) {
            const uint64_t key = cand_key(x[k], place(e, k));
            best = key > best ? key : best;
          }
      }
      __syncthreads();
      uint64_t least = 1;
      if (more_sh > BS_KEPT - K) {
        // Too many: a bar that K to 2 K threads' best logits reach, by bisection on the keys.  At least K logits
        // reach it, and at most BS_PER of each of those threads.
        uint64_t hi = ~0ull;
        if (__syncthreads_count(best >= least) >= 2 * K)
          while (hi - least > 1) {
            const uint64_t mid = least + (hi - least) / 2;
            const int c = __syncthreads_count(best >= mid);
            if (c >= K) {
              least = mid;
              if (c <= 2 * K) break;
            } else {
              hi = mid;
            }
          }
      }
      if (best >= least && mine) {
#pragma unroll
        for (int k = 0; k < BS_PER; ++k)
          if (x[k] > bar) {
            const uint64_t key = cand_key(x[k], place(e, k));
            if (key >= least) {
              const int at = atomicAdd(&n_sh, 1);
              if (at < BS_LIST) list[cur][at] = key;    // (there is room, see above)
            }
          }
      }
      __syncthreads();
      n = min(n_sh, BS_LIST);
      if (n > K + 64 || (n > K && !floor)) {            // back to the K best, in order
        for (int i = tid; i < n; i += BS_THREADS) {
          const uint64_t key = list[cur][i];
          int rank = 0;
          for (int j = 0; j < n; ++j) rank += list[cur][j] > key;
          if (rank < K) list[cur ^ 1][rank] = key;
        }
        __syncthreads();
        cur ^= 1;
        n = K;
        floor = list[cur][K - 1];
      }
      if (tid == 0) { n_sh = n; more_sh = 0; }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < BS_PER; ++k) x[k] = next[k];
  }
  // the part's list in order, and its maximum and sum
  const int64_t at = (int64_t)row * p.parts + part;
  const bool in = in_extent(at, 1, (int64_t)p.B * p.W * p.parts);
  for (int i = tid; i < n; i += BS_THREADS) {
    const uint64_t key = list[cur][i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[cur][j] > key;
    if (rank < K && in) p.keys[at * K + rank] = key;
  }
  for (int i = n + tid; i < K; i += BS_THREADS)
    if (in) p.keys[at * K + i] = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join_sums(m, s, m2, s2);
  }
  if (lane == 0) { red[0][warp] = m; red[1][warp] = s; }
  __syncthreads();
  if (tid == 0 && in) {
    for (int w = 1; w < BS_WARPS; ++w) join_sums(m, s, red[0][w], red[1][w]);
    p.stat[at] = make_float2(m, s);
  }
}

// Joins the parts of a request's rows: each part's list is in order, so a candidate below the n_out-th best of the lists'
// heads is none of the n_out best; the others are ranked against each other.
constexpr int BM_MOST = BS_MAX_K * BS_MAX_K;   // candidates at most: n_out lists (or fewer lists than n_out) of n_out
constexpr int BM_SMEM = BM_MOST * (int)(sizeof(double) + sizeof(int));

__global__ void __launch_bounds__(BS_THREADS) beam_merge_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ double score[];                      // [BM_MOST], then their places
  int* place = reinterpret_cast<int*>(score + BM_MOST);
  __shared__ double lsum[kBeamMaxW], bar_sh;   // log of a row's sum of exp(z - its maximum)
  __shared__ float base_sh[kBeamMaxW], top[kBeamMaxW];
  __shared__ int kind[kBeamMaxW], n_sh, bar_at;
  const int b = blockIdx.x, tid = threadIdx.x, K = p.K, lists = p.W * p.parts;
  pdl_wait();
  // kind: 0 no candidates, 1 logits, 2 finished
  for (int w = tid; w < p.W; w += BS_THREADS) {
    const int row = b * p.W + w;
    const float base = p.scores[row];
    const bool done = p.finished && p.finished[row];
    int kd = base > -INFINITY ? (done ? 2 : 1) : 0;
    float m = -INFINITY;
    if (kd == 1) {
      for (int q = 0; q < p.parts; ++q) m = fmaxf(m, p.stat[(int64_t)row * p.parts + q].x);
      double s = 0.0;
      for (int q = 0; q < p.parts; ++q) {
        const float2 st = p.stat[(int64_t)row * p.parts + q];
        if (st.x > -INFINITY) s += (double)(st.y * expf(st.x - m));
      }
      if (m > -INFINITY) lsum[w] = log(s);
      else kd = 0;
    }
    top[w] = m;
    base_sh[w] = base;
    kind[w] = kd;
  }
  if (tid == 0) { n_sh = 0; bar_sh = -INFINITY; bar_at = INT_MAX; }
  __syncthreads();
  // candidate c: entry c % K of list c / K; its score, -inf for none
  auto value = [&](int c) -> double {
    const int l = c / K, w = l / p.parts;
    if (kind[w] == 0) return -INFINITY;
    if (kind[w] == 2) return c == w * p.parts * K ? (double)base_sh[w] : -INFINITY;
    const uint64_t key = p.keys[((int64_t)b * lists + l) * K + c % K];
    return key ? (double)base_sh[w] + (((double)key_logit(key) - (double)top[w]) - lsum[w]) : -INFINITY;
  };
  // equal scores: the lower beam; within a beam the logits decide, whatever the score's size leaves of them
  auto key_of = [&](int c) { return kind[c / K / p.parts] == 1 ? p.keys[((int64_t)b * lists + c / K) * K + c % K] : 0ull; };
  auto beats = [&](double s, int c, double s2, int c2) {
    if (s != s2) return s > s2;
    const int w = c / K / p.parts, w2 = c2 / K / p.parts;
    if (w != w2) return w < w2;
    return c != c2 && key_of(c) > key_of(c2);
  };
  if (lists >= K) {   // the K-th best head
    for (int l = tid; l < lists; l += BS_THREADS) score[l] = value(l * K);
    __syncthreads();
    for (int l = tid; l < lists; l += BS_THREADS) {
      const double s = score[l];
      if (s == -INFINITY) continue;
      int rank = 0;
      for (int j = 0; j < lists; ++j) rank += beats(score[j], j * K, s, l * K);
      if (rank == K - 1) { bar_sh = s; bar_at = l * K; }
    }
    __syncthreads();
  }
  const double bar = bar_sh;
  const int at_bar = bar_at;
  for (int c = tid; c < lists * K; c += BS_THREADS) {
    const double s = value(c);
    if (s > -INFINITY && (at_bar == INT_MAX || c == at_bar || !beats(bar, at_bar, s, c))) {
      const int i = atomicAdd(&n_sh, 1);
      if (i < BM_MOST) { score[i] = s; place[i] = c; }
    }
  }
  __syncthreads();
  const int n = min(n_sh, BM_MOST);
  const int64_t out = (int64_t)b * K;
  const bool in = in_extent(out, K, (int64_t)p.B * K);
  for (int i = tid; i < n; i += BS_THREADS) {
    const double s = score[i];
    const int c = place[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += beats(score[j], place[j], s, c);
    if (rank < K && in) {
      const int w = c / K / p.parts;
      p.parents[out + rank] = w;
      p.tokens[out + rank] = kind[w] == 2 ? p.pad : key_token(key_of(c));
      p.out[out + rank] = (float)s;
    }
  }
  for (int i = n + tid; i < K; i += BS_THREADS)
    if (in) { p.parents[out + i] = -1; p.tokens[out + i] = -1; p.out[out + i] = -INFINITY; }
}

// Parts of a row: the count at which the last wave of CTAs is fullest, parts of a batch at least, the fewest at equal waste.
int select_parts(int64_t rows, int64_t V, int sms) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(BS_MAX_PARTS, (V + BS_BATCH - 1) / BS_BATCH));
  const int64_t room = (int64_t)BS_CTAS_PER_SM * sms;
  int best = 1;
  double least = 1e300;
  for (int64_t n = 1; n <= most; ++n) {
    // waves of parts, each with what a part costs before and after its share of the row (about a batch)
    const double cost = (double)((rows * n + room - 1) / room) * ((double)V / n + BS_BATCH);
    if (cost < least) { least = cost; best = (int)n; }
  }
  return best;
}

// --------------------------------------------------------------------------------------- reorder
constexpr int BR_THREADS = 256;
constexpr int BR_MAX_W = (int)kBeamMaxW;
constexpr int BR_MAX_POOLS = kBeamMaxPools;
constexpr int BR_CTAS_PER_SM = 4;
constexpr int BR_DEEP = 4;           // loads of a thread in flight

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

// One request per CTA: its new table rows, the copies its new beams need, and its dead pages in order.
__global__ void __launch_bounds__(BR_THREADS) beam_plan_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ int n[BR_MAX_W], par[BR_MAX_W], tile[BR_MAX_W][BR_THREADS], wsum[BR_THREADS / 32];
  __shared__ unsigned kept_sh;
  __shared__ int most_sh, n_copy_sh;
  __shared__ int64_t vecs_sh;
  const int b = blockIdx.x, W = p.W, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t P = p.max_pages;
  pdl_trigger();
  const int* old = p.table + (int64_t)b * W * P;
  int* out = p.table_out + (int64_t)b * W * P;
  bool bad = false;
  if (warp == 0) {
    int c = 0, q = -1;
    if (lane < W) {
      c = p.n_cached[b * W + lane];
      q = p.parents[b * W + lane];
      if (c < 0 || c > P * 128) { bad = true; c = 0; }
      if (q < -1 || q >= W) { bad = true; q = -1; }
    }
    n[lane] = c;
    par[lane] = q;
    __syncwarp();
    int most = c, mine = q >= 0 ? n[q] : 0;   // positions of the new beam
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    unsigned kept = 0;
    for (int w = 0; w < W; ++w)
      if (par[w] >= 0) kept |= 1u << par[w];
    // open pages that an earlier new beam already ends in
    int page = -2 - lane;
    const bool open = mine % 128 != 0;
    if (open) page = old[(int64_t)q * P + mine / 128];
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
      BeamCopy c2;
      c2.src = page;
      c2.rows = mine % 128;
      c2.beam = lane;
      c2.column = mine / 128;
      for (int k = 0; k < p.n_pools; ++k) vecs += (int64_t)p.pool[k].runs * run_vecs(p.pool[k], c2.rows);
      if (in_extent((int64_t)b * W + __popc(copies & ((1u << lane) - 1)), 1, (int64_t)p.B * W))
        p.copies[(int64_t)b * W + __popc(copies & ((1u << lane) - 1))] = c2;
    }
    if (lane < W && in_extent(b * W + lane, 1, (int64_t)p.B * W)) p.n_cached_out[b * W + lane] = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) vecs += __shfl_xor_sync(0xffffffffu, vecs, o);
    if (lane == 0) { kept_sh = kept; most_sh = (most + 127) / 128; n_copy_sh = __popc(copies); vecs_sh = vecs; }
  }
  __syncthreads();
  const unsigned kept = kept_sh;
  int n_dead = 0;
  for (int j0 = 0; j0 < most_sh; j0 += BR_THREADS) {
    const int j = j0 + threadIdx.x;
    unsigned dead = 0;
    if (j < most_sh) {
      for (int w = 0; w < W; ++w) tile[w][threadIdx.x] = j * 128 < n[w] ? old[w * P + j] : -1;
      for (int w = 0; w < W; ++w) {
        if (j * 128 >= n[w]) continue;
        const int page = tile[w][threadIdx.x];
        if (page < 0 || page >= p.n_pages) { bad = true; continue; }
        bool gone = !((kept >> w) & 1);
        for (int v = 0; gone && v < W; ++v)
          if (v != w && tile[v][threadIdx.x] == page && (v < w || ((kept >> v) & 1))) gone = false;
        if (gone) dead |= 1u << w;
      }
      for (int w = 0; w < W; ++w)
        if (par[w] >= 0 && j * 128 < n[par[w]] && in_extent((int64_t)(b * W + w) * P + j, 1, (int64_t)p.B * W * P))
          out[w * P + j] = tile[par[w]][threadIdx.x];
    }
    // dead pages in the order of columns, then beams
    const int c = __popc(dead);
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = n_dead, all = 0;
    for (int w = 0; w < BR_THREADS / 32; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    int at = before + x - c;
    for (int w = 0; w < W; ++w)
      if ((dead >> w) & 1) {
        const int64_t i = (int64_t)b * W * P + at++;
        if (in_extent(i, 1, (int64_t)p.B * W * P)) p.dead[i] = tile[w][threadIdx.x];
      }
    n_dead += all;
    __syncthreads();
  }
  if (threadIdx.x == 0 && in_extent(b, 1, p.B)) p.found[b] = BeamFound{n_copy_sh, n_dead, vecs_sh};
  if (bad) atomicOr(p.status, STATUS_BAD_PLAN);
}

// Where copy i of request b goes: a dead page of its own, then a free one; -1 if there is none or the source is none.
__device__ __forceinline__ int copy_target(const ReorderParams& p, int b, int i, int n_dead, int first_taken, int src) {
  int dst = -1;
  if (i < n_dead) dst = p.dead[(int64_t)b * p.W * p.max_pages + i];
  else if (first_taken + i - n_dead < p.n_free) dst = p.free_pages[first_taken + i - n_dead];
  return src >= 0 && dst >= 0 && dst < p.n_pages ? dst : -1;
}

// Bound by HBM for many copies, by the latency of a few dependent loads for few.  Every CTA sums up the requests' pages
// taken, pages left over and vectors to copy; entries and freed pages are dealt out by request, and the vectors of
// all copies, one after the other, are cut into equal ranges, one per CTA.
__global__ void __launch_bounds__(BR_THREADS, BR_CTAS_PER_SM) beam_copy_kernel(const __grid_constant__ ReorderParams p) {
  extern __shared__ int64_t v0[];   // [B + 1] first vector of each request; then [2][B + 1]: first page taken, first page freed
  int* t0 = reinterpret_cast<int*>(v0 + p.B + 1);
  int* f0 = t0 + p.B + 1;
  __shared__ int64_t wsum[3][BR_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
      if ((int64_t)f0[b] + i < p.freed_room) p.freed[f0[b] + i] = p.dead[(int64_t)b * p.W * p.max_pages + v.copies + i];
  }
  // this CTA's range of vectors
  int64_t x = (int64_t)blockIdx.x * all[0] / gridDim.x;
  const int64_t x1 = (int64_t)(blockIdx.x + 1) * all[0] / gridDim.x;
  if (x >= x1) return;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {   // the last request whose first vector is not behind x
    const int mid = (lo + hi) >> 1;
    if (v0[mid] <= x) lo = mid; else hi = mid;
  }
  int b = lo, i = 0, k = 0;
  int64_t first = v0[b];   // of copy i's part in pool k
  while (x < x1) {
    const int copies = p.found[b].copies;
    if (i == copies) { ++b; i = 0; continue; }
    const BeamCopy c = p.copies[(int64_t)b * p.W + i];
    const int dst = copy_target(p, b, i, p.found[b].dead, t0[b], c.src);
    for (k = 0; k < p.n_pools && x < x1; ++k) {
      const BeamPool& q = p.pool[k];
      const int nv = run_vecs(q, c.rows), bytes = c.rows * q.row_bytes;
      const int64_t total = (int64_t)q.runs * nv;
      if (x >= first + total) { first += total; continue; }
      const int v_from = (int)(x - first), v_to = (int)min(total, x1 - first);
      const char* src = q.base + (int64_t)c.src * q.page_bytes;
      char* to = q.base + (int64_t)dst * q.page_bytes;
      for (int v = v_from + tid; dst >= 0 && v < v_to; v += BR_THREADS * BR_DEEP) {
        uint4 w[BR_DEEP];
        int64_t o[BR_DEEP];
        int left[BR_DEEP];
#pragma unroll
        for (int j = 0; j < BR_DEEP; ++j) {
          const int vj = v + j * BR_THREADS;
          left[j] = 0;
          if (vj < v_to) {
            const int run = vj / nv, r = vj - run * nv, layer = run / q.parts, part = run - layer * q.parts;
            o[j] = layer * q.layer_bytes + (int64_t)part * 128 * q.row_bytes + (int64_t)r * 16;
            left[j] = bytes - r * 16;
            if (left[j] >= 16) w[j] = *reinterpret_cast<const uint4*>(src + o[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < BR_DEEP; ++j) {
          if (left[j] >= 16) *reinterpret_cast<uint4*>(to + o[j]) = w[j];
          else
            for (int y = 0; y < left[j]; y += 4) *reinterpret_cast<uint32_t*>(to + o[j] + y) = *reinterpret_cast<const uint32_t*>(src + o[j] + y);
        }
      }
      x = first + v_to;
      first += total;
    }
    ++i;
  }
}

}  // namespace

bool beam_select_supported(int64_t B, int64_t W) { return W <= kBeamMaxW && B < ((int64_t)1 << 22) && B * W < ((int64_t)1 << 22); }
constexpr int kMaxSms = 256;   // sizes the workspace, so that it does not depend on the device
size_t beam_select_ws_bytes(int64_t B, int64_t W, int64_t V) {
  // as many parts as any device may take
  const size_t lists = (size_t)(B * W) * std::max<int64_t>(1, std::min<int64_t>(BS_MAX_PARTS, (V + BS_BATCH - 1) / BS_BATCH));
  return round256(lists * kBeamMaxOut * sizeof(uint64_t)) + round256(lists * sizeof(float2));
}

int launch_beam_select(const BeamSelectDesc& d, int num_sms, cudaStream_t st) {
  SelectParams p;
  p.z = d.logits; p.ld = d.ld;
  p.B = (int)d.B; p.W = (int)d.W; p.V = (int)d.V; p.K = (int)d.n_out;
  p.parts = select_parts(d.B * d.W, d.V, num_sms);
  p.part_len = (int)(((d.V + p.parts - 1) / p.parts + 3) & ~(int64_t)3);
  p.scores = d.scores; p.finished = d.finished; p.pad = d.pad_token;
  p.parents = d.parents; p.tokens = d.tokens; p.out = d.out_scores;
  p.keys = static_cast<uint64_t*>(d.ws);
  const size_t lists = (size_t)(d.B * d.W) * p.parts;
  p.stat = reinterpret_cast<float2*>(static_cast<char*>(d.ws) + round256(lists * p.K * sizeof(uint64_t)));
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return -1;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BM_SMEM) != cudaSuccess) return -1;
    attr_set[dev] = true;
  }
  const unsigned grid = (unsigned)(d.B * d.W * p.parts);
  const bool vec = ((reinterpret_cast<uintptr_t>(d.logits) | (uintptr_t)(d.ld * 4)) & 15) == 0;
  if (vec) beam_part_kernel<true><<<grid, BS_THREADS, 0, st>>>(p);
  else beam_part_kernel<false><<<grid, BS_THREADS, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
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
  const int per_request = (int)(sizeof(int64_t) + 2 * sizeof(int));
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(beam_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kPlanMaxSeqs + 1) * per_request) !=
        cudaSuccess)
      return -1;
    attr_set[dev] = true;
  }
  if (d.B > 0) {
    beam_plan_kernel<<<(unsigned)d.B, BR_THREADS, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -1;
  }
  // CTAs for a few thousand vectors each, were every beam but one of each request to copy a whole page
  const int64_t work = std::max<int64_t>(d.B, (d.B * (d.W - 1) * vecs + 4 * BR_THREADS * BR_DEEP - 1) / (4 * BR_THREADS * BR_DEEP));
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(BR_CTAS_PER_SM * num_sms, work));
  return launch_after(beam_copy_kernel, dim3(grid), dim3(BR_THREADS), (size_t)(d.B + 1) * per_request, st, p) == cudaSuccess ? 0 : -1;
}

LLAMA_DEFINE_BOUNDS_READER(beam)

}  // namespace llama
