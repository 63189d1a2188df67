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
constexpr int BS_THREADS = 256;

struct SelectParams {
  const float* z;
  int64_t ld;
  int B, W, V, K;
  const float* scores;
  const int* finished;
  int pad;
  int *parents, *tokens;
  float* out;
  uint64_t* keys;   // [B W, K] the best tokens of a row, best first (0: none)
  float2* stat;     // [B W] maximum and sum of exp(z - maximum)
};

// Logits as integers that order as they do, the token below: larger is better, 0 is no candidate.
__device__ __forceinline__ uint64_t cand_key(float z, int i) {
  const uint32_t u = __float_as_uint(z);
  const uint32_t ord = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return z > -INFINITY ? ((uint64_t)ord << 32) | (uint32_t)~i : 0;
}
__device__ __forceinline__ float key_logit(uint64_t k) {
  const uint32_t ord = (uint32_t)(k >> 32);
  return __uint_as_float((ord & 0x80000000u) ? ord & 0x7FFFFFFFu : ~ord);
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T* buf, F f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < BS_THREADS / 32; ++w) v = f(v, buf[w]);
  return v;
}

__global__ void __launch_bounds__(BS_THREADS) beam_row_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint64_t buf[BS_THREADS / 32];
  __shared__ float fbuf[BS_THREADS / 32];
  const int row = blockIdx.x;
  const float* z = p.z + (int64_t)row * p.ld;
  if (p.finished && p.finished[row]) return;
  float m = -INFINITY;
  for (int i = threadIdx.x; i < p.V; i += BS_THREADS) m = fmaxf(m, z[i]);
  m = block_reduce(m, fbuf, [](float a, float b) { return fmaxf(a, b); });
  float s = 0.f;
  for (int i = threadIdx.x; i < p.V; i += BS_THREADS) s += z[i] > -INFINITY ? __expf(z[i] - m) : 0.f;
  s = block_reduce(s, fbuf, [](float a, float b) { return a + b; });
  if (threadIdx.x == 0) p.stat[row] = make_float2(m, s);
  uint64_t prev = ~0ull;
  for (int k = 0; k < p.K; ++k) {
    uint64_t best = 0;
    for (int i = threadIdx.x; i < p.V; i += BS_THREADS) {
      const uint64_t c = cand_key(z[i], i);
      if (c < prev && c > best) best = c;
    }
    best = block_reduce(best, buf, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    if (threadIdx.x == 0 && in_extent((int64_t)row * p.K + k, 1, (int64_t)p.B * p.W * p.K)) p.keys[(int64_t)row * p.K + k] = best;
    prev = best;
  }
}

__global__ void __launch_bounds__(BS_THREADS) beam_merge_kernel(const __grid_constant__ SelectParams p) {
  __shared__ double sbuf[BS_THREADS / 32];
  __shared__ int ibuf[BS_THREADS / 32];
  const int b = blockIdx.x, n = p.W * p.K;
  double last = INFINITY;
  int last_at = -1;
  for (int k = 0; k < p.K; ++k) {
    double best = -INFINITY;
    int at = INT_MAX;
    for (int c = threadIdx.x; c < n; c += BS_THREADS) {
      const int w = c / p.K, row = b * p.W + w;
      const float base = p.scores[row];
      double s = -INFINITY;
      int token = p.pad;
      if (p.finished && p.finished[row]) {
        if (c % p.K == 0) s = base;
      } else if (const uint64_t key = p.keys[(int64_t)row * p.K + c % p.K]) {
        const float2 st = p.stat[row];
        s = (double)base + (((double)key_logit(key) - st.x) - log((double)st.y));
        token = ~(int)(uint32_t)key;
      }
      // candidates in order: larger score, then lower place (beam, rank)
      if (s > -INFINITY && (s < last || (s == last && c > last_at)) && (s > best || (s == best && c < at))) { best = s; at = c; }
      (void)token;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double s2 = __shfl_xor_sync(0xffffffffu, best, o);
      const int a2 = __shfl_xor_sync(0xffffffffu, at, o);
      if (s2 > best || (s2 == best && a2 < at)) { best = s2; at = a2; }
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) { sbuf[threadIdx.x >> 5] = best; ibuf[threadIdx.x >> 5] = at; }
    __syncthreads();
    for (int w = 0; w < BS_THREADS / 32; ++w)
      if (sbuf[w] > best || (sbuf[w] == best && ibuf[w] < at)) { best = sbuf[w]; at = ibuf[w]; }
    if (threadIdx.x == 0 && in_extent((int64_t)b * p.K + k, 1, (int64_t)p.B * p.K)) {
      int parent = -1, token = -1;
      if (at != INT_MAX) {
        parent = at / p.K;
        const int row = b * p.W + parent;
        token = p.finished && p.finished[row] ? p.pad : ~(int)(uint32_t)p.keys[(int64_t)row * p.K + at % p.K];
      }
      p.parents[(int64_t)b * p.K + k] = parent;
      p.tokens[(int64_t)b * p.K + k] = token;
      p.out[(int64_t)b * p.K + k] = at != INT_MAX ? (float)best : -INFINITY;
    }
    last = best;
    last_at = at;
  }
}

// --------------------------------------------------------------------------------------- reorder
constexpr int BR_THREADS = 256;
constexpr int BR_MAX_W = (int)kBeamMaxW;
constexpr int BR_MAX_POOLS = kBeamMaxPools;
constexpr int BR_UNIT = 1024;        // 16-byte vectors of a copy that a CTA takes at once

struct BeamPool {
  char* base;
  int64_t page_bytes;                // parts * 128 * row_bytes
  int parts, row_bytes, part_vecs;   // 8 * row_bytes vectors of 16 bytes in a part
  int units;                         // of one page
};

struct BeamCopy { int src, rows, slot, pad; };   // slot: sequence * max_pages + column of the table entry

struct ReorderParams {
  const int *parents, *n_cached, *table, *free_pages;
  int *n_cached_out, *table_out, *freed, *counts;
  int B, W, n_free, n_pages;
  int64_t max_pages, freed_room;
  int2* found;        // [B] (copies, dead pages)
  BeamCopy* copies;   // [B, W]
  int* dead;          // [B, W max_pages]
  BeamPool pool[BR_MAX_POOLS];
  int n_pools, units_per_copy;                 // units of a copy over all pools and layers
  int pool_first[BR_MAX_POOLS + 1];            // first unit of each pool
  unsigned* status;
};

// One request per CTA: its new table rows, the copies its new beams need, and its dead pages in order.
__global__ void __launch_bounds__(BR_THREADS) beam_plan_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ int n[BR_MAX_W], par[BR_MAX_W], tile[BR_MAX_W][BR_THREADS], wsum[BR_THREADS / 32];
  __shared__ unsigned kept_sh;
  __shared__ int most_sh, n_copy_sh;
  const int b = blockIdx.x, W = p.W, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t P = p.max_pages;
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
    if (copy) {
      BeamCopy c2;
      c2.src = page;
      c2.rows = mine % 128;
      c2.slot = lane;
      c2.pad = mine / 128;
      if (in_extent((int64_t)b * W + __popc(copies & ((1u << lane) - 1)), 1, (int64_t)p.B * W))
        p.copies[(int64_t)b * W + __popc(copies & ((1u << lane) - 1))] = c2;
    }
    if (lane < W && in_extent(b * W + lane, 1, (int64_t)p.B * W)) p.n_cached_out[b * W + lane] = mine;
    if (lane == 0) { kept_sh = kept; most_sh = (most + 127) / 128; n_copy_sh = __popc(copies); }
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
  if (threadIdx.x == 0 && in_extent(b, 1, p.B)) p.found[b] = make_int2(n_copy_sh, n_dead);
  if (bad) atomicOr(p.status, STATUS_BAD_PLAN);
}

// Every CTA sums up the requests' copies, pages taken and pages left over; units of copies, table entries
// and freed pages are dealt out over the grid.
__global__ void __launch_bounds__(BR_THREADS) beam_copy_kernel(const __grid_constant__ ReorderParams p) {
  extern __shared__ int pre[];   // [3][B + 1]: first copy, first page taken, first page freed of each request
  int *c0 = pre, *t0 = pre + p.B + 1, *f0 = pre + 2 * (p.B + 1);
  if (threadIdx.x == 0) {
    int c = 0, t = 0, f = 0;
    for (int b = 0; b <= p.B; ++b) {
      c0[b] = c; t0[b] = t; f0[b] = f;
      if (b < p.B) {
        const int2 v = p.found[b];
        c += v.x;
        t += max(0, v.x - v.y);
        f += max(0, v.y - v.x);
      }
    }
  }
  __syncthreads();
  const int n_copies = c0[p.B];
  bool bad = t0[p.B] > p.n_free || f0[p.B] > p.freed_room;
  if (blockIdx.x == 0 && threadIdx.x == 0 && in_extent(0, 2, 2)) { p.counts[0] = t0[p.B]; p.counts[1] = f0[p.B]; }
  // freed pages
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int first = c0[b + 1] - c0[b], cnt = f0[b + 1] - f0[b];
    for (int i = threadIdx.x; i < cnt; i += BR_THREADS)
      if (f0[b] + i < p.freed_room) p.freed[f0[b] + i] = p.dead[(int64_t)b * p.W * p.max_pages + first + i];
  }
  const int64_t total = (int64_t)n_copies * p.units_per_copy;
  for (int64_t u = blockIdx.x; u < max(total, (int64_t)n_copies); u += gridDim.x) {
    const int per = max(1, p.units_per_copy);
    const int c = (int)(u / per);
    int r = (int)(u % per);
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (c0[mid] <= c) lo = mid; else hi = mid;
    }
    const int b = lo, i = c - c0[b];
    const BeamCopy cp = p.copies[(int64_t)b * p.W + i];
    const int n_dead = (c0[b + 1] - c0[b]) - (t0[b + 1] - t0[b]) + (f0[b + 1] - f0[b]);
    int dst = -1;
    if (i < n_dead) dst = p.dead[(int64_t)b * p.W * p.max_pages + i];
    else if (t0[b] + i - n_dead < p.n_free) dst = p.free_pages[t0[b] + i - n_dead];
    if (dst < 0 || dst >= p.n_pages || cp.src < 0) { bad = bad || cp.src >= 0; dst = -1; }
    if (r == 0 && threadIdx.x == 0) {
      const int64_t at = ((int64_t)b * p.W + cp.slot) * p.max_pages + cp.pad;
      if (in_extent(at, 1, (int64_t)p.B * p.W * p.max_pages)) p.table_out[at] = dst;
    }
    if (dst < 0 || total == 0) continue;
    int k = 0;
    while (r >= p.pool_first[k + 1]) ++k;
    r -= p.pool_first[k];
    const BeamPool& pool = p.pool[k];
    const int layer = r / pool.units, unit = r % pool.units;
    const int64_t lbase = (int64_t)layer * p.n_pages;
    const char* src = pool.base + (lbase + cp.src) * pool.page_bytes;
    char* to = pool.base + (lbase + dst) * pool.page_bytes;
    const int bytes = cp.rows * pool.row_bytes;      // of each part
    for (int v = unit * BR_UNIT + threadIdx.x; v < min((unit + 1) * BR_UNIT, pool.parts * pool.part_vecs); v += BR_THREADS) {
      const int part = v / pool.part_vecs, o = (v % pool.part_vecs) * 16;
      const int64_t at = (int64_t)part * pool.part_vecs * 16 + o;
      if (o + 16 <= bytes) *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(src + at);
      else
        for (int x = o; x < bytes; x += 4) *reinterpret_cast<uint32_t*>(to + at + x - o) = *reinterpret_cast<const uint32_t*>(src + at + x - o);
    }
  }
  if (bad && threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_PLAN);
}

}  // namespace

bool beam_select_supported(int64_t B, int64_t W) { return W <= kBeamMaxW && B < ((int64_t)1 << 22) && B * W < ((int64_t)1 << 22); }
size_t beam_select_ws_bytes(int64_t B, int64_t W, int64_t V) {
  (void)V;
  return round256((size_t)(B * W) * kBeamMaxOut * sizeof(uint64_t)) + round256((size_t)(B * W) * sizeof(float2));
}

int launch_beam_select(const BeamSelectDesc& d, int num_sms, cudaStream_t st) {
  (void)num_sms;
  SelectParams p;
  p.z = d.logits; p.ld = d.ld;
  p.B = (int)d.B; p.W = (int)d.W; p.V = (int)d.V; p.K = (int)d.n_out;
  p.scores = d.scores; p.finished = d.finished; p.pad = d.pad_token;
  p.parents = d.parents; p.tokens = d.tokens; p.out = d.out_scores;
  p.keys = static_cast<uint64_t*>(d.ws);
  p.stat = reinterpret_cast<float2*>(static_cast<char*>(d.ws) + round256((size_t)(d.B * d.W) * kBeamMaxOut * sizeof(uint64_t)));
  beam_row_kernel<<<(unsigned)(d.B * d.W), BS_THREADS, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  beam_merge_kernel<<<(unsigned)d.B, BS_THREADS, 0, st>>>(p);
  return 0;
}

int64_t beam_copy_units(const llama_page_pool* pools, int n_pools) {
  int64_t units = 0;
  for (int k = 0; k < n_pools; ++k)
    units += (pools[k].parts * 8 * pools[k].row_bytes + BR_UNIT - 1) / BR_UNIT * pools[k].n_layers;
  return units;
}

size_t beam_reorder_ws_bytes(int64_t B, int64_t W, int64_t max_pages) {
  return round256((size_t)B * sizeof(int2)) + round256((size_t)(B * W) * sizeof(BeamCopy)) +
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
  p.found = reinterpret_cast<int2*>(ws);
  ws += round256((size_t)d.B * sizeof(int2));
  p.copies = reinterpret_cast<BeamCopy*>(ws);
  ws += round256((size_t)(d.B * d.W) * sizeof(BeamCopy));
  p.dead = reinterpret_cast<int*>(ws);
  p.n_pools = d.n_pools;
  int64_t units = 0;
  for (int k = 0; k < d.n_pools; ++k) {
    BeamPool& q = p.pool[k];
    q.base = static_cast<char*>(d.pools[k].base);
    q.parts = (int)d.pools[k].parts;
    q.row_bytes = (int)d.pools[k].row_bytes;
    q.part_vecs = 8 * q.row_bytes;
    q.page_bytes = d.pools[k].parts * 128 * d.pools[k].row_bytes;
    q.units = (int)(((int64_t)q.parts * q.part_vecs + BR_UNIT - 1) / BR_UNIT);
    p.pool_first[k] = (int)units;
    units += (int64_t)q.units * d.pools[k].n_layers;
    p.pool_first[k + 1] = (int)units;
  }
  p.units_per_copy = (int)units;
  p.status = status;
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return -1;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(beam_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(3 * (kPlanMaxSeqs + 1) * sizeof(int))) != cudaSuccess)
      return -1;
    attr_set[dev] = true;
  }
  if (d.B > 0) beam_plan_kernel<<<(unsigned)d.B, BR_THREADS, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(4 * num_sms, std::max<int64_t>(d.B, d.B * d.W * std::max<int64_t>(1, units))));
  beam_copy_kernel<<<(unsigned)most, BR_THREADS, 3 * (d.B + 1) * sizeof(int), st>>>(p);
  return 0;
}

LLAMA_DEFINE_BOUNDS_READER(beam)

}  // namespace llama
