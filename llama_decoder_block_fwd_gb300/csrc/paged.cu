// The two steps that put new tokens into a paged KV cache ("LLaMA-3 8B ...", section 七: the cache
// grows by one K and one V row per token and layer): planning where each token goes, and writing it.
//
// plan: sequence b holds c_b positions and brings n_b tokens.  It has ceil(c_b / 128) pages and needs
//   ceil((c_b + n_b) / 128); the missing ones are taken from the free list in sequence order.
//   Token i of b sits at position c_b + i, in row (position mod 128) of page position / 128.
// append: q' = R(position) q, K[slot] = R(position) k, V[slot] = v, R the RoPE rotation.
#include <algorithm>
#include <climits>
#include <cstring>

#include "kernels.h"

namespace llama {
namespace {

// ------------------------------------------------------------------------------------------ plan
// A few hundred bytes to a megabyte move, so the launch and the latency of dependent loads are
// what it costs.  Every CTA scans the whole batch's lengths into its own shared memory (two loads
// per sequence and a block scan, cheaper than a second launch), then finds the owner of each token
// row and of each new page by bisection there.  64 sequences with drafts 3.2 us, 1024 sequences of which one
// brings 8192 tokens 4.1 us (a launch alone takes about 2).
constexpr int PL_THREADS = 512;

struct PlanParams {
  const int *n_cached, *n_new, *free_pages;
  int B, n_free, n_pages, max_pages;
  int* block_table;      // [B, max_pages]
  int n_tokens;
  int *cu_new, *positions, *slots, *pages_used;
  unsigned* status;
};

// Exclusive prefix sums of (a, b) over the block; *ta, *tb get the totals.
__device__ __forceinline__ void scan2_excl(int64_t& a, int64_t& b, int64_t* buf, int64_t* ta, int64_t* tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int W = PL_THREADS / 32;
  int64_t xa = a, xb = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ya = __shfl_up_sync(0xffffffffu, xa, o), yb = __shfl_up_sync(0xffffffffu, xb, o);
    if (lane >= o) { xa += ya; xb += yb; }
  }
  if (lane == 31) { buf[warp] = xa; buf[W + warp] = xb; }
  __syncthreads();
  int64_t pa = 0, pb = 0, sa = 0, sb = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == warp) { pa = sa; pb = sb; }
    sa += buf[w];
    sb += buf[W + w];
  }
  *ta = sa;
  *tb = sb;
  a = pa + xa - a;
  b = pb + xb - b;
}

// The last b with pre[b] <= x (pre[0] = 0, non-decreasing; x < pre[B]): the owner of entry x.
__device__ __forceinline__ int owner(const int* pre, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(PL_THREADS) paged_plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int pre[];          // [2][B + 1]: first token row, first new page of each sequence
  __shared__ int64_t buf[2 * PL_THREADS / 32];
  int* first_row = pre;
  int* first_page = pre + p.B + 1;
  // thread t scans the contiguous sequences [t * per, t * per + per)
  const int per = (p.B + PL_THREADS - 1) / PL_THREADS;
  const int s0 = min(p.B, (int)threadIdx.x * per), s1 = min(p.B, s0 + per);
  const int64_t room = (int64_t)p.max_pages * 128;
  bool bad = false;
  // a sequence whose lengths cannot be right brings nothing
  auto lengths = [&](int b, int& c, int& n) {
    c = __ldg(p.n_cached + b);
    n = __ldg(p.n_new + b);
    if (c < 0 || n < 0 || (int64_t)c + n > room) { bad = true; c = 0; n = 0; }
  };
  int64_t rows = 0, pages = 0;
  for (int b = s0; b < s1; ++b) {
    int c, n;
    lengths(b, c, n);
    rows += n;
    pages += (c + n + 127) / 128 - (c + 127) / 128;
  }
  int64_t all_rows, all_pages;
  scan2_excl(rows, pages, buf, &all_rows, &all_pages);
  for (int b = s0; b < s1; ++b) {
    int c, n;
    lengths(b, c, n);
    first_row[b] = (int)min(rows, (int64_t)p.n_tokens);
    first_page[b] = (int)min(pages, (int64_t)p.n_free);
    rows += n;
    pages += (c + n + 127) / 128 - (c + 127) / 128;
  }
  if (threadIdx.x == 0) {
    first_row[p.B] = (int)min(all_rows, (int64_t)p.n_tokens);
    first_page[p.B] = (int)min(all_pages, (int64_t)p.n_free);
    bad = bad || all_rows > p.n_tokens || all_pages > p.n_free;
    if (blockIdx.x == 0 && in_extent(0, 1, 1)) p.pages_used[0] = (int)min(all_pages, (int64_t)INT32_MAX);
  }
  __syncthreads();
  const int T = first_row[p.B], P = first_page[p.B];
  const int tid = blockIdx.x * PL_THREADS + threadIdx.x, step = gridDim.x * PL_THREADS;
  for (int b = tid; b <= p.B; b += step)
    if (in_extent(b, 1, (int64_t)p.B + 1)) p.cu_new[b] = first_row[b];
  for (int i = tid; i < P; i += step) {
    const int b = owner(first_page, p.B, i);
    const int j = (__ldg(p.n_cached + b) + 127) / 128 + i - first_page[b];
    const int page = __ldg(p.free_pages + i);
    if (page < 0 || page >= p.n_pages) bad = true;
    if (in_extent(j, 1, p.max_pages)) p.block_table[(int64_t)b * p.max_pages + j] = page;
  }
  for (int t = tid; t < p.n_tokens; t += step) {
    int pos = -1, slot = -1;
    if (t < T) {
      const int b = owner(first_row, p.B, t);
      const int c = __ldg(p.n_cached + b);
      pos = c + t - first_row[b];
      const int j = pos / 128, have = (c + 127) / 128;
      int page = -1;
      if (j < have) {
        page = p.block_table[(int64_t)b * p.max_pages + j];   // an entry this call does not write
      } else if (first_page[b] + j - have < p.n_free) {
        page = __ldg(p.free_pages + first_page[b] + j - have);
      }
      if (page >= 0 && page < p.n_pages) slot = page * 128 + pos % 128;
      else bad = true;
    }
    if (in_extent(t, 1, p.n_tokens)) {
      p.positions[t] = pos;
      p.slots[t] = slot;
    }
  }
  if (bad) atomicOr(p.status, STATUS_BAD_PLAN);
}

// ---------------------------------------------------------------------------------------- append
// HBM bound: every row is read once and written once, in 16-byte pieces.  A CTA takes TOK tokens,
// forms each token's hd/2 cosines and sines once in shared memory (all heads share them), then
// walks the tokens' q, k and v vectors, the next ones on their way.  8192 tokens of 32/8 heads x 128, 201 MB:
// 33.4 us = 6.0 TB/s (a persistent grid, other token counts and 3 to 6 CTAs per SM: no faster, up to 9% slower);
// 300 tokens 3.2 us.  RA_TOK tokens share a pass over the row where every SM gets them, else one.  RA_TOK
// against one, back to back: 300 tokens 4.0 / 3.2 us, 608 4.1 / 4.0, 1216 5.3 / 6.2, 8192 33.3 / 36.2.
constexpr int RA_THREADS = 256;
constexpr int RA_TOK = 4;

struct AppendParams {
  const uint16_t *q, *k, *v;             // [T] rows of n_q / n_kv / n_kv heads x hd, row strides below
  int64_t q_stride, k_stride, v_stride;  // elements
  const int *positions, *slots;
  uint16_t *q_out, *k_pool, *v_pool;
  int T, hd, q_vec, kv_vec;              // 16-byte vectors per token in q and in each of k and v
  int64_t n_slots;
  unsigned* status;
  RopeFreq freq[kMaxRopePairs];
};

__device__ __forceinline__ uint32_t rotate_pair(uint32_t w, float2 cs) {
  const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xFFFF0000u);
  return pack_bf2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

template <int TOK>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ __align__(16) float2 cs[TOK][kMaxRopePairs];
  __shared__ int slot_sh[TOK];
  const int half = p.hd / 2, vph = p.hd / 8;                 // vectors per head
  const int total = p.q_vec + 2 * p.kv_vec;
  const int t0 = blockIdx.x * TOK, n = min(TOK, p.T - t0);
  // vector i of the tokens: which part of the row it belongs to, and where it comes from
  auto load = [&](int i, uint4 (&w)[TOK]) {
    if (i >= total) return;
    const bool is_q = i < p.q_vec, is_v = i >= p.q_vec + p.kv_vec;
    const int o = is_q ? i : i - p.q_vec - (is_v ? p.kv_vec : 0);
    const uint16_t* src = is_q ? p.q : is_v ? p.v : p.k;
    const int64_t stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
#pragma unroll
    for (int tk = 0; tk < TOK; ++tk)
      if (tk < n) w[tk] = *reinterpret_cast<const uint4*>(src + (t0 + tk) * stride + o * 8);
  };
  // the first vectors are on their way while the angles are formed
  uint4 w[TOK];
  load(threadIdx.x, w);
  if (threadIdx.x < TOK) {
    const int t = t0 + threadIdx.x;
    int slot = -1;
    if (t < p.T) {
      slot = __ldg(p.slots + t);
      const int pos = __ldg(p.positions + t);
      if (slot >= 0 && (slot >= p.n_slots || pos < 0 || pos >= (1 << 24))) {
        atomicOr(p.status, STATUS_BAD_PLAN);
        slot = -1;
      }
    }
    slot_sh[threadIdx.x] = slot;
  }
  // neighbouring threads take the tokens of one pair: a warp then reads few different frequencies,
  // which come from the kernel's parameters one address at a time
  for (int i = threadIdx.x; i < TOK * half; i += RA_THREADS) {
    const int tk = i % TOK, j = i / TOK;
    if (tk < n) rope_sincos((float)__ldg(p.positions + t0 + tk), p.freq[j], cs[tk][j].y, cs[tk][j].x);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += RA_THREADS) {
    uint4 next[TOK];
    load(i + RA_THREADS, next);
    const bool is_q = i < p.q_vec, is_v = i >= p.q_vec + p.kv_vec;
    const int o = is_q ? i : i - p.q_vec - (is_v ? p.kv_vec : 0);   // vector within its part
    const int j = (o % vph) * 4;                                    // first pair
    uint16_t* dst = is_q ? p.q_out : is_v ? p.v_pool : p.k_pool;
#pragma unroll
    for (int tk = 0; tk < TOK; ++tk) {
      const int slot = slot_sh[tk];
      if (slot < 0) continue;
      if (!is_v) {
        const float4 c0 = *reinterpret_cast<const float4*>(&cs[tk][j]), c1 = *reinterpret_cast<const float4*>(&cs[tk][j + 2]);
        w[tk].x = rotate_pair(w[tk].x, make_float2(c0.x, c0.y));
        w[tk].y = rotate_pair(w[tk].y, make_float2(c0.z, c0.w));
        w[tk].z = rotate_pair(w[tk].z, make_float2(c1.x, c1.y));
        w[tk].w = rotate_pair(w[tk].w, make_float2(c1.z, c1.w));
      }
      const int64_t at = is_q ? (int64_t)(t0 + tk) * p.q_vec + o : (int64_t)slot * p.kv_vec + o;
      if (in_extent(at, 1, is_q ? (int64_t)p.T * p.q_vec : p.n_slots * p.kv_vec))
        *reinterpret_cast<uint4*>(dst + at * 8) = w[tk];
    }
#pragma unroll
    for (int tk = 0; tk < TOK; ++tk) w[tk] = next[tk];
  }
}

}  // namespace

int launch_paged_plan(const int* n_cached, const int* n_new, const int* free_pages, int64_t B, int64_t n_free,
                      int64_t n_pages, int64_t max_pages, int* block_table, int64_t n_tokens, int* cu_new,
                      int* positions, int* slots, int* pages_used, int num_sms, unsigned* status, cudaStream_t st) {
  PlanParams p;
  p.n_cached = n_cached; p.n_new = n_new; p.free_pages = free_pages;
  p.B = (int)B; p.n_free = (int)n_free; p.n_pages = (int)n_pages; p.max_pages = (int)max_pages;
  p.block_table = block_table;
  p.n_tokens = (int)n_tokens;
  p.cu_new = cu_new; p.positions = positions; p.slots = slots; p.pages_used = pages_used;
  p.status = status;
  const size_t smem = (size_t)2 * (B + 1) * sizeof(int);
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return -1;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(2 * (kPlanMaxSeqs + 1) * sizeof(int))) != cudaSuccess)
      return -1;
    attr_set[dev] = true;
  }
  const int64_t work = std::max(B + 1, n_tokens);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(num_sms, (work + PL_THREADS - 1) / PL_THREADS));
  paged_plan_kernel<<<grid, PL_THREADS, smem, st>>>(p);
  return 0;
}

int launch_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, const int* positions, const int* slots, void* q_out, void* k_pool,
                       void* v_pool, int64_t T, int64_t n_q, int64_t n_kv, int hd, int64_t n_pages,
                       const RopeFreq* freq, int num_sms, unsigned* status, cudaStream_t st) {
  AppendParams p;
  p.q = static_cast<const uint16_t*>(q); p.k = static_cast<const uint16_t*>(k); p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.positions = positions; p.slots = slots;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_pool = static_cast<uint16_t*>(k_pool);
  p.v_pool = static_cast<uint16_t*>(v_pool);
  p.T = (int)T; p.hd = hd;
  p.q_vec = q ? (int)(n_q * hd / 8) : 0;
  p.kv_vec = k ? (int)(n_kv * hd / 8) : 0;
  p.n_slots = n_pages * 128;
  p.status = status;
  memcpy(p.freq, freq, sizeof(RopeFreq) * (hd / 2));
  if (T >= (int64_t)RA_TOK * num_sms) rope_append_kernel<RA_TOK><<<(unsigned)((T + RA_TOK - 1) / RA_TOK), RA_THREADS, 0, st>>>(p);
  else rope_append_kernel<1><<<(unsigned)T, RA_THREADS, 0, st>>>(p);
  return 0;
}

LLAMA_DEFINE_BOUNDS_READER(paged)

}  // namespace llama
