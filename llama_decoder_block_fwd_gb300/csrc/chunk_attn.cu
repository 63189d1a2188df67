// Causal GQA attention of ragged chunks of new tokens over a paged KV cache ("Llama Architecture
// ...", Mathematical Foundations 4; "LLaMA-3 8B ...", section 四.4): token i of sequence b sits at
// position c_b + i and attends to positions 0 .. c_b + i of its sequence,
//     o = sum_j softmax_j(q . k_j / sqrt(hd)) v_j,
// taken over 128-key tiles (one page each) with a running maximum and sum.
//
// One form for every mix of lengths, from one token against a long cache (bound by reading K and V
// once) to long prompts (bound by the tensor cores):
//   * A Q tile is 128 rows: (128 / r) consecutive tokens x the r query heads of one KV group.  An item is
//     a pair of adjacent Q tiles of one (sequence, KV group), which share every K/V tile staged, or one Q
//     tile: a sequence's only or odd last one, and every one of a batch too small to fill the SMs with pairs.
//     A single tile's key tiles alternate between the two softmax groups (even tiles, odd tiles), each with
//     its own O, merged at the end, so that the two groups still take turns with the tensor core.
//   * chunk_plan_kernel cuts the items' key ranges into units: a sequence's tiles into n_chunk equal
//     parts of at least one tile, as many as make the units come out even over the SMs (see there).
//   * chunk_attn_kernel: one CTA per SM takes units from a counter.  Warp 0 fetches units and runs TMA
//     (Q tiles through two slots, K and V tiles through one ring of slots, across unit borders), warp 1
//     issues the MMAs, warps 4-7 / 8-11 are the softmax groups, one thread per row (TMEM lane).  A unit
//     that holds all of its item's keys stores o; otherwise it leaves (m, l, O) in the workspace.
//   * chunk_combine_kernel merges the parts of the rows that were cut.
// Measured (one call, plan and merge included, back to back for over a second): 2048 tokens after 30720, 32/8
// heads x 128, 687-700 us = 1520-1550 TFLOP/s at the 1.76-1.85 GHz that the power cap leaves (a few calls after
// a pause 643-653 us, the attention kernel alone 620 at 1.89 GHz, tensor pipe 73% active, its softmax warps'
// instructions in the way of the rest); 64 sequences of 3-5 tokens after 2-8 K, 1.28 GB of K and V, 208 us, the
// attention kernel 197-200 = 6.4 TB/s; three single tokens 14.0 us (plan 5, attention 6, merge 2.5).
// TMEM: S_0 [0,128), S_1 [128,256), O_0 [256,384), O_1 [384,512).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "attn_common.cuh"
#include "kernels.h"

namespace llama {
namespace {

// Three warpgroups: warp 0 TMA, warp 1 MMA (2 and 3 leave), then the two softmax groups.  Launched with 168
// registers a thread (384 x 168 = 64512), of which the first warpgroup gives up what the others take.
constexpr int CA_THREADS = 384;
constexpr int CA_REGS_ISSUE = 88, CA_REGS_SOFTMAX = 208;
static_assert(CA_REGS_ISSUE + 2 * CA_REGS_SOFTMAX <= 3 * 168, "register split");
constexpr uint32_t CA_TMEM_COLS = 512;
constexpr int CP_THREADS = 1024, CP_WARPS = CP_THREADS / 32;
constexpr int kMaxGrid = 256;            // attention CTAs at most (one per SM; sizes the workspace)

// Per sequence, written by the plan.
struct ChunkSeq {
  int unit0;          // first unit
  int lo, n, c;       // first packed row, new tokens, cached positions
  int np, wp;         // items per KV group; the last wp of them are not cut
  int span;           // tokens per item: two Q tiles' or one's
  int nc, ct;         // key chunks of the others and tiles per chunk
  int cut_n;          // tokens with partial rows (0 if nc = 1): those of the items that are cut
  int part0;          // first partial row: token i's in chunk k is part0 + k * cut_n + i
  int split0;         // cut_n of the sequences before this one
};
struct ChunkHead {
  int n_units, counter, n_split, pad;
};

// One unit, as the roles of a CTA see it.
struct __align__(16) ChunkUnit {
  int live;            // 0: no more units
  int t0;              // first key tile
  int n0, n1;          // rounds of groups 0 and 1
  int lone;            // 1: one Q tile, key tiles alternate between the groups
  int row0, row1;      // first packed row of each group's Q tile
  int end;             // the sequence's end row
  int pos_off;         // position = packed row + pos_off
  int g;               // KV group
  int kv_len;          // keys of the sequence
  int clean;           // tiles from here on hold keys that some row of the unit does not see
  int part;            // partial row = packed row + part; INT_MIN: store o
  int b;
  int pad0, pad1;
};
static_assert(sizeof(ChunkUnit) == 64, "unit record");

struct ChunkParams {   // 128-byte aligned by its tensor maps
  CUtensorMap tmQ;     // [T, n_q, hd], box (64, r, tpt)
  CUtensorMap tmK;     // [n_pages, 128, n_kv, hd], box (64, 1, 128, 1)
  CUtensorMap tmV;
  uint16_t* o;         // [T, n_q, hd]
  const uint16_t* v_pool;
  const int *block_table, *cu_new, *n_cached;
  int B, T, n_q, n_kv, r, tpt, n_pages, max_pages, max_pos;
  float scale_log2;    // log2(e) / sqrt(hd)
  ChunkHead* head;
  ChunkUnit* first;    // [grid]
  ChunkSeq* seq;       // [B]
  float* part_o;       // [part_rows, n_q, hd]
  float2* part_ml;     // [part_rows, n_q]  (m in log2 units, l)
  int part_rows, grid;
  unsigned inv_q, inv_kv, inv_grid, inv_pair, inv_tile;   // floor(2^32 / x) of n_q, n_kv, grid, 2 tpt and tpt
  unsigned* status;
};

// The arithmetic of the work split runs on the host too, where its tests call it.
#define LLAMA_BOTH __host__ __device__ __forceinline__
LLAMA_BOTH int cdiv(int a, int b) { return (a + b - 1) / b; }

// The last b of B (a power-of-32 search by one warp) with key(b) <= x; key is non-decreasing, key(0) <= x.
template <typename F>
__device__ __forceinline__ int warp_search(int B, int x, F&& key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = cdiv(n, 32), at = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < n && key(lo + at) <= x);
    const int k = 31 - __clz(le);     // lane 0 always holds
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// ------------------------------------------------------------------------------------------ plan
// A sequence of n new tokens after c cached has np = ceil(n / (2 tpt)) items per KV group of nt =
// ceil((c + n) / 128) key tiles or less.  With at most C tiles per unit a range is cut into nc =
// ceil(nt / C).  Of the items that share their K and V with others of their sequence the first `whole`
// (whole rounds of one per CTA, or none) are not cut, only what is left over after them; K and V that one
// item reads alone are read once however it is cut.  With less than a round of items, items of one Q tile
// are the other choice: twice the items, each tile of them kSingleTile of a pair's, its key tiles taken by
// both groups in turn (32/8 heads x 128: 200 tokens 16.7 -> 14.6 us, 2 x 100 after 1000 25.8 -> 21.1, 4 x 64
// after 500 22.6 -> 18.2; forced on 1500 tokens among 40 decodes, 107 against 99.6).  (C, whole or single) is
// the candidate of least estimated time,
// in units of one tile's time (1.4 us for a pair at hd 128).  A unit costs kUnitCost more than its tiles
// (its pipeline fills and drains); one that leaves partials kCutCost, and kRowCost for 256 rows of them,
// written and read again; the merge kMergeCost.  Units of about one size go in rounds of one per CTA;
// others fill up to half of the longest one, and no round takes more than its longest.  C takes 32 values, one
// per warp: 1, 1, 2, 3, 4, 6, 8, 12, .. 32768 tiles and all (1 stands twice: 2^(w/2) rounded down; those past the
// longest range cut nothing, like the last, and are skipped); candidates whose partials do not fit the
// workspace are out, the last C (nothing cut) always fits.
//
// One CTA does this while all the others wait: a chain of dependent steps (loads, scans, estimate, scans,
// records) of about 8000 cycles, whose length is what counts: divisions go through reciprocals (integer and
// IEEE divisions cost 1.6 us of it), and 512 threads or a warm instruction cache change nothing.
constexpr float kSingleTile = 0.62f, kUnitCost = 1.5f, kCutCost = 1.0f, kRowCost = 2.0f, kMergeCost = 2.0f;
// Sequences whose shapes are kept in shared memory (one per thread).  Beyond them every estimate reads the lengths
// from memory, a warp's 32 sequences after another, and nothing is left whole: the plan takes 23 us for 1024
// single tokens, 27 for 1025 and 217 for 8192 (of calls of 269, 274 and 2117 us), 35 against 30 with a prompt of
// 2000 tokens among them (312 against 308 us).
constexpr int CP_SEQS = CP_THREADS;

#ifndef LLAMA_HOST_RCP
#define LLAMA_HOST_RCP(x) (1.f / (x))
#endif
LLAMA_BOTH float rcp(float x) {
#ifdef __CUDA_ARCH__
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
#else
  return LLAMA_HOST_RCP(x);
#endif
}
LLAMA_BOTH unsigned mul_high(unsigned a, unsigned b) {
#ifdef __CUDA_ARCH__
  return __umulhi(a, b);
#else
  return (unsigned)(((uint64_t)a * b) >> 32);
#endif
}
// floor(a / b) for 0 <= a < 2^22, 0 < b, inv within a few ulp of 1 / b
LLAMA_BOTH int div_by(int a, int b, float inv) {
  int q = (int)((float)a * inv);
  if (q * b > a) --q;
  if ((q + 1) * b <= a) ++q;
  return q;
}
// floor(a / b), a >= 0, inv = floor(2^32 / b): a * inv / 2^32 is less than 1 + a / 2^32 below a / b
LLAMA_BOTH int div_inv(int a, int b, unsigned inv) {
  const int q = (int)mul_high((unsigned)a, inv);
  return b == 1 ? a : q + ((q + 1) * b <= a);
}
LLAMA_BOTH int cdiv_by(int a, int b, float inv) { return div_by(a + b - 1, b, inv); }

struct SeqShape { int lo, n, c, np, nt; };
// cu, n_cached -> the sequence's shape; lengths that cannot be right bring nothing and set bad
__device__ __forceinline__ SeqShape seq_shape(const ChunkParams& p, int b, bool& bad) {
  SeqShape s;
  s.lo = __ldg(p.cu_new + b);
  const int hi = __ldg(p.cu_new + b + 1);
  s.c = __ldg(p.n_cached + b);
  s.n = hi - s.lo;
  const bool wrong = s.lo < 0 || s.n < 0 || hi > p.T || (s.n > 0 && (s.c < 0 || (int64_t)s.c + s.n - 1 > p.max_pos));
  bad = bad || wrong;
  if (wrong || s.n == 0) { s.n = 0; s.c = 0; }
  s.np = div_inv(s.n + 2 * p.tpt - 1, 2 * p.tpt, p.inv_pair);
  s.nt = (s.c + s.n + 127) >> 7;
  return s;
}

// floor(2^32 / x), for div_inv
unsigned inverse(int64_t x) { return (unsigned)std::min<uint64_t>((1ull << 32) / (uint64_t)x, UINT32_MAX); }

// nt tiles in chunks of at most C (inv = 1 / C): their number and their tiles
LLAMA_BOTH void cut(int nt, int C, float inv, int& nc, int& ct) {
  nc = nt <= C ? 1 : cdiv_by(nt, C, inv);
  const float inv_nc = rcp((float)nc);
  ct = max(1, cdiv_by(nt, nc, inv_nc));
  nc = max(1, cdiv_by(nt, ct, rcp((float)ct)));
}
// candidate w of 32: 2^(w / 2) tiles, 1.5 x 2^((w - 1) / 2) for odd w (rounded down), the last one unbounded
LLAMA_BOTH int candidate(int w) {
  return w == 31 ? 1 << 20 : (w & 1) ? (3 << (w >> 1)) >> 1 : 1 << (w >> 1);
}

// Unit u of sequence b (seq[b].unit0 <= u); false if no row of it sees its keys.
LLAMA_BOTH bool make_unit(const ChunkParams& p, const ChunkSeq& s, int b, int u, ChunkUnit& d) {
  // first the uncut items, the longest first, then the others chunk by chunk
  const int x = u - s.unit0, item = div_inv(x, p.n_kv, p.inv_kv), y = item < s.wp ? item : item - s.wp, nq = s.np - s.wp;
  const bool uncut = item < s.wp;
  const int chunk = uncut || s.nc == 1 ? 0 : div_by(y, nq, rcp((float)nq));   // parts are bounded, so y is
  const int pair = uncut ? s.np - 1 - y : nq - 1 - (y - chunk * nq);
  const int first = pair * s.span;                                          // token of the earlier Q tile
  const int nt1 = cdiv(s.c + min(s.n, first + p.tpt), 128), nt0 = cdiv(s.c + min(s.n, first + s.span), 128);
  const int t0 = chunk * s.ct, t1 = uncut ? nt0 : min(t0 + s.ct, nt0);
  d.live = t0 < t1;
  d.t0 = t0;
  d.lone = min(s.n - first, s.span) <= p.tpt;
  d.n0 = d.lone ? (t1 - t0 + 1) / 2 : t1 - t0;
  d.n1 = d.lone ? (t1 - t0) / 2 : max(0, min(t1, nt1) - t0);
  d.row1 = s.lo + first;
  d.row0 = d.lone ? d.row1 : d.row1 + p.tpt;
  d.end = s.lo + s.n;
  d.pos_off = s.c - s.lo;
  d.g = x - item * p.n_kv;
  d.kv_len = s.c + s.n;
  d.clean = (s.c + first + 1) / 128;
  d.part = !uncut && s.cut_n > 0 ? s.part0 + chunk * s.cut_n - s.lo : INT_MIN;
  d.b = b;
  d.pad0 = d.pad1 = 0;
  return d.live;
}

// Inclusive prefix sums over a warp of N integers per lane, their chains side by side.
template <int N>
__device__ __forceinline__ void warp_scan(int (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    int y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __shfl_up_sync(0xffffffffu, v[i], o);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane >= o) v[i] += y[i];
  }
}

// What a lane, then a warp, adds up for one candidate: items left whole and pieces of the others, their
// time, the longest, partial rows.
struct Estimate {
  float nw = 0.f, cw = 0.f, lw = 0.f, nu = 0.f, cu = 0.f, lu = 0.f;
  float rows = 0.f;   // exact below 2^24, beyond it too many
  // v: (n, items, nt, tiles of the shortest item), cut in nc chunks of ct tiles but for wp items left whole;
  // an item has `span` tokens, and a tile of it takes `tile`
  __device__ __forceinline__ void add(const ChunkParams& p, const int4& v, int nc, int ct, int wp, int span, float tile) {
    const float n_kv = (float)p.n_kv, nt = (float)v.z, lo = (float)v.w;
    const float step = __fdividef(nt - lo, (float)max(v.y - 1, 1));
    if (wp > 0) {
      const float items = (float)wp * n_kv;
      nw += items;
      cw += items * (nt - 0.5f * step * (float)(wp - 1) + kUnitCost);
      lw = fmaxf(lw, nt + kUnitCost);
    }
    if (v.y > wp) {
      const float mean = 0.5f * (nt - step * (float)wp + lo);
      // chunks that hold keys, on average over the items: their tiles are spread over lo .. nt
      const float part = __fdividef(mean, (float)ct), spread = nt - step * (float)wp - lo;
      const float k = nc > 1 ? fminf((float)nc, spread < (float)ct ? ceilf(part) : part + 0.5f) : 1.f;
      const float row_cost = kRowCost / 256.f * (float)p.r;
      const float over = kUnitCost + (nc > 1 ? kCutCost + row_cost * (float)min(v.x, span) : 0.f);
      const float items = (float)(v.y - wp) * n_kv;
      nu += items * k;
      cu += items * (mean * tile + k * over);
      lu = fmaxf(lu, (float)min(ct, v.z) * tile + over);
      if (nc > 1) rows += (float)nc * (float)min(v.x, (v.y - wp) * span);
    }
  }
  // summed over the lanes, of which the first `lanes` hold something
  __device__ __forceinline__ float time(const ChunkParams& p, bool some_whole, int lanes) {
    for (int o = lanes > 16 ? 16 : lanes > 4 ? 8 : 2; o > 0; o >>= 1) {
      const float y0 = __shfl_xor_sync(0xffffffffu, nu, o), y1 = __shfl_xor_sync(0xffffffffu, cu, o);
      const float y2 = __shfl_xor_sync(0xffffffffu, rows, o);
      if (some_whole) {
        const float y3 = __shfl_xor_sync(0xffffffffu, nw, o), y4 = __shfl_xor_sync(0xffffffffu, cw, o);
        nw += y3;
        cw += y4;
      }
      nu += y0;
      cu += y1;
      rows += y2;
    }
    // (not negative, so ordered as their bits)
    if (some_whole) lw = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(lw)));
    lu = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(lu)));
    const float g = rcp((float)p.grid), mw = nw > 0.f ? __fdividef(cw, nw) : 0.f, mu = nu > 0.f ? __fdividef(cu, nu) : 0.f;
    const float e = lw <= 1.2f * mw && lu <= 1.2f * mu ? ceilf(nw * g - 0.01f) * mw + ceilf(nu * g - 0.01f) * mu
                                                       : fminf((cw + cu) * g + 0.5f * (nu > 0.f ? lu : lw),
                                                               ceilf((nw + nu) * g - 0.01f) * fmaxf(lw, lu));
    return rows <= (float)p.part_rows ? fmaxf(e, fmaxf(lw, lu)) + (rows > 0.f ? kMergeCost : 0.f) : INFINITY;
  }
};

__global__ void __launch_bounds__(CP_THREADS) chunk_plan_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ int4 shapes[CP_SEQS];  // (n, np, nt, tiles of the shortest item)
  __shared__ int4 places[CP_SEQS];  // (first packed row, cached positions, first partial row, items left whole)
  __shared__ int before[CP_SEQS];   // items per KV group that may be left whole, in the sequences before of the same 32
  __shared__ int unit0[CP_SEQS];
  __shared__ float est[64];
  __shared__ int most[CP_WARPS], shares[CP_WARPS], sums[3][CP_WARPS];   // per warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  bool bad = false;
  const int per = cdiv(p.B, CP_THREADS);                              // contiguous runs of sequences
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  const bool active = warp * 32 * per < p.B;                          // this warp has sequences
  const bool table = p.B <= CP_SEQS;
  const int tpt2 = 2 * p.tpt;
  SeqShape mine = {0, 0, 0, 0, 0};                                    // the first of this thread's
  if (b0 < b1) mine = seq_shape(p, b0, bad);
  auto shape = [&](int b) { return b == b0 ? mine : seq_shape(p, b, bad); };
  auto shape4 = [&](const SeqShape& s) { return make_int4(s.n, s.np, s.nt, (s.c + min(s.n, tpt2) + 127) >> 7); };
  int nt_max = 0, share = 0;
  bool several_tiles = false;
  if (active) {
    for (int b = b0; b < b1; ++b) {
      const SeqShape s = shape(b);
      nt_max = max(nt_max, s.nt);
      several_tiles = several_tiles || s.n > p.tpt;
    }
    nt_max = __reduce_max_sync(0xffffffffu, nt_max);
    if (table) {   // one sequence per thread
      const int own = mine.np > 1 ? mine.np : 0;
      int incl[1] = {own};
      warp_scan(incl);
      share = incl[0];
      if (b0 < b1) {
        shapes[b0] = shape4(mine);
        before[b0] = share - own;
      }
    }
  }
  if (lane == 31) {
    most[warp] = nt_max;
    shares[warp] = share;
  }
  if (tid < 64) est[tid] = INFINITY;
  const bool several = __syncthreads_or(several_tiles);   // a sequence of more than one Q tile
  nt_max = __reduce_max_sync(0xffffffffu, lane < CP_WARPS ? most[lane] : 0);
  // whole rounds of items that share their K and V with others, one per CTA (batches beyond the table: none)
  const int all = __reduce_add_sync(0xffffffffu, lane < CP_WARPS ? shares[lane] : 0) * p.n_kv;
  const int rounds_whole = div_inv(div_inv(all, p.grid, p.inv_grid) * p.grid, p.n_kv, p.inv_kv);
  // with less than a round of them, items of one Q tile are looked at instead
  const bool singles = rounds_whole == 0 && several;
  auto tiles_of = [&](int n) { return div_inv(n + p.tpt - 1, p.tpt, p.inv_tile); };
  for (int w = warp; w < 32; w += CP_WARPS) {
    const int C_est = candidate(w);
    if (C_est >= nt_max && w != 31) continue;   // from the longest range on they all cut nothing
    const float inv_C = rcp((float)C_est);
    Estimate e0, e1;
    for (int k = 0, base = 0; 32 * k < p.B; ++k) {
      const int b = 32 * k + lane;
      if (b < p.B) {
        const int4 v = table ? shapes[b] : shape4(seq_shape(p, b, bad));
        if (v.x > 0) {
          int nc, ct;
          cut(v.z, C_est, inv_C, nc, ct);
          e0.add(p, v, nc, ct, 0, tpt2, 1.f);
          if (rounds_whole > 0)
            e1.add(p, v, nc, ct, v.y > 1 ? min(max(rounds_whole - base - before[b], 0), v.y) : 0, tpt2, 1.f);
          else if (singles)
            e1.add(p, make_int4(v.x, tiles_of(v.x), v.z, v.w), nc, ct, 0, p.tpt, v.x > p.tpt ? kSingleTile : 1.f);
        }
      }
      if (rounds_whole > 0) base += shares[k];
    }
    const float t0 = e0.time(p, false, p.B), t1 = rounds_whole > 0 || singles ? e1.time(p, !singles, p.B) : INFINITY;
    if (lane == 0) {
      est[w] = t0;
      est[32 + w] = t1;
    }
  }
  __syncthreads();
  // the least estimate, the larger C of equals (every warp finds it for itself)
  const bool second = est[32 + lane] < est[lane];
  const unsigned bits = __float_as_uint(second ? est[32 + lane] : est[lane]);
  const unsigned least = __reduce_min_sync(0xffffffffu, bits);
  const int pick = __reduce_max_sync(0xffffffffu, bits == least ? lane + (second ? 32 : 0) : 0);
  const int C = candidate(pick & 31), whole = pick >= 32 ? rounds_whole : 0;
  const int span = pick >= 32 && singles ? p.tpt : tpt2;
  const float inv = rcp((float)C);
  // ---- the sequences' records; prefix sums of (units, partial rows, cut tokens)
  const int share0 = __reduce_add_sync(0xffffffffu, lane < warp ? shares[lane] : 0);
  auto record = [&](int b) {
    const SeqShape s = shape(b);
    ChunkSeq r;
    cut(s.nt, C, inv, r.nc, r.ct);
    r.lo = s.lo; r.n = s.n; r.c = s.c; r.span = span;
    r.np = span == tpt2 ? s.np : tiles_of(s.n);
    r.wp = whole && s.np > 1 ? min(max(whole - share0 - before[b], 0), s.np) : 0;
    r.cut_n = r.nc > 1 ? min(s.n, (r.np - r.wp) * span) : 0;
    return r;
  };
  int v[3] = {0, 0, 0};
  ChunkSeq mine_r;
  auto count = [&](const ChunkSeq& r) {
    v[0] += (r.wp + r.nc * (r.np - r.wp)) * p.n_kv;
    v[1] += r.nc * r.cut_n;
    v[2] += r.cut_n;
  };
  for (int b = b0; b < b1; ++b) {
    const ChunkSeq r = record(b);
    if (b == b0) mine_r = r;
    count(r);
  }
  if (bad) atomicOr(p.status, STATUS_BAD_PLAN);
  int incl[3] = {v[0], v[1], v[2]};
  if (active) warp_scan(incl);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (lane == 31) sums[i][warp] = incl[i];
    v[i] = incl[i] - v[i];
  }
  __syncthreads();
  const int n_units = __reduce_add_sync(0xffffffffu, lane < CP_WARPS ? sums[0][lane] : 0);
  if (active) {
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] += __reduce_add_sync(0xffffffffu, lane < warp ? sums[i][lane] : 0);
    for (int b = b0; b < b1; ++b) {
      ChunkSeq r = b == b0 ? mine_r : record(b);
      r.unit0 = v[0];
      r.part0 = v[1];
      r.split0 = v[2];
      if (in_extent(b, 1, p.B)) p.seq[b] = r;
      if (table) {
        unit0[b] = v[0];
        places[b] = make_int4(r.lo, r.c, r.part0, r.wp);
      }
      count(r);
    }
  }
  if (warp == CP_WARPS - 1) {
    const int n_split = __reduce_add_sync(0xffffffffu, lane < CP_WARPS ? sums[2][lane] : 0);
    if (lane == 0) {
      ChunkHead h;
      h.n_units = n_units;
      h.counter = p.grid;      // unit i < grid is CTA i's first
      h.n_split = n_split;
      h.pad = 0;
      *p.head = h;
    }
  }
  // ---- the CTAs' first units, ready to use: found here in parallel, not each by its own CTA's chain of loads
  __syncthreads();
  for (int u = tid; u < p.grid; u += CP_THREADS) {
    ChunkUnit d;
    d.live = 0;
    if (u < n_units) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((table ? unit0[mid] : p.seq[mid].unit0) <= u) lo = mid; else hi = mid;
      }
      ChunkSeq r;
      if (table) {
        const int4 a = shapes[lo], q = places[lo];
        cut(a.z, C, inv, r.nc, r.ct);
        r.unit0 = unit0[lo]; r.lo = q.x; r.n = a.x; r.c = q.y; r.wp = q.w; r.part0 = q.z; r.span = span;
        r.np = span == tpt2 ? a.y : tiles_of(a.x);
        r.cut_n = r.nc > 1 ? min(a.x, (r.np - q.w) * span) : 0;
      } else {
        r = p.seq[lo];
      }
      make_unit(p, r, lo, u, d);
    }
    if (in_extent(u, 1, p.grid)) p.first[u] = d;
  }
}

// ------------------------------------------------------------------------------------- attention
// Tiles before a unit's last copies at which its CTA takes the next one: late, so that what is left goes to
// those who are done (taken at the unit's start: 1248 tokens of 32/4 heads x 128 from an empty cache 33.2 us
// against 29.3, 1216 28.6 both, 64 sequences of 3-5 tokens 213 against 208, nine ragged prompts 18.2 against
// 16.9), but early enough to hide the look-up.
constexpr int kAskTiles = 2;
template <int HD>
struct CaSmem {
  static constexpr uint32_t TILE = 128 * HD * 2;             // one Q, K or V tile
  static constexpr int SLOTS = HD == 128 ? 5 : 10;           // K/V ring: 160 KB
  static constexpr uint32_t OFF_Q = 0;                       // 2 Q tiles
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_ML = OFF_KV + SLOTS * TILE;  // group 1's (m, l) of a lone Q tile
  static constexpr uint32_t OFF_UNIT = OFF_ML + 128 * 8;     // 2 unit records
  static constexpr uint32_t OFF_BAR = OFF_UNIT + 2 * 64;
  static constexpr uint32_t TOTAL = OFF_BAR + 384 + 1024;
};

// Barriers, one arrival each unless noted.
enum : int {
  BAR_Q_FULL = 0,    // [2] per Q slot
  BAR_Q_EMPTY = 2,   // [2]
  BAR_U_FULL = 4,    // [2] per unit record
  BAR_U_EMPTY = 6,   // [2] MMA warp and 8 softmax warps
  BAR_S_FULL = 8,    // [2] per group
  BAR_O_DONE = 10,   // [2]
  BAR_P_FULL = 12,   // [2][2] per group and half of P; 128 threads
  BAR_O_FREE = 16,   // [2] 128 threads
  BAR_ML_FULL = 18,  // 128 threads
  BAR_DRAIN = 19,
  BAR_KV_FULL = 20,  // [NS], then [NS] empty ones
};

// Element-wise: non-finite bf16 values of a 16-byte piece replaced by 0; returns whether there were any.
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
  const uint32_t f = nonfinite_bits(w);
  if (f & 0x8000u) w &= 0xFFFF0000u;
  if (f & 0x80000000u) w &= 0x0000FFFFu;
  return w;
}

// Keys past the last visible one of a row's 32 scores.
__device__ __forceinline__ void mask_keys(uint32_t (&v)[32], int seen) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (k > seen) v[k] = __float_as_uint(-INFINITY);
}
__device__ __forceinline__ float row_max(const uint32_t (&v)[32]) {
  float m0 = __uint_as_float(v[0]), m1 = __uint_as_float(v[1]);
#pragma unroll
  for (int k = 2; k < 30; k += 4) {
    m0 = max3(m0, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
    m1 = max3(m1, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
  }
  return fmaxf(max3(m0, __uint_as_float(v[30]), __uint_as_float(v[31])), m1);
}
// 32 scores of a row -> 16 bf16 pairs of P = 2^(s * scale - m); the fp32 values are added to the row sums.  P is
// rounded (2^-9 of each weight) because the tensor core takes both operands of the second product in V's type.
__device__ __forceinline__ void exp_pack(const uint32_t (&v)[32], uint32_t* w, float scale, float m, float& ls0,
                                         float& ls1) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a0, a1;
    fma_f32x2(a0, a1, __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]), scale, scale, -m, -m);
    const float p0 = ex2(a0);
    const float p1 = ex2(a1);
    add_f32x2(ls0, ls1, p0, p1);
    w[e] = pack_bf16x2(p0, p1);
  }
}

// The non-finite values among keys j0..j1 of sequence b, added to the row stored at `at` (which was summed
// without them).  Called for tiles at a sequence's end only, and only when one was met.
template <int HD>
__device__ __noinline__ void add_nonfinite(const ChunkParams& p, int b, int g, int j0, int j1, int64_t at, bool part) {
  for (int j = j0; j <= j1; ++j) {
    const int page = p.block_table[(int64_t)b * p.max_pages + j / 128];
    if (page < 0 || page >= p.n_pages) continue;
    const uint16_t* vr = p.v_pool + (((int64_t)page * 128 + j % 128) * p.n_kv + g) * HD;
    for (int k = 0; k < HD; ++k) {
      const float a = bf2f(vr[k]);
      if (fabsf(a) < INFINITY) continue;
      if (part) p.part_o[at * HD + k] += a;
      else p.o[at * HD + k] = f2bf(bf2f(p.o[at * HD + k]) + a);
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(CA_THREADS, 1) chunk_attn_kernel(const __grid_constant__ ChunkParams p) {
  using L = CaSmem<HD>;
  constexpr int HALVES = HD / 64;
  constexpr int NS = L::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars + BAR_Q_FULL;
  uint64_t* q_empty = bars + BAR_Q_EMPTY;
  uint64_t* u_full = bars + BAR_U_FULL;
  uint64_t* u_empty = bars + BAR_U_EMPTY;
  uint64_t* s_full = bars + BAR_S_FULL;
  uint64_t* o_done = bars + BAR_O_DONE;
  uint64_t* p_full = bars + BAR_P_FULL;
  uint64_t* o_free = bars + BAR_O_FREE;
  uint64_t* ml_full = bars + BAR_ML_FULL;
  uint64_t* kv_full = bars + BAR_KV_FULL;
  uint64_t* kv_empty = kv_full + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + NS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* dirty = reinterpret_cast<volatile int*>(tmem_slot + 2);   // serial of the last unit with non-finite V
  volatile ChunkUnit* units = reinterpret_cast<volatile ChunkUnit*>(smem + L::OFF_UNIT);
  float2* ml = reinterpret_cast<float2*>(smem + L::OFF_ML);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < BAR_KV_FULL + 2 * NS; ++i)
      mbar_init(&bars[i], i >= BAR_U_EMPTY && i < BAR_U_EMPTY + 2 ? 9
                          : i >= BAR_P_FULL && i <= BAR_ML_FULL   ? 128
                                                                  : 1);
    *abort_flag = 0;
    *dirty = -1;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmQ);
    tma_prefetch_desc(&p.tmK);
    tma_prefetch_desc(&p.tmV);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, CA_TMEM_COLS); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  pdl_wait();      // the plan
  pdl_trigger();   // the merge may start: what it reads before its own wait is the plan's

  if (warp < 4) {
    regs_give<CA_REGS_ISSUE>();
    if (warp == 0) {  // ---------------------------------------------------- units and TMA (whole warp)
      ChunkUnit d = p.first[blockIdx.x];
      const int n_units = p.head->n_units;
      const bool more = n_units > p.grid;   // units besides every CTA's first
      int next = 0, hint = 0, serial = 0, qi = 0, e = 0;
      bool ok = true, asked = false;
      const uint32_t q_bytes = (uint32_t)(HALVES * p.r * p.tpt * 128);
      while (ok) {
        while (!d.live && more) {   // the next unit that has keys
          if (!asked && lane == 0) next = atomicAdd(&p.head->counter, 1);
          asked = false;
          const int u = __shfl_sync(0xffffffffu, next, 0);
          if (u >= n_units) break;
          hint += warp_search(p.B - hint, u, [&](int b) { return p.seq[hint + b].unit0; });
          make_unit(p, p.seq[hint], hint, u, d);
        }
        // the page ids come 32 at a time, the first on their way while the unit is handed over
        const int nt = d.lone ? d.n0 + d.n1 : d.n0;
        const int* pages = p.block_table + (int64_t)d.b * p.max_pages + d.t0;
        int page_reg = d.live && lane < nt ? __ldg(pages + lane) : 0;
        // ---- hand the unit over
        const int us = serial & 1;
        if (lane == 0) {
          ok = mbar_wait(&u_empty[us], ((serial >> 1) & 1) ^ 1, abort_flag, p.status);
          if (ok) {
            volatile int* dst = reinterpret_cast<volatile int*>(units + us);
            const int* src = reinterpret_cast<const int*>(&d);
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[i] = src[i];
            mbar_arrive(&u_full[us]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok || !d.live) break;
        ++serial;
        // ---- Q tiles
        for (int x = 0; ok && x < (d.lone ? 1 : 2); ++x) {
          if (!d.lone && x == 1 && d.n1 == 0) break;
          if (lane == 0) {
            const int qs = qi & 1, row = x == 0 ? d.row0 : d.row1;
            ok = mbar_wait(&q_empty[qs], ((qi >> 1) & 1) ^ 1, abort_flag, p.status);
            if (ok && !box_in(0, HD, (int64_t)d.g * p.r, p.n_q, row, p.T)) { *abort_flag = 1; ok = false; }
            if (ok) {
              mbar_arrive_expect_tx(&q_full[qs], q_bytes);
              for (int hh = 0; hh < HALVES; ++hh)
                tma_load_3d(sbase + L::OFF_Q + qs * L::TILE + hh * 16384, &p.tmQ, &q_full[qs], hh * 64, d.g * p.r, row);
            }
          }
          if (ok) ++qi;
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // ---- K and V tiles
        for (int t = 0; ok && t < nt; ++t) {
          if (more && t == max(0, nt - kAskTiles)) {   // the next unit is asked for now and looked at later
            if (lane == 0) next = atomicAdd(&p.head->counter, 1);
            asked = true;
          }
          if ((t & 31) == 0) {
            if (t > 0) page_reg = t + lane < nt ? __ldg(pages + t + lane) : 0;
            if (page_reg < 0 || page_reg >= p.n_pages) {
              atomicOr(p.status, STATUS_BAD_PLAN);
              page_reg = p.n_pages;            // outside the tensor: the copy fills the tile with zeros
            }
          }
          const int page = __shfl_sync(0xffffffffu, page_reg, t & 31);
          if (lane == 0) {
            for (int kv = 0; ok && kv < 2; ++kv, ++e) {
              const int slot = e % NS;
              ok = mbar_wait(&kv_empty[slot], ((e / NS) & 1) ^ 1, abort_flag, p.status);
              if (ok && !box_in(0, HD, d.g, p.n_kv, 0, 128, page, (int64_t)p.n_pages + 1)) { *abort_flag = 1; ok = false; }
              if (!ok) break;
              mbar_arrive_expect_tx(&kv_full[slot], L::TILE);
              for (int hh = 0; hh < HALVES; ++hh)
                tma_load_4d(sbase + L::OFF_KV + slot * L::TILE + hh * 16384, kv ? &p.tmV : &p.tmK, &kv_full[slot], hh * 64,
                            d.g, 0, page);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        d.live = 0;
      }
      // every copy issued has landed before the CTA leaves (at once, unless a wait ran out)
      if (lane == 0) {
        int no_abort = 0;
        for (int k = max(0, e - NS); k < e; ++k) mbar_wait(&kv_full[k % NS], (k / NS) & 1, &no_abort, p.status);
        for (int k = max(0, qi - 2); k < qi; ++k) mbar_wait(&q_full[k & 1], (k >> 1) & 1, &no_abort, p.status);
      }
    } else if (warp == 1) {  // ------------------------------------------ MMA issuer (whole warp)
      // Every lane runs the loop and one elected lane's instructions take effect, and every wait ends by a
      // vote: the control flow stays uniform, so descriptors live in uniform registers.  Issued from a
      // one-lane branch, 8 MMAs took 600-900 cycles against the 512 they execute in (clock stamps, hd 128):
      // 2048 tokens after 30720 took 1014 us, 807 from the whole warp, 756 with P in halves and votes.
      const uint32_t one = elect_one();
      const uint32_t idesc_s = idesc_bf16(128, 128);
      const uint32_t idesc_o = idesc_bf16(128, HD, /*b_mn_major=*/true);
      const uint64_t kdesc = sdesc_sw128(sbase + L::OFF_KV, 16, 1024);
      const uint64_t vdesc = sdesc_sw128(sbase + L::OFF_KV, 16384, 1024);
      const uint64_t qdesc = sdesc_sw128(sbase + L::OFF_Q, 16, 1024);
      constexpr int TILE16 = (int)(L::TILE >> 4);
      constexpr int BAR_KV_EMPTY = BAR_KV_FULL + NS;
      const uint32_t bar = smem_u32(bars);
      auto B = [&](int i) { return bar + 8u * (uint32_t)i; };
      auto wait = [&](int i, int parity) { return mbar_wait_warp(B(i), (uint32_t)parity, abort_flag, p.status); };
      int qi = 0;                            // Q tiles so far
      int ks = 0, kph = 0, vs = 1, vph = 0;  // ring slot and phase of the next K and V tile
      int rounds[2] = {0, 0}, used[2] = {0, 0};   // per group: rounds, and units with any
      bool ok = true;
      for (int serial = 0; ok; ++serial) {
        const int us = serial & 1;
        if (!wait(BAR_U_FULL + us, (serial >> 1) & 1)) break;
        volatile const ChunkUnit* d = units + us;
        const int live = __shfl_sync(0xffffffffu, d->live, 0), lone = __shfl_sync(0xffffffffu, d->lone, 0);
        const int n0 = __shfl_sync(0xffffffffu, d->n0, 0), n1 = __shfl_sync(0xffffffffu, d->n1, 0);
        if (!live) break;
        if (one) mbar_arrive(bars + BAR_U_EMPTY + us);   // its fields are in registers
        const int nq = lone || n1 == 0 ? 1 : 2;
        // S_x = Q_x K^T of the next K tile; `last`: no other group reads the tile
        auto issue_s = [&](int x, int i, bool last) -> bool {
          if ((x == 0 || lone) && !wait(BAR_KV_FULL + ks, kph)) return false;
          tc_fence_after();
          const int qs = (qi + (lone ? 0 : x)) & 1;
          const uint64_t ad0 = qdesc + (uint64_t)(qs * TILE16);
          const uint64_t bd0 = kdesc + (uint64_t)(ks * TILE16);
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint64_t off = (uint64_t)(((k >> 2) * 16384 + (k & 3) * 32) >> 4);
            tc_mma_if(one, tmem + x * 128, ad0 + off, bd0 + off, idesc_s, k > 0 ? 1u : 0u);
          }
          tc_commit_if(one, B(BAR_S_FULL + x));
          if (last) {
            tc_commit_if(one, B(BAR_KV_EMPTY + ks));
            ks += 2;
            if (ks >= NS) { ks -= NS; kph ^= 1; }
          }
          if (lone ? 2 * i + x == n0 + n1 - 1 : i == (x ? n1 : n0) - 1) tc_commit_if(one, B(BAR_Q_EMPTY + qs));
          return true;
        };
        // O_x += P_x V of the next V tile
        auto issue_pv = [&](int x, int i, bool last) -> bool {
          if ((x == 0 || lone) && !wait(BAR_KV_FULL + vs, vph)) return false;
          const uint64_t bd0 = vdesc + (uint64_t)(vs * TILE16);
#pragma unroll
          for (int half = 0; half < 2; ++half) {   // P comes in two halves of 64 keys
            if (!wait(BAR_P_FULL + 2 * x + half, rounds[x] & 1)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)   // 16 keys per step: TMEM columns 8k..8k+7 of P_x
              tc_mma_ts_if(one, tmem + 256 + x * 128, tmem + x * 128 + k * 8, bd0 + (uint64_t)(k * 2048 >> 4), idesc_o,
                           k > 0 ? 1u : (i > 0 ? 1u : 0u));
          }
          if (i == (x ? n1 : n0) - 1) tc_commit_if(one, B(BAR_O_DONE + x));
          ++rounds[x];
          if (last) {
            tc_commit_if(one, B(BAR_KV_EMPTY + vs));
            vs += 2;
            if (vs >= NS) { vs -= NS; vph ^= 1; }
          }
          return true;
        };
        ok = wait(BAR_Q_FULL + (qi & 1), (qi >> 1) & 1) &&
             (nq == 1 || wait(BAR_Q_FULL + ((qi + 1) & 1), ((qi + 1) >> 1) & 1));
        if (ok) ok = issue_s(0, 0, lone || n1 == 0);
        if (ok && n1 > 0) ok = issue_s(1, 0, true);
        // the first P V of a unit overwrites O_x: what the last unit that used it left must have been
        // read (o_free counts those units only: a phase is never completed before it is waited for)
        if (ok) ok = wait(BAR_O_FREE, (used[0]++ & 1) ^ 1);
        if (ok && n1 > 0) ok = wait(BAR_O_FREE + 1, (used[1]++ & 1) ^ 1);
        for (int i = 0; ok && i < n0; ++i) {
          ok = issue_pv(0, i, lone || i >= n1);
          if (ok && i + 1 < n0) ok = issue_s(0, i + 1, lone || i + 1 >= n1);
          if (!ok || i >= n1) continue;
          ok = issue_pv(1, i, true);
          if (ok && i + 1 < n1) ok = issue_s(1, i + 1, true);
        }
        qi += nq;
      }
      int no_abort = 0;
      tc_commit_if(one, B(BAR_DRAIN));
      mbar_wait(bars + BAR_DRAIN, 0, &no_abort, p.status);
    }
  } else {  // ------------------------------------------------------------ softmax groups
    regs_take<CA_REGS_SOFTMAX>();
    const int x = (warp - 4) >> 2;
    const int qw = warp & 3;
    const int row = qw * 32 + lane;                     // TMEM lane = Q tile row
    const uint32_t lane_off = (uint32_t)(qw * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off;
    const uint32_t tO = tmem + 256 + x * 128 + lane_off;
    const int tok_in = row / p.r, head_in = row - tok_in * p.r;
    const bool row_used = row < p.r * p.tpt;
    int rc = 0, unit_count = 0, lone_count = 0;         // rounds of this group, units with any, lone units with n1 > 0
    int e = 0;                                          // ring entries of the units before
    bool ok = true;
    for (int serial = 0; ok; ++serial) {
      const int us = serial & 1;
      if (!mbar_wait_short(smem_u32(&u_full[us]), (serial >> 1) & 1, abort_flag, p.status)) break;
      // read from shared memory where it is used, and released at the unit's end: registers are short
      const volatile ChunkUnit& d = units[us];
      if (!d.live) break;
      const int n1 = d.n1, n = x ? n1 : d.n0, lone = d.lone;
      const int tok = (x ? d.row1 : d.row0) + tok_in;   // packed row of the token
      const int qpos = tok + d.pos_off;
      const int full = (qpos - tok_in + 1) / 128;       // tiles every row of the Q tile sees
      float m_ref = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i, ++rc) {
        const int jt = lone ? 2 * i + x : i, j = d.t0 + jt;
        if (!mbar_wait_short(smem_u32(&s_full[x]), rc & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after();
        const int kbase = j * 128;
        const int seen = j >= full ? qpos - kbase : 127;   // keys 0..seen of the tile are visible
        // Tiles with keys that some row does not see: P is 0 there, and 0 x V must stay 0.  Rows past
        // the sequence's end are zeroed; non-finite elements of the others too, and what they add to
        // the rows that do see them is added at the end (below).  Thread `row` takes key `row`.
        if (j >= d.clean) {
          const int en = e + 2 * jt + 1, slot = en % NS;
          if (!mbar_wait_short(smem_u32(&kv_full[slot]), (en / NS) & 1, abort_flag, p.status)) { ok = false; break; }
          uint8_t* vrow = smem + L::OFF_KV + slot * L::TILE + row * 128;
          const bool past = kbase + row >= d.kv_len;
#pragma unroll
          for (int c = 0; c < HD / 8; ++c) {   // pieces in an order that spreads the banks
            uint4* at = reinterpret_cast<uint4*>(vrow + (c >> 3) * 16384 + ((c ^ row) & 7) * 16);
            if (past) {
              *at = make_uint4(0, 0, 0, 0);
            } else {
              const uint4 w = *at;
              const uint32_t f = nonfinite_bits(w.x) | nonfinite_bits(w.y) | nonfinite_bits(w.z) | nonfinite_bits(w.w);
              if (f) {   // the mark first: who finds the values gone finds the mark
                *dirty = serial;
                __threadfence_block();
                *at = make_uint4(drop_nonfinite(w.x), drop_nonfinite(w.y), drop_nonfinite(w.z), drop_nonfinite(w.w));
              }
            }
          }
          fence_proxy_async_smem();
        }
        // A unit's first tile finds its maximum before anything else, a tile with unseen keys has them
        // masked in place: one rolled pass over the scores in TMEM, off the common path.
        if (i == 0 || j >= full) {
          float m = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t t[32];
            tmem_ld32(tS + c, t);
            tc_wait_ld();
            if (j >= full) {
              mask_keys(t, seen - c);
              tmem_st32(tS + c, t);
            }
            m = fmaxf(m, row_max(t));
          }
          tc_wait_st();
          if (i == 0) m_ref = m * p.scale_log2;
        }
        // P in two halves, each handed over as soon as it is stored: the first half's P V runs while the
        // second half is formed.  The first half is formed against the reference maximum so far while
        // the tile's maximum is found (exp2 and max run in different pipes); the rare tile that grows
        // it by more than 2^8 forms it again.
        uint32_t va[32], vb[32], vc[32], vd[32], w[32];
        float l0, l1, l2, l3;
        for (;;) {
          // a row that has seen no key yet keeps m = -inf; its P is 0
          const float mb = m_ref == -INFINITY ? 0.f : m_ref;
          tmem_ld32(tS, va);
          tmem_ld32(tS + 32, vb);
          tmem_ld32(tS + 64, vc);
          tmem_ld32(tS + 96, vd);
          tc_wait_ld();
          l0 = l1 = l2 = l3 = 0.f;
          float m = row_max(va);
          exp_pack(va, w, p.scale_log2, mb, l0, l1);
          m = fmaxf(m, fmaxf(row_max(vb), row_max(vc)));
          exp_pack(vb, w + 16, p.scale_log2, mb, l2, l3);
          const float mt = fmaxf(m, row_max(vd)) * p.scale_log2;
          const bool grow = mt > m_ref + kRescaleLog2;
          if (!__any_sync(0xffffffffu, grow)) break;
          // (i > 0: the first tile's reference is its maximum)  S of this round having arrived, O holds
          // the P V of all the tiles before it
          const float alpha = grow ? ex2(m_ref - mt) : 1.f;
          if (grow) m_ref = mt;
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t ov[16];
            tmem_ld16_at(tO + c * 16, ov);
            tc_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
            tmem_st16(tO + c * 16, ov);
          }
          tc_wait_st();
        }
        if (!ok) break;
        tmem_st32(tS, w);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[2 * x]);
        const float mb = m_ref == -INFINITY ? 0.f : m_ref;
        float l4 = 0.f, l5 = 0.f, l6 = 0.f, l7 = 0.f;
        exp_pack(vc, w, p.scale_log2, mb, l4, l5);
        exp_pack(vd, w + 16, p.scale_log2, mb, l6, l7);
        tmem_st32(tS + 32, w);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[2 * x + 1]);
        l += ((l0 + l1) + (l2 + l3)) + ((l4 + l5) + (l6 + l7));
      }
      const int n_tiles = lone ? d.n0 + n1 : d.n0;
      if (!ok) break;
      // ---- the unit's result
      if (n > 0 && !mbar_wait_short(smem_u32(&o_done[x]), unit_count++ & 1, abort_flag, p.status)) { ok = false; break; }
      e += 2 * n_tiles;
      tc_fence_after();
      if (lone && x == 1) {                         // hand (m, l, O_1) to group 0
        if (n > 0) {
          ml[row] = make_float2(m_ref, l);
          tc_fence_before();
          mbar_arrive(ml_full);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_empty[us]);
        continue;
      }
      float w0 = 1.f, w1 = 0.f;
      const bool merge = lone && n1 > 0;
      if (merge) {
        if (!mbar_wait_short(smem_u32(ml_full), lone_count & 1, abort_flag, p.status)) { ok = false; break; }
        ++lone_count;
        tc_fence_after();
        const float2 o = ml[row];
        const float m = fmaxf(m_ref, o.x);
        const float mu = m == -INFINITY ? 0.f : m;
        w0 = ex2(m_ref - mu);
        w1 = ex2(o.x - mu);
        l = l * w0 + o.y * w1;
        m_ref = m;
      }
      const bool store_part = d.part != INT_MIN;
      const bool live = row_used && tok < d.end && n > 0;
      const int h = d.g * p.r + head_in;
      if (!store_part) {
        const float inv = 1.f / l;
        w0 *= inv;
        w1 *= inv;
      }
      const int64_t at = store_part ? (int64_t)(tok + d.part) * p.n_q + h : (int64_t)tok * p.n_q + h;
      const int64_t extent = store_part ? (int64_t)p.part_rows * p.n_q : (int64_t)p.T * p.n_q;
      const bool inside = !live || in_extent(at, 1, extent);
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tO + c * 32, v);
        if (merge) {
          uint32_t v1[32];
          tmem_ld32(tO + 128 + c * 32, v1);
          tc_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            v[k] = __float_as_uint(fmaf(__uint_as_float(v1[k]), w1, __uint_as_float(v[k]) * w0));
        } else {
          tc_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * w0);
        }
        if (live && inside && store_part) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(p.part_o + at * HD + c * 32);   // whole sectors: 32 bytes each
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + k), "r"(v[k]), "r"(v[k + 1]),
                         "r"(v[k + 2]), "r"(v[k + 3]), "r"(v[k + 4]), "r"(v[k + 5]), "r"(v[k + 6]), "r"(v[k + 7])
                         : "memory");
        } else if (live && inside) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + at * HD + c * 32);
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            dst[k / 4] = make_uint4(pack_bf16x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])),
                                    pack_bf16x2(__uint_as_float(v[2 * k + 2]), __uint_as_float(v[2 * k + 3])),
                                    pack_bf16x2(__uint_as_float(v[2 * k + 4]), __uint_as_float(v[2 * k + 5])),
                                    pack_bf16x2(__uint_as_float(v[2 * k + 6]), __uint_as_float(v[2 * k + 7])));
        }
      }
      tc_fence_before();
      if (n > 0) mbar_arrive(&o_free[x]);
      if (merge) mbar_arrive(&o_free[1]);
      if (live && inside) {
        if (store_part) p.part_ml[at] = make_float2(m_ref, l);
        // (a later serial: group 1 met such values in its next unit already; then this looks without need)
        if (*dirty >= serial)
          add_nonfinite<HD>(p, d.b, d.g, max(d.clean, d.t0) * 128, min(qpos, (d.t0 + (lone ? n_tiles : n)) * 128 - 1), at,
                            store_part);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&u_empty[us]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, CA_TMEM_COLS);
  }
}

// ----------------------------------------------------------------------------------------- merge
// o = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k over the chunks k that hold keys the token sees.
// A warp takes one head of a token of the cut sequences, the loads of CC_CHUNKS of its parts in flight
// together (each waiting for its own, 45 us for the 136 MB of parts of 2048 tokens x 32 heads; now 17).  Four
// heads a warp, to have as many loads in flight from few chunks, cost registers and lost everywhere: 64
// sequences of 3-5 tokens 224 us for the whole call against 217, three single tokens 19.5 against 14.6.
constexpr int CC_CHUNKS = 4;

template <int HD>
__global__ void __launch_bounds__(256, 4) chunk_combine_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int PER = HD / 32;
  using Vec = typename std::conditional<PER == 4, float4, float2>::type;
  const int lane = threadIdx.x & 31, warps = gridDim.x * 8;
  const int total = p.head->n_split * p.n_q;   // no more than the parts
  bool waited = false;
  for (int w = blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += warps) {
    const int x = div_inv(w, p.n_q, p.inv_q), h = w - x * p.n_q;
    // sequences that were not cut hold no split rows, so the last one starting at or before x is it
    const int b = warp_search(p.B, x, [&](int i) { return p.seq[i].split0; });
    const ChunkSeq s = p.seq[b];
    const int i = x - s.split0;
    const int nk = min(s.nc, cdiv((s.c + i) / 128 + 1, s.ct));
    const int64_t stride = (int64_t)s.cut_n * p.n_q, row0 = (int64_t)(s.part0 + i) * p.n_q + h;
    if (!waited) pdl_wait();   // the parts
    waited = true;
    float2 a = lane < nk ? p.part_ml[row0 + lane * stride] : make_float2(-INFINITY, 0.f);
    float M = a.x;
    for (int k = lane + 32; k < nk; k += 32) M = fmaxf(M, p.part_ml[row0 + k * stride].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;
    float l = 0.f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < nk; k0 += 32) {
      if (k0 > 0) a = k0 + lane < nk ? p.part_ml[row0 + (k0 + lane) * stride] : make_float2(-INFINITY, 0.f);
      const float wl = ex2(a.x - M);   // 0 past the last chunk
      l += wl * a.y;
      const int kn = min(32, nk - k0);
      for (int k = 0; k < kn; k += CC_CHUNKS) {
        const float* src = p.part_o + (row0 + (k0 + k) * stride) * HD + lane * PER;
        Vec v[CC_CHUNKS];
#pragma unroll
        for (int q = 0; q < CC_CHUNKS; ++q)
          if (k + q < kn) v[q] = *reinterpret_cast<const Vec*>(src + q * stride * HD);
#pragma unroll
        for (int q = 0; q < CC_CHUNKS; ++q) {
          const float wk = __shfl_sync(0xffffffffu, wl, (k + q) & 31);
          if (k + q < kn) {
            const float* f = reinterpret_cast<const float*>(&v[q]);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(wk, f[e], acc[e]);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = 1.f / l;
    const int64_t at = ((int64_t)(s.lo + i) * p.n_q + h) * HD + lane * PER;
    if (!in_extent(at, PER, (int64_t)p.T * p.n_q * HD)) continue;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + at);
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  }
  if (!waited) pdl_wait();   // every CTA of the merge outlives the attention: the next call may reuse the workspace
}

size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

// Partial rows the workspace holds: no more than every token in chunks of one tile, and no more than
// about 8 x 152 units of two full Q tiles (162 MB at hd 128), past which cutting pays no more.
int64_t part_rows_of(int64_t T, int64_t n_q, int64_t max_pos) {
  const int64_t tiles = max_pos / 128 + 1;
  if (tiles < 2) return 0;
  return std::min(T * tiles, std::max<int64_t>(1, 8 * 152 * 256 / n_q));
}

template <int HD>
int launch_hd(const ChunkAttnDesc& a, int num_sms, cudaStream_t st) {
  ChunkParams p;
  memset(&p, 0, sizeof(p));
  const int r = (int)(a.n_q / a.n_kv), tpt = 128 / r;
  if (!encode_tmap_3d_bf16(&p.tmQ, a.q, HD, (uint64_t)a.n_q, (uint64_t)a.T, HD * 2, (uint64_t)a.n_q * HD * 2, 64,
                           (uint32_t)r, (uint32_t)tpt))
    return -1;
  const uint64_t dims[4] = {HD, (uint64_t)a.n_kv, 128, (uint64_t)a.n_pages};
  const uint64_t strides[3] = {HD * 2, (uint64_t)a.n_kv * HD * 2, (uint64_t)128 * a.n_kv * HD * 2};
  const uint32_t box[4] = {64, 1, 128, 1};
  if (!encode_tmap_4d_bf16(&p.tmK, a.k_pool, dims, strides, box) || !encode_tmap_4d_bf16(&p.tmV, a.v_pool, dims, strides, box))
    return -1;
  p.o = static_cast<uint16_t*>(a.o);
  p.v_pool = static_cast<const uint16_t*>(a.v_pool);
  p.block_table = a.block_table; p.cu_new = a.cu_new; p.n_cached = a.n_cached;
  p.B = (int)a.B; p.T = (int)a.T; p.n_q = (int)a.n_q; p.n_kv = (int)a.n_kv; p.r = r; p.tpt = tpt;
  p.n_pages = (int)a.n_pages; p.max_pages = (int)a.max_pages; p.max_pos = (int)a.max_pos;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part_rows = (int)part_rows_of(a.T, a.n_q, a.max_pos);
  char* ws = static_cast<char*>(a.ws);
  p.head = reinterpret_cast<ChunkHead*>(ws);
  p.first = reinterpret_cast<ChunkUnit*>(ws + 256);
  ws += 256 + kMaxGrid * sizeof(ChunkUnit);
  p.seq = reinterpret_cast<ChunkSeq*>(ws);
  ws += round256((size_t)a.B * sizeof(ChunkSeq));
  ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));   // 32-byte stores
  p.part_o = reinterpret_cast<float*>(ws);
  ws += round256((size_t)p.part_rows * a.n_q * HD * 4);
  p.part_ml = reinterpret_cast<float2*>(ws);
  p.grid = std::min(num_sms, kMaxGrid);
  p.inv_q = inverse(a.n_q);
  p.inv_kv = inverse(a.n_kv);
  p.inv_grid = inverse(p.grid);
  p.inv_pair = inverse(2 * tpt);
  p.inv_tile = inverse(tpt);
  p.status = a.status;
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return -1;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(chunk_attn_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, CaSmem<HD>::TOTAL) !=
        cudaSuccess)
      return -1;
    attr_set[dev] = true;
  }
  // launched plainly: the merge reads the plan's records before its own dependency wait, and they are complete
  // when the attention triggers it, because the attention has waited for the plan and the plan for all before
  chunk_plan_kernel<<<1, CP_THREADS, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  // the attention's set-up overlaps the plan, and the merge's launch the attention
  const bool pdl = pdl_enabled();
  set_pdl(true);
  cudaError_t e = launch_k(chunk_attn_kernel<HD>, dim3(p.grid), dim3(CA_THREADS), CaSmem<HD>::TOTAL, st, p);
  if (e == cudaSuccess && p.part_rows > 0) {
    const int64_t warps = (a.T * a.n_q + 7) / 8;
    e = launch_k(chunk_combine_kernel<HD>, dim3((unsigned)std::min<int64_t>(warps, 8 * num_sms)), dim3(256), 0, st, p);
  }
  set_pdl(pdl);
  return e == cudaSuccess ? 0 : -1;
}

}  // namespace

// Units are counted in 32 bits.
bool chunk_attn_supported(int64_t B, int64_t T, int64_t n_q, int64_t n_kv) {
  const int64_t tpt = 128 / (n_q / n_kv);
  return T <= INT32_MAX / 2 && B <= INT32_MAX / 256 && (T / (2 * tpt) + B) * n_kv <= (int64_t)1 << 28 && n_q <= 65536;
}

size_t chunk_attn_ws_bytes(int64_t B, int64_t T, int64_t n_q, int64_t, int64_t hd, int64_t max_pos) {
  const size_t rows = (size_t)part_rows_of(T, n_q, max_pos) * n_q;
  return 256 + kMaxGrid * sizeof(ChunkUnit) + round256((size_t)B * sizeof(ChunkSeq)) + round256(rows * hd * 4) + 32 +
         round256(rows * 8);
}

int launch_chunk_attn(const ChunkAttnDesc& a, int num_sms, cudaStream_t st) {
  return a.hd == 128 ? launch_hd<128>(a, num_sms, st) : launch_hd<64>(a, num_sms, st);
}

LLAMA_DEFINE_BOUNDS_READER(chunk_attn)

}  // namespace llama
