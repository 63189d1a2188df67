// One-token GQA attention over an 8-bit paged cache with a scale per position and KV head ("LLaMA-3 8B ...", section 九:
// a decode step reads every cached key and value once; 8-bit rows halve that).
//
//   o_h = sum_j exp(s_hj) vs_j c_j / sum_j exp(s_hj),   s_hj = ks_j (q_h . kc_j) / sqrt(hd)
//
// kc_j, c_j the E4M3 codes of key and value j of the query head's KV head, ks_j, vs_j their scales.
//
// What bounds it: the codes and scales are read once, 2 (hd + 4) bytes per position and KV head, at a few operations
// per byte, so HBM does, where there are enough tiles, and the latency of one tile's chain where there are few.  64 sequences
// of 2-8 K positions, 32/8 heads x 128 (671 MB): 109.0 us = 6.2 TB/s, 92% of a copy's rate; one of 131000 (277 MB) 48.0 us,
// 86%; three of 100 to 900: 9.2 us.  With 8 query heads and more per KV head the softmax comes nearest to it (64 sequences of 64/8
// heads 124 us), and with 16 over one KV head it sets the pace (16/1 heads 35 us where the bytes take 14).
//
// Tiles.  A tile is one page (128 positions) by 128 bytes of a row: one KV head of 128, or two of 64 side by side, which
//   one product serves (each head's query rows hold zeros in the other's bytes).  tcgen05 kind::f8f6f4 reads the codes as
//   TMA lands them: S^T = K Q^T (M = 128 keys) and O^T += V^T P^T (M = 128 bytes of the row, V as the MN-major operand).
//   One thread per key does the softmax of its tile; the scales come with the tile by bulk copies, a head's 128
//   scales of a page being contiguous.
// Operands.  The other side has 8 bits an element too.  q enters as x = hi + 2^-5 lo in E4M3, hi = e4m3(x), lo = e4m3(32 (x - hi)): all
//   of a bf16's bits down to 2^-14 of the row's largest, off by 2^-22 of that below.  P enters as three E5M2 values, x = a + b/16 + c/256, each the
//   rounding of what the ones before it leave: off by 2^-11 of x (2^-3 after the first, 2^-4 more with each further one) down to 2^-25
//   of the row's largest, by 2^-38 of that below.  So a tail of 2^24 small weights beside a heavy one keeps its sum, where
//   E4M3's few binades lose it (two E4M3 parts: a tail that is 30% of the row, off by 14% of itself).  The further rows ride
//   in the padding of the operand's N = 16 (P: 32 for 8 rows, 48 for 16).
// Scales.  A key's scale multiplies its row of S^T.  A value's scale cannot leave the sum over keys, so P holds
//   w_j = exp(s_j) vs_j, as 2^(s_j + log2 vs_j - m) with m the running maximum of that exponent: the largest
//   product, not the largest weight, has the format's full precision.  The weights themselves, for their sum, are exponentials of
//   their own against the same m, 2^(s_j - m): where value scales lie far apart a key of small values may have most of the
//   weight.  For scales of 2^-100 .. 2^100 the largest weight lies in 2^-100 .. 2^102, so that 2^24 of them, and twice that, are
//   finite in fp32, and what is 2^-49 of the largest is still there (the exponential keeps subnormal results).  Sums are brought
//   to a new m by its square root twice, since 2^(m - m') may be nothing where the sum is large.
// Split.  The pages of all sequences, one after the other, are cut into equal ranges; range i of head group g is CTA
//   i * groups + g, so the CTAs that run side by side read all heads of the same pages (a page's rows are contiguous
//   over heads).  A sequence inside one range is finished there; of one that a cut goes through, each range leaves a part
//   (m, l, O) in the workspace, at most two parts a range, and a second kernel joins them.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "e4m3.cuh"
#include "kernels.h"

namespace llama {
namespace {

// Threads: warp 0 TMA and q -> E4M3 hi / lo, warp 1 MMA, then SG groups of four softmax warps.  With 8 rows and more the softmax
// sets the pace, so two groups share the rows of a tile (a thread has one key of four or eight rows); a warp of its own for q
// would leave two such CTAs 80 registers a thread, and eight rows' state spills there.
constexpr int dp_threads(int SG) { return 64 + 128 * SG; }
// two CTAs per SM (2 x 114 KB of shared memory), so that one's hand-offs overlap the other's
constexpr int DP_KSTAGES = 3;
constexpr int DP_VSTAGES = 2;
constexpr int DP_SSTAGES = 4;     // scales
constexpr int DP_CTAS_PER_SM = 2;
constexpr uint32_t DP_TMEM_COLS = 128;   // S^T 2 x NQ (cols 0..63), O^T NP (cols 64..111)
// O and l keep their reference until a tile's maximum exceeds it by 2 (log2), so w <= 4 before the 2^13 below
// and w * 2^13 <= 2^15 stays under E5M2's 57344 (kDpOut takes the factors out of O / l); half a step there is 2^11, so 16 (x - a) <= 2^15 too.
constexpr float kDpRescaleLog2 = 2.0f;
constexpr float kDpPScaleLog2 = 13.0f;
constexpr float kDpLScaleLog2 = 1.0f;                        // l's weights are 2^1 2^(s - m)
constexpr float kDpOut = 1.f / 4096.f;                       // O / l to the row: 2^(1 - 13)
constexpr float kDpLo = 32.0f;      // q's second part
constexpr float kDpStep = 16.0f;    // each further part of P

struct SplitInfo { int b, last; };   // the sequence whose first part is this range's tail (-1: none), the range of its last part

struct DecodeAttn8pParams {   // 128-byte aligned by its tensor maps
  CUtensorMap tmK;   // codes as [n_pages * 128, n_kv * hd] bytes, box (128, 128), 128-byte swizzle
  CUtensorMap tmV;
  const uint16_t* q;
  const float *k_scale, *v_scale;
  const int *block_table, *seq_pos;
  uint16_t* o;
  float* part_o;       // [2 n_ranges, groups, R, 128]
  float2* part_ml;     // [2 n_ranges, groups, R]  (m in log2 units, l)
  SplitInfo* split;    // [n_ranges]
  int B, n_q, n_kv, r, hd, n_pages, max_pos;
  int n_ranges, groups, subs;   // group = (packed KV heads, block of their query heads)
  int64_t max_pages;
  float scale_log2;
  unsigned* status;
};

struct DpSmem {
  static constexpr uint32_t F8 = 128 * 128;     // one code tile
  static constexpr uint32_t OPB = 32 * 128;     // q operand: up to 32 rows of 128 codes
  static constexpr uint32_t PB = 48 * 128;      // P operand
  static constexpr uint32_t SC = 4 * 512;       // scales of a tile: K of two heads, V of two heads
  static constexpr uint32_t OFF_K8 = 0;
  static constexpr uint32_t OFF_V8 = OFF_K8 + DP_KSTAGES * F8;
  static constexpr uint32_t OFF_Q = OFF_V8 + DP_VSTAGES * F8;  // 2 buffers
  static constexpr uint32_t OFF_P = OFF_Q + 2 * OPB;           // 2 buffers
  static constexpr uint32_t OFF_SC = OFF_P + 2 * PB;
  static constexpr uint32_t OFF_RED = OFF_SC + DP_SSTAGES * SC;      // [2 groups][3][4][16] floats
  static constexpr uint32_t OFF_QS = OFF_RED + 2 * 3 * 4 * 16 * 4;   // inverse q scales [2][16]
  static constexpr uint32_t OFF_BAR = OFF_QS + 2 * 16 * 4;
  static constexpr uint32_t TOTAL = OFF_BAR + 512 + 1024;
};
static_assert(DP_CTAS_PER_SM * (DpSmem::TOTAL + 1024) <= 233472, "two CTAs per SM");

enum : int {   // barrier slots
  P_KF = 0, P_VF = 3, P_KE = 5, P_VE = 8, P_QR = 10, P_QE = 12, P_SF = 14, P_SFREE = 16, P_PF = 18, P_OD = 20, P_OFREE = 22,
  P_DRAIN = 23, P_QC = 24, P_SCF = 26, P_SCE = 30, P_COUNT = 34
};

__device__ __forceinline__ void tmem_ld16_dp(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
// N columns of 32-bit TMEM cells, 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "columns");
  if constexpr (N == 4) tmem_ld4(taddr, v);
  else if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
  else tmem_ld16_dp(taddr, v);
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&v)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "columns");
  if constexpr (N == 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
  else if constexpr (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  else tmem_st16(taddr, v);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void softmax_sync_dp(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ float warp_max_dp(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Instruction descriptor for kind::f8f6f4 with E4M3 A (format 0), E4M3 or E5M2 B (1) and an fp32 accumulator.
enum : uint32_t { B_E4M3 = 0, B_E5M2 = 1 };
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, uint32_t b_format, bool a_mn_major = false) {
  return (1u << 4) | (b_format << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// x = hi + lo / 32 in E4M3 (a first): returns hi codes, sets lo codes.
__device__ __forceinline__ uint32_t split_fine(float a, float b, uint32_t& lo) {
  const uint32_t hi = e4m3x2(a, b);
  const float2 h = e4m3x2_to_f2(hi);
  lo = e4m3x2((a - h.x) * kDpLo, (b - h.y) * kDpLo);
  return hi;
}
// Two floats to two E5M2 codes (round to nearest even, saturating): a in the low byte; and back, an E5M2 code being the upper byte of
// a half.
__device__ __forceinline__ uint32_t e5m2x2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}
__device__ __forceinline__ float2 e5m2x2_to_f2(uint32_t c) {
  const uint32_t h = __byte_perm(c, 0, 0x1404);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// x = p0 + p1 / 16 + p2 / 256 in E5M2 (a's codes in the low bytes).
__device__ __forceinline__ void split_weights(float a, float b, uint32_t (&p)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    p[k] = e5m2x2(a, b);
    const float2 h = e5m2x2_to_f2(p[k]);
    a = (a - h.x) * kDpStep;
    b = (b - h.y) * kDpStep;
  }
}
// Byte offset of (row n, byte c) in a K-major operand of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128_at(int n, int c) {
  return (uint32_t)(n * 128 + ((((c >> 4) ^ (n & 7))) << 4) + (c & 15));
}

// mbar_wait in few instructions: the roles' loops wait in many places, and together they have to fit the instruction cache.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* status) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) [[likely]] return true;
  const unsigned long long t0 = globaltimer_ns();
  do {
    if (mbar_try_wait(a, parity)) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) [[unlikely]] {
      atomicOr(status, STATUS_TIMEOUT);
      *abort = 1;
    }
  } while (!*abort);
  return false;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_full(float x) {   // with subnormal results
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---- the work split
__device__ __forceinline__ int good_pos(int pos, int max_pos) { return pos < -1 || pos > max_pos ? -1 : pos; }
__device__ __forceinline__ int tiles_at(const DecodeAttn8pParams& p, int b) {
  return (good_pos(__ldg(p.seq_pos + b), p.max_pos) + 128) / 128;
}
__device__ __forceinline__ int64_t range_first(int64_t T, int n, int i) { return (int64_t)i * T / n; }
// The range that holds tile x.
__device__ __forceinline__ int range_with(int64_t T, int n, int64_t x) {
  int i = (int)min((int64_t)n - 1, x * n / T);
  while (i + 1 < n && range_first(T, n, i + 1) <= x) ++i;
  while (i > 0 && range_first(T, n, i) > x) --i;
  return i;
}

// The pieces of a CTA's range: tiles [t0, t1) of sequence b, n_keys positions in all.
struct Pieces { int b, t; int64_t left; int next_pos; };
__device__ __forceinline__ bool next_piece(const DecodeAttn8pParams& p, Pieces& s, int& b, int& t0, int& t1, int& nt, int& n_keys) {
  if (s.left <= 0) return false;
  int pos = good_pos(s.next_pos, p.max_pos);
  while (pos < 0 && s.b + 1 < p.B) pos = good_pos(__ldg(p.seq_pos + ++s.b), p.max_pos);   // empty sequences have no tiles
  if (pos < 0) return false;
  b = s.b;
  t0 = s.t;
  nt = (pos + 128) / 128;
  t1 = (int)min((int64_t)nt, t0 + s.left);
  n_keys = pos + 1;
  s.left -= t1 - t0;
  s.t = 0;
  if (s.left > 0 && s.b + 1 < p.B) s.next_pos = __ldg(p.seq_pos + ++s.b);   // on its way while this piece runs
  return true;
}

// R query rows per CTA: R / PACK query heads of each of its PACK KV heads.
constexpr int dp_groups(int R) { return R >= 8 ? 2 : 1; }
template <int R, int PACK>
__global__ void __launch_bounds__(dp_threads(dp_groups(R)), DP_CTAS_PER_SM) decode_attn8p_kernel(const __grid_constant__ DecodeAttn8pParams p) {
  using L = DpSmem;
  constexpr int HD = 128 / PACK, RH = R / PACK;
  constexpr int SG = dp_groups(R), RT = R / SG, DP_THREADS = dp_threads(SG);   // softmax groups, rows of each
  constexpr int NQ = R <= 8 ? 16 : 32;              // q's operand rows: hi 0..R-1, lo R..2R-1, zero padding
  constexpr int NP = (3 * R + 15) / 16 * 16;        // P's: its parts 0..R-1, R..2R-1, 2R..3R-1, zero padding
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + P_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* start = reinterpret_cast<int*>(tmem_slot + 2);                  // first sequence and tile of the range
  int64_t* wsum = reinterpret_cast<int64_t*>(bars + P_COUNT + 2);      // [warps]
  float* red = reinterpret_cast<float*>(smem + L::OFF_RED);
  float* qinv = reinterpret_cast<float*>(smem + L::OFF_QS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int range = blockIdx.x / p.groups, group = blockIdx.x % p.groups;
  const int g0 = group / p.subs * PACK, sub = group % p.subs;          // first KV head, block of query heads
  // query head of row h, -1 for a padding row
  auto head_of = [&](int h) {
    const int g = g0 + h / RH, i = sub * RH + h % RH;
    return g < p.n_kv && i < p.r ? g * p.r + i : -1;
  };
  if (threadIdx.x < P_COUNT) {
    const int i = threadIdx.x;
    const bool softmax = i == P_SFREE || i == P_SFREE + 1 || i == P_PF || i == P_PF + 1 || i == P_OFREE || i == P_QC || i == P_QC + 1 ||
                         (i >= P_SCE && i < P_SCE + DP_SSTAGES);
    mbar_init(&bars[i], softmax ? 128 * SG : i == P_QR || i == P_QR + 1 ? 32 : 1);
    if (i == 0) *abort_flag = 0;
    fence_mbar_init();
  } else if (threadIdx.x == 64) {
    tma_prefetch_desc(&p.tmK);
    tma_prefetch_desc(&p.tmV);
  }
  // the padding rows and, of packed heads, the other head's bytes stay zero in the q and P operands
  for (int i = threadIdx.x; i < (int)(L::OFF_SC - L::OFF_Q) / 16; i += DP_THREADS)
    reinterpret_cast<uint4*>(smem + L::OFF_Q)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) { tmem_alloc(tmem_slot, DP_TMEM_COLS); tmem_relinquish(); }

  pdl_wait();   // nothing of the caller's is read or written before
  pdl_trigger();
  // tiles of all sequences: thread i adds up the contiguous sequences [i * per, (i + 1) * per)
  const int per = (p.B + DP_THREADS - 1) / DP_THREADS;
  const int s0 = min(p.B, (int)threadIdx.x * per), s1 = min(p.B, s0 + per);
  int64_t mine = 0;
  for (int b = s0; b < s1; ++b) {
    const int pos = __ldg(p.seq_pos + b);
    const int nt = (good_pos(pos, p.max_pos) + 128) / 128;
    mine += nt;
    if (blockIdx.x == 0 && pos != good_pos(pos, p.max_pos)) atomicOr(p.status, STATUS_BAD_PLAN);
    if (nt == 0 && b % p.n_ranges == range) {   // nothing to attend to: this group's rows are zeros
      for (int h = 0; h < R; ++h) {
        const int64_t at = ((int64_t)b * p.n_q + head_of(h)) * HD;
        if (head_of(h) >= 0 && in_extent(at, HD, (int64_t)p.B * p.n_q * HD))
          for (int i = 0; i < HD / 8; ++i) reinterpret_cast<uint4*>(p.o + at)[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
  int64_t T = 0, first = upto - mine;
  for (int w = 0; w < DP_THREADS / 32; ++w) {
    if (w < warp) first += wsum[w];
    T += wsum[w];
  }
  // no more ranges than tiles, so that each of them has some and leaves its parts; CTAs past them have nothing to do
  const int n_ranges = (int)min((int64_t)p.n_ranges, T);
  const int64_t x0 = range < n_ranges ? range_first(T, n_ranges, range) : 0;
  const int64_t x1 = range < n_ranges ? range_first(T, n_ranges, range + 1) : 0;
  if (x0 < x1) {
    if (first <= x0 && x0 < first + mine) {
      int64_t off = first;
      int b = s0, nt = tiles_at(p, b);
      while (off + nt <= x0) { off += nt; nt = tiles_at(p, ++b); }
      start[0] = b;
      start[1] = (int)(x0 - off);
    }
    if (group == 0 && first <= x1 - 1 && x1 - 1 < first + mine) {
      int64_t off = first;
      int b = s0, nt = tiles_at(p, b);
      while (off + nt <= x1 - 1) { off += nt; nt = tiles_at(p, ++b); }
      SplitInfo s{-1, 0};
      if (off >= x0 && off + nt > x1) { s.b = b; s.last = range_with(T, n_ranges, off + nt - 1); }
      if (in_extent(range, 1, p.n_ranges)) p.split[range] = s;
    }
  } else if (group == 0 && threadIdx.x == 0 && in_extent(range, 1, p.n_ranges)) {
    p.split[range] = SplitInfo{-1, 0};
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem;          // S^T buffers: columns 0..NQ-1 and NQ..2NQ-1
  const uint32_t tO = tmem + 64;     // O^T: columns 64..64+NP-1
  const uint32_t sbase = smem_u32(smem);
  Pieces it0;
  it0.left = x1 - x0;
  it0.b = x0 < x1 ? start[0] : 0;
  it0.t = x0 < x1 ? start[1] : 0;
  it0.next_pos = x0 < x1 ? __ldg(p.seq_pos + it0.b) : -1;
  int b, t0, t1, nt, n_keys;

  if (warp == 0) {  // -------------------------------------------------------- TMA producer
    // V(j) is requested one tile after K(j): P V needs it only after S^T and the softmax of its tile
    const int n_sc = min(PACK, p.n_kv - g0);        // heads whose scales there are
    int tile = 0, v_page = 0, k_sent = 0, v_sent = 0;
    bool ok = true;
    auto issue_v = [&](int gt) -> bool {
      const int vs = gt % DP_VSTAGES;
      if (!wait_for(&bars[P_VE + vs], ((gt / DP_VSTAGES) & 1) ^ 1, abort_flag, p.status)) return false;
      if (!box_in(g0 * HD, p.n_kv * HD, (int64_t)v_page * 128, (int64_t)p.n_pages * 128)) { *abort_flag = 1; return false; }
      mbar_arrive_expect_tx(&bars[P_VF + vs], L::F8);
      tma_load_2d(sbase + L::OFF_V8 + vs * L::F8, &p.tmV, &bars[P_VF + vs], g0 * HD, v_page * 128);
      v_sent = gt + 1;
      return true;
    };
    // the query rows of piece `it` as hi and lo codes, by the whole warp
    auto put_q = [&](int it) -> bool {
      constexpr int VH = HD / 8;                  // 8-element chunks of a row
      constexpr int NCH = R * VH;
      constexpr int PER = (NCH + 31) / 32;
      const int qb = it & 1;
      uint4 w[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int c = lane + 32 * j, head = c < NCH ? head_of(c / VH) : -1;
        w[j] = head >= 0 ? *reinterpret_cast<const uint4*>(p.q + ((int64_t)b * p.n_q + head) * HD + c % VH * 8)
                         : make_uint4(0, 0, 0, 0);
      }
      // the buffer is free once the MMAs of piece it - 2 have read it and the softmax warps its scales; the lanes go on together or
      // not at all (the row maxima are the whole warp's)
      const bool free = wait_for(&bars[P_QE + qb], ((it >> 1) & 1) ^ 1, abort_flag, p.status) &&
                        wait_for(&bars[P_QC + qb], ((it >> 1) & 1) ^ 1, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, free)) return false;
      uint8_t* qop = smem + L::OFF_Q + qb * L::OPB;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int c = lane + 32 * j, h = c / VH;
        const uint32_t e[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
#pragma unroll
        for (int o = VH / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // a power of two per row: amax * qs in [128, 256)
        const int ex = (int)(__float_as_uint(amax) >> 23) - 127;
        const int up = min(max(7 - ex, -126), 126);
        const float qs = ex > 127 ? __uint_as_float(0x7FC00000u) : exp2_int(up);   // an infinity makes the row NaN, as its scores are
        if (c < NCH) {
          const int d = c % VH * 8 + h / RH * HD;
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            hi[k] = split_fine(__uint_as_float(e[k] << 16) * qs, __uint_as_float(e[k] & 0xFFFF0000u) * qs, lo[k]);
          *reinterpret_cast<uint2*>(qop + sw128_at(h, d)) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(qop + sw128_at(R + h, d)) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          if (c % VH == 0) qinv[qb * 16 + h] = exp2_int(-up);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      mbar_arrive(&bars[P_QR + qb]);
      return true;
    };
    int it = 0;
    Pieces s = it0;
    for (; ok && next_piece(p, s, b, t0, t1, nt, n_keys); ++it) {
      const int* row = p.block_table + (int64_t)b * p.max_pages;
      int ids = 0;
      for (int t = t0; t < t1; ++t, ++tile) {
        if (((t - t0) & 31) == 0) {                 // the pages of the next 32 tiles, one per lane
          ids = t + lane < t1 ? __ldg(row + t + lane) : 0;
          if (ids < 0 || ids >= p.n_pages) { atomicOr(p.status, STATUS_BAD_PLAN); ids = 0; }
        }
        const int page = __shfl_sync(0xffffffffu, ids, (t - t0) & 31);
        if (lane == 0) {
          const int ks = tile % DP_KSTAGES, sc = tile % DP_SSTAGES;
          ok = wait_for(&bars[P_KE + ks], ((tile / DP_KSTAGES) & 1) ^ 1, abort_flag, p.status) &&
               wait_for(&bars[P_SCE + sc], ((tile / DP_SSTAGES) & 1) ^ 1, abort_flag, p.status);
          if (ok && !(box_in(g0 * HD, p.n_kv * HD, (int64_t)page * 128, (int64_t)p.n_pages * 128) &&
                      in_extent(((int64_t)page * p.n_kv + g0) * 128, n_sc * 128, (int64_t)p.n_pages * p.n_kv * 128))) {
            *abort_flag = 1;
            ok = false;
          }
          if (ok) {
            mbar_arrive_expect_tx(&bars[P_KF + ks], L::F8);
            tma_load_2d(sbase + L::OFF_K8 + ks * L::F8, &p.tmK, &bars[P_KF + ks], g0 * HD, page * 128);
            const uint32_t bytes = n_sc * 512, dst = sbase + L::OFF_SC + sc * L::SC;
            const int64_t at = ((int64_t)page * p.n_kv + g0) * 128;
            mbar_arrive_expect_tx(&bars[P_SCF + sc], 2 * bytes);
            bulk_load(dst, p.k_scale + at, bytes, &bars[P_SCF + sc]);
            bulk_load(dst + 1024, p.v_scale + at, bytes, &bars[P_SCF + sc]);
            k_sent = tile + 1;
            if (tile > 0) ok = issue_v(tile - 1);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        if (!ok) break;
        v_page = page;
        if (t == t0 && !(ok = put_q(it))) break;   // behind the piece's first K, which is on its way meanwhile
      }
    }
    if (lane == 0) {
      if (ok && tile > 0) issue_v(tile - 1);
      int no_abort = 0;   // a CTA that gives up does not leave while its copies are on their way
      for (int k = max(0, k_sent - DP_KSTAGES); k < k_sent; ++k) wait_for(&bars[P_KF + k % DP_KSTAGES], (k / DP_KSTAGES) & 1, &no_abort, p.status);
      for (int k = max(0, k_sent - DP_SSTAGES); k < k_sent; ++k) wait_for(&bars[P_SCF + k % DP_SSTAGES], (k / DP_SSTAGES) & 1, &no_abort, p.status);
      for (int k = max(0, v_sent - DP_VSTAGES); k < v_sent; ++k) wait_for(&bars[P_VF + k % DP_VSTAGES], (k / DP_VSTAGES) & 1, &no_abort, p.status);
    }
  } else if (warp == 1) {
    if (lane == 0) {  // ---------------------------------------------------- MMA issuer
      const uint32_t idesc_s = idesc_f8(128, NQ, B_E4M3);
      const uint32_t idesc_o = idesc_f8(128, NP, B_E5M2, /*a_mn_major=*/true);
      Pieces s = it0;
      // S^T of tile gt, the first of piece it or a later one
      auto issue_s = [&](int gt, int it, bool first) -> bool {
        const int st = gt % DP_KSTAGES, sb = gt & 1, qb = it & 1;
        if (first && !wait_for(&bars[P_QR + qb], (it >> 1) & 1, abort_flag, p.status)) return false;
        if (!wait_for(&bars[P_KF + st], (gt / DP_KSTAGES) & 1, abort_flag, p.status)) return false;
        if (!wait_for(&bars[P_SFREE + sb], ((gt >> 1) & 1) ^ 1, abort_flag, p.status)) return false;
        tc_fence_after();
        const uint64_t qd0 = sdesc_sw128(sbase + L::OFF_Q + qb * L::OPB, 16, 1024);
        const uint64_t kd0 = sdesc_sw128(sbase + L::OFF_K8 + st * L::F8, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)   // 32 bytes of the row per step
          tc_mma_f8(tS + sb * NQ, kd0 + (uint64_t)(2 * k), qd0 + (uint64_t)(2 * k), idesc_s, k > 0 ? 1u : 0u);
        tc_commit(&bars[P_SF + sb]);
        tc_commit(&bars[P_KE + st]);
        return true;
      };
      auto issue_pv = [&](int gt, int it, bool first) -> bool {
        const int st = gt % DP_VSTAGES, pb = gt & 1;
        if (!wait_for(&bars[P_PF + pb], (gt >> 1) & 1, abort_flag, p.status)) return false;
        if (!wait_for(&bars[P_VF + st], (gt / DP_VSTAGES) & 1, abort_flag, p.status)) return false;
        if (first && !wait_for(&bars[P_OFREE], (it & 1) ^ 1, abort_flag, p.status)) return false;
        tc_fence_after();
        // V^T: M = bytes of the row (MN-major), 8-key groups 1024 bytes apart
        const uint64_t vd0 = sdesc_sw128(sbase + L::OFF_V8 + st * L::F8, 16384, 1024);
        const uint64_t pd0 = sdesc_sw128(sbase + L::OFF_P + pb * L::PB, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)   // 32 keys per step
          tc_mma_f8(tO, vd0 + (uint64_t)(k * 4096 >> 4), pd0 + (uint64_t)(2 * k), idesc_o, (!first || k > 0) ? 1u : 0u);
        tc_commit(&bars[P_OD + pb]);
        tc_commit(&bars[P_VE + st]);
        return true;
      };
      // the next tile's S^T goes out before this one's P V, the next piece's first tile included
      int tile = 0, it = 0;
      bool ok = next_piece(p, s, b, t0, t1, nt, n_keys) && issue_s(0, 0, true);
      while (ok) {
        const int n = t1 - t0;
        bool more = false;
        for (int j = 0; ok && j < n; ++j, ++tile) {
          if (j + 1 < n) {
            ok = issue_s(tile + 1, it, false);
          } else {
            tc_commit(&bars[P_QE + (it & 1)]);
            more = next_piece(p, s, b, t0, t1, nt, n_keys);
            if (more) ok = issue_s(tile + 1, it + 1, true);
          }
          ok = ok && issue_pv(tile, it, j == 0);
        }
        ++it;
        ok = ok && more;
      }
      int no_abort = 0;
      tc_commit(&bars[P_DRAIN]);
      wait_for(&bars[P_DRAIN], 0, &no_abort, p.status);
    }
  } else {  // ------------------------------------------------------------ softmax warps
    // A wait that is given up (another one then was, and the rows are undefined) changes nothing of a thread's way: the threads of a
    // group meet at its barrier and in shuffles, so one that left would hold up the others for good.  After the abort no wait
    // lasts, and the tiles that are left are gone through in a moment.
    const int sg = (warp - 2) >> 2, qw = warp & 3;   // a warp reaches TMEM lanes 32 * (warp % 4) ..
    const int t = qw * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qw * 32) << 16;
    const int h0 = sg * RT;                          // this group's first row
    // scales: of packed heads one for each half of the rows, which a group of two has to itself
    constexpr int NSC = PACK / SG > 1 ? 2 : 1;
    const int sc0 = PACK == 2 && SG == 2 ? sg : 0;
    // columns of this group's rows: the parts side by side (one group), or blocks of RT columns R apart
    constexpr int LD = SG == 1 ? 16 : RT, QL = SG == 1 ? 1 : 2, PL = SG == 1 ? 1 : 3;   // columns of a load, loads of S^T, of O^T
    auto load = [&](uint32_t base, auto& v) {
#pragma unroll
      for (int k = 0; k < (int)(sizeof(v) / sizeof(v[0])); ++k) tmem_ld_cols<LD>(base + k * R + h0 + lane_off, v[k]);
      tc_wait_ld();
    };
    // part k of row i of what was loaded
    auto at = [](auto& v, int k, int i) -> uint32_t& { return SG == 1 ? v[0][(k * R + i) % LD] : v[k * (SG - 1)][i % LD]; };
    float* red_g = red + sg * 192;
    int tile = 0, it = 0;
    Pieces s = it0;
    auto await = [&](int bar, int parity) { wait_for(&bars[bar], (uint32_t)parity, abort_flag, p.status); };
    for (; next_piece(p, s, b, t0, t1, nt, n_keys); ++it) {
      const int qb = it & 1;
      await(P_QR + qb, (it >> 1) & 1);
      float m_ref[RT], lsum[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        m_ref[i] = -INFINITY;
        lsum[i] = 0.f;
      }
      for (int tt = t0; tt < t1; ++tt, ++tile) {
        const int sb = tile & 1, ss = tile % DP_SSTAGES;
        const bool valid = tt * 128 + t < n_keys;
        await(P_SCF + ss, (tile / DP_SSTAGES) & 1);
        float ks[NSC], lvs[NSC];
        {
          const float* scales = reinterpret_cast<const float*>(smem + L::OFF_SC + ss * L::SC) + sc0 * 128;
#pragma unroll
          for (int k = 0; k < NSC; ++k) {
            ks[k] = scales[k * 128 + t] * p.scale_log2;
            const float vs = scales[256 + k * 128 + t];
            const float v = vs < 7.88860905e-31f ? 7.88860905e-31f : vs;   // 2^-100: a zero scale has a logarithm too; a NaN stays
            lvs[k] = valid ? lg2(v) : 0.f;
          }
        }
        mbar_arrive(&bars[P_SCE + ss]);
        await(P_SF + sb, (tile >> 1) & 1);
        tc_fence_after();
        uint32_t st[QL][LD];
        load(tS + sb * NQ, st);
        tc_fence_before();
        mbar_arrive(&bars[P_SFREE + sb]);
        float e[RT];   // log2 of weight * value scale
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int k = NSC == 2 ? i / RH : 0;
          const float score = fmaf(__uint_as_float(at(st, 1, i)), 1.f / kDpLo, __uint_as_float(at(st, 0, i)));
          e[i] = valid ? fmaf(score, qinv[qb * 16 + h0 + i] * ks[k], lvs[k]) : -INFINITY;
        }
        float* rbuf = red_g + (tile & 1) * 64;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float v = warp_max_dp(e[i]);
          if (lane == i) rbuf[qw * 16 + i] = v;
        }
        softmax_sync_dp(sg);
        auto tile_max = [&](int i) { return fmaxf(fmaxf(rbuf[i], rbuf[16 + i]), fmaxf(rbuf[32 + i], rbuf[48 + i])); };
        bool resc = false;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float tm = tile_max(i);
          if (m_ref[i] == -INFINITY) m_ref[i] = tm;
          else resc = resc || tm - m_ref[i] > kDpRescaleLog2;   // (a sum would round to more than 2 above a large m_ref)
        }
        const int pb = tile & 1;
        if (tile >= 2) await(P_OD + pb, ((tile - 2) >> 1) & 1);
        if (resc) [[unlikely]] {   // the same in all 128 threads of the group, which saw the same maxima
          await(P_OD + ((tile - 1) & 1), ((tile - 1) >> 1) & 1);
          tc_fence_after();
          float alpha[RT];
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float tm = tile_max(i);
            const bool up = tm - m_ref[i] > kDpRescaleLog2;
            const float half = up ? ex2(0.5f * (m_ref[i] - tm)) : 1.f;
            alpha[i] = half * half;
            if (up) m_ref[i] = tm;
            lsum[i] = lsum[i] * half * half;
          }
#pragma unroll
          for (int k = 0; k < PL; ++k) {
            uint32_t ot[LD];
            tmem_ld_cols<LD>(tO + k * R + h0 + lane_off, ot);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < (SG == 1 ? 3 * R : RT); ++i) ot[i] = __float_as_uint(__uint_as_float(ot[i]) * alpha[i % RT]);
            tmem_st_cols<LD>(tO + k * R + h0 + lane_off, ot);
          }
          tc_wait_st();
        }
        // P^T rows h, R + h and 2R + h, this thread's key in byte t of each; two rows are converted at a time
        uint8_t* pbase = smem + L::OFF_P + pb * L::PB;
#pragma unroll
        for (int i = 0; i < RT; i += 2) {
          float w[2] = {0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (i + j < RT) {
              const float d = e[i + j] - m_ref[i + j];   // (first: large scores keep their digits)
              w[j] = ex2(d + kDpPScaleLog2);
              lsum[i + j] += ex2_full(d - (lvs[NSC == 2 ? (i + j) / RH : 0] - kDpLScaleLog2));
            }
          uint32_t part[3];
          split_weights(w[0], w[1], part);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (i + j < RT) {
#pragma unroll
              for (int k = 0; k < 3; ++k) pbase[sw128_at(k * R + h0 + i + j, t)] = (uint8_t)(part[k] >> (8 * j));
            }
        }
        if (sg == 0 && (tt + 1) * 128 > n_keys) [[unlikely]] {   // rows behind the last key may hold anything, NaN codes too: zeros for the product
          const int vs = tile % DP_VSTAGES;
          await(P_VF + vs, (tile / DP_VSTAGES) & 1);
          if (!valid) {
            uint4* vrow = reinterpret_cast<uint4*>(smem + L::OFF_V8 + vs * L::F8 + t * 128);
#pragma unroll
            for (int i = 0; i < 8; ++i) vrow[i] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars[P_PF + pb]);
      }
      mbar_arrive(&bars[P_QC + qb]);   // the q scales have been read
      await(P_OD + ((tile - 1) & 1), ((tile - 1) >> 1) & 1);
      tc_fence_after();
      uint32_t ot[PL][LD];
      load(tO, ot);
      tc_fence_before();
      mbar_arrive(&bars[P_OFREE]);
      float* lbuf = red_g + 128;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float v = lsum[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == i) lbuf[qw * 16 + i] = v;
      }
      softmax_sync_dp(sg);
      const bool whole = t0 == 0 && t1 == nt;
      const int64_t part = ((int64_t)(2 * range + (t0 == 0 ? 1 : 0)) * p.groups + group) * R;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int h = h0 + i;
        const float l = (lbuf[i] + lbuf[16 + i]) + (lbuf[32 + i] + lbuf[48 + i]);
        const float fine = fmaf(__uint_as_float(at(ot, 2, i)), 1.f / kDpStep, __uint_as_float(at(ot, 1, i)));
        const float sum = fmaf(fine, 1.f / kDpStep, __uint_as_float(at(ot, 0, i)));
        const bool own = h / RH == t / HD;      // lane t holds byte t of the row: another head's, for half the rows
        if (whole) {
          const int head = head_of(h);
          const int64_t to = ((int64_t)b * p.n_q + head) * HD + t % HD;
          if (own && head >= 0 && in_extent(to, 1, (int64_t)p.B * p.n_q * HD)) p.o[to] = f2bf(sum / l * kDpOut);
        } else if (in_extent(part + h, 1, (int64_t)2 * p.n_ranges * p.groups * R)) {
          if (own) p.part_o[(part + h) * HD + t % HD] = sum;
          if (t == 0) p.part_ml[part + h] = make_float2(m_ref[i], l);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, DP_TMEM_COLS);
  }
}

// Joins the parts of the sequences that cuts go through: o = kDpOut sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i (the l_i by square
// roots, see Scales above).  Block (x, group, z):
// RB rows of sequence x, whose place among the ranges it finds from the lengths while the first kernel still runs; where there
// are more sequences than ranges, of the sequence whose first part is range x's tail.  The latency of its dependent loads is what
// it costs: a lane has one part's statistics, and the parts' rows come four elements per lane, eight rows' loads in flight.  Up to
// 16 parts, a warp takes a row; of more, the NW warps share each row's.
template <int NW, int RB, bool BY_SEQ>
__global__ void __launch_bounds__(32 * NW) decode_join8p_kernel(const __grid_constant__ DecodeAttn8pParams p, int R, int pack) {
  __shared__ float4 sum[NW][32];
  __shared__ float mx[NW], ls[NW];
  __shared__ int64_t all[NW], ahead[NW];
  const int group = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int RH = R / pack;
  int range = blockIdx.x;
  SplitInfo s{-1, 0};
  if (BY_SEQ) {   // (the lengths were complete before the first kernel, which triggered past its own wait)
    const int b = blockIdx.x;
    int64_t x = 0, y = 0;
    for (int k = threadIdx.x; k < p.B; k += 32 * NW) {
      const int nt = tiles_at(p, k);
      x += nt;
      if (k < b) y += nt;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    if (lane == 0) { all[warp] = x; ahead[warp] = y; }
    __syncthreads();
    int64_t T = 0, off = 0;
    for (int w = 0; w < NW; ++w) { T += all[w]; off += ahead[w]; }
    const int nt = tiles_at(p, b), n_ranges = (int)min((int64_t)p.n_ranges, T);
    if (nt > 0) {
      range = range_with(T, n_ranges, off);
      s.last = range_with(T, n_ranges, off + nt - 1);
      if (s.last > range) s.b = b;
    }
  }
  pdl_wait();
  pdl_trigger();
  if (!BY_SEQ) s = p.split[range];
  if (s.b < 0 || s.b >= p.B || s.last >= p.n_ranges) return;
  const int n = s.last - range + 1;      // parts: the tail of `range`, then the first of each range up to `last`
  const bool in = lane * 4 < p.hd;
  // query head of row h, -1 for a padding row
  auto head_of = [&](int h) {
    const int g = group / p.subs * pack + h / RH, i = group % p.subs * RH + h % RH;
    return h < R && g < p.n_kv && i < p.r ? g * p.r + i : -1;
  };
  // parts w0, w0 + step, .. of row h: their maximum, sum and weighted rows
  auto gather = [&](int h, int w0, int step, float& m, float& l, float4& acc) {
    auto slot = [&](int k) { return ((int64_t)(k == 0 ? 2 * range + 1 : 2 * (range + k)) * p.groups + group) * R + h; };
    m = -INFINITY;
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = w0; k0 < n; k0 += 32 * step) {
      const int mine = k0 + lane * step, cnt = min(32, (n - k0 + step - 1) / step);
      const float2 ml = mine < n ? p.part_ml[slot(mine)] : make_float2(-INFINITY, 0.f);
      float top = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m2 = fmaxf(m, top), h0 = m > -INFINITY ? exp2f(0.5f * (m - m2)) : 0.f, a = h0 * h0;
      l = l * h0 * h0;
      acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
      m = m2;
      const float half = mine < n ? exp2f(0.5f * (ml.x - m)) : 0.f, w = half * half;
      l += ml.y * half * half;
      for (int j0 = 0; j0 < cnt; j0 += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = in && j0 + j < cnt ? reinterpret_cast<const float4*>(p.part_o + slot(k0 + (j0 + j) * step) * p.hd)[lane]
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
          acc.x = fmaf(wj, v[j].x, acc.x);
          acc.y = fmaf(wj, v[j].y, acc.y);
          acc.z = fmaf(wj, v[j].z, acc.z);
          acc.w = fmaf(wj, v[j].w, acc.w);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  };
  auto store = [&](int head, float l, const float4& acc) {
    const int64_t at = ((int64_t)s.b * p.n_q + head) * p.hd + lane * 4;
    if (in && in_extent(at, 4, (int64_t)p.B * p.n_q * p.hd))
      *reinterpret_cast<uint2*>(p.o + at) = make_uint2(pack_bf2(acc.x / l * kDpOut, acc.y / l * kDpOut), pack_bf2(acc.z / l * kDpOut, acc.w / l * kDpOut));
  };
  float m, l;
  float4 acc;
  if (RB > 1 && n <= 16) {
    const int h = blockIdx.z * RB + warp;
    if (warp >= RB || head_of(h) < 0) return;
    gather(h, 0, 1, m, l, acc);
    store(head_of(h), l, acc);
    return;
  }
  for (int r = 0; r < RB; ++r) {
    const int h = blockIdx.z * RB + r, head = head_of(h);
    if (head < 0) continue;
    gather(h, warp, NW, m, l, acc);
    sum[warp][lane] = acc;
    if (lane == 0) { mx[warp] = m; ls[warp] = l; }
    __syncthreads();
    if (warp == 0) {
      float M = mx[0];
      for (int w = 1; w < NW; ++w) M = fmaxf(M, mx[w]);
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
      for (int w = 0; w < min(NW, n); ++w) {       // (warps past n have no parts)
        const float half = exp2f(0.5f * (mx[w] - M)), a = half * half;
        const float4 v = sum[w][lane];
        l += ls[w] * half * half;
        acc.x = fmaf(a, v.x, acc.x); acc.y = fmaf(a, v.y, acc.y); acc.z = fmaf(a, v.z, acc.z); acc.w = fmaf(a, v.w, acc.w);
      }
      store(head, l, acc);
    }
    __syncthreads();
  }
}

// Query rows of a CTA, head groups and, at most, ranges.
struct Shape { int R, pack, subs, groups; };
Shape shape_of(int64_t n_q, int64_t n_kv, int64_t hd) {
  Shape s;
  s.pack = hd == 64 ? 2 : 1;
  const int64_t r = n_q / n_kv, most = 16 / s.pack;
  int64_t rh = 1;
  while (rh < most && rh < r) rh *= 2;
  s.R = (int)rh * s.pack;
  s.subs = (int)((r + rh - 1) / rh);
  s.groups = (int)((n_kv + s.pack - 1) / s.pack) * s.subs;
  return s;
}
int ranges_of(const Shape& s, int64_t B, int64_t max_pos, int sms) {
  const int64_t tiles = B * ((max_pos + 128) / 128);
  return (int)std::max<int64_t>(1, std::min<int64_t>(DP_CTAS_PER_SM * sms / s.groups, tiles));
}
constexpr size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
struct Parts { size_t ml, split, total; };
Parts parts_of(const Shape& s, int ranges, int64_t hd) {
  const size_t rows = ranges > 1 ? (size_t)2 * ranges * s.groups * s.R : 0;   // one range cuts nothing
  Parts a;
  a.ml = round256(rows * hd * sizeof(float));
  a.split = a.ml + round256(rows * sizeof(float2));
  a.total = a.split + round256((size_t)ranges * sizeof(SplitInfo));
  return a;
}
constexpr int kMaxSms = 256;   // sizes the workspace, so that it does not depend on the device

template <int R, int PACK>
int launch_attn(const DecodeAttn8pParams& p, int dev, cudaStream_t st) {
  static bool attr_set[64] = {};
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(decode_attn8p_kernel<R, PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, DpSmem::TOTAL) != cudaSuccess)
      return -1;
    attr_set[dev] = true;
  }
  return launch_after(decode_attn8p_kernel<R, PACK>, dim3((unsigned)(p.n_ranges * p.groups)), dim3(dp_threads(dp_groups(R))), DpSmem::TOTAL, st, p) ==
                 cudaSuccess
             ? 0
             : -1;
}

}  // namespace

bool decode_attn8p_supported(int64_t B, int64_t n_q, int64_t n_kv, int64_t hd) {
  return (hd == 64 || hd == 128) && n_q <= 65536 && B * n_kv < ((int64_t)1 << 24) && B <= 65535;
}

size_t decode_attn8p_ws_bytes(int64_t B, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_pos) {
  const Shape s = shape_of(n_q, n_kv, hd);
  return parts_of(s, ranges_of(s, B, max_pos, kMaxSms), hd).total;
}

int launch_decode_attn8p(const DecodeAttn8pDesc& d, int num_sms, cudaStream_t st) {
  DecodeAttn8pParams p;
  memset(&p, 0, sizeof(p));
  const Shape s = shape_of(d.n_q, d.n_kv, d.hd);
  const int ranges = ranges_of(s, d.B, d.max_pos, std::min(num_sms, kMaxSms));
  const Parts parts = parts_of(s, ranges, d.hd);
  const uint64_t inner = (uint64_t)(d.n_kv * d.hd), rows = (uint64_t)d.n_pages * 128;
  if (!encode_tmap_2d_u8(&p.tmK, d.k_codes, inner, rows, inner, 128, 128)) return -1;
  if (!encode_tmap_2d_u8(&p.tmV, d.v_codes, inner, rows, inner, 128, 128)) return -1;
  p.q = static_cast<const uint16_t*>(d.q);
  p.k_scale = d.k_scale; p.v_scale = d.v_scale;
  p.block_table = d.block_table; p.seq_pos = d.seq_pos;
  p.o = static_cast<uint16_t*>(d.o);
  char* ws = static_cast<char*>(d.ws);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + parts.ml);
  p.split = reinterpret_cast<SplitInfo*>(ws + parts.split);
  p.B = (int)d.B; p.n_q = (int)d.n_q; p.n_kv = (int)d.n_kv; p.r = (int)(d.n_q / d.n_kv); p.hd = (int)d.hd;
  p.n_pages = (int)d.n_pages;
  p.max_pos = (int)d.max_pos;
  p.n_ranges = ranges; p.groups = s.groups; p.subs = s.subs;
  p.max_pages = d.max_pages;
  p.scale_log2 = d.scale * 1.4426950408889634f;
  p.status = d.status;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return -1;
  int rc = -1;
  if (s.pack == 1) {
    switch (s.R) {
      case 1: rc = launch_attn<1, 1>(p, dev, st); break;
      case 2: rc = launch_attn<2, 1>(p, dev, st); break;
      case 4: rc = launch_attn<4, 1>(p, dev, st); break;
      case 8: rc = launch_attn<8, 1>(p, dev, st); break;
      case 16: rc = launch_attn<16, 1>(p, dev, st); break;
    }
  } else {
    switch (s.R) {
      case 2: rc = launch_attn<2, 2>(p, dev, st); break;
      case 4: rc = launch_attn<4, 2>(p, dev, st); break;
      case 8: rc = launch_attn<8, 2>(p, dev, st); break;
      case 16: rc = launch_attn<16, 2>(p, dev, st); break;
    }
  }
  if (rc != 0 || ranges == 1) return rc;   // one range cuts nothing
  // By the parts that a sequence has if all are alike: a warp per row up to 4, a block per row above, a large one above 16.
  const bool by_seq = d.B < ranges;
  const int64_t each = ranges / d.B;
  const int rows_each = by_seq && each > 4 ? 1 : 4;
  const dim3 grid((unsigned)(by_seq ? d.B : ranges - 1), (unsigned)s.groups, (unsigned)((s.R + rows_each - 1) / rows_each));
  const cudaError_t e = !by_seq     ? launch_after(decode_join8p_kernel<4, 4, false>, grid, dim3(128), 0, st, p, s.R, s.pack)
                        : each <= 4 ? launch_after(decode_join8p_kernel<4, 4, true>, grid, dim3(128), 0, st, p, s.R, s.pack)
                        : each <= 16 ? launch_after(decode_join8p_kernel<4, 1, true>, grid, dim3(128), 0, st, p, s.R, s.pack)
                                     : launch_after(decode_join8p_kernel<16, 1, true>, grid, dim3(512), 0, st, p, s.R, s.pack);
  return e == cudaSuccess ? 0 : -1;
}

LLAMA_DEFINE_BOUNDS_READER(decode_attn8p)

}  // namespace llama
