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
// HBM bound: phase 1 reads every judged row of z and y once and leaves (max, sum of exponentials)
// of each 8192-logit part; phase 2 (a cluster of CTAs per sequence) merges the parts, finds the
// first rejection and reads one row of z, y and e again for the race.  A part's sums are formed in a
// fixed order and merged in a fixed order, and the race keeps (score, lowest id), so the result does
// not depend on timing.
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
constexpr int VF_UNITS = 8;                               // float4 units per thread in a part
constexpr int VF_PART = VF_THREADS * VF_UNITS * 4;        // logits per part
constexpr int VF_CLUSTER = 8;
using u64 = unsigned long long;

struct VerifyParams {
  const float *z, *y;              // [T, ld], [T, ld_y]; y may be null
  int64_t ld, ld_y, ld_e;
  int T, V, B, parts, greedy;
  float c_hi, c_lo;                // log2(e) / T as an unevaluated sum of two floats
  float d_min;                     // (z - m) below this has no weight
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
// exp((z - m) / T) for z <= m; the exponent is formed to about 2^-24 relative before ex2 (2^-22).  A
// masked logit (-inf) has weight 0; differences are cut off where the weight is below 2^-1000, so
// that masks of the type's lowest value stay finite on the way.
__device__ __forceinline__ float vf_exp(const VerifyParams& p, float z, float m) {
  const float d = fmaxf(z - m, p.d_min);
  return z == -INFINITY ? 0.f : vf_ex2(fmaf(d, p.c_hi, d * p.c_lo));
}

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

// one CTA per (row, part) of z (blockIdx.y = 0) and of y (blockIdx.y = 1)
__global__ void __launch_bounds__(VF_THREADS) verify_stats_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ float red_m[VF_THREADS / 32], red_s[VF_THREADS / 32];
  __shared__ int red_i[VF_THREADS / 32];
  const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool draft = blockIdx.y == 1;
  const float* src = draft ? p.y + (int64_t)row * p.ld_y : p.z + (int64_t)row * p.ld;
  const bool vec = vf_aligned(src);
  const int i0 = part * VF_PART;
  pdl_trigger();
  // rows behind the last sequence hold nothing, and the last row of a sequence judges no draft
  bool skip = row >= __ldg(p.cu + p.B);
  if (draft)
    for (int b = tid; b < p.B; b += VF_THREADS) skip = skip || __ldg(p.cu + b + 1) - 1 == row;
  if (__syncthreads_or(skip)) return;
  float4 w[VF_UNITS];
#pragma unroll
  for (int j = 0; j < VF_UNITS; ++j) w[j] = vf_load4(src, i0 + (j * VF_THREADS + tid) * 4, p.V, vec);
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < VF_UNITS; ++j) m = fmaxf(m, fmaxf(fmaxf(w[j].x, w[j].y), fmaxf(w[j].z, w[j].w)));
  float mw = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
  if (lane == 0) red_m[warp] = mw;
  __syncthreads();
  float mb = red_m[0];
#pragma unroll
  for (int k = 1; k < VF_THREADS / 32; ++k) mb = fmaxf(mb, red_m[k]);
  float2* stat = (draft ? p.stat_y : p.stat_z) + (int64_t)row * p.parts + part;
  if (p.greedy) {   // the lowest id that holds the maximum
    int id = INT_MAX;
#pragma unroll
    for (int j = VF_UNITS - 1; j >= 0; --j) {
      const int i = i0 + (j * VF_THREADS + tid) * 4;
      if (w[j].w == mb && i + 3 < p.V) id = i + 3;
      if (w[j].z == mb && i + 2 < p.V) id = i + 2;
      if (w[j].y == mb && i + 1 < p.V) id = i + 1;
      if (w[j].x == mb && i < p.V) id = i;
    }
    id = __reduce_min_sync(0xffffffffu, id);
    if (lane == 0) red_i[warp] = id;
    __syncthreads();
    if (tid == 0) {
      for (int k = 1; k < VF_THREADS / 32; ++k) id = min(id, red_i[k]);
      *stat = make_float2(mb, __int_as_float(id));
    }
    return;
  }
  const float mu = mb == -INFINITY ? 0.f : mb;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < VF_UNITS; ++j)
    s += (vf_exp(p, w[j].x, mu) + vf_exp(p, w[j].y, mu)) + (vf_exp(p, w[j].z, mu) + vf_exp(p, w[j].w, mu));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red_s[warp] = s;
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < VF_THREADS / 32; ++k) s += red_s[k];
    *stat = make_float2(mb, s);
  }
}

// A row's (max, 1 / sum) from its parts, by one warp.
__device__ __forceinline__ float2 merge_parts(const VerifyParams& p, const float2* stat) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int i = lane; i < p.parts; i += 32) m = fmaxf(m, stat[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = 0.f;
  for (int i = lane; i < p.parts; i += 32)
    if (stat[i].y > 0.f) s += stat[i].y * vf_exp(p, stat[i].x, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return make_float2(m, 1.f / s);
}
// A row's argmax from its parts (greedy), by one warp.
__device__ __forceinline__ int merge_argmax(const VerifyParams& p, const float2* stat) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  int id = INT_MAX;
  for (int i = lane; i < p.parts; i += 32)
    if (stat[i].x > m) { m = stat[i].x; id = __float_as_int(stat[i].y); }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o);
    const int oi = __shfl_xor_sync(0xffffffffu, id, o);
    if (om > m || (om == m && oi < id)) { m = om; id = oi; }
  }
  return id == INT_MAX ? 0 : id;
}

// (score, id) as one word: larger score first, then the lower id.  Scores are >= 0; NaN loses.
__device__ __forceinline__ u64 race_key(float s, int i) {
  return s >= 0.f ? ((u64)(__float_as_uint(s) + 1u) << 32) | (0xFFFFFFFFu - (uint32_t)i) : 0ull;
}

__global__ void __launch_bounds__(VF_THREADS) verify_pick_kernel(const __grid_constant__ VerifyParams p) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cl = cg::this_cluster();
  const int P = (int)cl.num_blocks(), cr = (int)cl.block_rank(), b = blockIdx.x / P;
  __shared__ int stop_sh;
  __shared__ float2 sz_sh, sy_sh;
  __shared__ int top_sh;
  __shared__ u64 best[2], wbest[2][VF_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  const int lo = max(0, __ldg(p.cu + b)), hi = min(p.T, __ldg(p.cu + b + 1));
  if (hi <= lo) {           // a sequence without rows (the whole cluster leaves)
    if (cr == 0 && tid == 0 && in_extent(b, 1, p.B)) p.n_acc[b] = 0;
    return;
  }
  if (tid == 0) stop_sh = hi - 1;
  __syncthreads();
  // ---- the first row whose draft is turned down (the last row if none is)
  for (int row = lo + warp; row < hi - 1; row += VF_THREADS / 32) {
    const int d = __ldg(p.tokens + row + 1);
    const bool real = d >= 0 && d < p.V;
    bool ok;
    if (p.greedy) {
      ok = merge_argmax(p, p.stat_z + (int64_t)row * p.parts) == d;
    } else {
      const float2 sz = merge_parts(p, p.stat_z + (int64_t)row * p.parts);
      float qd = 1.f, pd = 0.f;
      if (p.y) {
        const float2 sy = merge_parts(p, p.stat_y + (int64_t)row * p.parts);
        if (real) qd = vf_exp(p, __ldg(p.y + (int64_t)row * p.ld_y + d), sy.x) * sy.y;
      }
      if (real) pd = vf_exp(p, __ldg(p.z + (int64_t)row * p.ld + d), sz.x) * sz.y;
      float u = __ldg(p.u + row);
      u = (u >= 0.f) ? fminf(u, 0.99999994f) : 0.f;
      ok = (double)u * (double)qd < (double)pd;   // the product is exact
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
  if (p.greedy) {
    if (warp == 0) {
      const int id = merge_argmax(p, p.stat_z + (int64_t)stop * p.parts);
      if (lane == 0) top_sh = id;
    }
    __syncthreads();
    token = top_sh;
  } else {
    if (warp == 0) {
      const float2 s = merge_parts(p, p.stat_z + (int64_t)stop * p.parts);
      if (lane == 0) sz_sh = s;
    }
    if (warp == 1 && p.y && rejected) {
      const float2 s = merge_parts(p, p.stat_y + (int64_t)stop * p.parts);
      if (lane == 0) sy_sh = s;
    }
    __syncthreads();
    // ---- the race over this CTA's share of the vocabulary: key[0] over the remainder
    //      max(p - q, 0), key[1] over p (taken when nothing was rejected or nothing remains)
    const float* z = p.z + (int64_t)stop * p.ld;
    const float* y = p.y && rejected ? p.y + (int64_t)stop * p.ld_y : nullptr;
    const float* e = p.e + (int64_t)b * p.ld_e;
    const bool vz = vf_aligned(z), vy = y && vf_aligned(y), ve = vf_aligned(e);
    const int d = rejected ? __ldg(p.tokens + stop + 1) : -1;
    const float2 sz = sz_sh, sy = y ? sy_sh : make_float2(0.f, 0.f);
    u64 k0 = 0ull, k1 = 0ull;
    const int units = (p.V + 3) >> 2;
    for (int q0 = cr * VF_THREADS + tid; q0 < units; q0 += P * VF_THREADS) {
      const int i = q0 * 4;
      const float4 a = vf_load4(z, i, p.V, vz), n = vf_load4(e, i, p.V, ve);
      const float4 c = y ? vf_load4(y, i, p.V, vy) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float za[4] = {a.x, a.y, a.z, a.w}, ya[4] = {c.x, c.y, c.z, c.w}, ea[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (i + t >= p.V) break;
        const float pi = vf_exp(p, za[t], sz.x) * sz.y;
        float w = pi;
        if (y) w = fmaxf(pi - vf_exp(p, ya[t], sy.x) * sy.y, 0.f);
        else if (i + t == d) w = 0.f;
        const u64 a0 = race_key(__fdividef(w, ea[t]), i + t), a1 = race_key(__fdividef(pi, ea[t]), i + t);
        if (a0 > k0 && w > 0.f) k0 = a0;
        if (a1 > k1) k1 = a1;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const u64 o0 = __shfl_xor_sync(0xffffffffu, k0, o), o1 = __shfl_xor_sync(0xffffffffu, k1, o);
      k0 = o0 > k0 ? o0 : k0;
      k1 = o1 > k1 ? o1 : k1;
    }
    if (lane == 0) { wbest[0][warp] = k0; wbest[1][warp] = k1; }
    __syncthreads();
    if (tid < 2) {
      u64 k = wbest[tid][0];
      for (int i = 1; i < VF_THREADS / 32; ++i) k = wbest[tid][i] > k ? wbest[tid][i] : k;
      best[tid] = k;
    }
    cl.sync();
    if (cr == 0) {
      k0 = k1 = 0ull;
      for (int r = 0; r < P; ++r) {
        const u64* o = cl.map_shared_rank(best, r);
        k0 = o[0] > k0 ? o[0] : k0;
        k1 = o[1] > k1 ? o[1] : k1;
      }
    }
    cl.sync();   // the others' shared memory stays until the leader has read it
    const u64 k = k0 ? k0 : k1;
    token = k ? (int)(0xFFFFFFFFu - (uint32_t)k) : 0;
  }
  if (cr != 0) return;
  if (tid == 0 && in_extent(b, 1, p.B)) p.n_acc[b] = stop - lo;
  for (int row = lo + tid; row < hi; row += VF_THREADS)
    if (in_extent(row, 1, p.T)) p.out[row] = row < stop ? __ldg(p.tokens + row + 1) : row == stop ? token : -1;
}

size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
int64_t parts_of(int64_t V) { return (V + VF_PART - 1) / VF_PART; }

}  // namespace

bool verify_supported(int64_t T, int64_t V) { return T * parts_of(V) <= INT32_MAX; }   // one CTA per part

size_t verify_ws_bytes(int64_t T, int64_t V) { return 2 * round256((size_t)T * parts_of(V) * sizeof(float2)); }

int launch_verify(const VerifyDesc& d, int, unsigned* status, cudaStream_t st) {
  VerifyParams p;
  p.z = d.logits; p.y = d.temperature > 0.f ? d.draft_logits : nullptr;
  p.ld = d.ld; p.ld_y = d.draft_ld; p.ld_e = d.noise_ld;
  p.T = (int)d.T; p.V = (int)d.V; p.B = (int)d.B;
  p.parts = (int)parts_of(d.V);
  p.greedy = !(d.temperature > 0.f);
  const double c = p.greedy ? 0.0 : 1.4426950408889634074 / (double)d.temperature;
  p.c_hi = (float)c;
  p.c_lo = (float)(c - (double)p.c_hi);
  p.d_min = (float)std::max(-1000.0 / c, -(double)FLT_MAX);   // T = inf: c = 0, no cut
  p.cu = d.cu_new; p.tokens = d.tokens; p.u = d.u; p.e = d.noise;
  p.n_acc = d.n_accepted; p.out = d.out_tokens;
  p.stat_z = static_cast<float2*>(d.ws);
  p.stat_y = reinterpret_cast<float2*>(static_cast<char*>(d.ws) + round256((size_t)d.T * p.parts * sizeof(float2)));
  p.status = status;
  if (d.T > 0) verify_stats_kernel<<<dim3((unsigned)(p.parts * d.T), p.y ? 2 : 1), VF_THREADS, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  const int P = p.greedy ? 1 : VF_CLUSTER;
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
