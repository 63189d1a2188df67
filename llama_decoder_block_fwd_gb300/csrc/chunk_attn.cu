// Causal GQA attention of ragged chunks of new tokens over a paged KV cache ("Llama Architecture
// ...", Mathematical Foundations 4; "LLaMA-3 8B ...", section 四.4): token i of sequence b sits at
// position c_b + i and attends to positions 0 .. c_b + i of its sequence.
#include <cmath>
#include <cstring>

#include "kernels.h"

namespace llama {
namespace {

// One warp per (token, query head), lanes over the head dimension, running maximum and sum.
__global__ void chunk_attn_simt_kernel(const __grid_constant__ ChunkAttnDesc a) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int t = (int)(w / a.n_q), h = (int)(w % a.n_q), g = h / (int)(a.n_q / a.n_kv);
  if (t >= a.T || t >= a.cu_new[a.B]) return;
  int b = 0;
  while (b + 1 < a.B && a.cu_new[b + 1] <= t) ++b;
  const int pos = a.n_cached[b] + t - a.cu_new[b];
  if (pos < 0 || pos > a.max_pos) {
    if (lane == 0) atomicOr(a.status, STATUS_BAD_PLAN);
    return;
  }
  const int hd = (int)a.hd, per = hd / 32;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((int64_t)t * a.n_q + h) * hd;
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < per; ++e) qv[e] = bf2f(q[lane + 32 * e]) * a.scale;
  for (int j = 0; j <= pos; ++j) {
    const int page = a.block_table[(int64_t)b * a.max_pages + j / 128];
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) atomicOr(a.status, STATUS_BAD_PLAN);
      return;
    }
    const int64_t row = (((int64_t)page * 128 + j % 128) * a.n_kv + g) * hd;
    float s = 0.f;
    for (int e = 0; e < per; ++e) s += qv[e] * bf2f(static_cast<const uint16_t*>(a.k_pool)[row + lane + 32 * e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s), c = expf(m - mn), pv = expf(s - mn);
    m = mn;
    l = l * c + pv;
    for (int e = 0; e < per; ++e)
      acc[e] = acc[e] * c + pv * bf2f(static_cast<const uint16_t*>(a.v_pool)[row + lane + 32 * e]);
  }
  uint16_t* o = static_cast<uint16_t*>(a.o) + ((int64_t)t * a.n_q + h) * hd;
  for (int e = 0; e < per; ++e) o[lane + 32 * e] = f2bf(acc[e] / l);
}

}  // namespace

size_t chunk_attn_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 256; }

int launch_chunk_attn(const ChunkAttnDesc& a, int, cudaStream_t st) {
  const int64_t warps = a.T * a.n_q;
  chunk_attn_simt_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(a);
  return 0;
}

LLAMA_DEFINE_BOUNDS_READER(chunk_attn)

}  // namespace llama
