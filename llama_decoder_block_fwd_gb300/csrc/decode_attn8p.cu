// One-token GQA attention over an 8-bit paged cache with a scale per position and KV head.
//
//   o_h = sum_j exp(s_hj) vs_j c_j / sum_j exp(s_hj),   s_hj = ks_j (q_h . kc_j) / sqrt(hd)
//
// kc_j, c_j the E4M3 codes of key and value j of the query head's KV head, ks_j, vs_j their scales.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "e4m3.cuh"
#include "kernels.h"

namespace llama {
namespace {

struct DecodeAttn8pParams {
  const uint16_t* q;
  const uint8_t *k_codes, *v_codes;
  const float *k_scale, *v_scale;
  const int *block_table, *seq_pos;
  uint16_t* o;
  int B, n_q, n_kv, n_pages;
  int64_t max_pages;
  int max_pos;
  float scale_log2;
  unsigned* status;
};

// One CTA per (sequence, query head); thread t scores key t of each page and keeps output element t.
template <int HD>
__global__ void __launch_bounds__(128) decode_attn8p_kernel(const __grid_constant__ DecodeAttn8pParams p) {
  __shared__ float q[HD], w[128], red[4];
  const int b = blockIdx.y, h = blockIdx.x, g = h / (p.n_q / p.n_kv), t = threadIdx.x;
  int pos = __ldg(p.seq_pos + b);
  if (pos < -1 || pos > p.max_pos) {
    if (t == 0) atomicOr(p.status, STATUS_BAD_PLAN);
    pos = -1;
  }
  if (t < HD) q[t] = bf2f(p.q[((int64_t)b * p.n_q + h) * HD + t]) * p.scale_log2;
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j = 0; j * 128 <= pos; ++j) {
    const int page = __ldg(p.block_table + (int64_t)b * p.max_pages + j);
    if (page < 0 || page >= p.n_pages) {
      if (t == 0) atomicOr(p.status, STATUS_BAD_PLAN);
      continue;
    }
    const int n = min(128, pos + 1 - j * 128);
    const int64_t row0 = (int64_t)page * 128, s0 = ((int64_t)page * p.n_kv + g) * 128;
    float s = -INFINITY;
    if (t < n) {
      const uint4* kc = reinterpret_cast<const uint4*>(p.k_codes + ((row0 + t) * p.n_kv + g) * HD);
      float d = 0.f;
      for (int i = 0; i < HD / 16; ++i) {
        const uint4 c = kc[i];
        const uint32_t e[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = e4m3x2_to_f2(e[k] & 0xFFFFu), hi = e4m3x2_to_f2(e[k] >> 16);
          d += q[i * 16 + k * 4] * lo.x + q[i * 16 + k * 4 + 1] * lo.y + q[i * 16 + k * 4 + 2] * hi.x + q[i * 16 + k * 4 + 3] * hi.y;
        }
      }
      s = d * p.k_scale[s0 + t];
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((t & 31) == 0) red[t >> 5] = mx;
    __syncthreads();
    mx = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float alpha = exp2f(m - mx);
    m = mx;
    const float e = t < n ? exp2f(s - m) : 0.f;
    l = l * alpha + e;
    w[t] = t < n ? e * p.v_scale[s0 + t] : 0.f;
    __syncthreads();
    acc *= alpha;
    if (t < HD) {
      const uint8_t* vc = p.v_codes + (row0 * p.n_kv + g) * HD + t;
      for (int i = 0; i < n; ++i) acc += w[i] * e4m3x2_to_f2(vc[(int64_t)i * p.n_kv * HD]).x;
    }
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if ((t & 31) == 0) red[t >> 5] = l;
  __syncthreads();
  l = red[0] + red[1] + red[2] + red[3];
  const int64_t at = ((int64_t)b * p.n_q + h) * HD + t;
  if (t < HD && in_extent(at, 1, (int64_t)p.B * p.n_q * HD)) p.o[at] = f2bf(pos >= 0 ? acc / l : 0.f);
}

}  // namespace

bool decode_attn8p_supported(int64_t B, int64_t n_q, int64_t n_kv, int64_t hd) {
  return (hd == 64 || hd == 128) && n_q <= 65536 && B * n_kv < ((int64_t)1 << 24) && B <= 65535;
}

size_t decode_attn8p_ws_bytes(int64_t B, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_pos) {
  (void)B; (void)n_q; (void)n_kv; (void)hd; (void)max_pos;
  return 256;
}

int launch_decode_attn8p(const DecodeAttn8pDesc& d, int num_sms, cudaStream_t st) {
  (void)num_sms;
  DecodeAttn8pParams p;
  p.q = static_cast<const uint16_t*>(d.q);
  p.k_codes = static_cast<const uint8_t*>(d.k_codes); p.v_codes = static_cast<const uint8_t*>(d.v_codes);
  p.k_scale = d.k_scale; p.v_scale = d.v_scale;
  p.block_table = d.block_table; p.seq_pos = d.seq_pos;
  p.o = static_cast<uint16_t*>(d.o);
  p.B = (int)d.B; p.n_q = (int)d.n_q; p.n_kv = (int)d.n_kv; p.n_pages = (int)d.n_pages;
  p.max_pages = d.max_pages;
  p.max_pos = (int)d.max_pos;
  p.scale_log2 = d.scale * 1.4426950408889634f;
  p.status = d.status;
  const dim3 grid((unsigned)d.n_q, (unsigned)d.B);
  if (d.hd == 128) decode_attn8p_kernel<128><<<grid, 128, 0, st>>>(p);
  else decode_attn8p_kernel<64><<<grid, 128, 0, st>>>(p);
  return 0;
}

LLAMA_DEFINE_BOUNDS_READER(decode_attn8p)

}  // namespace llama
