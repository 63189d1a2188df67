// The 8-bit paged cache ("LLaMA-3 8B ...", section 七 sizes the cache): writing K and V rows as E4M3 codes
// with a scale per position and KV head, and reading pages back to bf16.
//
// write: x the rotated K row or the V row of one head, u = max |v_i| for V and max (|a| + |b|) over the
//   pairs for K (a rotation keeps a pair inside that circle, so the scale is the same at every
//   position and no code saturates); scale 2^e, e the smallest with u <= 448 * 2^e; code = E4M3(x * 2^-e).
//   A power of two costs a floating-point code nothing, and code * scale has a bf16 value.
// read: x = code * scale.
#include <algorithm>
#include <climits>
#include <cstring>

#include "e4m3.cuh"
#include "kernels.h"

namespace llama {
namespace {

constexpr int A8_THREADS = 256;

struct Append8Params {
  const uint16_t *q, *k, *v;             // [T] rows of n_q / n_kv / n_kv heads x hd, row strides below
  int64_t q_stride, k_stride, v_stride;  // elements
  const int *positions, *slots;
  uint16_t* q_out;
  uint8_t *k_codes, *v_codes;            // [n_pages, 128, n_kv, hd]
  float *k_scale, *v_scale;              // [n_pages, n_kv, 128]
  int T, hd, n_q, n_kv;
  int64_t n_slots;
  unsigned* status;
  RopeFreq freq[kMaxRopePairs];
};

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(e[i] << 16);
    x[2 * i + 1] = __uint_as_float(e[i] & 0xFFFF0000u);
  }
}

// One token per CTA, one head per warp at a time.
__global__ void __launch_bounds__(A8_THREADS) rope_append8_kernel(const __grid_constant__ Append8Params p) {
  __shared__ float2 cs[kMaxRopePairs];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.hd / 2, vph = p.hd / 8;
  const int slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);
  if (slot < 0) return;
  if (slot >= p.n_slots || pos < 0 || pos >= (1 << 24)) {
    if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_PLAN);
    return;
  }
  for (int j = threadIdx.x; j < half; j += A8_THREADS) rope_sincos((float)pos, p.freq[j], cs[j].y, cs[j].x);
  __syncthreads();
  const int n_q = p.q ? p.n_q : 0;
  for (int h = warp; h < n_q + 2 * p.n_kv; h += A8_THREADS / 32) {
    const bool is_q = h < n_q, is_v = h >= n_q + p.n_kv;
    const int g = is_q ? h : is_v ? h - n_q - p.n_kv : h - n_q;
    const uint16_t* src = is_q ? p.q + t * p.q_stride : is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride;
    float x[8];
    float u = 0.f;
    if (lane < vph) {
      unpack8(*reinterpret_cast<const uint4*>(src + (int64_t)g * p.hd + lane * 8), x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        u = fmaxf(u, is_v ? fmaxf(fabsf(a), fabsf(b)) : fabsf(a) + fabsf(b));
        if (!is_v) {
          const float2 c = cs[lane * 4 + i];
          x[2 * i] = a * c.x - b * c.y;
          x[2 * i + 1] = a * c.y + b * c.x;
        }
      }
    }
    if (is_q) {
      const int64_t at = ((int64_t)t * p.n_q + g) * p.hd + lane * 8;
      if (lane < vph && in_extent(at, 8, (int64_t)p.T * p.n_q * p.hd))
        *reinterpret_cast<uint4*>(p.q_out + at) =
            make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
      continue;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
    const int e = row_scale_exp(u);
    const float inv = exp2_int(-e);
    if (lane < vph) {
      const int64_t at = ((int64_t)slot * p.n_kv + g) * p.hd + lane * 8;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
      if (in_extent(at, 8, p.n_slots * p.n_kv * p.hd))
        *reinterpret_cast<uint2*>((is_v ? p.v_codes : p.k_codes) + at) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    const int64_t sat = ((int64_t)(slot / 128) * p.n_kv + g) * 128 + slot % 128;
    if (lane == 0 && in_extent(sat, 1, p.n_slots * p.n_kv)) (is_v ? p.v_scale : p.k_scale)[sat] = exp2_int(e);
  }
}

struct Dequant8Params {
  const uint8_t *k_codes, *v_codes;
  const float *k_scale, *v_scale;
  uint16_t *k_pool, *v_pool;
  const int *block_table, *n_pos;
  int B, hd, n_kv, n_pages;
  int64_t max_pages;
  unsigned* status;
};

// One CTA per page at a time: blockIdx.y is the sequence, blockIdx.x strides over its pages.
__global__ void __launch_bounds__(256) dequant8_kernel(const __grid_constant__ Dequant8Params p) {
  const int b = blockIdx.y, n = __ldg(p.n_pos + b);
  if (n < 0 || n > p.max_pages * 128) {
    if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_PLAN);
    return;
  }
  const int vph = p.hd / 8;
  for (int j = blockIdx.x; j * 128 < n; j += gridDim.x) {
    const int page = __ldg(p.block_table + (int64_t)b * p.max_pages + j);
    if (page < 0 || page >= p.n_pages) {
      if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_PLAN);
      continue;
    }
    const int total = min(128, n - j * 128) * p.n_kv * vph;
    for (int i = threadIdx.x; i < 2 * total; i += 256) {
      const bool is_v = i >= total;
      const int o = is_v ? i - total : i;
      const int row = o / (p.n_kv * vph), g = o / vph % p.n_kv;
      const int64_t at = ((int64_t)page * 128 * p.n_kv * vph + o) * 8;
      const uint2 c = *reinterpret_cast<const uint2*>((is_v ? p.v_codes : p.k_codes) + at);
      const float s = (is_v ? p.v_scale : p.k_scale)[((int64_t)page * p.n_kv + g) * 128 + row];
      const float2 a0 = e4m3x2_to_f2(c.x & 0xFFFFu), a1 = e4m3x2_to_f2(c.x >> 16);
      const float2 a2 = e4m3x2_to_f2(c.y & 0xFFFFu), a3 = e4m3x2_to_f2(c.y >> 16);
      if (in_extent(at, 8, (int64_t)p.n_pages * 128 * p.n_kv * p.hd))
        *reinterpret_cast<uint4*>((is_v ? p.v_pool : p.k_pool) + at) =
            make_uint4(pack_bf2(a0.x * s, a0.y * s), pack_bf2(a1.x * s, a1.y * s), pack_bf2(a2.x * s, a2.y * s),
                       pack_bf2(a3.x * s, a3.y * s));
    }
  }
}

}  // namespace

int launch_rope_append8(const Append8Desc& d, const RopeFreq* freq, int num_sms, unsigned* status, cudaStream_t st) {
  (void)num_sms;
  Append8Params p;
  p.q = static_cast<const uint16_t*>(d.q); p.k = static_cast<const uint16_t*>(d.k); p.v = static_cast<const uint16_t*>(d.v);
  p.q_stride = d.q_stride; p.k_stride = d.k_stride; p.v_stride = d.v_stride;
  p.positions = d.positions; p.slots = d.slots;
  p.q_out = static_cast<uint16_t*>(d.q_out);
  p.k_codes = static_cast<uint8_t*>(d.k_codes); p.v_codes = static_cast<uint8_t*>(d.v_codes);
  p.k_scale = d.k_scale; p.v_scale = d.v_scale;
  p.T = (int)d.T; p.hd = (int)d.hd; p.n_q = (int)d.n_q; p.n_kv = (int)d.n_kv;
  p.n_slots = d.n_pages * 128;
  p.status = status;
  memcpy(p.freq, freq, sizeof(RopeFreq) * (d.hd / 2));
  rope_append8_kernel<<<(unsigned)d.T, A8_THREADS, 0, st>>>(p);
  return 0;
}

int launch_kv_dequant_paged(const Dequant8Desc& d, int num_sms, unsigned* status, cudaStream_t st) {
  Dequant8Params p;
  p.k_codes = static_cast<const uint8_t*>(d.k_codes); p.v_codes = static_cast<const uint8_t*>(d.v_codes);
  p.k_scale = d.k_scale; p.v_scale = d.v_scale;
  p.k_pool = static_cast<uint16_t*>(d.k_pool); p.v_pool = static_cast<uint16_t*>(d.v_pool);
  p.block_table = d.block_table; p.n_pos = d.n_pos;
  p.B = (int)d.B; p.hd = (int)d.hd; p.n_kv = (int)d.n_kv; p.n_pages = (int)d.n_pages;
  p.max_pages = d.max_pages;
  p.status = status;
  const int64_t x = std::max<int64_t>(1, std::min<int64_t>(d.max_pages, (4 * num_sms + d.B - 1) / d.B));
  dequant8_kernel<<<dim3((unsigned)x, (unsigned)d.B), 256, 0, st>>>(p);
  return 0;
}

LLAMA_DEFINE_BOUNDS_READER(paged8)

}  // namespace llama
