// The 8-bit paged cache ("LLaMA-3 8B ...", section 七 sizes the cache): writing K and V rows as E4M3 codes
// with a scale per position and KV head, and reading pages back to bf16.
//
// write: x the rotated K row or the V row of one head, u = max |v_i| for V and max (|a| + |b|) over the
//   pairs for K (a rotation keeps a pair inside that circle, so the scale is the same at every
//   position and no code saturates; summed upwards, so that what is above 448 * 2^e does not round onto it); scale 2^e, e the smallest with u <= 448 * 2^e; code = E4M3(x * 2^-e).
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
constexpr int A8_FEW = 2, A8_MANY = 4;       // tokens of a CTA
constexpr int A8_MANY_CTAS_PER_SM = 6;

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

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
}

// A row whose slot can be written: its slot, else -1 (latching what cannot be).
__device__ __forceinline__ int checked_slot(const Append8Params& p, int t) {
  if (t >= p.T) return -1;
  const int slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);
  if (slot >= 0 && (slot >= p.n_slots || pos < 0 || pos >= (1 << 24))) {
    atomicOr(p.status, STATUS_BAD_PLAN);
    return -1;
  }
  return slot;
}

// Where a token's rows go.
struct TokenOut {
  uint16_t* q;
  uint8_t *k, *v;
  float *ks, *vs;      // its scale in head 0
  int slot;            // -1: nothing is written
};

// One 16-byte vector of a head's row, VPH of them in VPH neighbouring lanes: rotated, and for K and V (`scales`: some lane of the
// warp has one) encoded with the scale that the lanes agree on.  Every lane of the warp calls it; `live` says which have a
// vector: number o of part 0 (q), 1 (k) or 2 (v).
template <int VPH>
__device__ __forceinline__ void store_vector(const Append8Params& p, uint4 w, bool live, bool scales, int part, int o,
                                             const TokenOut& out, const float2* cs) {
  float x[8];
  unpack8(w, x);
  float u = 0.f;
  if (scales) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float a = fabsf(x[i]), b = fabsf(x[i + 1]);
      u = fmaxf(u, part == 2 ? fmaxf(a, b) : __fadd_ru(a, b));
    }
#pragma unroll
    for (int k = VPH / 2; k > 0; k >>= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, k));
  }
  if (!live || out.slot < 0) return;
  const int j = o % VPH;
  if (part != 2) {
    const float4 c0 = reinterpret_cast<const float4*>(cs)[2 * j], c1 = reinterpret_cast<const float4*>(cs)[2 * j + 1];
    const float2 c[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i].x - b * c[i].y;
      x[2 * i + 1] = a * c[i].y + b * c[i].x;
    }
  }
  if (part == 0) {
    if (in_extent(out.q + o * 8 - p.q_out, 8, (int64_t)p.T * p.n_q * p.hd)) *reinterpret_cast<uint4*>(out.q + o * 8) = pack8(x);
    return;
  }
  const int e = row_scale_exp(u);
  uint8_t* codes = part == 2 ? out.v : out.k;
  if (in_extent(codes + o * 8 - (part == 2 ? p.v_codes : p.k_codes), 8, p.n_slots * p.n_kv * p.hd))
    *reinterpret_cast<uint2*>(codes + o * 8) = encode8(x, exp2_int(-e));
  float* scale = (part == 2 ? out.vs : out.ks) + o / VPH * 128;
  if (j == 0 && in_extent(scale - (part == 2 ? p.v_scale : p.k_scale), 1, p.n_slots * p.n_kv)) *scale = exp2_int(e);
}

// HBM bound: every row is read once in 16-byte pieces and written once.  A CTA takes TOK tokens, forms each token's hd / 2
// cosines and sines once, then walks the vectors of their q, k and v heads: vector i of all its tokens at a time, so that what
// belongs to a place in the row is found once, the next ones on their way; the lanes of a head (VPH = hd / 8, a power
// of two) agree on its scale by shuffles.  8192 tokens of 32/8 heads x 128 (185 MB): 31.3 us = 5.9 TB/s with four tokens per
// CTA, 32.9 with two, 34.1 with one; 2048 of 32/32: 16.7, 16.1, 17.8; 1000 of 32/8: 6.5, 6.2, 6.0; 300: 3.4.  So four where
// that leaves every SM several CTAs, two where it leaves it one.  (A warp per head and token 59 us.)
template <int VPH, int TOK>
__global__ void __launch_bounds__(A8_THREADS) rope_append8_kernel(const __grid_constant__ Append8Params p) {
  __shared__ __align__(16) float2 cs[TOK][VPH * 4];
  __shared__ TokenOut out[TOK];
  const int q_vec = p.q ? p.n_q * VPH : 0, kv_vec = p.n_kv * VPH, total = q_vec + 2 * kv_vec;
  const int t0 = blockIdx.x * TOK, n = min(TOK, p.T - t0);
  auto place = [&](int i, int& part, int& o) {
    part = i < q_vec ? 0 : i < q_vec + kv_vec ? 1 : 2;
    o = part == 0 ? i : i - q_vec - (part == 2 ? kv_vec : 0);
  };
  auto load = [&](int i, uint4 (&w)[TOK]) {
    if (i >= total) return;
    int part, o;
    place(i, part, o);
    const uint16_t* src = part == 0 ? p.q : part == 2 ? p.v : p.k;
    const int64_t stride = part == 0 ? p.q_stride : part == 2 ? p.v_stride : p.k_stride;
    src += t0 * stride + o * 8;
#pragma unroll
    for (int tk = 0; tk < TOK; ++tk)
      if (tk < n) w[tk] = *reinterpret_cast<const uint4*>(src + tk * stride);
  };
  uint4 w[TOK];
  load(threadIdx.x, w);   // on their way while the angles are formed
  if (threadIdx.x < TOK) {
    TokenOut r;
    r.slot = checked_slot(p, t0 + threadIdx.x);
    const int64_t at = max(r.slot, 0), row = at * p.n_kv * p.hd, head0 = at / 128 * p.n_kv * 128 + at % 128;
    r.q = p.q_out + (int64_t)(t0 + threadIdx.x) * p.n_q * p.hd;
    r.k = p.k_codes + row;
    r.v = p.v_codes + row;
    r.ks = p.k_scale + head0;
    r.vs = p.v_scale + head0;
    out[threadIdx.x] = r;
  }
  for (int i = threadIdx.x; i < TOK * VPH * 4; i += A8_THREADS) {
    const int tk = i % TOK, j = i / TOK;
    if (tk < n) rope_sincos((float)__ldg(p.positions + t0 + tk), p.freq[j], cs[tk][j].y, cs[tk][j].x);
  }
  __syncthreads();
  for (int i0 = 0; i0 < total; i0 += A8_THREADS) {   // whole warps stay together for the shuffles
    const int i = i0 + threadIdx.x;
    uint4 next[TOK];
    load(i + A8_THREADS, next);
    int part, o;
    place(i, part, o);
    const bool live = i < total, scales = (i | 31) >= q_vec;   // (the warp's last vector is no query's)
#pragma unroll
    for (int tk = 0; tk < TOK; ++tk)
      if (tk < n) store_vector<VPH>(p, w[tk], live, scales, part, live ? o : 0, out[tk], cs[tk]);
#pragma unroll
    for (int tk = 0; tk < TOK; ++tk) w[tk] = next[tk];
  }
}

// Other head widths: one token per CTA, one head per warp at a time, a lane per vector.
__global__ void __launch_bounds__(A8_THREADS) rope_append8_any_kernel(const __grid_constant__ Append8Params p) {
  __shared__ float2 cs[kMaxRopePairs];
  __shared__ int slot_sh;
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.hd / 2, vph = p.hd / 8;
  if (threadIdx.x == 0) slot_sh = checked_slot(p, t);
  const int pos = __ldg(p.positions + t);
  for (int j = threadIdx.x; j < half; j += A8_THREADS) rope_sincos((float)pos, p.freq[j], cs[j].y, cs[j].x);
  __syncthreads();
  const int slot = slot_sh;
  if (slot < 0) return;
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
        u = fmaxf(u, is_v ? fmaxf(fabsf(a), fabsf(b)) : __fadd_ru(fabsf(a), fabsf(b)));
        if (!is_v) {
          const float2 c = cs[lane * 4 + i];
          x[2 * i] = a * c.x - b * c.y;
          x[2 * i + 1] = a * c.y + b * c.x;
        }
      }
    }
    if (is_q) {
      const int64_t at = ((int64_t)t * p.n_q + g) * p.hd + lane * 8;
      if (lane < vph && in_extent(at, 8, (int64_t)p.T * p.n_q * p.hd)) *reinterpret_cast<uint4*>(p.q_out + at) = pack8(x);
      continue;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
    const int e = row_scale_exp(u);
    if (lane < vph) {
      const int64_t at = ((int64_t)slot * p.n_kv + g) * p.hd + lane * 8;
      if (in_extent(at, 8, p.n_slots * p.n_kv * p.hd))
        *reinterpret_cast<uint2*>((is_v ? p.v_codes : p.k_codes) + at) = encode8(x, exp2_int(-e));
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

// HBM bound.  A unit is DQ_ROWS rows of a page of K or of V; the CTAs take the units of all sequences, one after the
// other, in turn, so that at any time they work on neighbouring ones.  16 ragged sequences of 1000-6000 positions, 8 heads
// x 128 (337 MB): 56.3 us = 6.0 TB/s, 90% of a copy's rate; a contiguous range per CTA 57.6 us, 16-byte stores
// 67 us, 4 and 6 CTAs per SM 57-62 us, streaming loads 3-4 us more.
constexpr int DQ_THREADS = 256;
constexpr int DQ_ROWS = 32;
constexpr int DQ_UNITS = 2 * 128 / DQ_ROWS;   // of a page
constexpr int DQ_CTAS_PER_SM = 3;
constexpr int DQ_DEEP = 4;                    // loads of a thread in flight

// VEC codes of one head's row, as a load.
template <int VEC> struct Codes;
template <> struct Codes<16> { uint4 w; };
template <> struct Codes<8> { uint2 w; };

__device__ __forceinline__ uint4 decode8(uint32_t c0, uint32_t c1, float s) {
  const float2 a0 = e4m3x2_to_f2(c0 & 0xFFFFu), a1 = e4m3x2_to_f2(c0 >> 16);
  const float2 a2 = e4m3x2_to_f2(c1 & 0xFFFFu), a3 = e4m3x2_to_f2(c1 >> 16);
  return make_uint4(pack_bf2(a0.x * s, a0.y * s), pack_bf2(a1.x * s, a1.y * s), pack_bf2(a2.x * s, a2.y * s),
                    pack_bf2(a3.x * s, a3.y * s));
}
__device__ __forceinline__ void store_decoded(uint16_t* dst, const Codes<8>& c, float s) {
  *reinterpret_cast<uint4*>(dst) = decode8(c.w.x, c.w.y, s);
}
__device__ __forceinline__ void store_decoded(uint16_t* dst, const Codes<16>& c, float s) {   // 32 bytes, aligned
  const uint4 a = decode8(c.w.x, c.w.y, s), b = decode8(c.w.z, c.w.w, s);
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// VEC: 16 where heads are that wide a multiple, else 8
template <int VEC>
__global__ void __launch_bounds__(DQ_THREADS, DQ_CTAS_PER_SM) dequant8_kernel(const __grid_constant__ Dequant8Params p) {
  __shared__ int64_t wsum[DQ_THREADS / 32];
  __shared__ int start[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto pages_of = [&](int b, bool tell) {
    const int n = __ldg(p.n_pos + b);
    const bool bad = n < 0 || n > p.max_pages * 128 || n > (1 << 24);
    if (bad && tell) atomicOr(p.status, STATUS_BAD_PLAN);
    return bad ? 0 : (n + 127) / 128;
  };
  const int per = (p.B + DQ_THREADS - 1) / DQ_THREADS;
  const int s0 = min(p.B, (int)threadIdx.x * per), s1 = min(p.B, s0 + per);
  int64_t mine = 0;
  for (int b = s0; b < s1; ++b) mine += pages_of(b, blockIdx.x == 0);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
  int64_t all = 0, first = upto - mine;
  for (int w = 0; w < DQ_THREADS / 32; ++w) {
    if (w < warp) first += wsum[w];
    all += wsum[w];
  }
  const int64_t u0 = blockIdx.x, u1 = all * DQ_UNITS;
  if (u0 >= u1) return;
  if (first <= u0 / DQ_UNITS && u0 / DQ_UNITS < first + mine) {
    int64_t off = first;
    int b = s0, n = pages_of(b, false);
    while (off + n <= u0 / DQ_UNITS) { off += n; n = pages_of(++b, false); }
    start[0] = b;
    start[1] = (int)(u0 / DQ_UNITS - off);
  }
  __syncthreads();
  int b = start[0], j = start[1], n = __ldg(p.n_pos + b);
  int64_t pg = u0 / DQ_UNITS;
  const unsigned vph = p.hd / VEC, row_vecs = p.n_kv * vph;
  for (int64_t u = u0; u < u1; u += gridDim.x) {
    j += (int)(u / DQ_UNITS - pg);
    pg = u / DQ_UNITS;
    while (j * 128 >= n) {   // the sequence that holds it
      j -= pages_of(b, false);
      n = pages_of(++b, false) ? __ldg(p.n_pos + b) : 0;
    }
    const int part = (int)(u % DQ_UNITS);
    const int page = __ldg(p.block_table + (int64_t)b * p.max_pages + j);
    const bool is_v = part >= DQ_UNITS / 2;
    const int row0 = part % (DQ_UNITS / 2) * DQ_ROWS, rows = min(DQ_ROWS, n - j * 128 - row0);
    if (page < 0 || page >= p.n_pages) {
      if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_PLAN);
    } else if (rows > 0) {
      const int64_t at = ((int64_t)page * 128 + row0) * row_vecs;   // in vectors of VEC elements
      const Codes<VEC>* src = reinterpret_cast<const Codes<VEC>*>(is_v ? p.v_codes : p.k_codes) + at;
      uint16_t* dst = (is_v ? p.v_pool : p.k_pool) + at * VEC;
      const float* scale = (is_v ? p.v_scale : p.k_scale) + (int64_t)page * p.n_kv * 128 + row0;
      const unsigned total = rows * row_vecs;
      for (unsigned i0 = threadIdx.x; i0 < total; i0 += DQ_THREADS * DQ_DEEP) {
        Codes<VEC> c[DQ_DEEP];
        float s[DQ_DEEP];
#pragma unroll
        for (int k = 0; k < DQ_DEEP; ++k) {
          const unsigned i = i0 + k * DQ_THREADS;
          if (i < total) {
            c[k].w = __ldg(&src[i].w);
            const unsigned row = i / row_vecs, g = (i - row * row_vecs) / vph;
            s[k] = __ldg(scale + (int64_t)g * 128 + row);
          }
        }
#pragma unroll
        for (int k = 0; k < DQ_DEEP; ++k) {
          const unsigned i = i0 + k * DQ_THREADS;
          if (i < total && in_extent(at + i, 1, (int64_t)p.n_pages * 128 * row_vecs)) store_decoded(dst + (int64_t)i * VEC, c[k], s[k]);
        }
      }
    }
  }
}

}  // namespace

int launch_rope_append8(const Append8Desc& d, const RopeFreq* freq, int num_sms, unsigned* status, cudaStream_t st) {
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
  const int tok = d.T >= (int64_t)A8_MANY * A8_MANY_CTAS_PER_SM * num_sms ? A8_MANY : d.T >= (int64_t)A8_FEW * num_sms ? A8_FEW : 1;
  const unsigned grid = (unsigned)((d.T + tok - 1) / tok);
  if (d.hd == 64)
    (tok == A8_MANY  ? rope_append8_kernel<8, A8_MANY>
     : tok == A8_FEW ? rope_append8_kernel<8, A8_FEW>
                     : rope_append8_kernel<8, 1>)<<<grid, A8_THREADS, 0, st>>>(p);
  else if (d.hd == 128)
    (tok == A8_MANY  ? rope_append8_kernel<16, A8_MANY>
     : tok == A8_FEW ? rope_append8_kernel<16, A8_FEW>
                     : rope_append8_kernel<16, 1>)<<<grid, A8_THREADS, 0, st>>>(p);
  else rope_append8_any_kernel<<<(unsigned)d.T, A8_THREADS, 0, st>>>(p);
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
  const int64_t units = std::min<int64_t>(d.B * d.max_pages, INT32_MAX) * DQ_UNITS;
  const unsigned grid = (unsigned)std::min<int64_t>(units, DQ_CTAS_PER_SM * num_sms);
  // 32-byte stores need the pools on 32 bytes too
  const bool wide = d.hd % 16 == 0 && ((reinterpret_cast<uintptr_t>(d.k_pool) | reinterpret_cast<uintptr_t>(d.v_pool)) & 31) == 0;
  if (wide) dequant8_kernel<16><<<grid, DQ_THREADS, 0, st>>>(p);
  else dequant8_kernel<8><<<grid, DQ_THREADS, 0, st>>>(p);
  return 0;
}

LLAMA_DEFINE_BOUNDS_READER(paged8)

}  // namespace llama
