// Device helpers shared by the flash-attention kernels whose softmax owns one TMEM lane (score row) per
// thread: dense prefill (attn_tc.cu) and chunks over a paged cache (chunk_attn.cu).
#pragma once

#include "common.cuh"

namespace llama {

// O in TMEM is rescaled only when a row's maximum grew by more than 2^8
constexpr float kRescaleLog2 = 8.0f;

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^x with one MUFU instruction (PTX ex2.approx.ftz: relative error about 2^-22, subnormal
// results flushed to zero -- exact enough for P, which is rounded to bf16).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void tmem_ld16_at(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// Packed pairs of fp32 (sm_100 and later): (d0, d1) = (a0 b0 + c0, a1 b1 + c1) in one instruction,
// and (s0, s1) += (a0, a1).
__device__ __forceinline__ void fma_f32x2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0,
                                          float c1) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add_f32x2(float& s0, float& s1, float a0, float a1) {
  asm("{\n\t.reg .b64 ra, rs;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rs, {%0, %1};\n\t"
      "add.rn.f32x2 rs, rs, ra;\n\tmov.b64 {%0, %1}, rs;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(a0), "f"(a1));
}

// 32 scores of a row -> 16 bf16 pairs of P = 2^(s * scale - m) stored at TMEM column `col`; the
// fp32 values are added to the row sums.  The scaling and the sums run on packed pairs.
__device__ __forceinline__ void exp_chunk(const uint32_t (&v)[32], uint32_t col, float scale, float m, float& ls0,
                                          float& ls1) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a0, a1;
    fma_f32x2(a0, a1, __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]), scale, scale, -m, -m);
    const float p0 = ex2(a0);
    const float p1 = ex2(a1);
    add_f32x2(ls0, ls1, p0, p1);
    w[e] = pack_bf16x2(p0, p1);
  }
  tmem_st16(col, w);
}

// mbar_wait in few instructions (what a warp executes between two waits has to come from the
// instruction cache): only every 64th failed try leaves the loop, to look at the abort flag and the
// clock.  Returns false when the wait was given up, as mbar_wait does.
static __device__ __noinline__ unsigned long long wait_check(unsigned long long t0, volatile int* abort, unsigned* status) {
  if (*abort) return 0;
  const unsigned long long t = globaltimer_ns();
  if (t0 == 0) return t;
  if (t - t0 <= kWaitLimitNs) return t0;
  atomicOr(status, STATUS_TIMEOUT);
  *abort = 1;
  return 0;
}
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* status) {
  unsigned long long t0 = 0;
  uint32_t tries = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++tries & 63u) == 0 && !(t0 = wait_check(t0, abort, status))) return false;
  }
  return true;
}

// The same for a whole warp whose control flow is to stay uniform: the loop's exit is a vote.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* status) {
  uint32_t tries = 0;
  unsigned long long t0 = 0;
  while (__ballot_sync(0xffffffffu, mbar_try_wait(bar, parity)) != 0xffffffffu) {
    if ((++tries & 63u) == 0) {
      if (__ballot_sync(0xffffffffu, *abort != 0) != 0u) return false;
      const unsigned long long t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (__ballot_sync(0xffffffffu, t - t0 > kWaitLimitNs) != 0u) {
        atomicOr(status, STATUS_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
  }
  return true;
}

// ---- tcgen05 issued from a whole warp: every lane runs the instruction stream, the lane with `one` != 0
//      issues.  The flow stays uniform, so operands stay in uniform registers.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void tc_mma_if(uint32_t one, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts_if(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(one)
      : "memory");
}

// Registers per thread of a warpgroup, moved between warpgroups of a running block.
template <int N> __device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

}  // namespace llama
