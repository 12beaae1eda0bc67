// Instructions of the attention kernels on tcgen05: products with an operand in Tensor Memory, its loads and stores, and
// paired fp32 arithmetic.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "ptx.cuh"

namespace moe {

// Bounded wait: the thread sleeps until the phase completes, and gives up after limit_ns, or once another thread of the block
// has given up. The one that gives up leaves `code` in *abort, which the kernel records at its end (these kernels run five
// kinds of warps side by side, and their code has to share the instruction cache).
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* abort,
                                         uint32_t code) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort = code;
      return false;
    }
  }
}

// D (+)= A B with A from Tensor Memory (bf16, two a column).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

#define MOE_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                     "=r"(r[i + 6]), "=r"(r[i + 7])
#define MOE_RW8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
                      "+r"(r[i + 6]), "+r"(r[i + 7])
#define MOE_RI8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                      "r"(r[i + 6]), "r"(r[i + 7])

// 32 lanes x 32 columns from r[i] on / back.
template <int N>
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[N], int i) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : MOE_R8(r, i), MOE_R8(r, i + 8), MOE_R8(r, i + 16), MOE_R8(r, i + 24) : "r"(taddr) : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[N]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::MOE_RI8(r, 0), MOE_RI8(r, 8), "r"(taddr) : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[N], int i) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      ::MOE_RI8(r, i), MOE_RI8(r, i + 8), MOE_RI8(r, i + 16), MOE_RI8(r, i + 24), "r"(taddr) : "memory");
}
// No use of r[i..i+31] is scheduled before this point.
template <int N>
__device__ __forceinline__ void reg_fence32(uint32_t (&r)[N], int i) {
  asm volatile("" : MOE_RW8(r, i), MOE_RW8(r, i + 8), MOE_RW8(r, i + 16), MOE_RW8(r, i + 24));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The factor of a score s in its weight's exponent, s c - m c in one fused operation, which keeps what rounding m c has left out: up
// to 16 below 2^29, which fp32 and bf16 weights can bear, but more than either at 2^32. From 2^29 on two scores that differ at all
// differ by 32 or more, so the power of two below c takes c's place: its products are exact, m's own exponent is 0, and the
// others' are below -16 still.
__device__ __forceinline__ float weight_factor(float m, float c) {
  return fabsf(m * c) < 0x1p29f ? c : __uint_as_float(__float_as_uint(c) & 0x7F800000u);
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// a b + c of two bf16 each.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace moe
