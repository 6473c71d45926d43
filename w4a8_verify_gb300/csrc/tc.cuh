// tcgen05 by inline PTX, as the attention kernels over the caches use it: f16 products with A in tensor memory, loads and
// stores of tensor memory, and the turns of mbarrier rings.
#pragma once
#include "common.cuh"

namespace w4a8 {

__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
// f16 x f16 -> f32, both operands K-major, M = 128
__host__ __device__ constexpr uint32_t tc_idesc(int N) { return 1u << 4 | (uint32_t)(N / 8) << 17 | (128u / 16) << 24; }
// Shared-memory operand, low word: K-major rows of 128 bytes; high word: eight rows 1024 bytes apart, 128-byte swizzle
__device__ __forceinline__ uint32_t tc_desc(uint32_t addr) { return (addr >> 4 & 0x3fffu) | 1u << 16; }
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
// D[128][N] (+)= A (tensor memory) B (shared memory), one k-step of 16, by one thread of a converged warp: the operands
// are uniform values, and no branch around the instruction keeps the compiler from holding them as such
template <int N>
__device__ __forceinline__ void tc_mma(uint32_t leader, uint32_t d, uint32_t a, uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %0, 0;\n mov.b64 b, {%3, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %5, p;\n}\n" ::"r"(leader), "r"(d), "r"(a), "r"(desc),
      "r"((uint32_t)add), "r"(tc_idesc(N)), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %0, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}\n" ::"r"(leader), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
#define W4A8_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define W4A8_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tc_load32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;\n"
      : W4A8_R8(v, 0), W4A8_R8(v, 8), W4A8_R8(v, 16), W4A8_R8(v, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_load16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n tcgen05.wait::ld.sync.aligned;\n"
      : W4A8_R8(v, 0), W4A8_R8(v, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_store16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::W4A8_I8(
                   v, 0),
               W4A8_I8(v, 8), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The nearest whole number of |x| < 2^22 (NaN stays)
__device__ __forceinline__ float whole(float x) { return __fadd_rn(__fadd_rn(x, 12582912.0f), -12582912.0f); }

// Use n of a ring of mbarriers: entry and phase parity.
template <int N>
struct Turn {
  int i, ph;
  __device__ explicit Turn(unsigned n = 0) : i((int)(n % N)), ph((int)(n / N & 1u)) {}
  __device__ void next() {
    if (++i == N) i = 0, ph ^= 1;
  }
};

}  // namespace w4a8
