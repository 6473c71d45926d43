// Warp-level f16 matrix products and the ranges of work, as the attention kernels over the caches use them.
#pragma once
#include "common.cuh"

namespace w4a8 {

// Workers of U units: ng for each CTA, W <= U in all.
struct Kv8Workers {
  int ng, W;
};
__device__ __forceinline__ Kv8Workers kv8_workers(int U, int ctas, int most) {
  const int ng = min(most, (U + ctas - 1) / ctas);
  return {ng, min(U, ctas * ng)};
}
// First unit of worker w of W <= U over U units, and the worker of unit u.
__device__ __forceinline__ int worker_begin(int w, int W, int U) { return (int)((int64_t)w * U / W); }
__device__ __forceinline__ int worker_of(int u, int W, int U) { return (int)((((int64_t)u + 1) * W - 1) / U); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// power of two that takes a largest magnitude into [2^10, 2^11) (1 where it is not finite)
__device__ __forceinline__ float f16_scale(float amax) {
  const int ex = (int)(__float_as_uint(amax) >> 23) & 255;
  return ex == 255 ? 1.0f : __uint_as_float((uint32_t)min(254, 264 - ex) << 23);
}

}  // namespace w4a8
