// The 8-bit key/value cache: geometry of a page, bounds of a cache and the device checks that
// every kernel on it shares.
#pragma once
#include <cuda_bf16.h>

#include <atomic>
#include <climits>

#include "common.cuh"

namespace w4a8 {

constexpr int kPage = 64;              // tokens of a page (one scale each for its keys and its values)
constexpr int kKv8MaxSeqs = 4096;
constexpr int kKv8MaxHeads = 1024;
constexpr int kKv8MaxPages = 16384;    // a million tokens; the selection keeps a head's scores in shared memory
constexpr int kKv8MaxRows = 64;        // new rows of one sequence in an attention call (one 64-bit mask)
constexpr int kKv8MaxGroup = 16;       // query heads per KV head

// Lets a kernel use that much dynamic shared memory: once for each device (a host call of a microsecond).
template <auto Kern>
inline cudaError_t kv8_smem(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

inline w4a8_status kv8_dims(const w4a8_kv8_cache* c) {
  if (!c) return W4A8_ERR_ARG;
  if (c->n_seqs < 1 || c->n_seqs > kKv8MaxSeqs || c->n_kv_heads < 1 || c->n_kv_heads > kKv8MaxHeads ||
      (c->head_dim != 64 && c->head_dim != 128) || c->max_pages < 1 || c->max_pages > kKv8MaxPages ||
      (int64_t)c->n_seqs * c->n_kv_heads * c->max_pages >= ((int64_t)1 << 31))
    return W4A8_ERR_SHAPE;
  return W4A8_OK;
}
inline w4a8_status kv8_valid(const w4a8_kv8_cache* c) {
  const w4a8_status st = kv8_dims(c);
  if (st != W4A8_OK) return st;
  if (!c->codes || !c->scales || !c->sums || !c->tail || !c->table || !c->len || !c->ctl) return W4A8_ERR_ARG;
  if (!aligned(c->codes, 128) || !aligned(c->tail, 16) || !aligned(c->sums, 16) || !aligned(c->scales, 16) ||
      !aligned(c->table, 4) || !aligned(c->len, 4) || !aligned(c->ctl, 4))
    return W4A8_ERR_ARG;
  return W4A8_OK;
}
inline bool kv8_dtype(int t) { return t == W4A8_F32 || t == W4A8_BF16; }
inline size_t kv8_elem(int t) { return t == W4A8_F32 ? 4 : 2; }

// Whether groups of eight elements can be read 16 bytes at a time.
inline bool kv8_vec_rows(const w4a8_rows& r, int dtype) {
  const int64_t e = 16 / (int64_t)kv8_elem(dtype);
  return aligned(r.data, 16) && r.seq % e == 0 && r.row % e == 0 && r.head % e == 0;
}

// (sequence, KV head) pair index and page addresses: 64-bit, a long cache passes 4 GB
__device__ __forceinline__ size_t kv8_pair(const w4a8_kv8_cache& c, int s, int h) { return (size_t)s * c.n_kv_heads + h; }
__device__ __forceinline__ size_t kv8_page(const w4a8_kv8_cache& c, size_t pair, int phys) {
  return pair * c.max_pages + phys;
}

// Committed length of sequence s, or -1 (and the status bit) where it is out of range.
__device__ __forceinline__ int kv8_len(const w4a8_kv8_cache& c, const int32_t* len, int s) {
  const int L = __ldcg(len + s);  // from L2: a kernel that starts early reads it before it waits for the last one
  if (L < 0 || L > kPage * c.max_pages + kPage - 1) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    return -1;
  }
  return L;
}
// Rows of sequence s in a call of n, or -1 (and the status bit) where the count is out of range.
__device__ __forceinline__ int kv8_count(const w4a8_kv8_cache& c, const int32_t* counts, int s, int n) {
  if (!counts) return n;
  const int v = __ldcg(counts + s);
  if (v < 0 || v > n) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    return -1;
  }
  return v;
}
// Physical page of logical page p of a pair, or -1 (and the status bit) where the entry is out of range.
__device__ __forceinline__ int kv8_phys(const w4a8_kv8_cache& c, size_t pair, int p) {
  const int v = c.table[pair * c.max_pages + p];
  if (v < 0 || v >= c.max_pages) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_TREE);
    return -1;
  }
  return v;
}

__device__ __forceinline__ float kv8_float(float v) { return v; }
__device__ __forceinline__ float kv8_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ float kv8_load(const T* p) {
  return kv8_float(*p);
}
template <typename T>
__device__ __forceinline__ void kv8_store(T* p, float v);
template <>
__device__ __forceinline__ void kv8_store<float>(float* p, float v) {
  *p = v;
}
template <>
__device__ __forceinline__ void kv8_store<__nv_bfloat16>(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

// max that keeps a NaN (an absmax with a NaN among the values is NaN)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// scale of values whose largest magnitude is amax (NaN where a value was not finite)
__device__ __forceinline__ float kv8_scale(float amax) {
  return amax <= 3.402823466e38f ? __fdiv_rn(amax, 127.0f) : __int_as_float(0x7fffffff);
}
// code of a finite x at scale s > 0
__device__ __forceinline__ int kv8_code(float x, float s) {
  const float r = rintf(__fdiv_rn(x, s));
  return (int)fminf(fmaxf(r, -127.0f), 127.0f);
}

}  // namespace w4a8
