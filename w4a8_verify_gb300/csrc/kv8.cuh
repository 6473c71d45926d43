// The 8-bit key/value cache: geometry of a page, bounds of a cache and the device checks that
// every kernel on it shares.
#pragma once
#include <cuda_bf16.h>

#include <algorithm>
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
constexpr int64_t kMaxDifferences = 1 << 16;  // of strides that do not nest, in a host's check

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

// Whether two of the S x n x heads rows of D elements lie on one another.  Strides that nest (each at least the extent of
// the smaller ones) do not; else a difference of up to two of the indexes is followed by the nearest of the third (more than
// `most` such differences: taken as overlapping).
inline bool rows_overlap(const w4a8_rows& r, int S, int n, int heads, int D, int64_t most = INT64_MAX) {
  using Wide = __int128;
  struct Axis {
    Wide stride;
    int size;
  } ax[3] = {{r.seq, S}, {r.row, n}, {r.head, heads}};
  for (Axis& x : ax) x.stride = x.size == 1 ? 0 : x.stride < 0 ? -x.stride : x.stride;
  std::sort(ax, ax + 3, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  Wide extent = D;
  bool nested = true;
  for (const Axis& x : ax) {
    nested = nested && (x.size == 1 || x.stride >= extent);
    extent += (Wide)(x.size - 1) * x.stride;
  }
  if (nested) return false;
  if ((int64_t)ax[1].size * ax[2].size > most) return true;
  for (const Axis& x : ax)
    if (x.size > 1 && x.stride < D) return true;
  // a row of other indexes closer than D: i, j the differences in the two wider axes, k in the narrowest
  for (int i = 0; i < ax[2].size; ++i)
    for (int j = i ? 1 - ax[1].size : 1; j < ax[1].size; ++j) {
      const Wide at = i * ax[2].stride + j * ax[1].stride;
      const Wide k = ax[0].size == 1 ? 0 : at / ax[0].stride;
      for (Wide y = k - 1; y <= k + 1; ++y) {
        const Wide d = at - y * ax[0].stride;
        if (y > -ax[0].size && y < ax[0].size && d > -D && d < D) return true;
      }
    }
  return false;
}

// Whether the rows of two views, S x n x their heads x D elements of one size, may share memory: not where their address
// ranges are apart, nor where they are different heads of one tensor whose rows do not lie on one another.
inline bool rows_meet(const w4a8_rows& x, int heads_x, const w4a8_rows& y, int heads_y, int S, int n, int D, size_t el) {
  using Wide = __int128;
  auto range = [&](const w4a8_rows& r, int heads, Wide& lo, Wide& hi) {
    lo = hi = (Wide)reinterpret_cast<uintptr_t>(r.data);
    const Wide steps[3] = {(Wide)(S - 1) * r.seq, (Wide)(n - 1) * r.row, (Wide)(heads - 1) * r.head};
    for (Wide step : steps) (step < 0 ? lo : hi) += step * (Wide)el;
    hi += (Wide)D * (Wide)el;
  };
  Wide a0, a1, b0, b1;
  range(x, heads_x, a0, a1);
  range(y, heads_y, b0, b1);
  if (a1 <= b0 || b1 <= a0) return false;
  if ((S > 1 && x.seq != y.seq) || (n > 1 && x.row != y.row)) return true;
  // y's first head is head m of a tensor whose head 0 is x's first
  const int64_t head = heads_x > 1 ? x.head : y.head;
  if (heads_x > 1 && heads_y > 1 && x.head != y.head) return true;
  const Wide d = (Wide)reinterpret_cast<uintptr_t>(y.data) - (Wide)reinterpret_cast<uintptr_t>(x.data);
  if (!head || d % ((Wide)head * (Wide)el)) return true;
  const Wide m = d / ((Wide)head * (Wide)el);
  if (m > -heads_y && m < heads_x) return true;
  const Wide all = m > 0 ? m + heads_y : heads_x - m;
  w4a8_rows whole = x;
  whole.head = head;
  return all > (Wide)1 << 20 || rows_overlap(whole, S, n, (int)all, D, kMaxDifferences);
}

// Whether the a bytes at p and the b bytes at q share one (NULL: no).
inline bool bytes_meet(const void* p, size_t a, const void* q, size_t b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  return p && q && x < y + b && y < x + a;
}
// Whether one of the S x n x heads rows of D elements of el bytes lies on the bytes at p (NULL: no).  Where the address ranges
// cross, the first row behind p - D el is looked for along the longest axis, for each pair of the others' indexes (more than
// kMaxDifferences pairs: taken as touching).
inline bool rows_touch(const w4a8_rows& r, int heads, int S, int n, int D, size_t el, const void* p, size_t bytes) {
  using Wide = __int128;
  struct Axis {
    Wide stride;
    int size;
  } ax[3] = {{(Wide)r.seq * (Wide)el, S}, {(Wide)r.row * (Wide)el, n}, {(Wide)r.head * (Wide)el, heads}};
  const Wide row = (Wide)D * (Wide)el, lo = (Wide)reinterpret_cast<uintptr_t>(p), hi = lo + (Wide)bytes;
  Wide base = (Wide)reinterpret_cast<uintptr_t>(r.data), extent = row;
  for (Axis& x : ax) {  // from the lowest row on, upwards
    const Wide all = (x.size - 1) * x.stride;
    if (all < 0) base += all, x.stride = -x.stride;
    extent += all < 0 ? -all : all;
  }
  if (!p || !r.data || base + extent <= lo || hi <= base) return false;
  std::sort(ax, ax + 3, [](const Axis& x, const Axis& y) { return x.size > y.size; });
  if ((int64_t)ax[1].size * ax[2].size > kMaxDifferences) return true;
  for (int i = 0; i < ax[1].size; ++i)
    for (int j = 0; j < ax[2].size; ++j) {
      const Wide at = base + i * ax[1].stride + j * ax[2].stride, d = lo - row - at;
      const Wide k = d < 0 ? 0 : ax[0].stride ? d / ax[0].stride + 1 : ax[0].size;
      if (k < ax[0].size && at + k * ax[0].stride < hi) return true;
    }
  return false;
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

// Eight elements of a row, as they are, and in fp32.
template <typename T>
struct Eight {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) reinterpret_cast<T*>(u)[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p, bool wide) const {
    if (wide) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = reinterpret_cast<const T*>(u)[i];
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = kv8_load(reinterpret_cast<const T*>(u) + i);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) kv8_store(reinterpret_cast<T*>(u) + i, x[i]);
  }
};

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
