// The 4-bit key/value cache: geometry of a page, the scale's eight bits, bounds of a cache and the device checks that
// every kernel on it shares.
//
// A row of 32 dims is c s, c a whole number -7 .. 7 and s = (8 + m) 2^(e - 18) with three bits of m: c s has seven
// significant bits at most, so it is exact as f16 (the tensor cores' operand) and as bf16 (what a read may return), and no
// kernel has to carry scales behind its products.  s to the nearest of those numbers costs no error of a code: the
// largest value is at most 7.4375 s, which the code 7 holds as well as any other value its own (but for scales below
// 2^-14, whose steps are coarser, and the largest).
#pragma once
#include "kv8.cuh"

namespace w4a8 {

constexpr float kKv4MaxScale = 240.0f;       // 264 s, the offset of a code in f16, stays finite
constexpr int kKv4Nan = 255;                 // scale byte of a group with a value that is not finite
constexpr int kKv4MaxRows = 64;              // new rows of one sequence in an attention call (one 64-bit mask)

// Bytes of a page of one head: codes of the keys, of the values, scales of the keys, of the values.
template <int D>
struct Kv4Page {
  static constexpr int V = 32 * D, KS = 64 * D, VS = 66 * D, BYTES = 68 * D;
};

inline w4a8_status kv4_dims(const w4a8_kv4_cache* c) {
  if (!c) return W4A8_ERR_ARG;
  if (c->n_seqs < 1 || c->n_seqs > kKv8MaxSeqs || c->n_kv_heads < 1 || c->n_kv_heads > kKv8MaxHeads ||
      (c->head_dim != 64 && c->head_dim != 128) || c->max_pages < 1 || c->max_pages > kKv8MaxPages || c->n_pages < 1 ||
      (int64_t)c->n_pages * c->n_kv_heads >= ((int64_t)1 << 31) ||
      (int64_t)c->n_seqs * c->n_kv_heads * c->max_pages >= ((int64_t)1 << 31))
    return W4A8_ERR_SHAPE;
  return W4A8_OK;
}
inline w4a8_status kv4_valid(const w4a8_kv4_cache* c) {
  const w4a8_status st = kv4_dims(c);
  if (st != W4A8_OK) return st;
  if (!c->pages || !c->table || !c->len || !c->ctl) return W4A8_ERR_ARG;
  if (!aligned(c->pages, 128) || !aligned(c->table, 4) || !aligned(c->len, 4) || !aligned(c->ctl, 4)) return W4A8_ERR_ARG;
  return W4A8_OK;
}

inline size_t kv4_pool_bytes(const w4a8_kv4_cache& c) { return (size_t)c.n_pages * c.n_kv_heads * 68 * (size_t)c.head_dim; }

// Committed length of sequence s, or -1 (and the status bit) where it is out of range.
__device__ __forceinline__ int kv4_len(const w4a8_kv4_cache& c, const int32_t* len, int s) {
  const int L = __ldcg(len + s);  // from L2: a kernel that starts early reads it before it waits for the last one
  if (L < 0 || L > kPage * c.max_pages) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    return -1;
  }
  return L;
}
// Rows of sequence s in a call of n, or -1 (and the status bit) where the count is out of range.
__device__ __forceinline__ int kv4_count(const w4a8_kv4_cache& c, const int32_t* counts, int s, int n) {
  if (!counts) return n;
  const int v = __ldcg(counts + s);
  if (v < 0 || v > n) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    return -1;
  }
  return v;
}
// Page of the pool that holds page p of sequence s, or -1 (and the status bit) where the entry is out of range.
__device__ __forceinline__ int kv4_phys(const w4a8_kv4_cache& c, int s, int p) {
  const int v = __ldcg(c.table + (size_t)s * c.max_pages + p);
  if (v < 0 || v >= c.n_pages) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_TREE);
    return -1;
  }
  return v;
}
template <int D>
__device__ __forceinline__ uint8_t* kv4_page(const w4a8_kv4_cache& c, int phys, int h) {
  return c.pages + ((size_t)phys * c.n_kv_heads + h) * Kv4Page<D>::BYTES;
}

// Scale of a group whose largest magnitude is amax, and its byte: amax / 7 by IEEE division, then to the nearest (half to
// even) of (8 + m) 2^(e - 18), or m 2^-17 below 2^-14.
__device__ __forceinline__ float kv4_scale(float amax, uint32_t& byte) {
  if (!(amax <= 3.402823466e38f)) {
    byte = kKv4Nan;
    return __int_as_float(0x7fffffff);
  }
  const float t = __fdiv_rn(amax, 7.0f);
  if (t < 6.103515625e-5f) {  // 2^-14
    const float r = rintf(t * 131072.0f);
    byte = (uint32_t)r;
    return r * 7.62939453125e-6f;
  }
  uint32_t u = __float_as_uint(fminf(t, kKv4MaxScale));
  u = (u + 0x7ffffu + (u >> 20 & 1u)) >> 20;
  byte = u - (112u << 3);
  return __uint_as_float(u << 20);
}
// The four 4-bit fields of a 16-bit word lie two bits to the left of their natural place, the last one's upper half
// around the end: two of them are then whole f16 mantissa fields (bits 2..5 under the exponent of 256, bits 6..9 under that
// of 16), and the other two after the word's bytes change places.
__device__ __forceinline__ uint32_t kv4_turn(uint32_t two) {  // both 16-bit halves of natural fields
  return (two << 2 & 0xfffcfffcu) | (two >> 14 & 0x00030003u);
}
__device__ __forceinline__ uint32_t kv4_unturn(uint32_t two) {
  return (two >> 2 & 0x3fff3fffu) | (two << 14 & 0xc000c000u);
}

// (a & b) | c as one instruction: two immediates would make two of it
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

}  // namespace w4a8
