// Writing and reading the 4-bit key/value cache.
//
// A warp takes a tile, the 16 tokens x head_dim keys or values of one head: the unit whose words no other tile shares, so
// whoever adds a token to a page changes its 4-bit fields without atomics.  Each 32-dim group of a row is quantised
// on its own, in registers: four lanes (keys) or two (values) hold it, and exchange nothing but its largest magnitude.
#include "kv4.cuh"

#include <type_traits>

using namespace w4a8;

namespace {

constexpr int kTile = 16;                // tokens of a tile
constexpr int kMaxIndexed = 1024;        // rows of an append that takes its source rows from a list
constexpr int kBigThreads = 256;         // four tiles of keys, four of values
constexpr int kSmallThreads = 512;

struct Source {                          // new rows of one of keys and values
  w4a8_rows rows;
  int wide;                              // eight elements may be read 16 bytes at a time
};

// New length of a sequence, or -1 where the call leaves it as it was.
__device__ int append_end(const w4a8_kv4_cache& c, const int32_t* counts, int s, int n, int L) {
  const int cnt = kv4_count(c, counts, s, n);
  if (L < 0 || cnt < 0) return -1;
  if (L + (int64_t)cnt > (int64_t)kPage * c.max_pages) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    return -1;
  }
  return L + cnt;
}
// Whether every source row of the sequence's list is in range (all threads of the block).
__device__ bool append_index_ok(const w4a8_kv4_cache& c, const int32_t* index, int s, int n, int n_src, int cnt) {
  bool ok = true;
  for (int j = threadIdx.x; j < cnt; j += blockDim.x) {
    const int r = index[(size_t)s * n + j];
    ok = ok && r >= 0 && r < n_src;
  }
  ok = __syncthreads_and(ok);
  if (!ok && threadIdx.x == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TOKEN);
  return ok;
}

// Largest magnitude of N vectors of eight elements; NaN where one is among them.
template <int N>
__device__ __forceinline__ float largest(const Eight<float> (&x)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8 * N; ++i) m = max_nan(m, fabsf(reinterpret_cast<const float*>(x)[i]));
  return m;
}
template <int N>
__device__ __forceinline__ float largest(const Eight<__nv_bfloat16> (&x)[N]) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(x);
  __nv_bfloat162 m = __habs2(p[0]);
#pragma unroll
  for (int i = 1; i < 4 * N; ++i) m = __hmax2_nan(m, __habs2(p[i]));
  return max_nan(__low2float(m), __high2float(m));
}

// Codes are held as the bits of the fp32 number 1.5 2^23 + 8 + code: adding that constant makes a whole number, ties to
// even, in the low bits.  A word of eight fields is then a sum of products (kFields takes the constant's bits out).
constexpr float kMagic = 12582920.0f;
constexpr uint32_t kMagicBits = 0x4b400000u, kFields = 0u - kMagicBits * 0x11111111u;

// Scale of a group, its byte, and the codes of N of its values.
//
// fp32: rint of the IEEE quotient without a division.  f = rint(x fl(1 / s)) is the nearest whole number or, close to a half,
// its neighbour; x - f s is exact (f s has seven bits), so comparing it with s / 2 decides: x and s / 2 odd multiples
// are a unit of x apart at least, which the quotient's rounding keeps on its side.
template <int N>
__device__ __forceinline__ uint32_t quantise(const Eight<float> (&v)[N], float amax, uint32_t (&u)[8 * N]) {
  const float* x = reinterpret_cast<const float*>(v);
  uint32_t byte;
  const float s = kv4_scale(amax, byte);
  if (!(s > 0.0f)) {
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) u[i] = kMagicBits + 8;
    return byte;
  }
  const float inv = __fdividef(1.0f, s), half = 0.5f * s, top = 7.0f * s;
  float off = amax > 7.4375f * s ? half : 0.0f;  // the largest scale and the smallest ones: some are clamped
#pragma unroll
  for (int i = 0; i < 8 * N; ++i) {
    const float r = fmaf(x[i], inv, kMagic);
    off = fmaxf(off, fabsf(fmaf(-__fadd_rn(r, -kMagic), s, x[i])));
    u[i] = __float_as_uint(r);
  }
  if (off >= half) {
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) {
      const float y = fminf(fmaxf(x[i], -top), top);
      const float r = fmaf(y, inv, kMagic), f = __fadd_rn(r, -kMagic);
      const float d = fmaf(-f, s, y);
      const bool over = fabsf(d) > half || (fabsf(d) == half && (__float_as_uint(r) & 1u));
      u[i] = __float_as_uint(over ? __fadd_rn(r, copysignf(1.0f, d)) : r);
    }
  }
  return byte;
}
// bf16: a value of eight bits over a scale of four is exactly half way between two codes (one value in a hundred is), or
// 2^-9 of itself away from there and more.  So both neighbours of a half are found, by factors 2^-20 below and above 1 / s, and
// the even one is taken; elsewhere they are the same.  The scale, to four bits, of a largest magnitude over 7 likewise.
template <int N>
__device__ __forceinline__ uint32_t quantise(const Eight<__nv_bfloat16> (&v)[N], float amax, uint32_t (&u)[8 * N]) {
  constexpr float kBelow = 0.99999904632568359375f, kAbove = 1.00000095367431640625f;  // 1 -+ 2^-20
  float s;
  uint32_t byte;
  if (amax > 5e-4f && amax < 1670.0f) {  // normal scales below the largest: 7 2^-14, 7 240
    const uint32_t a = (__float_as_uint(amax * (kBelow / 7.0f)) + 0x80000u) >> 20;
    const uint32_t b = (__float_as_uint(amax * (kAbove / 7.0f)) + 0x80000u) >> 20, t = a & 1u ? b : a;
    byte = t - (112u << 3);
    s = __uint_as_float(t << 20);
  } else {
    s = kv4_scale(amax, byte);
  }
  if (!(s > 0.0f)) {
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) u[i] = kMagicBits + 8;
    return byte;
  }
  float x[8 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i].get(*reinterpret_cast<float(*)[8]>(x + 8 * i));
  if (amax > 7.4375f * s) {  // the largest scale and the smallest ones: some are clamped
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) x[i] = fminf(fmaxf(x[i], -7.0f * s), 7.0f * s);
  }
  const float inv = __fdividef(1.0f, s), below = inv * kBelow, above = inv * kAbove;
#pragma unroll
  for (int i = 0; i < 8 * N; ++i) {
    const uint32_t a = __float_as_uint(fmaf(x[i], below, kMagic)), b = __float_as_uint(fmaf(x[i], above, kMagic));
    u[i] = a & 1u ? b : a;
  }
  return byte;
}

// Keys: lane (g, t) has tokens g and g + 8, dims 8 t .. 8 t + 7 of each group: two words of the page order, whole.
template <typename T, int D>
__device__ __forceinline__ void put_keys(uint8_t* page, int tile, const T* const (&row)[2], const bool (&is_new)[2], bool wide) {
  const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
  uint32_t scale[2][D / 32];
  const uint32_t keep = kv4_turn((is_new[0] ? 0u : 0x0f0f0f0fu) | (is_new[1] ? 0u : 0xf0f0f0f0u));
  Eight<T> x[D / 32][2][1];  // every load on its way
#pragma unroll
  for (int k = 0; k < D / 32; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (is_new[i]) {
        x[k][i][0].load(row[i] + 32 * k + 8 * t, wide);
      } else {
        x[k][i][0] = Eight<T>{};
      }
    }
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int kh = 0; kh < 2; ++kh) {
      uint32_t u[2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float m = largest(x[2 * j + kh][i]);
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
        scale[i][2 * j + kh] = quantise(x[2 * j + kh][i], m, u[i]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t nat = kFields;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i) nat += u[i][4 * p + e] * (1u << (16 * (e & 1) + 8 * (e >> 1) + 4 * i));
        w[2 * kh + p] = kv4_turn(nat);
      }
    }
    uint4* to = reinterpret_cast<uint4*>(page) + (tile * (D / 64) + j) * 32 + lane;
    if (keep) {
      const uint4 old = *to;
      w[0] = (w[0] & ~keep) | (old.x & keep), w[1] = (w[1] & ~keep) | (old.y & keep);
      w[2] = (w[2] & ~keep) | (old.z & keep), w[3] = (w[3] & ~keep) | (old.w & keep);
    }
    if (is_new[0] || is_new[1]) *to = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (t == 0) {
    uint8_t* to = page + Kv4Page<D>::KS + (tile * 8 + g) * (D / 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!is_new[i]) continue;
      if (D == 128) {
        *reinterpret_cast<uint32_t*>(to + 4 * i) = scale[i][0] | scale[i][1] << 8 | scale[i][D / 32 - 2] << 16 | scale[i][D / 32 - 1] << 24;
      } else {
        *reinterpret_cast<uint16_t*>(to + 2 * i) = (uint16_t)(scale[i][0] | scale[i][1] << 8);
      }
    }
  }
}

// Values: lane (j, t, i) has the tokens 2 t, 2 t + 1 and those plus 8, dims 16 (4 j + i) .. + 15: eight words of the page
// order, whole; neighbouring i make 16 bytes, those of a store instruction 64.
template <typename T, int D>
__device__ __forceinline__ void put_values(uint8_t* page, int tile, const T* const (&row)[4], const bool (&is_new)[4], bool wide) {
  const int lane = threadIdx.x & 31, i = lane & 3, t = lane >> 2 & 3, j = lane >> 4;
  const bool mine = j < D / 64;
  const int dt = 4 * j + i;
  Eight<T> x[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (mine && is_new[k]) {
      x[k][0].load(row[k] + 16 * dt, wide);
      x[k][1].load(row[k] + 16 * dt + 8, wide);
    } else {
      x[k][0] = x[k][1] = Eight<T>{};
    }
  }
  uint32_t nat[8], bytes[4], kept = 0;
#pragma unroll
  for (int g = 0; g < 8; ++g) nat[g] = kFields;
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // token 2 t + (k & 1) + 8 (k >> 1)
    float m = largest(x[k]);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    uint32_t u[16];
    bytes[k] = quantise(x[k], m, u);
    if (!is_new[k]) kept |= 0x0f0fu << (16 * (k & 1) + 4 * (k >> 1));
#pragma unroll
    for (int e = 0; e < 16; ++e) nat[e & 7] += u[e] * (1u << (16 * (k & 1) + 8 * (e >> 3) + 4 * (k >> 1)));
  }
  if (!mine || !(is_new[0] || is_new[1] || is_new[2] || is_new[3])) return;
  kept = kv4_turn(kept);
  uint32_t* to = reinterpret_cast<uint32_t*>(page + Kv4Page<D>::V) + ((tile * (D / 64) + j) * 32 + t) * 4 + i;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    uint32_t w = kv4_turn(nat[g]);
    if (kept) w = (w & ~kept) | (to[16 * g] & kept);
    to[16 * g] = w;
  }
  if (!(i & 1)) {
    uint8_t* sc = page + Kv4Page<D>::VS + ((tile * 4 + t) * (D / 32) + dt / 2) * 4;
    if (!kept) {
      *reinterpret_cast<uint32_t*>(sc) = bytes[0] | bytes[1] << 8 | bytes[2] << 16 | bytes[3] << 24;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (is_new[k]) sc[k] = (uint8_t)bytes[k];
    }
  }
}

// Tile `tile` (of sequence s, counted from its first token) of one head takes its new rows [L, end).
template <typename T, int D, bool WIDE>
__device__ __forceinline__ void append_tile(const w4a8_kv4_cache& c, const Source& src, bool val, int s, int h, int tile, int L,
                                            int end, int n, const int32_t* index) {
  const int lane = threadIdx.x & 31, p0 = tile * kTile;
  const int phys = kv4_phys(c, s, tile >> 2);
  if (phys < 0) return;
  uint8_t* page = kv4_page<D>(c, phys, h);
  const T* base = static_cast<const T*>(src.rows.data) + (int64_t)s * src.rows.seq + (int64_t)h * src.rows.head;
  auto row = [&](int pos, bool& is_new) {
    is_new = pos >= L && pos < end;
    const int j = is_new ? pos - L : 0;
    return base + (int64_t)(index && is_new ? index[(size_t)s * n + j] : j) * src.rows.row;
  };
  if (!val) {
    bool is_new[2];
    const T* r[2];
    for (int i = 0; i < 2; ++i) r[i] = row(p0 + (lane >> 2) + 8 * i, is_new[i]);
    put_keys<T, D>(page, tile & 3, r, is_new, WIDE || src.wide);
  } else {
    bool is_new[4];
    const T* r[4];
    for (int i = 0; i < 4; ++i) r[i] = row(p0 + 2 * (lane >> 2 & 3) + (i & 1) + 8 * (i >> 1), is_new[i]);
    put_values<T, D>(page, tile & 3, r, is_new, WIDE || src.wide);
  }
}

// Many rows: one CTA per (four tiles, head, sequence), a warp per tile of keys or values.  WIDE: rows are read 16 bytes
// at a time, known at compile time.  Bound by instructions, 19 a value (conversion, two roundings and a choice, packing), and
// by fetching them: 24600 bf16 rows of 8 heads of 128, keys and values, 40 us, 3.2 TB/s (a correction pass behind one rounding
// took 35 a value and 85 us).  fp32 rows, 95 registers: by latency, 16 warps an SM (57 us, 4.0 TB/s).
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kBigThreads) k_kv4_append(w4a8_kv4_cache c, Source k, Source v, int n_src, int n,
                                                            const int32_t* counts, const int32_t* index, int32_t* len_out,
                                                            bool store_len) {
  griddep_enter();
  const int h = blockIdx.y, s = blockIdx.z, warp = threadIdx.x >> 5;
  const int L = kv4_len(c, c.len, s);
  int end = append_end(c, counts, s, n, L);
  if (index && end >= 0 && !append_index_ok(c, index, s, n, n_src, end - L)) end = -1;
  if (store_len && blockIdx.x == 0 && h == 0 && threadIdx.x == 0) len_out[s] = end >= 0 ? end : c.len[s];
  if (end <= L) return;
  const int64_t tile = (int64_t)(L / kTile & ~3) + blockIdx.x * 4 + (warp & 3);  // a CTA's tiles are of one page
  if (tile < L / kTile || tile * kTile >= end) return;
  append_tile<T, D, WIDE>(c, warp >> 2 ? v : k, warp >> 2, s, h, (int)tile, L, end, n, index);
}
// A few rows (decode steps, accepted paths): one CTA per sequence takes all heads and then stores the length, so the call is one
// launch.  Bound by latency: length, table, rows and old words one after the other, for each round of the CTA's warps over its tiles.
template <typename T, int D>
__global__ void __launch_bounds__(kSmallThreads) k_kv4_append_few(w4a8_kv4_cache c, Source k, Source v, int n_src, int n,
                                                                  const int32_t* counts, const int32_t* index, int32_t* len_out) {
  griddep_enter();
  const int s = blockIdx.x;
  const int L = kv4_len(c, c.len, s);
  int end = append_end(c, counts, s, n, L);
  if (index && end >= 0 && !append_index_ok(c, index, s, n, n_src, end - L)) end = -1;
  const int tiles = end > L ? (end - 1) / kTile - L / kTile + 1 : 0;
  for (int x = threadIdx.x >> 5; x < tiles * 2 * c.n_kv_heads; x += kSmallThreads / 32) {
    const int h = (x >> 1) % c.n_kv_heads, tile = L / kTile + (x >> 1) / c.n_kv_heads;
    append_tile<T, D, false>(c, x & 1 ? v : k, x & 1, s, h, tile, L, end, n, index);
  }
  __syncthreads();  // every warp has read the old length
  if (threadIdx.x == 0 && (end >= 0 || len_out != c.len)) len_out[s] = end >= 0 ? end : c.len[s];
}

// Whether a call of up to 16 rows is k_kv4_append_few's: where a warp has one tile (one launch instead of two), or the heads of
// all sequences are so many that their CTAs would queue.  R rounds of a warp cost about 2 + 4 R us whatever the sequences,
// k_kv4_append and the lengths behind it 6 us and 1 for every 85 (fp32) to 150 (bf16) heads.  Measured (us, heads of 128, sequences
// x heads, few / many; caches of 50 to 300 tokens that advance):
//   fp32, 1 row:   1 x 8  6.5 / 6.1,  64 x 8  6.8 / 11.2,  16 x 16  10.5 / 7.3,  64 x 16  10.5 / 18.1,  1 x 32  17.5 / 6.3,  1 x 1024  477 / 17
//   fp32, 8 rows:  16 x 4  6.7 / 7.2,  1 x 8  10.7 / 6.7,  64 x 8  10.9 / 12.6,  64 x 16  18.2 / 19.2,  256 x 16  34 / 61
//   bf16, 8 rows:  16 x 4  7.0 / 7.8,  1 x 8  10.9 / 7.3,  64 x 8  11.3 / 11.2,  64 x 16  19.6 / 15.7,  256 x 16  37 / 45
inline bool append_few(const w4a8_kv4_cache& c, int n) {
  if (n > kTile) return false;
  const int tiles = 2 * c.n_kv_heads * (n > 1 ? 2 : 1), warps = kSmallThreads / 32, rounds = (tiles + warps - 1) / warps;
  return rounds == 1 || c.n_seqs * c.n_kv_heads >= 256 * rounds;
}

// The new lengths of an append that advances its own cache: behind the kernel whose CTAs all read the old ones.
__global__ void k_kv4_append_len(w4a8_kv4_cache c, int n_src, int n, const int32_t* counts, const int32_t* index) {
  griddep_enter();
  const int s = blockIdx.x;
  const int L = kv4_len(c, c.len, s);
  int end = append_end(c, counts, s, n, L);
  if (index && end >= 0 && !append_index_ok(c, index, s, n, n_src, end - L)) end = -1;
  __syncthreads();
  if (threadIdx.x == 0 && end >= 0) c.len[s] = end;
}

__global__ void k_kv4_reset(w4a8_kv4_cache c) {
  griddep_enter();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < (int64_t)c.n_seqs * c.max_pages) c.table[i] = i < c.n_pages ? (int)i : -1;  // no page for two sequences
  if (i < c.n_seqs) c.len[i] = 0;
  if (i == 0) *c.ctl = 0;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}
// The values of the 4-bit fields at bit `at` of two 16-bit halves, times s: neighbours lo, hi of a vector.  A field below the
// leading bit of 128 (bf16) or 16 (fp32) is a number; c s and, in fp32, 24 s are exact.
__device__ __forceinline__ void put_pair(Eight<__nv_bfloat16>& x, int pair, uint32_t w, int at, float s) {
  uint32_t v = and_or(w >> at, 0x000f000fu, 0x43004300u);
  const __nv_bfloat162 c = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), __float2bfloat162_rn(136.0f));
  reinterpret_cast<__nv_bfloat162*>(x.u)[pair] = __hmul2(c, __float2bfloat162_rn(s));
}
__device__ __forceinline__ void put_pair(Eight<float>& x, int pair, uint32_t w, int at, float s) {
  const uint32_t a = at <= 19 ? w << (19 - at) : w >> (at - 19), b = at + 16 <= 19 ? w << (3 - at) : w >> (at - 3 < 0 ? 0 : at - 3);
  float* f = reinterpret_cast<float*>(x.u) + 2 * pair;
  f[0] = fmaf(__uint_as_float(and_or(a, 0x00780000u, 0x41800000u)), s, -24.0f * s);
  f[1] = fmaf(__uint_as_float(and_or(b, 0x00780000u, 0x41800000u)), s, -24.0f * s);
}

// One CTA per (four tiles, head, sequence), a warp per tile of keys or values, in the lanes of the append.
// Bound by the writes: 32768 bf16 rows of 8 heads of 128, keys and values, 30 us, 5.4 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_kv4_read(w4a8_kv4_cache c, const int32_t* first, const int32_t* len, int n,
                                                  T* __restrict__ k_out, T* __restrict__ v_out) {
  griddep_enter();
  const int h = blockIdx.y, s = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = c.n_kv_heads;
  const bool val = warp >> 2;
  const int F = first[s];
  int L = kv4_len(c, len, s);
  if (F < 0) {
    if (threadIdx.x == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    L = 0;
  }
  const int64_t f = F < 0 ? 0 : F, stop = f + n;
  const int64_t tile = f / kPage * 4 + blockIdx.x * 4 + (warp & 3), p0 = tile * kTile;
  if (p0 + kTile <= f || p0 >= stop) return;
  int phys = -1;
  if (p0 < L) phys = kv4_phys(c, s, (int)(tile >> 2));
  T* out = (val ? v_out : k_out) + ((size_t)s * n * H + h) * D;
  auto put = [&](int64_t pos, int d, const Eight<T>& x) {
    if (pos < f || pos >= stop) return;
    const Eight<T> zero{};
    (phys >= 0 && pos < L ? x : zero).store(out + (size_t)(pos - f) * H * D + d, true);
  };
  const uint8_t* page = kv4_page<D>(c, phys < 0 ? 0 : phys, h);
  const int tl = (int)(tile & 3);
  if (!val) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* sc = page + Kv4Page<D>::KS + (tl * 8 + g) * (D / 16);
    uint4 w[D / 64];
    uint32_t b[2][D / 32];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) w[j] = reinterpret_cast<const uint4*>(page)[(tl * (D / 64) + j) * 32 + lane];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < D / 32; ++k) b[i][k] = sc[i * (D / 32) + k];
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        const uint32_t n0 = kv4_unturn(kh ? w[j].z : w[j].x), n1 = kv4_unturn(kh ? w[j].w : w[j].y);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float s0 = scale_value(b[i][2 * j + kh]);
          Eight<T> x;
#pragma unroll
          for (int e = 0; e < 4; ++e) put_pair(x, e, e < 2 ? n0 : n1, 8 * (e & 1) + 4 * i, s0);
          put(p0 + g + 8 * i, 32 * (2 * j + kh) + 8 * t, x);
        }
      }
  } else {
    const int i = lane & 3, t = lane >> 2 & 3, j = lane >> 4, dt = 4 * j + i;
    if (j >= D / 64) return;
    const uint32_t* from = reinterpret_cast<const uint32_t*>(page + Kv4Page<D>::V) + ((tl * (D / 64) + j) * 32 + t) * 4 + i;
    const uint32_t sc = *reinterpret_cast<const uint32_t*>(page + Kv4Page<D>::VS + ((tl * 4 + t) * (D / 32) + dt / 2) * 4);
    uint32_t w[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) w[g] = from[16 * g];
#pragma unroll
    for (int g = 0; g < 8; ++g) w[g] = kv4_unturn(w[g]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float s0 = scale_value(sc >> (8 * k) & 255u);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        Eight<T> x;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          put_pair(x, g, __byte_perm(w[2 * g], w[2 * g + 1], k & 1 ? 0x7632 : 0x5410), 8 * q + 4 * (k >> 1), s0);
        put(p0 + 2 * t + (k & 1) + 8 * (k >> 1), 16 * dt + 8 * q, x);
      }
    }
  }
}

}  // namespace

W4A8_API w4a8_status w4a8_kv4_bytes(const w4a8_kv4_cache* c, size_t bytes[4]) {
  const w4a8_status st = kv4_dims(c);
  if (st != W4A8_OK) return st;
  if (!bytes) return W4A8_ERR_ARG;
  bytes[0] = kv4_pool_bytes(*c);
  bytes[1] = (size_t)c->n_seqs * c->max_pages * 4;
  bytes[2] = (size_t)c->n_seqs * 4;
  bytes[3] = 4;
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv4_reset(const w4a8_kv4_cache* c, void* stream) {
  const w4a8_status st = kv4_valid(c);
  if (st != W4A8_OK) return st;
  const int64_t total = (int64_t)c->n_seqs * c->max_pages;  // >= n_seqs
  W4A8_CUDA_TRY(launch_pdl(k_kv4_reset, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, as_stream(stream), *c));
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv4_check(const w4a8_kv4_cache* c, uint32_t* flags) {
  const w4a8_status st = kv4_valid(c);
  if (st != W4A8_OK) return st;
  if (!flags) return W4A8_ERR_ARG;
  W4A8_CUDA_TRY(cudaMemcpy(flags, c->ctl, 4, cudaMemcpyDeviceToHost));
  return *flags ? W4A8_ERR_DEVICE_FLAG : W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv4_append(const w4a8_kv4_cache* c, const w4a8_rows* k, const w4a8_rows* v, int dtype,
                                     int n_src, int n, const int32_t* counts, const int32_t* index, int32_t* len_out,
                                     void* stream) {
  const w4a8_status ok = kv4_valid(c);
  if (ok != W4A8_OK) return ok;
  if (!k || !v || !k->data || !v->data || !len_out || !kv8_dtype(dtype) || n < 1 || n_src < 1) return W4A8_ERR_ARG;
  if (index ? n > kMaxIndexed : n_src < n) return W4A8_ERR_SHAPE;
  if (!aligned(k->data, kv8_elem(dtype)) || !aligned(v->data, kv8_elem(dtype)) || !aligned(counts, 4) ||
      !aligned(index, 4) || !aligned(len_out, 4))
    return W4A8_ERR_ARG;
  // new lengths on what the call writes, or other CTAs of it still read (they may take the place of the old ones); rows on what it writes
  const size_t S4 = 4 * (size_t)c->n_seqs, pool = kv4_pool_bytes(*c);
  auto on = [&](const void* p, size_t bytes) { return bytes_meet(p, bytes, len_out, S4); };
  auto written = [&](const w4a8_rows& r) {
    const size_t el = kv8_elem(dtype);
    return rows_touch(r, c->n_kv_heads, c->n_seqs, n_src, c->head_dim, el, len_out, S4) ||
           rows_touch(r, c->n_kv_heads, c->n_seqs, n_src, c->head_dim, el, c->pages, pool);
  };
  if (on(counts, S4) || on(index, S4 * n) || on(c->table, S4 * c->max_pages) || on(c->ctl, 4) || on(c->pages, pool) ||
      (len_out != c->len && on(c->len, S4)) || written(*k) || written(*v))
    return W4A8_ERR_ARG;
  if (n > kPage * c->max_pages) return W4A8_ERR_CAPACITY;
  cudaStream_t st = as_stream(stream);
  const bool own = len_out == c->len, f32 = dtype == W4A8_F32, d64 = c->head_dim == 64;
  const Source ks{*k, kv8_vec_rows(*k, dtype)}, vs{*v, kv8_vec_rows(*v, dtype)};
  if (append_few(*c, n)) {
    auto run = [&](auto kern) {
      return launch_pdl(kern, dim3((unsigned)c->n_seqs), dim3(kSmallThreads), 0, st, *c, ks, vs, n_src, n, counts, index, len_out);
    };
    W4A8_CUDA_TRY(f32 ? (d64 ? run(k_kv4_append_few<float, 64>) : run(k_kv4_append_few<float, 128>))
                      : (d64 ? run(k_kv4_append_few<__nv_bfloat16, 64>) : run(k_kv4_append_few<__nv_bfloat16, 128>)));
    return W4A8_OK;
  }
  const dim3 grid((unsigned)((n + kPage - 1 + kPage - 1) / kPage), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs);
  auto run = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(kBigThreads), 0, st, *c, ks, vs, n_src, n, counts, index, len_out, !own);
  };
  auto typed = [&](auto t, auto all) {
    using T = decltype(t);
    constexpr bool WIDE = decltype(all)::value;
    return d64 ? run(k_kv4_append<T, 64, WIDE>) : run(k_kv4_append<T, 128, WIDE>);
  };
  const std::true_type yes{};
  const std::false_type no{};
  const bool all = ks.wide && vs.wide;
  if (f32) W4A8_CUDA_TRY(all ? typed(float{}, yes) : typed(float{}, no));
  else W4A8_CUDA_TRY(all ? typed(__nv_bfloat16{}, yes) : typed(__nv_bfloat16{}, no));
  if (own)
    W4A8_CUDA_TRY(launch_pdl(k_kv4_append_len, dim3((unsigned)c->n_seqs), dim3(index ? 128 : 32), 0, st, *c, n_src, n,
                             counts, index));
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv4_read(const w4a8_kv4_cache* c, const int32_t* first, const int32_t* len, int n, int dtype,
                                   void* k_out, void* v_out, void* stream) {
  const w4a8_status ok = kv4_valid(c);
  if (ok != W4A8_OK) return ok;
  if (!first || !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(first, 4) || !aligned(len, 4) ||
      n < 1 || !kv8_dtype(dtype))
    return W4A8_ERR_ARG;
  if (n > kPage * c->max_pages) return W4A8_ERR_CAPACITY;
  const size_t S4 = 4 * (size_t)c->n_seqs, bytes = (size_t)c->n_seqs * n * c->n_kv_heads * c->head_dim * kv8_elem(dtype);
  for (const void* out : {k_out, v_out})  // on one another, or on what other CTAs still read
    if (bytes_meet(out, bytes, c->pages, kv4_pool_bytes(*c)) || bytes_meet(out, bytes, c->table, S4 * c->max_pages) ||
        bytes_meet(out, bytes, c->len, S4) || bytes_meet(out, bytes, c->ctl, 4) || bytes_meet(out, bytes, first, S4) ||
        bytes_meet(out, bytes, len, S4) || bytes_meet(k_out, bytes, v_out, bytes))
      return W4A8_ERR_ARG;
  const dim3 grid((unsigned)((n + kPage - 1 + kPage - 1) / kPage), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs);
  const int32_t* L = len ? len : c->len;
  cudaStream_t st = as_stream(stream);
  auto run = [&](auto kern, auto* k, auto* v) {
    return launch_pdl(kern, grid, dim3(256), 0, st, *c, first, L, n, k, v);
  };
  const bool d64 = c->head_dim == 64;
  if (dtype == W4A8_F32) {
    float *k = static_cast<float*>(k_out), *v = static_cast<float*>(v_out);
    W4A8_CUDA_TRY(d64 ? run(k_kv4_read<float, 64>, k, v) : run(k_kv4_read<float, 128>, k, v));
  } else {
    __nv_bfloat16 *k = static_cast<__nv_bfloat16*>(k_out), *v = static_cast<__nv_bfloat16*>(v_out);
    W4A8_CUDA_TRY(d64 ? run(k_kv4_read<__nv_bfloat16, 64>, k, v) : run(k_kv4_read<__nv_bfloat16, 128>, k, v));
  }
  return W4A8_OK;
}
