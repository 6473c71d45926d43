// Writing, reading and thinning the 8-bit key/value cache.
//
// append: a page is quantised once, when its last row arrives: absmax over its 64 * D values, one
// IEEE division for the scale, one per value, round half even (the rule of w4a8_quantize_rows).
// The rows of the open page wait in the fp32 tail.
#include "kv8.cuh"

using namespace w4a8;

namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxIndexed = 1024;  // rows of an append that takes its source rows from a list

// New length of a sequence, or -1 where the call leaves it as it was.
__device__ int append_end(const w4a8_kv8_cache& c, const int32_t* counts, int s, int n, int L) {
  const int cnt = kv8_count(c, counts, s, n);
  if (L < 0 || cnt < 0) return -1;
  if (L + (int64_t)cnt > (int64_t)kPage * c.max_pages + kPage - 1) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    return -1;
  }
  return L + cnt;
}
// Whether every source row of the sequence's list is in range.
__device__ bool append_index_ok(const w4a8_kv8_cache& c, const int32_t* index, int s, int n, int n_src, int cnt) {
  bool ok = true;
  for (int j = threadIdx.x; j < cnt; j += blockDim.x) {
    const int r = index[(size_t)s * n + j];
    ok = ok && r >= 0 && r < n_src;
  }
  ok = __syncthreads_and(ok);
  if (!ok && threadIdx.x == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TOKEN);
  return ok;
}

// Codes + 128 of eight values at scale s > 0 (|x| <= 127 s up to rounding), four to a word: rint of the IEEE quotient,
// mostly without the division.  x fl(1 / s) is within 1.2e-5 of fl(x / s) (127 2^-24 of the reciprocal's rounding, half of
// that of the quotient's), so only one that close to a half needs it; added to 1.5 2^23 in one rounding it becomes a whole
// number in the low bits.  inv is 0 where 1 / s is not a good factor (subnormal s).
__device__ __forceinline__ void codes8(const float (&x)[8], float s, float inv, uint32_t (&word)[2]) {
  uint32_t n[8];
  float off = inv == 0.0f ? 1.0f : 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float r = fmaf(x[e], inv, 12582912.0f);
    off = fmaxf(off, fabsf(fmaf(x[e], inv, -__fadd_rn(r, -12582912.0f))));
    n[e] = __float_as_uint(r);
  }
  if (off > 0.5f - 6e-5f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = (uint32_t)kv8_code(x[e], s);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    word[i] = __byte_perm(__byte_perm(n[4 * i], n[4 * i + 1], 0x0040), __byte_perm(n[4 * i + 2], n[4 * i + 3], 0x0040), 0x5410) ^
              0x80808080u;
}

constexpr int kVPad = 4;  // bytes between the token rows of a page's value codes in shared memory

// One CTA per (page of the call's window, KV head, sequence and keys/values).  A thread takes eight neighbouring
// dims of four (D = 128) rows, 16 or 32 bytes at a time where the rows allow it.  A page of whole new rows is read once,
// all loads in flight, and held in registers between the absmax and the quantisation; other pages (rows of the
// tail, of a list, unaligned) are read twice.  Key groups of 16 bytes are whole in a thread; value groups (eight tokens of
// two dims) are gathered from the codes in shared memory.  The CTA of the window's first page reads the old tail, so
// it alone writes the new one, afterwards.
// Bound by instructions (20 a value: absmax, rounding, packing, sums; 69% of the issue slots) and by the loads in flight:
// 32768 bf16 rows of 8 heads of 128, 134 MB in and 67 MB out, 58 us cold (3.5 TB/s) with six CTAs on an SM, 63 with four.
// Four pages a CTA with the next one's loads in flight (120 registers): 10 us more.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 ? 6 : 5) k_kv8_append(w4a8_kv8_cache c, w4a8_rows kr, w4a8_rows vr, int n_src,
                                                                int n, const int32_t* counts, const int32_t* index,
                                                                int32_t* len_out, bool store_len, int vec) {
  griddep_enter();
  constexpr int kChunks = kPage * D / 8 / kAppendThreads;
  __shared__ float red[kAppendThreads / 32];
  __shared__ uint32_t ksum[D / 2];  // sums of code + 128 of dims 4 i + j and 4 i + j + 2 in entry 2 i + j
  __shared__ __align__(16) uint8_t vs[kPage * (D + kVPad)];
  const int w = blockIdx.x, h = blockIdx.y, s = blockIdx.z >> 1;
  const bool val = blockIdx.z & 1;
  const int tid = threadIdx.x;
  const int L = kv8_len(c, c.len, s);
  int end = append_end(c, counts, s, n, L);
  if (index && end >= 0 && !append_index_ok(c, index, s, n, n_src, end - L)) end = -1;
  if (store_len && w == 0 && h == 0 && !val && tid == 0) len_out[s] = end >= 0 ? end : c.len[s];
  if (end < 0 || end == L) return;
  const w4a8_rows rows = val ? vr : kr;
  const bool wide = vec >> val & 1;
  const T* src = static_cast<const T*>(rows.data) + (int64_t)s * rows.seq + (int64_t)h * rows.head;
  const size_t pair = kv8_pair(c, s, h);
  float* tail = c.tail + (pair * 2 + val) * kPage * D;
  const int page = L / kPage + w, base = page * kPage;
  auto row_of = [&](int pos) -> const T* {  // source of a position at or behind L
    const int j = pos - L;
    return src + (int64_t)(index ? index[(size_t)s * n + j] : j) * rows.row;
  };
  // dims d .. d + 7 (d % 8 == 0) of a position
  auto load8 = [&](int pos, int d, float (&x)[8]) {
    if (pos < L) {
      const float4* p = reinterpret_cast<const float4*>(tail + (pos - base) * D + d);
      const float4 a = p[0], b = p[1];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
      return;
    }
    const T* p = row_of(pos) + d;
    if (wide) {
      uint4 u[sizeof(T) / 2];
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
      const T* e = reinterpret_cast<const T*>(u);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = kv8_load(e + i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = kv8_load(p + i);
    }
  };
  if (base + kPage <= end) {
    const int phys = kv8_phys(c, pair, page);
    // chunk i of a thread, keys: group gi = (i / 2) threads + tid of the page's order, its token g + 8 (i & 1);
    // values: the i-th of the page's eight-dim chunks in rows
    auto place = [&](int i, int& tok, int& d) {
      if (!val) {
        const int gi = (i >> 1) * kAppendThreads + tid, q = gi >> 5;
        tok = q / (D / 32) * 16 + (i & 1) * 8 + ((gi >> 2) & 7);
        d = q % (D / 32) * 32 + (gi & 3) * 8;
      } else {
        const int ci = i * kAppendThreads + tid;
        tok = ci / (D / 8), d = ci % (D / 8) * 8;
      }
    };
    const bool whole = wide && !index && base >= L;  // a page of whole new rows: the loads alone, all in flight
    uint4 u[kChunks][sizeof(T) / 2];
    float m = 0.0f;
    auto held = [&](int i, float (&y)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = kv8_load(reinterpret_cast<const T*>(u[i]) + e);
    };
    auto again = [&](int i, float (&y)[8]) {
      int tok, d;
      place(i, tok, d);
      load8(base + tok, d, y);
    };
    auto largest = [&](const float (&y)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(y[e]));
    };
    if (whole) {
      const T* from = src + (int64_t)(base - L) * rows.row;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        int tok, d;
        place(i, tok, d);
        const uint4* p = reinterpret_cast<const uint4*>(from + tok * rows.row + d);
#pragma unroll
        for (int y = 0; y < (int)sizeof(T) / 2; ++y) u[i][y] = __ldg(p + y);
      }
      if constexpr (sizeof(T) == 2) {  // of pairs
        __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __hmax2_nan(top, __habs2(reinterpret_cast<const __nv_bfloat162*>(u[i])[e]));
        m = max_nan(__low2float(top), __high2float(top));
      } else {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          float y[8];
          held(i, y);
          largest(y);
        }
      }
    } else {
#pragma unroll 2
      for (int i = 0; i < kChunks; ++i) {
        float y[8];
        again(i, y);
        largest(y);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    for (int d = tid; d < D / 2; d += kAppendThreads) ksum[d] = 0;
    __syncthreads();
    float amax = red[0];
#pragma unroll
    for (int i = 1; i < kAppendThreads / 32; ++i) amax = max_nan(amax, red[i]);
    const float sc = kv8_scale(amax);
    const float inv = sc > 1e-37f ? __fdiv_rn(1.0f, sc) : 0.0f;
    uint32_t word[kChunks][2];  // code + 128 of four dims each
#pragma unroll
    for (int i = 0; i < kChunks; ++i) word[i][0] = word[i][1] = 0x80808080u;
    if (sc > 0.0f && whole) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        float y[8];
        held(i, y);
        codes8(y, sc, inv, word[i]);
      }
    } else if (sc > 0.0f) {
#pragma unroll 1
      for (int i = 0; i < kChunks; ++i) {
        float y[8];
        uint32_t w[2];
        again(i, y);
        codes8(y, sc, inv, w);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) word[k][0] = k == i ? w[0] : word[k][0], word[k][1] = k == i ? w[1] : word[k][1];
      }
    }
    const size_t pg = kv8_page(c, pair, phys < 0 ? 0 : phys);
    uint4* out = reinterpret_cast<uint4*>(c.codes + (pg * 2 + val) * (size_t)(kPage * D));
    if (!val) {
      uint32_t sum[4] = {};  // dims e, e + 2 of a half of the thread's eight: sums of code + 128 in 16 bits each
#pragma unroll
      for (int i = 0; i < kChunks; i += 2) {
        if (phys >= 0) out[(i >> 1) * kAppendThreads + tid] = make_uint4(word[i][0], word[i + 1][0], word[i][1], word[i + 1][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int sh = 8 * (e & 1), half = e >> 1;
          sum[e] += (word[i][half] >> sh & 0x00ff00ffu) + (word[i + 1][half] >> sh & 0x00ff00ffu);
        }
      }
      // a thread's chunks are of the same dims: its groups are 8 (a multiple of D / 32) dim blocks apart
      const int t = tid & 3, kp = (tid >> 5) % (D / 32);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t v = sum[e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        // at most 64 * 255 in a half: no carry; integers: any order
        if (((tid >> 2) & 7) == 0) atomicAdd(&ksum[((kp * 4 + t) * 2 + (e >> 1)) * 2 + (e & 1)], v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int ci = i * kAppendThreads + tid;
        uint32_t* p = reinterpret_cast<uint32_t*>(vs + ci / (D / 8) * (D + kVPad) + ci % (D / 8) * 8);
        p[0] = word[i][0], p[1] = word[i][1];
      }
    }
    __syncthreads();
    if (phys >= 0) {
      if (tid == 0) c.scales[pg * 2 + val] = sc;
      if (!val) {
        for (int d = tid; d < D; d += kAppendThreads)
          c.sums[pg * D + d] = (int16_t)((int)(ksum[(d >> 2) * 2 + (d & 1)] >> (8 * (d & 2)) & 0xffffu) - 128 * kPage);
      } else {
        // a thread gathers four groups of one (tile, chunk, t): dims g .. g + 3 and + 8 of eight tokens, as words of
        // four dims that change places with four tokens
        for (int x = tid; x < kPage * D / 64; x += kAppendThreads) {
          const int t = x & 3, g4 = (x >> 2) & 1, q = x >> 3;
          const uint8_t* from = vs + ((q & 1) * 32 + t * 2) * (D + kVPad) + (q >> 1) * 16 + g4 * 4;
          uint32_t u[4][4];  // group, word: (ks, dim half): tokens + 16 ks + {0, 1, 8, 9}
#pragma unroll
          for (int wd = 0; wd < 4; ++wd) {
            uint32_t v[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
              v[b] = *reinterpret_cast<const uint32_t*>(from + ((wd >> 1) * 16 + (b >> 1) * 8 + (b & 1)) * (D + kVPad) + (wd & 1) * 8);
            const uint32_t a0 = __byte_perm(v[0], v[1], 0x5140), a1 = __byte_perm(v[2], v[3], 0x5140);
            const uint32_t b0 = __byte_perm(v[0], v[1], 0x7362), b1 = __byte_perm(v[2], v[3], 0x7362);
            u[0][wd] = __byte_perm(a0, a1, 0x5410), u[1][wd] = __byte_perm(a0, a1, 0x7632);
            u[2][wd] = __byte_perm(b0, b1, 0x5410), u[3][wd] = __byte_perm(b0, b1, 0x7632);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) out[(q * 8 + g4 * 4 + i) * 4 + t] = make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]);
        }
      }
    }
  }
  if (w == 0) {
    __syncthreads();  // the old tail has been read
    const int from = max(L, end / kPage * kPage);
    for (int i = tid; i < (end - from) * D; i += kAppendThreads) {
      const int pos = from + i / D, d = i % D;
      tail[(pos & (kPage - 1)) * D + d] = kv8_load(row_of(pos) + d);
    }
  }
}

// The new lengths of an append that advances its own cache: behind the kernel whose CTAs all read the old ones.
__global__ void k_kv8_append_len(w4a8_kv8_cache c, int n_src, int n, const int32_t* counts, const int32_t* index) {
  griddep_enter();
  const int s = blockIdx.x;
  const int L = kv8_len(c, c.len, s);
  int end = append_end(c, counts, s, n, L);
  if (index && end >= 0 && !append_index_ok(c, index, s, n, n_src, end - L)) end = -1;
  __syncthreads();
  if (threadIdx.x == 0 && end >= 0) c.len[s] = end;
}

__global__ void k_kv8_reset(w4a8_kv8_cache c) {
  griddep_enter();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t total = (int64_t)c.n_seqs * c.n_kv_heads * c.max_pages;
  if (i < total) c.table[i] = (int)(i % c.max_pages);
  if (i < c.n_seqs) c.len[i] = 0;
  if (i == 0) *c.ctl = 0;
}

// One CTA per (page of the window, KV head, sequence and keys/values): each value s * c with one rounding; positions
// of the open page come from the tail.  A thread writes eight neighbouring dims of a position, 32 bytes; the codes of
// value groups (eight tokens of two dims) change places in shared memory.  Bound by the writes: 32768 positions of
// 8 heads of 128, 67 MB in and 268 MB out, 61 us cold (5.5 TB/s).
template <int D>
__global__ void __launch_bounds__(256) k_kv8_read(w4a8_kv8_cache c, const int32_t* first, const int32_t* len, int n,
                                                   float* __restrict__ k_out, float* __restrict__ v_out) {
  griddep_enter();
  __shared__ __align__(16) uint8_t vs[kPage * (D + kVPad)];
  const int h = blockIdx.y, s = blockIdx.z >> 1, tid = threadIdx.x;
  const bool val = blockIdx.z & 1;
  const int F = first[s];
  int L = kv8_len(c, len, s);
  if (F < 0) {
    if (tid == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    L = 0;
  }
  if (L < 0) L = 0;
  const int64_t f = F < 0 ? 0 : F;
  const int64_t page = f / kPage + blockIdx.x, base = page * kPage;
  if (base >= f + n) return;
  const size_t pair = kv8_pair(c, s, h);
  float* out = (val ? v_out : k_out) + ((size_t)s * n * c.n_kv_heads + h) * D;
  auto put8 = [&](int tok, int d, const float (&x)[8]) {
    const int64_t j = base + tok - f;
    if (j < 0 || j >= n) return;
    float4* p = reinterpret_cast<float4*>(out + (size_t)j * c.n_kv_heads * D + d);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  };
  if (base + kPage > L) {
    const float* tail = c.tail + (pair * 2 + val) * kPage * D;
    for (int ci = tid; ci < kPage * D / 8; ci += 256) {
      const int tok = ci / (D / 8), d = ci % (D / 8) * 8;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = base + tok < L ? tail[tok * D + d + e] : 0.0f;
      put8(tok, d, x);
    }
    return;
  }
  const int phys = kv8_phys(c, pair, (int)page);
  const size_t pg = kv8_page(c, pair, phys < 0 ? 0 : phys);
  const float sc = phys < 0 ? 0.0f : c.scales[pg * 2 + val];
  const uint4* in = reinterpret_cast<const uint4*>(c.codes + (pg * 2 + val) * (size_t)(kPage * D));
  auto value = [&](uint32_t w, int e) { return sc * (float)((int)(w >> (8 * e) & 255u) - 128); };
#pragma unroll
  for (int i = 0; i < kPage * D / 16 / 256; ++i) {
    const int gi = i * 256 + tid, t = gi & 3, g = (gi >> 2) & 7, q = gi >> 5;
    const uint4 u = __ldg(in + gi);
    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
    if (!val) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = value(word[(e >> 2) * 2 + r], e & 3);
        put8(q / (D / 32) * 16 + r * 8 + g, q % (D / 32) * 32 + t * 8, x);
      }
    } else {
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        const int tok = (q & 1) * 32 + (b >> 3) * 16 + ((b >> 1) & 1) * 8 + t * 2 + (b & 1);
        vs[tok * (D + kVPad) + (q >> 1) * 16 + ((b >> 2) & 1) * 8 + g] = (uint8_t)(word[b >> 2] >> (8 * (b & 3)));
      }
    }
  }
  if (!val) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPage * D / 8 / 256; ++i) {
    const int ci = i * 256 + tid, tok = ci / (D / 8), d = ci % (D / 8) * 8;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(vs + tok * (D + kVPad) + d);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = value(p[e >> 2], e & 3);
    put8(tok, d, x);
  }
}

}  // namespace

W4A8_API w4a8_status w4a8_kv8_bytes(const w4a8_kv8_cache* c, size_t bytes[7]) {
  const w4a8_status st = kv8_dims(c);
  if (st != W4A8_OK) return st;
  if (!bytes) return W4A8_ERR_ARG;
  const size_t pairs = (size_t)c->n_seqs * c->n_kv_heads, pages = pairs * c->max_pages, D = (size_t)c->head_dim;
  bytes[0] = pages * 2 * kPage * D;
  bytes[1] = pages * 2 * 4;
  bytes[2] = pages * D * 2;
  bytes[3] = pairs * 2 * kPage * D * 4;
  bytes[4] = pages * 4;
  bytes[5] = (size_t)c->n_seqs * 4;
  bytes[6] = 4;
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_reset(const w4a8_kv8_cache* c, void* stream) {
  const w4a8_status st = kv8_valid(c);
  if (st != W4A8_OK) return st;
  const int64_t total = (int64_t)c->n_seqs * c->n_kv_heads * c->max_pages;  // >= n_seqs
  W4A8_CUDA_TRY(launch_pdl(k_kv8_reset, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, as_stream(stream), *c));
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_check(const w4a8_kv8_cache* c, uint32_t* flags) {
  const w4a8_status st = kv8_valid(c);
  if (st != W4A8_OK) return st;
  if (!flags) return W4A8_ERR_ARG;
  W4A8_CUDA_TRY(cudaMemcpy(flags, c->ctl, 4, cudaMemcpyDeviceToHost));
  return *flags ? W4A8_ERR_DEVICE_FLAG : W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_append(const w4a8_kv8_cache* c, const w4a8_rows* k, const w4a8_rows* v, int dtype,
                                     int n_src, int n, const int32_t* counts, const int32_t* index, int32_t* len_out,
                                     void* stream) {
  const w4a8_status ok = kv8_valid(c);
  if (ok != W4A8_OK) return ok;
  if (!k || !v || !k->data || !v->data || !len_out || !kv8_dtype(dtype) || n < 1 || n_src < 1) return W4A8_ERR_ARG;
  if (index ? n > kMaxIndexed : n_src < n) return W4A8_ERR_SHAPE;
  if (!aligned(k->data, kv8_elem(dtype)) || !aligned(v->data, kv8_elem(dtype)) || !aligned(counts, 4) ||
      !aligned(index, 4) || !aligned(len_out, 4))
    return W4A8_ERR_ARG;
  if (n > kPage * c->max_pages + kPage - 1) return W4A8_ERR_CAPACITY;
  cudaStream_t st = as_stream(stream);
  const dim3 grid((unsigned)((n + kPage - 1 + kPage - 1) / kPage), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs * 2);
  const bool own = len_out == c->len;
  const int vec = (kv8_vec_rows(*k, dtype) ? 1 : 0) | (kv8_vec_rows(*v, dtype) ? 2 : 0);
  auto run = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(kAppendThreads), 0, st, *c, *k, *v, n_src, n, counts, index, len_out, !own, vec);
  };
  if (dtype == W4A8_F32)
    W4A8_CUDA_TRY(c->head_dim == 64 ? run(k_kv8_append<float, 64>) : run(k_kv8_append<float, 128>));
  else
    W4A8_CUDA_TRY(c->head_dim == 64 ? run(k_kv8_append<__nv_bfloat16, 64>) : run(k_kv8_append<__nv_bfloat16, 128>));
  if (own)
    W4A8_CUDA_TRY(launch_pdl(k_kv8_append_len, dim3((unsigned)c->n_seqs), dim3(index ? 128 : 32), 0, st, *c, n_src, n,
                             counts, index));
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_read(const w4a8_kv8_cache* c, const int32_t* first, const int32_t* len, int n,
                                   float* k_out, float* v_out, void* stream) {
  const w4a8_status ok = kv8_valid(c);
  if (ok != W4A8_OK) return ok;
  if (!first || !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(first, 4) || !aligned(len, 4) || n < 1)
    return W4A8_ERR_ARG;
  if (n > kPage * c->max_pages + kPage - 1) return W4A8_ERR_CAPACITY;
  const dim3 grid((unsigned)((n + kPage - 1 + kPage - 1) / kPage), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs * 2);
  const int32_t* L = len ? len : c->len;
  cudaStream_t st = as_stream(stream);
  W4A8_CUDA_TRY(c->head_dim == 64
                    ? launch_pdl(k_kv8_read<64>, grid, dim3(256), 0, st, *c, first, L, n, k_out, v_out)
                    : launch_pdl(k_kv8_read<128>, grid, dim3(256), 0, st, *c, first, L, n, k_out, v_out));
  return W4A8_OK;
}
