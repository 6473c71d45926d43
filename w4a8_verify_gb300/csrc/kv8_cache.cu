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

// One CTA per (page of the call's window, KV head, sequence and keys/values).  A thread owns the
// 16-byte groups of the page's byte order, so the codes leave in 16-byte stores; the values of a
// group sit in registers between the absmax and the quantisation (one read of the rows).  The CTA of the
// window's first page reads the old tail, so it alone writes the new one, afterwards.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) k_kv8_append(w4a8_kv8_cache c, w4a8_rows kr, w4a8_rows vr, int n_src,
                                                                int n, const int32_t* counts, const int32_t* index,
                                                                int32_t* len_out, bool store_len) {
  griddep_enter();
  __shared__ float red[kAppendThreads / 32];
  __shared__ int ksum[D];
  const int w = blockIdx.x, h = blockIdx.y, s = blockIdx.z >> 1;
  const bool val = blockIdx.z & 1;
  const int tid = threadIdx.x;
  const int L = kv8_len(c, c.len, s);
  int end = append_end(c, counts, s, n, L);
  if (index && end >= 0 && !append_index_ok(c, index, s, n, n_src, end - L)) end = -1;
  if (store_len && w == 0 && h == 0 && !val && tid == 0) len_out[s] = end >= 0 ? end : c.len[s];
  if (end < 0 || end == L) return;
  const w4a8_rows rows = val ? vr : kr;
  const T* src = static_cast<const T*>(rows.data) + (int64_t)s * rows.seq + (int64_t)h * rows.head;
  const size_t pair = kv8_pair(c, s, h);
  float* tail = c.tail + (pair * 2 + val) * kPage * D;
  const int page = L / kPage + w, base = page * kPage;
  auto row_of = [&](int pos) -> const T* {  // source of a position at or behind L
    const int j = pos - L;
    return src + (int64_t)(index ? index[(size_t)s * n + j] : j) * rows.row;
  };
  auto value = [&](int tok, int d) -> float {
    const int pos = base + tok;
    return pos < L ? tail[tok * D + d] : kv8_load(row_of(pos) + d);
  };
  if (base + kPage <= end) {
    const int phys = kv8_phys(c, pair, page);
    constexpr int kGroups = 64 * D / 16 / kAppendThreads;  // 16-byte groups of a thread
    float x[kGroups][16];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int gi = i * kAppendThreads + tid, t = gi & 3, g = (gi >> 2) & 7, q = gi >> 5;
      if (!val) {  // q = (16-token tile, 32-dim chunk): tokens g, g + 8, dims 8t..8t+7
        const int mt = q / (D / 32), kp = q % (D / 32);
#pragma unroll
        for (int b = 0; b < 16; ++b)
          x[i][b] = value(mt * 16 + ((b >> 2) & 1) * 8 + g, kp * 32 + t * 8 + (b >> 3) * 4 + (b & 3));
      } else {  // q = (16-dim tile, 32-token chunk): dims g, g + 8, tokens 2t, 2t + 1, + 8, + 16, + 24
        const int dt = q >> 1, kp = q & 1;
#pragma unroll
        for (int b = 0; b < 16; ++b)
          x[i][b] = value(kp * 32 + (b >> 3) * 16 + ((b >> 1) & 1) * 8 + t * 2 + (b & 1),
                          dt * 16 + ((b >> 2) & 1) * 8 + g);
      }
#pragma unroll
      for (int b = 0; b < 16; ++b) m = max_nan(m, fabsf(x[i][b]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    for (int d = tid; d < D; d += kAppendThreads) ksum[d] = 0;
    __syncthreads();
    float amax = red[0];
#pragma unroll
    for (int i = 1; i < kAppendThreads / 32; ++i) amax = max_nan(amax, red[i]);
    const float sc = kv8_scale(amax);
    if (phys >= 0) {
      const size_t pg = kv8_page(c, pair, phys);
      uint4* out = reinterpret_cast<uint4*>(c.codes + (pg * 2 + val) * (size_t)(kPage * D));
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int gi = i * kAppendThreads + tid;
        uint32_t word[4] = {0, 0, 0, 0};
        int code[16];
#pragma unroll
        for (int b = 0; b < 16; ++b) {
          code[b] = sc > 0.0f ? kv8_code(x[i][b], sc) : 0;
          word[b >> 2] |= (uint32_t)(code[b] + 128) << (8 * (b & 3));
        }
        out[gi] = make_uint4(word[0], word[1], word[2], word[3]);
        if (!val) {
          const int t = gi & 3, kp = (gi >> 5) % (D / 32);
#pragma unroll
          for (int b = 0; b < 8; ++b) {  // dim 8t + b of the chunk: tokens g and g + 8, then the eight g
            int v = code[(b >> 2) * 8 + (b & 3)] + code[(b >> 2) * 8 + 4 + (b & 3)];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            if (((tid >> 2) & 7) == 0) atomicAdd(&ksum[kp * 32 + t * 8 + b], v);  // integers: any order
          }
        }
      }
      if (tid == 0) c.scales[pg * 2 + val] = sc;
      if (!val) {
        __syncthreads();
        for (int d = tid; d < D; d += kAppendThreads) c.sums[pg * D + d] = (int16_t)ksum[d];
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

// One CTA per (page of the window, KV head, sequence and keys/values): 16-byte groups of codes, each value
// s * c with one rounding; positions of the open page come from the tail.
template <int D>
__global__ void __launch_bounds__(256) k_kv8_read(w4a8_kv8_cache c, const int32_t* first, const int32_t* len, int n,
                                                   float* __restrict__ k_out, float* __restrict__ v_out) {
  griddep_enter();
  const int h = blockIdx.y, s = blockIdx.z >> 1;
  const bool val = blockIdx.z & 1;
  const int F = first[s];
  int L = kv8_len(c, len, s);
  if (F < 0) {
    if (threadIdx.x == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_CAPACITY);
    L = 0;
  }
  if (L < 0) L = 0;
  const int64_t f = F < 0 ? 0 : F;
  const int64_t page = f / kPage + blockIdx.x, base = page * kPage;
  const size_t pair = kv8_pair(c, s, h);
  float* out = val ? v_out : k_out;
  const size_t rs = (size_t)c.n_kv_heads * D;
  out += ((size_t)s * n * c.n_kv_heads + h) * D;
  auto put = [&](int tok, int d, float v) {
    const int64_t j = base + tok - f;
    if (j >= 0 && j < n) out[(size_t)j * rs + d] = v;
  };
  if (base + kPage <= L) {
    const int phys = kv8_phys(c, pair, (int)page);
    const size_t pg = kv8_page(c, pair, phys < 0 ? 0 : phys);
    const float sc = phys < 0 ? 0.0f : c.scales[pg * 2 + val];
    const uint4* in = reinterpret_cast<const uint4*>(c.codes + (pg * 2 + val) * (size_t)(kPage * D));
    for (int gi = threadIdx.x; gi < kPage * D / 16; gi += 256) {
      const uint4 u = in[gi];
      const uint32_t word[4] = {u.x, u.y, u.z, u.w};
      const int t = gi & 3, g = (gi >> 2) & 7, q = gi >> 5;
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        const float x = sc * (float)((int)((word[b >> 2] >> (8 * (b & 3))) & 255u) - 128);
        if (!val)
          put((q / (D / 32)) * 16 + ((b >> 2) & 1) * 8 + g, (q % (D / 32)) * 32 + t * 8 + (b >> 3) * 4 + (b & 3), x);
        else
          put((q & 1) * 32 + (b >> 3) * 16 + ((b >> 1) & 1) * 8 + t * 2 + (b & 1), (q >> 1) * 16 + ((b >> 2) & 1) * 8 + g,
              x);
      }
    }
  } else {
    const float* tail = c.tail + (pair * 2 + val) * kPage * D;
    for (int i = threadIdx.x; i < kPage * D; i += 256) put(i / D, i % D, base + i / D < L ? tail[i] : 0.0f);
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
  if (!aligned(k->data, kv8_elem(dtype)) || !aligned(v->data, kv8_elem(dtype))) return W4A8_ERR_ARG;
  if (n > kPage * c->max_pages + kPage - 1) return W4A8_ERR_CAPACITY;
  cudaStream_t st = as_stream(stream);
  const dim3 grid((unsigned)((n + kPage - 1 + kPage - 1) / kPage), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs * 2);
  const bool own = len_out == c->len;
  auto run = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(kAppendThreads), 0, st, *c, *k, *v, n_src, n, counts, index, len_out, !own);
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
  if (!first || !k_out || !v_out || n < 1) return W4A8_ERR_ARG;
  if (n > kPage * c->max_pages + kPage - 1) return W4A8_ERR_CAPACITY;
  const dim3 grid((unsigned)((n + kPage - 1 + kPage - 1) / kPage), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs * 2);
  const int32_t* L = len ? len : c->len;
  cudaStream_t st = as_stream(stream);
  W4A8_CUDA_TRY(c->head_dim == 64
                    ? launch_pdl(k_kv8_read<64>, grid, dim3(256), 0, st, *c, first, L, n, k_out, v_out)
                    : launch_pdl(k_kv8_read<128>, grid, dim3(256), 0, st, *c, first, L, n, k_out, v_out));
  return W4A8_OK;
}
