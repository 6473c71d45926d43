// Attention of new rows over the 8-bit key/value cache.
//
// For query head h of new row i of sequence s (KV head h / G):
//   l_t = scale * q . k_t,  out = sum_t exp(l_t - m) v_t / sum_t exp(l_t - m),  m = max_t l_t
// over the tokens t the row sees: whole pages (s * c), the open page's fp32 rows, visible new rows.
#include "kv8.cuh"

using namespace w4a8;

namespace {

constexpr int kWarps = 8;

struct AttnView {  // what a row sees: pages (all, or a list), open rows, new rows
  int whole, open, cnt, units;
  const int32_t* list;
};

// Logical page of unit u, or -1 where the list ends or is out of order.
__device__ int view_page(const w4a8_kv8_cache& c, const AttnView& v, int u) {
  if (!v.list) return u;
  const int p = v.list[u];
  if (p == -1) return -1;
  if (p < 0 || p >= v.whole || (u > 0 && v.list[u - 1] >= p) || (u > 0 && v.list[u - 1] < 0)) {
    atomicOr(c.ctl, (unsigned)FLAG_ERR_TREE);
    return -1;
  }
  return p;
}

// One CTA per (query head, new row, sequence); a warp takes every kWarps-th token, a lane every 32nd dim.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) k_kv8_attn(w4a8_kv8_cache c, w4a8_kv8_attn a, float2* __restrict__ ml) {
  griddep_enter();
  constexpr int E = D / 32;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
  const int hq = blockIdx.x, i = blockIdx.y, s = blockIdx.z, G = a.n_heads / c.n_kv_heads, h = hq / G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = kv8_len(c, c.len, s), cnt = kv8_count(c, a.counts, s, a.n);
  if (L < 0 || i >= cnt) return;
  AttnView v{L / kPage, L % kPage, cnt, L / kPage, nullptr};
  if (a.pages) {
    v.list = a.pages + (((size_t)s * a.n + i) * c.n_kv_heads + h) * a.top_k;
    v.units = min(a.top_k, v.whole);
  }
  const size_t pair = kv8_pair(c, s, h);
  const T* q = static_cast<const T*>(a.q.data) + s * a.q.seq + i * a.q.row + hq * a.q.head;
  const T* kn = static_cast<const T*>(a.k.data) + s * a.k.seq + h * a.k.head;
  const T* vn = static_cast<const T*>(a.v.data) + s * a.v.seq + h * a.v.head;
  const uint64_t mask = a.mask ? a.mask[(size_t)s * a.n + i] : (i >= 63 ? ~0ull : (1ull << (i + 1)) - 1);
  float qr[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qr[e] = kv8_load(q + lane + 32 * e) * a.scale;
    o[e] = 0.0f;
  }
  const int rows = v.open + (a.k.data ? cnt : 0);
  for (int t = warp; t < v.units * kPage + rows; t += kWarps) {
    float k[E], x[E];
    if (t < v.units * kPage) {
      const int p = view_page(c, v, t / kPage);
      const int phys = p < 0 ? -1 : kv8_phys(c, pair, p);
      if (phys < 0) continue;
      const size_t pg = kv8_page(c, pair, phys);
      const uint8_t* b = c.codes + pg * 2 * (size_t)(kPage * D);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = c.scales[pg * 2] * (float)((int)b[kv8_key_byte(D, t % kPage, lane + 32 * e)] - 128);
        x[e] = c.scales[pg * 2 + 1] * (float)((int)b[kPage * D + kv8_val_byte(t % kPage, lane + 32 * e)] - 128);
      }
    } else {
      const int r = t - v.units * kPage;
      if (r >= v.open && !(mask >> (r - v.open) & 1)) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = lane + 32 * e;
        k[e] = r < v.open ? c.tail[(pair * 2 * kPage + r) * D + d] : kv8_load(kn + (r - v.open) * a.k.row + d);
        x[e] = r < v.open ? c.tail[((pair * 2 + 1) * kPage + r) * D + d] : kv8_load(vn + (r - v.open) * a.v.row + d);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot = fmaf(qr[e], k[e], dot);
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, b);
    const float m1 = fmaxf(m, dot), base = m1 == -INFINITY ? 0.0f : m1;
    const float f = expf(m - base), w = expf(dot - base);
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[e], o[e] * f);
    m = m1;
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float M = -INFINITY, S = 0.0f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  const float base = M == -INFINITY ? 0.0f : M;
  for (int w = 0; w < kWarps; ++w) S += sm_l[w] * expf(sm_m[w] - base);
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float r = 0.0f;
    for (int w = 0; w < kWarps; ++w) r += sm_o[w][d] * expf(sm_m[w] - base);
    T* out = static_cast<T*>(a.out.data) + s * a.out.seq + i * a.out.row + hq * a.out.head;
    kv8_store(out + d, S == 0.0f ? 0.0f : r / S);
  }
  if (ml && threadIdx.x == 0) ml[((size_t)s * a.n + i) * a.n_heads + hq] = make_float2(base, S);
}

// The softmax weight on each whole page: one warp per page, the rows and heads in order.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) k_kv8_mass(w4a8_kv8_cache c, w4a8_kv8_attn a,
                                                          const float2* __restrict__ ml) {
  griddep_enter();
  constexpr int E = D / 32;
  const int p = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y, s = blockIdx.z, lane = threadIdx.x & 31;
  const int G = a.n_heads / c.n_kv_heads;
  if (p >= c.max_pages) return;
  const int L = kv8_len(c, c.len, s), cnt = kv8_count(c, a.counts, s, a.n);
  const size_t pair = kv8_pair(c, s, h);
  float sum = a.mass ? a.mass[pair * c.max_pages + p] : 0.0f;
  const int phys = L >= 0 && p < L / kPage ? kv8_phys(c, pair, p) : -1;
  if (phys >= 0) {
    const size_t pg = kv8_page(c, pair, phys);
    const uint8_t* b = c.codes + pg * 2 * (size_t)(kPage * D);
    for (int r = 0; r < cnt * G; ++r) {
      const int i = r / G, hq = h * G + r % G;
      const T* q = static_cast<const T*>(a.q.data) + s * a.q.seq + i * a.q.row + hq * a.q.head;
      const float2 st = ml[((size_t)s * a.n + i) * a.n_heads + hq];
      float w = 0.0f;
      for (int t = 0; t < kPage; ++t) {
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          dot = fmaf(kv8_load(q + lane + 32 * e) * a.scale,
                     c.scales[pg * 2] * (float)((int)b[kv8_key_byte(D, t, lane + 32 * e)] - 128), dot);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        w += expf(dot - st.x);
      }
      sum += w / st.y;
    }
  }
  if (lane == 0) a.mass_out[pair * c.max_pages + p] = sum;
}

w4a8_status attn_args(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a) {
  const w4a8_status ok = kv8_dims(c);
  if (ok != W4A8_OK) return ok;
  if (!a || !kv8_dtype(a->dtype) || !a->k.data != !a->v.data) return W4A8_ERR_ARG;
  if (a->n < 1 || a->n > kKv8MaxRows || a->n_heads < 1 || a->n_heads % c->n_kv_heads ||
      a->n_heads / c->n_kv_heads > kKv8MaxGroup || (a->pages && (a->top_k < 1 || a->top_k > c->max_pages)))
    return W4A8_ERR_SHAPE;
  if (a->pages && a->mass_out) return W4A8_ERR_UNSUPPORTED;
  return W4A8_OK;
}

}  // namespace

W4A8_API w4a8_status w4a8_kv8_attention_workspace_bytes(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a,
                                                        size_t* bytes) {
  const w4a8_status ok = attn_args(c, a);
  if (ok != W4A8_OK) return ok;
  if (!bytes) return W4A8_ERR_ARG;
  *bytes = (size_t)c->n_seqs * a->n * a->n_heads * 8;
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_attention(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  size_t need = 0;
  w4a8_status ok = w4a8_kv8_attention_workspace_bytes(c, a, &need);
  if (ok == W4A8_OK) ok = kv8_valid(c);
  if (ok != W4A8_OK) return ok;
  const size_t el = kv8_elem(a->dtype);
  if (!a->q.data || !a->out.data || !workspace || !aligned(workspace, 256) || !aligned(a->q.data, el) ||
      !aligned(a->out.data, el) || !aligned(a->k.data, el) || !aligned(a->v.data, el))
    return W4A8_ERR_ARG;
  if (workspace_bytes < need) return W4A8_ERR_CAPACITY;
  cudaStream_t st = as_stream(stream);
  float2* ml = a->mass_out ? static_cast<float2*>(workspace) : nullptr;
  const dim3 grid((unsigned)a->n_heads, (unsigned)a->n, (unsigned)c->n_seqs);
  const dim3 mgrid((unsigned)((c->max_pages + kWarps - 1) / kWarps), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs);
  auto run = [&](auto kern, auto mass) -> cudaError_t {
    cudaError_t e = launch_pdl(kern, grid, dim3(32 * kWarps), 0, st, *c, *a, ml);
    if (e != cudaSuccess || !ml) return e;
    return launch_pdl(mass, mgrid, dim3(32 * kWarps), 0, st, *c, *a, (const float2*)ml);
  };
  if (a->dtype == W4A8_F32)
    W4A8_CUDA_TRY(c->head_dim == 64 ? run(k_kv8_attn<float, 64>, k_kv8_mass<float, 64>)
                                    : run(k_kv8_attn<float, 128>, k_kv8_mass<float, 128>));
  else
    W4A8_CUDA_TRY(c->head_dim == 64 ? run(k_kv8_attn<__nv_bfloat16, 64>, k_kv8_mass<__nv_bfloat16, 64>)
                                    : run(k_kv8_attn<__nv_bfloat16, 128>, k_kv8_mass<__nv_bfloat16, 128>));
  return W4A8_OK;
}
