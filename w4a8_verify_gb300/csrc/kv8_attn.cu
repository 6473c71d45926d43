// Attention over the 8-bit key/value cache: joining the parts, the pages' mass, and the entry points.
#include "kv8_attn.cuh"

using namespace w4a8;

namespace {

constexpr int kJoinWarps = 8;

// One CTA per (row of a column block, segment): the parts of a cut segment, a warp takes every eighth of them,
// eight loads in flight; then the warps' sums.  Order fixed by the parts' places.  Segments of one worker are
// written already; rows that see nothing (no units) are zero.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) k_kv8_join(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo,
                                                              Kv8Scratch ws) {
  griddep_enter();
  constexpr int E = D / 32;
  __shared__ float sm_l[kJoinWarps];
  __shared__ float sm_o[kJoinWarps][D];
  const int H = c.n_kv_heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = blockIdx.y;
  int s, h, i, r, q;
  if (a.pages) {
    s = seg / H / a.n, h = seg % H, i = seg / H % a.n, r = blockIdx.x, q = seg % (a.n * H);
  } else {
    s = seg / geo.CB / H, h = seg / geo.CB % H, r = seg % geo.CB * geo.RB + blockIdx.x, i = r / geo.G;
    q = seg % (H * geo.CB);
  }
  const int L = kv8_len(c, c.len, s), cnt = kv8_count(c, a.counts, s, a.n);
  if (L < 0 || r >= geo.R || i >= cnt) return;
  const int hq = h * geo.G + (a.pages ? r : r % geo.G);
  T* out = static_cast<T*>(a.out.data) + s * a.out.seq + i * a.out.row + hq * a.out.head;
  float2* fin = ws.fin ? ws.fin + ((size_t)s * a.n + i) * a.n_heads + hq : nullptr;
  const int per = kv8_units(a, L, cnt).total();
  if (per == 0) {
    for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) kv8_store(out + d, 0.0f);
    if (fin && threadIdx.x == 0) *fin = make_float2(0.0f, 0.0f);
    return;
  }
  const int U = ws.prefix[c.n_seqs], W = min(geo.workers, U), u0 = ws.prefix[s] + q * per;
  const int w0 = worker_of(u0, W, U), parts = worker_of(u0 + per - 1, W, U) - w0 + 1;
  if (parts == 1) return;
  // the first worker's part is its range's last one unless it starts the range
  const int first = worker_begin(w0, W, U) == u0 ? 0 : 1;
  auto slot = [&](int p) { return (2 * (size_t)(w0 + p) + (p == 0 ? first : 0)) * geo.RB + blockIdx.x; };
  float M = -INFINITY;
  for (int p = lane; p < parts; p += 32) M = fmaxf(M, ws.ml[slot(p)].x);
  M = warp_max(M);
  const float base = M == -INFINITY ? 0.0f : M;
  float l = 0.0f, o[E] = {};
  constexpr int B = 8;
  for (int p0 = warp; p0 < parts; p0 += kJoinWarps * B) {
    float2 ml[B];
    float v[B][E];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int p = p0 + b * kJoinWarps;
      ml[b] = p < parts ? ws.ml[slot(p)] : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[b][e] = p < parts ? ws.o[slot(p) * D + e * 32 + lane] : 0.0f;
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const float w = ex2(ml[b].x - base);
      l = fmaf(ml[b].y, w, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(v[b][e], w, o[e]);
    }
  }
  if (lane == 0) sm_l[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][e * 32 + lane] = o[e];
  __syncthreads();
  float S = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) S += sm_l[w];
  if (threadIdx.x < D) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) v += sm_o[w][threadIdx.x];
    kv8_store(out + threadIdx.x, S == 0.0f ? 0.0f : v / S);
  }
  if (fin && threadIdx.x == 0) *fin = make_float2(base, S);
}

// Page weights onto the mass: one warp per page, a lane takes every 32nd row, the lanes' sums in a fixed tree.
__global__ void __launch_bounds__(256) k_kv8_mass(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo, Kv8Scratch ws) {
  griddep_enter();
  __shared__ float2 row[kKv8MaxRows * kKv8MaxGroup];  // maximum, 1 / sum
  const int h = blockIdx.y, s = blockIdx.z, lane = threadIdx.x & 31;
  const int L = kv8_len(c, c.len, s), cnt = kv8_count(c, a.counts, s, a.n);
  const int R = L < 0 || cnt < 0 ? 0 : cnt * geo.G;
  for (int r = threadIdx.x; r < R; r += 256) {
    const float2 f = ws.fin[((size_t)s * a.n + r / geo.G) * a.n_heads + h * geo.G + r % geo.G];
    row[r] = make_float2(f.x, f.y == 0.0f ? 0.0f : 1.0f / f.y);
  }
  __syncthreads();
  const size_t pair = kv8_pair(c, s, h);
  const int p = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (p >= c.max_pages) return;
  float sum = 0.0f;
  if (R > 0 && p < L / kPage && kv8_phys(c, pair, p) >= 0)
    for (int r = lane; r < R; r += 32) {
      const float2 f = ws.page[((pair * geo.CB + r / geo.RB) * c.max_pages + p) * geo.RB + r % geo.RB];
      sum = fmaf(f.y * ex2(f.x - row[r].x), row[r].y, sum);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) a.mass_out[pair * c.max_pages + p] = (a.mass ? a.mass[pair * c.max_pages + p] : 0.0f) + sum;
}

struct Plan {
  Kv8Geom geo;
  size_t segments, prefix, ml, o, fin, page, bytes;  // offsets
};

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

w4a8_status plan_of(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, Plan* p) {
  const w4a8_status ok = kv8_dims(c);
  if (ok != W4A8_OK) return ok;
  if (!a || !kv8_dtype(a->dtype) || !a->k.data != !a->v.data) return W4A8_ERR_ARG;
  if (a->n < 1 || a->n > kKv8MaxRows || a->n_heads < 1 || a->n_heads % c->n_kv_heads ||
      a->n_heads / c->n_kv_heads > kKv8MaxGroup || (a->pages && (a->top_k < 1 || a->top_k > kKv8MaxPages)))
    return W4A8_ERR_SHAPE;
  if (a->pages && a->mass_out) return W4A8_ERR_UNSUPPORTED;
  Kv8Geom& g = p->geo;
  g.n = a->n;
  g.G = a->n_heads / c->n_kv_heads;
  g.R = a->pages ? g.G : g.n * g.G;
  const Kv8Shape sh = kv8_shape(g.R, a->dtype);
  g.RB = sh.TW * sh.WC * (a->dtype == W4A8_F32 ? 4 : 8);
  g.CB = (g.R + g.RB - 1) / g.RB;
  p->segments = (size_t)c->n_seqs * c->n_kv_heads * (a->pages ? g.n : g.CB);
  const size_t units = p->segments * ((a->pages && a->top_k < c->max_pages ? a->top_k : c->max_pages) + 8);
  if (units >= (size_t)1 << 31) return W4A8_ERR_SHAPE;
  const int ng = kv8_warps(sh.TW) / sh.WC;
  const size_t ctas = (units + ng - 1) / ng;
  g.workers = (int)(ctas < (size_t)kKv8Ctas ? ctas : (size_t)kKv8Ctas) * ng;
  p->prefix = 0;
  p->ml = up256(((size_t)c->n_seqs + 1) * 4);
  p->o = up256(p->ml + (size_t)2 * g.workers * g.RB * 8);
  p->fin = up256(p->o + (size_t)2 * g.workers * g.RB * c->head_dim * 4);
  p->page = p->bytes = p->fin;
  if (a->mass_out) {
    p->page = up256(p->fin + (size_t)c->n_seqs * a->n * a->n_heads * 8);
    p->bytes = p->page + p->segments * c->max_pages * g.RB * 8;
  }
  return W4A8_OK;
}

// Whether groups of eight elements can be read 16 bytes at a time.
bool vec_rows(const w4a8_rows& r, int dtype) {
  const int64_t e = 16 / (int64_t)kv8_elem(dtype);
  return aligned(r.data, 16) && r.seq % e == 0 && r.row % e == 0 && r.head % e == 0;
}

}  // namespace

W4A8_API w4a8_status w4a8_kv8_attention_workspace_bytes(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a,
                                                        size_t* bytes) {
  Plan p;
  if (!bytes) return W4A8_ERR_ARG;
  const w4a8_status ok = plan_of(c, a, &p);
  if (ok == W4A8_OK) *bytes = p.bytes;
  return ok;
}

W4A8_API w4a8_status w4a8_kv8_attention(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  Plan p;
  w4a8_status ok = kv8_valid(c);
  if (ok == W4A8_OK) ok = plan_of(c, a, &p);
  if (ok != W4A8_OK) return ok;
  const size_t el = kv8_elem(a->dtype);
  if (!a->q.data || !a->out.data || !workspace || !aligned(workspace, 256) || !aligned(a->q.data, el) ||
      !aligned(a->out.data, el) || !aligned(a->k.data, el) || !aligned(a->v.data, el))
    return W4A8_ERR_ARG;
  if (workspace_bytes < p.bytes) return W4A8_ERR_CAPACITY;
  if (p.segments > 65535) return W4A8_ERR_SHAPE;
  char* base = static_cast<char*>(workspace);
  Kv8Scratch ws{reinterpret_cast<int*>(base + p.prefix), reinterpret_cast<float2*>(base + p.ml),
                reinterpret_cast<float*>(base + p.o), a->mass_out ? reinterpret_cast<float2*>(base + p.fin) : nullptr,
                a->mass_out ? reinterpret_cast<float2*>(base + p.page) : nullptr};
  p.geo.vec = (vec_rows(a->q, a->dtype) ? 1 : 0) | (vec_rows(a->k, a->dtype) ? 2 : 0);
  cudaStream_t st = as_stream(stream);
  const bool f32 = a->dtype == W4A8_F32, d64 = c->head_dim == 64;
  W4A8_CUDA_TRY((f32 ? d64 ? kv8_split_f32_d64 : kv8_split_f32_d128 : d64 ? kv8_split_bf16_d64 : kv8_split_bf16_d128)(
      *c, *a, p.geo, ws, st));
  const dim3 grid((unsigned)(p.geo.R < p.geo.RB ? p.geo.R : p.geo.RB), (unsigned)p.segments);
  auto join = [&](auto kern) { return launch_pdl(kern, grid, dim3(32 * kJoinWarps), 0, st, *c, *a, p.geo, ws); };
  if (f32)
    W4A8_CUDA_TRY(d64 ? join(k_kv8_join<float, 64>) : join(k_kv8_join<float, 128>));
  else
    W4A8_CUDA_TRY(d64 ? join(k_kv8_join<__nv_bfloat16, 64>) : join(k_kv8_join<__nv_bfloat16, 128>));
  if (a->mass_out)
    W4A8_CUDA_TRY(launch_pdl(k_kv8_mass,
                             dim3((unsigned)((c->max_pages + 7) / 8), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs),
                             dim3(256), 0, st, *c, *a, p.geo, ws));
  return W4A8_OK;
}
