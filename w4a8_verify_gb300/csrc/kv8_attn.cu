// Attention over the 8-bit key/value cache: joining the parts, the pages' mass, and the entry points.
#include "kv8_attn.cuh"

using namespace w4a8;

namespace {

constexpr int kJoinWarps = 8;

// The parts of a segment's rows, the split kernel's CTAs in their order, then the row tiles': RPC rows to a CTA, a warp
// takes every (kJoinWarps / RPC)th part of its row, B loads in flight; then the warps' sums.  No parts: zero.  The
// sum of a part that is not there, where a CTA's wait ran out, is NaN, and so is the row.
// Bound by latency: 32 rows of 28 parts 6.6 us cold, 4096 rows 8 us.
template <typename T, int D, int RPC>
__global__ void __launch_bounds__(32 * kJoinWarps) k_kv8_join(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo,
                                                              Kv8Scratch ws) {
  constexpr int E = D / 32, WPR = kJoinWarps / RPC;
  using Vec = std::conditional_t<E == 4, float4, float2>;
  __shared__ float2 sm_ml[kJoinWarps];
  __shared__ __align__(16) float sm_o[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = blockIdx.x;
  const int rb = blockIdx.y * RPC + warp / WPR, first = warp % WPR;
  const Kv8Segment sg = kv8_segment(c, a, geo, seg);
  const int r = sg.cb * geo.RB + rb, i = a.pages ? sg.i : r / geo.G, s = sg.s;
  const int L = kv8_len(c, c.len, s), cnt = kv8_count(c, a.counts, s, a.n);
  const bool mine = L >= 0 && rb < geo.RB && r < geo.R && i < cnt;
  // lengths and counts are older than the split kernel; its parts are waited for
  griddep_enter();
  float m = -INFINITY, l = 0.0f, o[E] = {};
  if (mine) {
    const Kv8Units un = kv8_units(a, L, cnt);
    int c0 = 0, held = 0, early = 0;  // CTAs that hold parts, and whether a worker ended it and went on
    if (un.pages > 0) {
      const int U = ws.prefix[c.n_seqs];
      const Kv8Workers wk = kv8_workers(U, geo.ctas, geo.ng);
      const int of = a.pages ? sg.i * c.n_kv_heads + sg.h : sg.h * kv8_blocks(geo, cnt) + sg.cb;  // segment of the sequence
      const int u0 = ws.prefix[s] + of * un.pages, u1 = u0 + un.pages;
      const int w0 = worker_of(u0, wk.W, U), w1 = worker_of(u1 - 1, wk.W, U);
      early = worker_begin(w1 + 1, wk.W, U) > u1;
      c0 = w0 / wk.ng;
      held = w1 - early < w0 ? 0 : (w1 - early) / wk.ng - c0 + 1;
    }
    const int tile0 = held + early, parts = tile0 + un.open + un.fresh;
    // place of part p: of the CTAs, the early one, the row tiles (those beyond the early one: another array)
    auto place = [&](int p) -> int64_t {
      if (p < held) return ((int64_t)c0 + p + seg) * geo.RB + rb;
      if (p < tile0) return ((int64_t)geo.ctas + geo.segments + seg) * geo.RB + rb;
      const int f = p - tile0 < un.open ? p - tile0 : kPage / kRowTile + p - tile0 - un.open;
      return ((int64_t)seg * geo.tiles + f) * geo.RB + rb;
    };
    constexpr int B = WPR == 1 ? 4 : 8;
    for (int p0 = first; p0 < parts; p0 += WPR * B) {
      float2 ml[B];
      Vec v[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int p = p0 + b * WPR;
        ml[b] = make_float2(-INFINITY, 0.0f);
        v[b] = {};
        if (p < parts) {
          const int64_t at = place(p);
          ml[b] = (p < tile0 ? ws.ml : ws.rml)[at];
          v[b] = *reinterpret_cast<const Vec*>((p < tile0 ? ws.o : ws.ro) + at * D + E * lane);
        }
      }
      float mx = m;
#pragma unroll
      for (int b = 0; b < B; ++b) mx = fmaxf(mx, ml[b].x);
      const float base = mx == -INFINITY ? 0.0f : mx, f = ex2(m - base);
      m = mx;
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float w = ex2(ml[b].x - base);
        const float* ve = reinterpret_cast<const float*>(&v[b]);
        l = fmaf(ml[b].y, w, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(ve[e], w, o[e]);
      }
    }
  }
  if (lane == 0) sm_ml[warp] = make_float2(m, l);
  *reinterpret_cast<Vec*>(&sm_o[warp][E * lane]) = *reinterpret_cast<Vec*>(o);
  __syncthreads();
  if (!mine || first > 0) return;
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < WPR; ++w) M = fmaxf(M, sm_ml[warp + w].x);
  const float base = M == -INFINITY ? 0.0f : M;
  l = 0.0f;
  float sum[E] = {};
#pragma unroll
  for (int w = 0; w < WPR; ++w) {
    const float2 ml = sm_ml[warp + w];
    const float f = ex2(ml.x - base);
    l = fmaf(ml.y, f, l);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = fmaf(sm_o[warp + w][E * lane + e], f, sum[e]);
  }
  const int hq = sg.h * geo.G + (a.pages ? r : r % geo.G);
  T* out = static_cast<T*>(a.out.data) + s * a.out.seq + i * a.out.row + hq * a.out.head + E * lane;
#pragma unroll
  for (int e = 0; e < E; ++e) kv8_store(out + e, l == 0.0f ? 0.0f : sum[e] / l);
  if (ws.fin && lane == 0) ws.fin[((size_t)s * a.n + i) * a.n_heads + hq] = make_float2(base, l);
}

// Page weights onto the mass: one warp per page, a lane takes every 32nd row, the lanes' sums in a fixed tree.  Bound by the
// reads of 8 bytes for each (row, page): 256 rows of 500 pages of 8 heads, 8.2 MB, 10 us cold.
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
  size_t segments, prefix, ml, o, rml, ro, fin, page, bytes;  // offsets
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
  const bool wide = kv8_is_wide(*c, *a, g.R);
  const int wc = kv8_split_warps(g.R, a->dtype);
  g.RB = wide ? kWideRows : wc * (a->dtype == W4A8_F32 ? 4 : 8);
  g.CB = (g.R + g.RB - 1) / g.RB;
  p->segments = (size_t)c->n_seqs * c->n_kv_heads * (a->pages ? g.n : g.CB);
  const size_t units = p->segments * (a->pages && a->top_k < c->max_pages ? a->top_k : c->max_pages);
  if (units >= (size_t)1 << 31 || p->segments >= (size_t)1 << 22) return W4A8_ERR_SHAPE;
  g.ng = wide ? 1 : kKv8Warps / wc;
  g.tiles = kPage / kRowTile + (a->k.data ? (g.n + kRowTile - 1) / kRowTile : 0);
  // CTAs for the pages, or (split kernel) for a round of its row warps' parts
  const size_t chunks = p->segments * ((g.R < g.RB ? g.R : g.RB) + kRowChunk - 1) / kRowChunk;
  // the fp32 rows by a kernel of their own where the row warps would take more than about two rounds (with half of an
  // open page): 38 sequences of 27 tokens, 7 fp32 rows, 2 heads of 64, 7 query heads each 30.1 -> 16.1 us; below that its
  // launch costs more
  g.apart = !wide && g.n * g.G > kRowsApart && chunks * (g.tiles - 2) > 2 * kKv8Ctas * kKv8RowWarps;
  const size_t parts = wide || g.apart ? 0 : chunks * g.tiles;
  const size_t ctas = units > parts / kKv8RowWarps ? units : parts / kKv8RowWarps;
  g.ctas = (int)(ctas < (size_t)kKv8Ctas ? ctas : (size_t)kKv8Ctas);
  p->prefix = 0;
  g.segments = (int)p->segments;
  const size_t slots = g.ctas + 2 * p->segments, rslots = p->segments * g.tiles, row = (size_t)g.RB * 4;
  p->ml = up256(((size_t)c->n_seqs + 1) * 4);
  p->o = up256(p->ml + slots * row * 2);
  p->rml = up256(p->o + slots * row * c->head_dim);
  p->ro = up256(p->rml + rslots * row * 2);
  p->fin = up256(p->ro + rslots * row * c->head_dim);
  p->page = p->bytes = p->fin;
  if (a->mass_out) {
    p->page = up256(p->fin + (size_t)c->n_seqs * a->n * a->n_heads * 8);
    p->bytes = p->page + p->segments * c->max_pages * g.RB * 8;
  }
  return W4A8_OK;
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

// withheld, wait_ns: see Kv8Geom.
static w4a8_status attend(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, void* workspace, size_t workspace_bytes,
                          void* stream, int withheld, uint64_t wait_ns) {
  Plan p;
  w4a8_status ok = kv8_valid(c);
  if (ok == W4A8_OK) ok = plan_of(c, a, &p);
  if (ok != W4A8_OK) return ok;
  const size_t el = kv8_elem(a->dtype);
  // rows of out that lie on one another would be written in any order
  if ((c->n_seqs > 1 && !a->out.seq) || (a->n > 1 && !a->out.row) || (a->n_heads > 1 && !a->out.head)) return W4A8_ERR_ARG;
  if (!a->q.data || !a->out.data || !workspace || !aligned(workspace, 256) || !aligned(a->q.data, el) ||
      !aligned(a->out.data, el) || !aligned(a->k.data, el) || !aligned(a->v.data, el) || !aligned(a->counts, 4) ||
      !aligned(a->mask, 8) || !aligned(a->pages, 4) || !aligned(a->mass, 4) || !aligned(a->mass_out, 4))
    return W4A8_ERR_ARG;
  if (workspace_bytes < p.bytes) return W4A8_ERR_CAPACITY;
  if (rows_overlap(a->out, c->n_seqs, a->n, a->n_heads, c->head_dim)) return W4A8_ERR_ARG;
  char* base = static_cast<char*>(workspace);
  Kv8Scratch ws{reinterpret_cast<int*>(base + p.prefix), reinterpret_cast<float2*>(base + p.ml),
                reinterpret_cast<float*>(base + p.o), reinterpret_cast<float2*>(base + p.rml),
                reinterpret_cast<float*>(base + p.ro), a->mass_out ? reinterpret_cast<float2*>(base + p.fin) : nullptr,
                a->mass_out ? reinterpret_cast<float2*>(base + p.page) : nullptr};
  p.geo.vec = (kv8_vec_rows(a->q, a->dtype) ? 1 : 0) | (kv8_vec_rows(a->k, a->dtype) ? 2 : 0) | (kv8_vec_rows(a->v, a->dtype) ? 4 : 0);
  p.geo.withheld = withheld;
  p.geo.wait_ns = wait_ns;
  cudaStream_t st = as_stream(stream);
  const bool f32 = a->dtype == W4A8_F32, d64 = c->head_dim == 64;
  if (kv8_is_wide(*c, *a, p.geo.R)) W4A8_CUDA_TRY(kv8_wide(*c, *a, p.geo, ws, st));
  else W4A8_CUDA_TRY((f32 ? d64 ? kv8_split_f32_d64 : kv8_split_f32_d128 : d64 ? kv8_split_bf16_d64 : kv8_split_bf16_d128)(
      *c, *a, p.geo, ws, st));
  if (p.geo.apart) W4A8_CUDA_TRY(kv8_rows(*c, *a, p.geo, ws, st));
  // Warps of a row: all eight of a CTA where rows are few (some CTAs for each SM) and parts may be many; one where
  // segments are so many that each has a few parts (64 sequences of 8 heads: 2.4 us less than with two); else two (one
  // sequence with 128 rows to a head: 2 us less than with one).
  const int rows = p.geo.R < p.geo.RB ? p.geo.R : p.geo.RB;
  const int rpc = (int64_t)rows * (int64_t)p.segments <= 4 * kKv8Ctas ? 1 : p.segments < (size_t)kKv8Ctas ? 4 : 8;
  auto join = [&](auto one, auto four, auto eight) {
    const dim3 grid((unsigned)p.segments, (unsigned)((rows + rpc - 1) / rpc));
    return launch_pdl(rpc == 1 ? one : rpc == 4 ? four : eight, grid, dim3(32 * kJoinWarps), 0, st, *c, *a, p.geo, ws);
  };
#define W4A8_JOIN(T, D) join(k_kv8_join<T, D, 1>, k_kv8_join<T, D, 4>, k_kv8_join<T, D, 8>)
  W4A8_CUDA_TRY(f32 ? (d64 ? W4A8_JOIN(float, 64) : W4A8_JOIN(float, 128))
                    : (d64 ? W4A8_JOIN(__nv_bfloat16, 64) : W4A8_JOIN(__nv_bfloat16, 128)));
#undef W4A8_JOIN
  if (a->mass_out)
    W4A8_CUDA_TRY(launch_pdl(k_kv8_mass,
                             dim3((unsigned)((c->max_pages + 7) / 8), (unsigned)c->n_kv_heads, (unsigned)c->n_seqs),
                             dim3(256), 0, st, *c, *a, p.geo, ws));
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_attention(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  return attend(c, a, workspace, workspace_bytes, stream, -1, kWaitLimitNs);
}

W4A8_API w4a8_status w4a8_kv8_attention_inject_timeout(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, void* workspace,
                                                       size_t workspace_bytes, int cta, void* stream) {
  if (cta < 0) return W4A8_ERR_ARG;
  return attend(c, a, workspace, workspace_bytes, stream, cta, 20000000ull);
}
