// Attention over the 4-bit key/value cache: the plan of a call and the entry points.
#include "kv4_attn.cuh"

using namespace w4a8;

namespace {

struct Plan {
  Kv4Geom geo;
  bool wide;
  size_t ml, o, prefix, rml, ro, bytes;  // offsets
};

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

w4a8_status plan_of(const w4a8_kv4_cache* c, const w4a8_kv4_attn* a, Plan* p) {
  const w4a8_status ok = kv4_dims(c);
  if (ok != W4A8_OK) return ok;
  if (!a || !kv8_dtype(a->dtype) || !a->k.data != !a->v.data) return W4A8_ERR_ARG;
  if (a->n < 1 || a->n > kKv4MaxRows || a->n_heads < 1 || a->n_heads % c->n_kv_heads ||
      a->n_heads / c->n_kv_heads > kKv8MaxGroup)
    return W4A8_ERR_SHAPE;
  Kv4Geom& g = p->geo;
  g = Kv4Geom{};
  g.n = a->n;
  g.G = a->n_heads / c->n_kv_heads;
  g.R = g.n * g.G;
  p->wide = kv4_is_wide(*c, g.R, a->dtype);
  g.RB = p->wide ? kKv4WideRows : kv4_split_tiles(g.R, a->dtype) * (a->dtype == W4A8_F32 ? 4 : 8);
  g.CB = (g.R + g.RB - 1) / g.RB;
  const size_t segments = (size_t)c->n_seqs * c->n_kv_heads * g.CB, units = segments * (p->wide ? c->max_pages : c->max_pages + 1);
  if (units >= (size_t)1 << 31 || segments >= (size_t)1 << 22) return W4A8_ERR_SHAPE;
  g.segments = (int)segments;
  size_t most_ctas = kKv4Ctas;
  if (p->wide && a->k.data) {  // a few CTAs for the new rows get SMs of their own, a sixth of them at most
    g.tiles = (g.n + kKv4RowTile - 1) / kKv4RowTile;
    const int64_t blocks = kv4_rows_blocks(*c, g);
    if (blocks >= (int64_t)1 << 31) return W4A8_ERR_SHAPE;
    if (blocks <= kKv4Ctas / 6) g.folded = (int)blocks, most_ctas -= g.folded;
  }
  const size_t workers = p->wide ? 1 : (size_t)kv4_split_warps(g.R, a->dtype) / 2, ctas = (units + workers - 1) / workers;
  g.ctas = (int)(ctas < most_ctas ? ctas : most_ctas);
  const size_t row = (size_t)g.RB * 4, D = (size_t)c->head_dim;
  const size_t slots = p->wide ? g.ctas + 2 * segments : 5 * g.ctas * workers;
  p->ml = W4A8_KV4_TICKETS;
  p->o = up256(p->ml + slots * row * 2);
  p->prefix = p->rml = p->ro = p->bytes = up256(p->o + slots * row * D);
  if (p->wide) {
    p->rml = up256(p->prefix + ((size_t)c->n_seqs + 1) * 4);
    p->ro = up256(p->rml + segments * g.tiles * row * 2);
    p->bytes = up256(p->ro + segments * g.tiles * row * D);
  }
  return W4A8_OK;
}

// withheld, wait_ns: see Kv4Geom.
w4a8_status attend(const w4a8_kv4_cache* c, const w4a8_kv4_attn* a, void* workspace, size_t workspace_bytes, void* stream,
                   int withheld, uint64_t wait_ns) {
  Plan p;
  w4a8_status ok = kv4_valid(c);
  if (ok == W4A8_OK) ok = plan_of(c, a, &p);
  if (ok != W4A8_OK) return ok;
  const size_t el = kv8_elem(a->dtype);
  if (!a->q.data || !a->out.data || !workspace || !aligned(workspace, 256) || !aligned(a->q.data, el) ||
      !aligned(a->out.data, el) || !aligned(a->k.data, el) || !aligned(a->v.data, el) || !aligned(a->counts, 4) ||
      !aligned(a->mask, 8))
    return W4A8_ERR_ARG;
  if (workspace_bytes < p.bytes) return W4A8_ERR_CAPACITY;
  const int S = c->n_seqs, n = a->n, D = c->head_dim, H = c->n_kv_heads;
  // rows of out that lie on one another, or on what is read, would be written in any order
  if (rows_overlap(a->out, S, n, a->n_heads, D, kMaxDifferences) || rows_meet(a->out, a->n_heads, a->q, a->n_heads, S, n, D, el) ||
      (a->k.data && (rows_meet(a->out, a->n_heads, a->k, H, S, n, D, el) || rows_meet(a->out, a->n_heads, a->v, H, S, n, D, el))))
    return W4A8_ERR_ARG;
  auto on = [&](const void* at, size_t bytes) { return rows_touch(a->out, a->n_heads, S, n, D, el, at, bytes); };
  if (on(c->pages, kv4_pool_bytes(*c)) || on(c->table, 4 * (size_t)S * c->max_pages) || on(c->len, 4 * (size_t)S) || on(c->ctl, 4) ||
      on(a->counts, 4 * (size_t)S) || on(a->mask, 8 * (size_t)S * n) || on(workspace, p.bytes))
    return W4A8_ERR_ARG;
  char* base = static_cast<char*>(workspace);
  const Kv4Scratch ws{reinterpret_cast<int*>(base),          reinterpret_cast<float2*>(base + p.ml),
                      reinterpret_cast<float*>(base + p.o),  reinterpret_cast<int*>(base + p.prefix),
                      reinterpret_cast<float2*>(base + p.rml), reinterpret_cast<float*>(base + p.ro)};
  p.geo.vec = (kv8_vec_rows(a->q, a->dtype) ? 1 : 0) | (kv8_vec_rows(a->k, a->dtype) ? 2 : 0) | (kv8_vec_rows(a->v, a->dtype) ? 4 : 0);
  p.geo.withheld = withheld;
  p.geo.wait_ns = wait_ns;
  const double l = (double)a->scale * 1.4426950408889634;
  p.geo.lhi = (float)l, p.geo.llo = (float)(l - (double)p.geo.lhi);
  const bool f32 = a->dtype == W4A8_F32, d64 = D == 64;
  if (p.wide) W4A8_CUDA_TRY(kv4_wide(*c, *a, p.geo, ws, as_stream(stream)));
  else W4A8_CUDA_TRY((f32 ? d64 ? kv4_split_f32_d64 : kv4_split_f32_d128 : d64 ? kv4_split_bf16_d64 : kv4_split_bf16_d128)(
      *c, *a, p.geo, ws, as_stream(stream)));
  return W4A8_OK;
}

}  // namespace

W4A8_API w4a8_status w4a8_kv4_attention_workspace_bytes(const w4a8_kv4_cache* c, const w4a8_kv4_attn* a,
                                                        size_t* bytes) {
  Plan p;
  if (!bytes) return W4A8_ERR_ARG;
  const w4a8_status ok = plan_of(c, a, &p);
  if (ok == W4A8_OK) *bytes = p.bytes;
  return ok;
}

W4A8_API w4a8_status w4a8_kv4_attention(const w4a8_kv4_cache* c, const w4a8_kv4_attn* a, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  return attend(c, a, workspace, workspace_bytes, stream, -1, kWaitLimitNs);
}

W4A8_API w4a8_status w4a8_kv4_attention_inject_timeout(const w4a8_kv4_cache* c, const w4a8_kv4_attn* a, void* workspace,
                                                       size_t workspace_bytes, int cta, void* stream) {
  if (cta < 0) return W4A8_ERR_ARG;
  return attend(c, a, workspace, workspace_bytes, stream, cta, 20000000ull);
}
