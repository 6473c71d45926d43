// Attention over the 4-bit cache for many query rows of a KV head (draft trees, prompt buckets): tcgen05.
//
// A segment is 128 query rows of one (sequence, KV head); its pages, end to end over the segments, are cut into equal
// ranges, one for each CTA.  Per page, in a pipeline of warps:
//   copy      one bulk copy brings the page (8.5 KB at D = 128) into a ring of four;
//   convert   codes and scales become the cached values in f16 (exact), keys [64 tokens][D] and values [D][64 tokens], in
//             the 128-byte-swizzled K-major layout of the tensor core's B operand;
//   products  S = Q K^T and O' = P V, tcgen05.mma with A (Q, P) in tensor memory, 128 x 64 x D and 128 x D x 64;
//   softmax   a thread holds one query row: no exchange between lanes.  P (scaled by 2^7) returns to tensor memory in the
//             token order of the values' chunks.  A page is tried with the row's old maximum, and done again with
//             its own when a logit passes that by 8 (log2);
//   values    O = O c + O' in registers, a thread half a row: fp32 additions, and nothing is rescaled in tensor memory.
// fp32 calls split Q and P into f16 hi + lo; the products of P's share an accumulator, those of Q's have one each.  The
// hi terms are the nearest whole numbers at a largest magnitude of 2^11 (P: scaled by 2^10, with the maximum of its own page), so
// that the products of one scale add up to multiples of its last bit, which the tensor core's truncating additions keep.
//
// Bound by the softmax warps, one to a scheduler: 64 rows over 32000 tokens of 8 heads of 128 with 4 query heads each take 86 us (bf16,
// tensor pipe 20%, issue slots 42%) or 128 (fp32, 25%), of which the new rows and the join 15; a tree of 16 rows over 4096 20 and 22 us,
// bound by the latency of the stages.
#include "kv4_attn.cuh"
#include "tc.cuh"

namespace w4a8 {
namespace {

// Two fp32 numbers in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Warp roles.  Softmax and value warps sit where their number modulo 4 names the tensor-memory lanes they may touch.
constexpr int kSoftWarps = 4, kSumWarps = 8, kConvWarps = 4;
constexpr int kSum0 = kSoftWarps, kConv0 = kSum0 + kSumWarps, kMmaWarp = kConv0 + kConvWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kWideThreads = 32 * (kCopyWarp + 1);
constexpr int kRing = 4;   // pages of codes
constexpr int kFac = 4;    // pages whose P and row factors may be on their way from the softmax to the value warps

template <typename T, int D>
struct Wide {
  static constexpr int NQ = sizeof(T) == 4 ? 2 : 1;         // f16 terms of Q and P
  static constexpr int NO = sizeof(T) == 4 ? 1 : 2;         // buffers of O'
  static constexpr int PAGE = Kv4Page<D>::BYTES, TILE = kPage * D * 2;  // bytes of a page, of an f16 tile
  // scale of P, and how far (log2) a logit may pass its row's maximum before that moves
  static constexpr float PSCALE = NQ == 2 ? 1024.0f : kP4Scale, SLACK = NQ == 2 ? 0.9f : kP4Slack;
  // buffers of P
  static constexpr int NP = NQ == 2 ? 1 : 2;
  // tensor memory columns: Q, S twice, the product with the lo term of Q (apart: a sum of whole numbers that
  // fractions are added to is truncated each time), P, O'
  static constexpr int cQ = 0, cS = cQ + NQ * D / 2, cL = cS + 2 * kPage, cP = cL + (NQ - 1) * kPage,
                       cO = cP + NP * NQ * kPage / 2;
  static_assert(cO + NO * D <= 512, "tensor memory");
  // shared memory
  static_assert(kRing * PAGE % 1024 == 0, "swizzle atoms");
  static constexpr int sK = kRing * PAGE, sV = sK + 2 * TILE, sBar = sV + 2 * TILE, sFac = sBar + 256;
  static constexpr int QROW = D * (int)sizeof(T) + 16;  // a staged query row: 16 bytes on, so that lanes of a row each do not collide
  static constexpr int sQ = sFac + kFac * kKv4WideRows * 4 + 64 + 16;
  static constexpr int sPrefix = sQ + kKv4WideRows * QROW;
};

// mbarriers.  A wait knows its phase by parity alone, so the phase after it must not complete before every warp has passed
// the wait.  Use n of an entry of depth d is waited for before use n + d can complete because that one needs, from the waiting warp:
//   code_full  code_empty(n)                                   code_empty  the copy of page n + kRing
//   k_full, v_full  S(n), O'(n), issued behind the wait        s_done, pv_done  k_full(n + 2), v_full(n + 2) (converters),
//   s_empty    S(n), lo_empty: L(n), issued behind the wait      p_full(n + 1) or p_full(n + 2) (softmax), o_empty(n) (values)
//   p_full     o_empty(n), by way of O'(n + 2), S(n + 4)       o_empty     O'(n + NO), issued behind the wait
//   q_full     q_empty of the run                              q_empty     the next run's copies
// p_full has kFac entries: with two, bf16 calls (two buffers of P and of O') let the softmax warps complete p_full(n) and
// p_full(n + 2) while a value warp was still at page n - 1; it then waited for p_full(n + 4), which needs its own o_empty(n).
struct Bars {
  uint64_t code_full[kRing], code_empty[kRing], k_full[2], v_full[2], s_done[2], s_empty[2], p_full[kFac], pv_done[2], o_empty[2], lo_empty, q_full, q_empty, drained;
};
static_assert(sizeof(Bars) + 4 <= 256, "barriers");

// The new rows of wide calls: 64 query rows by 16 tokens to a CTA of 256 threads, both products in registers: a thread
// holds the logits of two rows and two tokens, then D / 8 values of the two rows.  Rows 32 apart and tokens 8 apart
// belong to a thread, so that the lanes' 16-byte reads of neighbouring (padded) rows meet no bank twice.  Plain fp32.
// A few of them are CTAs of the wide kernel's own grid, which then leaves them SMs (a tree of 16 rows: 33 us as a kernel of
// its own behind, 22.5 us so); many are a kernel behind it, whose CTAs start as SMs become free: it reads (from L2) what the wide
// kernel waited for before it let this one start, so the wait for that kernel comes last, for the join that follows.
constexpr int kRowsThreads = 256, kRT = 8 * kKv4RowsRows / kRowsThreads;  // kRT rows of a thread
template <int D>
struct RowsSmem {
  float q[kKv4RowsRows][D + 4], k[kKv4RowTile][D + 4], v[kKv4RowTile][D], p[kKv4RowsRows][kKv4RowTile + 4];
  uint32_t see[kKv4RowsRows];
};
// whether x holds for one of the first kRowsThreads threads, which meet here
__device__ __forceinline__ bool rows_any(bool x) {
  unsigned r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((unsigned)x), "n"(kRowsThreads)
      : "memory");
  return r != 0;
}
// Block `number` of the call's; the CTA's first kRowsThreads threads.
template <typename T, int D>
__device__ __forceinline__ void rows_block(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo,
                                           const Kv4Scratch& ws, uint8_t* shared, int number) {
  RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>(shared);
  constexpr int V = D / 8;  // vectors of eight elements in a row
  const int tid = threadIdx.x, rg = tid >> 3, tg = tid & 7;
  const int blocks = (a.n * geo.G + kKv4RowsRows - 1) / kKv4RowsRows, x = number / blocks;
  const int fresh = x % geo.tiles, pair = x / geo.tiles;
  const struct { int s, h; } sg = {pair / c.n_kv_heads, pair % c.n_kv_heads};
  const int L = __ldcg(c.len + sg.s), cnt = a.counts ? __ldcg(a.counts + sg.s) : a.n;
  const int first = number % blocks * kKv4RowsRows;
  auto slot = [&](int r) {  // of row first + r of the KV head
    return (((size_t)pair * geo.CB + (first + r) / geo.RB) * geo.tiles + fresh) * geo.RB + (first + r) % geo.RB;
  };
  int nv = 0, rows = 0;
  if (L >= 0 && L <= kPage * c.max_pages && cnt > 0 && cnt <= a.n) {
    nv = min(kKv4RowTile, cnt - fresh * kKv4RowTile);
    rows = min(kKv4RowsRows, cnt * geo.G - first);
  }
  if (nv > 0 && rows > 0) {  // the same for the whole block
    const T* kn = static_cast<const T*>(a.k.data) + sg.s * a.k.seq + sg.h * a.k.head + (int64_t)fresh * kKv4RowTile * a.k.row;
    const T* vn = static_cast<const T*>(a.v.data) + sg.s * a.v.seq + sg.h * a.v.head + (int64_t)fresh * kKv4RowTile * a.v.row;
    // eight elements of a row of T; all of a loop's rows on their way
    auto load8 = [&](const T* p, int vec, float (&e)[8]) {
      if (vec) {
        uint4 w[sizeof(T) / 2];
#pragma unroll
        for (int y = 0; y < (int)sizeof(T) / 2; ++y) w[y] = __ldcg(reinterpret_cast<const uint4*>(p) + y);
#pragma unroll
        for (int y = 0; y < 8; ++y) e[y] = kv8_load(reinterpret_cast<const T*>(w) + y);
      } else {
#pragma unroll
        for (int y = 0; y < 8; ++y) e[y] = kv8_float(__ldcg(p + y));
      }
    };
    bool bad = false;  // a value that is not finite
#pragma unroll
    for (int y = tid; y < 2 * kKv4RowTile * V; y += kRowsThreads) {
      const int t = y / V % kKv4RowTile, d = y % V * 8;
      const bool val = y >= kKv4RowTile * V;
      float e[8] = {};
      if (t < nv) {
        load8(val ? vn + (int64_t)t * a.v.row + d : kn + (int64_t)t * a.k.row + d, geo.vec & (val ? 4 : 2), e);
      }
      float* to = val ? &sm.v[t][d] : &sm.k[t][d];
      *reinterpret_cast<float4*>(to) = *reinterpret_cast<float4*>(e);
      *reinterpret_cast<float4*>(to + 4) = *reinterpret_cast<float4*>(e + 4);
#pragma unroll
      for (int z = 0; z < 8; ++z) bad = bad || (val && !(fabsf(e[z]) <= 3.402823466e38f));
    }
#pragma unroll 4
    for (int y = tid; y < kKv4RowsRows * V; y += kRowsThreads) {
      const int r = y / V, d = y % V * 8, rr = first + min(r, rows - 1);
      float e[8];
      load8(static_cast<const T*>(a.q.data) + sg.s * a.q.seq + (rr / geo.G) * a.q.row +
                (sg.h * geo.G + rr % geo.G) * a.q.head + d, geo.vec & 1, e);
      *reinterpret_cast<float4*>(&sm.q[r][d]) = *reinterpret_cast<float4*>(e);
      *reinterpret_cast<float4*>(&sm.q[r][d + 4]) = *reinterpret_cast<float4*>(e + 4);
    }
    if (tid < kKv4RowsRows) {  // tokens that a row sees
      const int node = (first + min(tid, rows - 1)) / geo.G;
      const uint64_t mask = a.mask ? __ldcg(a.mask + (size_t)sg.s * a.n + node) : (node >= 63 ? ~0ull : (1ull << (node + 1)) - 1ull);
      sm.see[tid] = (uint32_t)(mask >> (fresh * kKv4RowTile)) & ((1u << nv) - 1u);
    }
    bad = rows_any(bad);
    float s[kRT][2] = {};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 k[2], q[kRT];
#pragma unroll
      for (int j = 0; j < 2; ++j) k[j] = *reinterpret_cast<const float4*>(&sm.k[8 * j + tg][d]);
#pragma unroll
      for (int i = 0; i < kRT; ++i) q[i] = *reinterpret_cast<const float4*>(&sm.q[kKv4RowsRows / kRT * i + rg][d]);
#pragma unroll
      for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          s[i][j] = fmaf(q[i].w, k[j].w, fmaf(q[i].z, k[j].z, fmaf(q[i].y, k[j].y, fmaf(q[i].x, k[j].x, s[i][j]))));
    }
    const float qscale = a.scale * 1.4426950408889634f;
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      const int r = kKv4RowsRows / kRT * i + rg;
      const uint32_t see = sm.see[r] >> tg;
      const float s0 = see & 1u ? s[i][0] * qscale : -INFINITY, s1 = see & 256u ? s[i][1] * qscale : -INFINITY;
      float m = fmaxf(s0, s1);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.0f : m;
      const float p0 = see & 1u ? ex2(s0 - base) : 0.0f, p1 = see & 256u ? ex2(s1 - base) : 0.0f;
      float l = p0 + p1;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      sm.p[r][tg] = p0, sm.p[r][8 + tg] = p1;
      if (tg == 0 && r < rows) ws.rml[slot(r)] = make_float2(m, l);
    }
    __syncwarp();  // a row's weights come from the lanes that read them
    float4 o[kRT][D / 32] = {};
#pragma unroll 1
    for (int t = 0; t < kKv4RowTile; t += 4) {
      float p[kRT][4];
#pragma unroll
      for (int i = 0; i < kRT; ++i) *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(&sm.p[kKv4RowsRows / kRT * i + rg][t]);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float4 v[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) v[e] = *reinterpret_cast<const float4*>(&sm.v[t + y][32 * e + 4 * tg]);
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
          if (bad && !(sm.see[kKv4RowsRows / kRT * i + rg] >> (t + y) & 1u)) continue;  // 0 times it would not be 0
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            o[i][e].x = fmaf(p[i][y], v[e].x, o[i][e].x), o[i][e].y = fmaf(p[i][y], v[e].y, o[i][e].y);
            o[i][e].z = fmaf(p[i][y], v[e].z, o[i][e].z), o[i][e].w = fmaf(p[i][y], v[e].w, o[i][e].w);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRT; ++i)
      if (kKv4RowsRows / kRT * i + rg < rows)
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
          *reinterpret_cast<float4*>(ws.ro + slot(kKv4RowsRows / kRT * i + rg) * D + 32 * e + 4 * tg) = o[i][e];
  }
}
template <typename T, int D>
__global__ void __launch_bounds__(kRowsThreads, 3) k_kv4_rows(w4a8_kv4_cache c, w4a8_kv4_attn a, Kv4Geom geo, Kv4Scratch ws) {
  griddep_launch();
  extern __shared__ __align__(16) uint8_t sm_raw[];
  rows_block<T, D>(c, a, geo, ws, sm_raw, blockIdx.x);
  // the grid has not ended before the kernel in front has; only one CTA keeps its place for that
  if (blockIdx.x == 0) griddep_wait();
}

template <typename T, int D>
__global__ void __launch_bounds__(kWideThreads, 1) k_kv4_wide(w4a8_kv4_cache c, w4a8_kv4_attn a, Kv4Geom geo, Kv4Scratch ws) {
  using C = Wide<T, D>;
  constexpr int NQ = C::NQ, NO = C::NO;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(16) uint8_t sm_raw[];
  if ((int)blockIdx.x >= geo.ctas) {  // a block of new rows
    griddep_enter();
    if (threadIdx.x < kRowsThreads) rows_block<T, D>(c, a, geo, ws, sm_raw, blockIdx.x - geo.ctas);
    return;
  }
  uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);  // swizzle atoms start at multiples of 1024
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + C::sBar + sizeof(Bars));
  Bars& bar = *reinterpret_cast<Bars*>(sm + C::sBar);
  float* fac = reinterpret_cast<float*>(sm + C::sFac);          // [kFac][rows] factor of the old values
  int* moved = reinterpret_cast<int*>(fac + kFac * kKv4WideRows);  // [kFac][softmax warp] whether one is not 1
  int* held = moved + kFac * kSoftWarps;                        // [kRing] tokens of a page (0: not there)
  int* prefix = reinterpret_cast<int*>(sm + C::sPrefix);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = c.n_seqs;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(&bar.code_full[i], 1), mbar_init(&bar.code_empty[i], kConvWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], kConvWarps / 2), mbar_init(&bar.v_full[i], kConvWarps / 2);
      mbar_init(&bar.s_done[i], 1), mbar_init(&bar.pv_done[i], 1);
      mbar_init(&bar.s_empty[i], kSoftWarps);
      mbar_init(&bar.o_empty[i], kSumWarps);
    }
    for (int i = 0; i < kFac; ++i) mbar_init(&bar.p_full[i], kSoftWarps);
    mbar_init(&bar.lo_empty, kSoftWarps);
    mbar_init(&bar.q_full, 1), mbar_init(&bar.q_empty, kSoftWarps), mbar_init(&bar.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  griddep_enter();
  // behind the wait: held while waiting, tensor memory could be what a CTA of the kernel in front still wants on this SM
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  kv4_prefix(c, a, geo, prefix, nullptr, [](int L) { return (L + kPage - 1) / kPage; });
  tc_before();
  __syncthreads();
  tc_after();
  if (blockIdx.x == 0)
    for (int s = tid; s <= S; s += kWideThreads) ws.prefix[s] = prefix[s];
  const uint32_t tmem = s_tmem;
  const int U = prefix[S];
  const Kv8Workers wk = kv8_workers(U, geo.ctas, 1);
  const int worker = blockIdx.x;
  const bool has = worker < wk.W;
  const int u0 = has ? worker_begin(worker, wk.W, U) : 0, u1 = has ? worker_begin(worker + 1, wk.W, U) : 0;

  // every role walks the range in the same way: runs of pages of one segment
  struct Run {
    int seg, first, pages;  // segment, its first page here, how many
    bool ends;              // whether the range goes on behind the run
    int s, h, cb, cnt, L;
  };
  auto run_at = [&](int x) {
    Run r;
    r.s = kv4_seq_of(prefix, S, x);
    r.cnt = a.counts ? a.counts[r.s] : a.n;
    r.L = c.len[r.s];
    const int per = (r.L + kPage - 1) / kPage, q = (x - prefix[r.s]) / per;
    r.first = (x - prefix[r.s]) % per;
    const int blocks = kv4_blocks(geo, r.cnt);
    r.h = q / blocks, r.cb = q % blocks;
    r.seg = (r.s * c.n_kv_heads + r.h) * geo.CB + r.cb;
    r.pages = min(per - r.first, u1 - x);
    r.ends = x + r.pages < u1;
    return r;
  };
  // 32 pages of a run, one for each lane: the pool's page, or -1 (left out)
  auto batch_at = [&](const Run& r, int p) {
    if (p + lane >= r.pages) return -1;
    const int v = c.table[(size_t)r.s * c.max_pages + r.first + p + lane];
    return v >= 0 && v < c.n_pages ? v : -1;
  };
  auto tokens_of = [&](const Run& r, int p, int phys) { return phys < 0 ? 0 : min(kPage, r.L - (r.first + p) * kPage); };
  bool ok = true;
  auto wait = [&](uint64_t* b, int parity) {
    ok = ok && __all_sync(FULL, mbar_wait(b, (unsigned)parity, geo.wait_ns));
    return ok;
  };

  // query row of the run's row `row`
  auto query_row = [&](const Run& r, int row) {
    const int rr = r.cb * kKv4WideRows + row;
    return static_cast<const T*>(a.q.data) + r.s * a.q.seq + (rr / geo.G) * a.q.row + (r.h * geo.G + rr % geo.G) * a.q.head;
  };
  auto rows_of = [&](const Run& r) { return max(0, min(kKv4WideRows, r.cnt * geo.G - r.cb * kKv4WideRows)); };
  if (warp == kCopyWarp) {
    Turn<kRing> e;
    int n = 0, runs = 0;
    for (int x = u0; x < u1 && ok; ++runs) {
      const Run r = run_at(x);
      if (geo.vec & 1) {  // the run's query rows
        const int rows = rows_of(r);
        if (runs > 0 && !wait(&bar.q_empty, (runs - 1) & 1)) break;
        if (lane == 0) mbar_expect_tx(&bar.q_full, rows * D * sizeof(T));
        __syncwarp();
        for (int row = lane; row < rows; row += 32)
          bulk_g2s(sm + C::sQ + row * C::QROW, query_row(r, row), D * sizeof(T), &bar.q_full);
        __syncwarp();
      }
      int now = -1, then = batch_at(r, 0);
      for (int p = 0; p < r.pages && ok; ++p, ++n, e.next()) {
        if ((p & 31) == 0) now = then, then = batch_at(r, p + 32);
        if (n >= kRing && !wait(&bar.code_empty[e.i], e.ph ^ 1)) break;
        const int phys = __shfl_sync(FULL, now, p & 31);
        if (lane == 0) {
          if (phys < 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TREE);
          held[e.i] = tokens_of(r, p, phys);  // for the converters; page 0 stands in for one that is not there
          mbar_expect_tx(&bar.code_full[e.i], C::PAGE);
          if (geo.withheld != (int)blockIdx.x)
            bulk_g2s(sm + e.i * C::PAGE, kv4_page<D>(c, max(phys, 0), r.h), C::PAGE, &bar.code_full[e.i]);
        }
        __syncwarp();
      }
      x += r.pages;
    }
    // no copy in flight when the CTA ends
    const WaitsWithin drain(geo.wait_ns);
    for (int i = max(0, n - kRing); i < n; ++i) (void)drain.wait(&bar.code_full[i % kRing], (unsigned)(i / kRing & 1));
    if ((geo.vec & 1) && runs > 0) (void)drain.wait(&bar.q_full, (unsigned)(runs - 1) & 1);
  } else if (warp >= kConv0 && warp < kMmaWarp) {
    // the first half of the warps takes the keys, the second the values
    constexpr int kHalf = kConvWarps / 2;
    const int v = (warp - kConv0) / kHalf, ct = (tid - kConv0 * 32) % (32 * kHalf);
    Turn<kRing> e;
    Turn<2> b;
    for (int i = 0; i < u1 - u0 && ok; ++i, e.next(), b.next()) {
      // the tile's last readers: the products of two pages ago
      if (i >= 2 && !wait(v ? &bar.pv_done[b.i] : &bar.s_done[b.i], b.ph ^ 1)) break;
      if (!wait(&bar.code_full[e.i], e.ph)) break;
      uint8_t* tile = sm + (v ? C::sV : C::sK) + b.i * C::TILE;
      const uint8_t* from = sm + e.i * C::PAGE;
      const int tokens = held[e.i];
      const int t = ct & 3, g = ct >> 2 & 7;
      // In either tile the rows of odd g take the other half of a row's 128 bytes: no bank conflict of a store's phases.
      if (!v) {
        // a 16-byte group of the page's order: four 16-byte chunks, of tokens g and g + 8 in two groups of 32 dims
#pragma unroll 2
        for (int q = ct >> 5; q < 4 * (D / 64); q += kHalf) {
          const int t16 = q / (D / 64), j = q % (D / 64);
          const uint4 w4 = reinterpret_cast<const uint4*>(from)[q * 32 + (ct & 31)];
          const uint8_t* sc = from + Kv4Page<D>::KS + (t16 * 8 + g) * (D / 16) + 2 * j;
          uint32_t s2[2] = {*reinterpret_cast<const uint16_t*>(sc), *reinterpret_cast<const uint16_t*>(sc + D / 32)};
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (16 * t16 + g + 8 * i >= tokens) s2[i] = 0;  // whatever the bytes of a token that is not there hold
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int kh = y ^ (g & 1);
            const uint32_t wa = kh ? w4.z : w4.x, wb = kh ? w4.w : w4.y, va = kv4_swap(wa), vb = kv4_swap(wb);
            const uint32_t s0 = kv4_scale_pair(s2[0] >> (8 * kh), 0, 0), s1 = kv4_scale_pair(s2[1] >> (8 * kh), 0, 0);
            const uint32_t b0 = mul_h2(s0, kMinus264), b1 = mul_h2(s1, kMinus24);
            const uint4 lo = make_uint4(fma_h2(kv4_f16_low(wa), s0, b0), fma_h2(kv4_f16_low(va), s0, b0),
                                        fma_h2(kv4_f16_low(wb), s0, b0), fma_h2(kv4_f16_low(vb), s0, b0));
            const uint4 hi = make_uint4(fma_h2(kv4_f16_high(wa), s1, b1), fma_h2(kv4_f16_high(va), s1, b1),
                                        fma_h2(kv4_f16_high(wb), s1, b1), fma_h2(kv4_f16_high(vb), s1, b1));
            // keys of D = 128 are two tiles of 64 dims
            uint8_t* to = tile + j * (kPage * 128) + (16 * t16 + g) * 128 + (((4 * kh + t) ^ g) << 4);
            *reinterpret_cast<uint4*>(to) = lo;
            *reinterpret_cast<uint4*>(to + 8 * 128) = hi;
          }
        }
      } else {
        // two such groups, of two tiles of 16 tokens: eight chunks, of dims g and g + 8 in four blocks of 16 dims; a chunk is the
        // tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of either tile, the order in which the softmax stores P
#pragma unroll 1
        for (int q = ct >> 5; q < 2 * (D / 64); q += kHalf) {
          const int pair = (q / (D / 64)) ^ (g & 1), j = q % (D / 64);
          uint32_t w[2][4], sw[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t16 = 2 * pair + i;
            const uint4 x = reinterpret_cast<const uint4*>(from + Kv4Page<D>::V)[(t16 * (D / 64) + j) * 32 + (ct & 31)];
            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
            const uint2 s = *reinterpret_cast<const uint2*>(from + Kv4Page<D>::VS + (t16 * 4 + t) * (D / 8) + 8 * j);
            sw[i][0] = s.x, sw[i][1] = s.y;
            if (tokens < kPage) {
              __syncwarp();
              uint32_t keep = 0;
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if (16 * t16 + 2 * t + (b & 1) + 8 * (b >> 1) < tokens) keep |= 255u << (8 * b);
              sw[i][0] &= keep, sw[i][1] &= keep;
            }
          }
#pragma unroll
          for (int gh = 0; gh < 2; ++gh) {
            uint32_t s0[2], s1[2], b0[2], b1[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s0[i] = kv4_scale_pair(sw[i][gh], 0, 1), s1[i] = kv4_scale_pair(sw[i][gh], 2, 3);
              b0[i] = mul_h2(s0[i], kMinus264), b1[i] = mul_h2(s1[i], kMinus24);
            }
#pragma unroll
            for (int dd = 0; dd < 2; ++dd) {
              const uint32_t wa = w[0][2 * gh + dd], wb = w[1][2 * gh + dd], va = kv4_swap(wa), vb = kv4_swap(wb);
              const uint4 lo = make_uint4(fma_h2(kv4_f16_low(wa), s0[0], b0[0]), fma_h2(kv4_f16_high(wa), s1[0], b1[0]),
                                          fma_h2(kv4_f16_low(wb), s0[1], b0[1]), fma_h2(kv4_f16_high(wb), s1[1], b1[1]));
              const uint4 hi = make_uint4(fma_h2(kv4_f16_low(va), s0[0], b0[0]), fma_h2(kv4_f16_high(va), s1[0], b1[0]),
                                          fma_h2(kv4_f16_low(vb), s0[1], b0[1]), fma_h2(kv4_f16_high(vb), s1[1], b1[1]));
              uint8_t* to = tile + (16 * (4 * j + 2 * gh + dd) + g) * 128 + (((4 * pair + t) ^ g) << 4);
              *reinterpret_cast<uint4*>(to) = lo;
              *reinterpret_cast<uint4*>(to + 8 * 128) = hi;
            }
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.code_empty[e.i]);
        mbar_arrive(v ? &bar.v_full[b.i] : &bar.k_full[b.i]);
      }
    }
  } else if (warp == kMmaWarp) {
    Turn<2> b;
    int n = 0;  // pages whose S is issued
    const uint32_t one = elect_one();
    auto values = [&](int i) {  // O' of page i (the one before the newest S)
      const Turn<2> pb(i);
      const Turn<NO> ob(i);
      const Turn<kFac> pf(i);
      if (!wait(&bar.p_full[pf.i], pf.ph) || !wait(&bar.v_full[pb.i], pb.ph)) return;
      if (i >= NO && !wait(&bar.o_empty[ob.i], ob.ph ^ 1)) return;
      tc_after();
      const uint32_t v = tc_desc(smem_u32(sm + C::sV + pb.i * C::TILE)), o = tmem + C::cO + ob.i * D;
      const uint32_t pa = tmem + C::cP + pb.i % C::NP * NQ * (kPage / 2);
#pragma unroll
      for (int k = 0; k < NQ * kPage / 16; ++k) tc_mma<D>(one, o, pa + k * 8, v + (k & 3) * 2, k > 0);
      tc_commit(one, &bar.pv_done[pb.i]);
    };
    for (int x = u0; x < u1 && ok;) {
      const Run r = run_at(x);
      for (int p = 0; p < r.pages && ok; ++p, ++n, b.next()) {
        // the softmax warps wait for a run's last products before they bring the next run's Q, and release s_empty
        // of both buffers when it is there
        if (!wait(&bar.k_full[b.i], b.ph) || !wait(&bar.s_empty[b.i], b.ph)) break;
        tc_after();
        // 16 dims are 32 bytes of a row; dims 64 .. 127 are another tile
        const uint32_t k0 = tc_desc(smem_u32(sm + C::sK + b.i * C::TILE));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma<kPage>(one, tmem + C::cS + b.i * kPage, tmem + C::cQ + k * 8, k0 + (k >> 2) * (kPage * 128 / 16) + (k & 3) * 2, k > 0);
        if (NQ == 2) {
          if (!wait(&bar.lo_empty, n & 1)) break;
          tc_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma<kPage>(one, tmem + C::cL, tmem + C::cQ + D / 2 + k * 8, k0 + (k >> 2) * (kPage * 128 / 16) + (k & 3) * 2, k > 0);
        }
        tc_commit(one, &bar.s_done[b.i]);
        if (p > 0) values(n - 1);
      }
      if (ok && r.pages > 0) values(n - 1);
      x += r.pages;
    }
  } else if (warp < kSoftWarps) {
    const int row = tid;  // 0..127
    const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
    Turn<2> b;
    Turn<kFac> fb;
    int n = 0, runs = 0, freed = 0;  // pages and runs done; S buffers released to the products (page n needs n + 1 of them)
    // the logit's factor is not negative (Q takes the scale's sign), so the largest logit is the largest S
    const float lhi = fabsf(geo.lhi), llo = a.scale < 0.0f ? -geo.llo : geo.llo;
    for (int x = u0; x < u1 && ok;) {
      const Run r = run_at(x);
      const int rows = rows_of(r);
      int now = -1, then = batch_at(r, 0);
      // Q of the run: the products of the run before are done (its last O' was waited for)
      float colfac, collow, m = -INFINITY, l = 0.0f;
      {
        const T* q = geo.vec & 1 ? reinterpret_cast<const T*>(sm + C::sQ + row * C::QROW) : query_row(r, min(row, max(rows - 1, 0)));
        if ((geo.vec & 1) && !wait(&bar.q_full, runs & 1)) break;
        float am = 0.0f;
        auto load8 = [&](int d, float (&v)[8]) {
          if (row >= rows) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
          } else if (geo.vec & 1) {
            uint4 w[sizeof(T) / 2];
#pragma unroll
            for (int e = 0; e < (int)sizeof(T) / 2; ++e) w[e] = reinterpret_cast<const uint4*>(q + d)[e];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = kv8_load(reinterpret_cast<const T*>(w) + e);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = kv8_load(q + d + e);
          }
        };
#pragma unroll 8
        for (int d = 0; d < D; d += 8) {
          float v[8];
          load8(d, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) am = max_nan(am, fabsf(v[e]));
        }
        const float up = a.scale < 0.0f ? -f16_scale(am) : f16_scale(am), down = 1.0f / f16_scale(am);
        colfac = lhi * down;
        collow = llo * down;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float v[8];
            load8(d + 8 * y, v);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float f0 = v[e] * up, f1 = v[e + 1] * up;
              if (NQ == 2) {
                const float w0 = whole(f0), w1 = whole(f1);
                hi[4 * y + e / 2] = pack_f16(w0, w1);
                lo[4 * y + e / 2] = pack_f16(f0 - w0, f1 - w1);
              } else {
                hi[4 * y + e / 2] = pack_f16(f0, f1);
              }
            }
          }
          tc_store16(mine + C::cQ + d / 2, hi);
          if (NQ == 2) tc_store16(mine + C::cQ + D / 2 + d / 2, lo);
        }
        tc_store_wait();
      }
      tc_before();
      __syncwarp();
      if ((geo.vec & 1) && lane == 0) mbar_arrive(&bar.q_empty);
      for (int y = 0; y < 2 && freed < n + r.pages; ++y, ++freed)
        if (lane == 0) mbar_arrive(&bar.s_empty[freed & 1]);
      if (NQ == 2 && lane == 0) mbar_arrive(&bar.lo_empty);
      for (int p = 0; p < r.pages && ok; ++p, ++n, b.next(), fb.next()) {
        if ((p & 31) == 0) now = then, then = batch_at(r, p + 32);
        const int tokens = tokens_of(r, p, __shfl_sync(FULL, now, p & 31));
        if (!wait(&bar.s_done[b.i], b.ph)) break;
        tc_after();
        const uint32_t sa = mine + C::cS + b.i * kPage;
        float f = 1.0f, ps, mx;
        // the run's first maximum; bf16 calls try later pages with the old one
        if (p == 0 || NQ == 2) {
          mx = -INFINITY;
#pragma unroll 1
          for (int y = 0; y < 2; ++y) {
            uint32_t v[32];
            tc_load32(sa + 32 * y, v);
            if (tokens < kPage) {
              __syncwarp();  // a branch: as predicated instructions it would cost every page its selects
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * y + e >= tokens) v[e] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(v[e]));
          }
          if (mx * colfac > m) {
            f = ex2(m - mx * colfac);
            m = mx * colfac;
            l *= f;
          }
        }
        // P's last readers; and the value warps are past page n - 4, whose row factors these replace
        if (n >= C::NP && !wait(&bar.pv_done[(n - C::NP) & 1], (n - C::NP) >> 1 & 1)) break;
#pragma unroll 1
        for (int again = 0;; ++again) {
          const float base = m == -INFINITY ? 0.0f : m;
          ps = 0.0f, mx = -INFINITY;
          const bool part = tokens < kPage;
#pragma unroll 1
          for (int y = 0; y < 2; ++y) {
            uint32_t v[32], hi[16], lo[16];
            tc_load32(sa + 32 * y, v);
            if (NQ == 2) {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                uint32_t w[16];
                tc_load16(mine + C::cL + 32 * y + 16 * z, w);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  v[16 * z + e] = __float_as_uint(__uint_as_float(v[16 * z + e]) + __uint_as_float(w[e]));
              }
            }
            if (part) {
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * y + e >= tokens) v[e] = __float_as_uint(-INFINITY);
            }
            float2 sum = make_float2(0.0f, 0.0f);
            float top[2] = {mx, mx};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 s = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              top[0] = fmaxf(top[0], s.x), top[1] = fmaxf(top[1], s.y);
              const float off = NQ == 2 ? -base : 7.0f - base;
              float2 y = fma2(s, make_float2(colfac, colfac), make_float2(off, off));
              if (NQ == 2) y = fma2(s, make_float2(collow, collow), y);
              v[e] = __float_as_uint(NQ == 2 ? ex2(y.x) * C::PSCALE : ex2(y.x));
              v[e + 1] = __float_as_uint(NQ == 2 ? ex2(y.y) * C::PSCALE : ex2(y.y));
            }
            if (part) {  // a factor of 0 makes NaN of what is not there
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * y + e >= tokens) v[e] = 0;
            }
            // register 4 t + 2 ks + h8 holds tokens 16 ks + 8 h8 + 2 t + {0, 1} of the 32: the values' chunk order
#pragma unroll
            for (int z = 0; z < 16; ++z) {
              const int tok = (z >> 1 & 1) * 16 + (z & 1) * 8 + (z >> 2) * 2;
              const float e0 = __uint_as_float(v[tok]), e1 = __uint_as_float(v[tok + 1]);
              sum = add2(sum, make_float2(e0, e1));
              if (NQ == 2) {
                const float w0 = whole(e0), w1 = whole(e1);
                hi[z] = pack_f16(w0, w1);
                lo[z] = pack_f16(e0 - w0, e1 - w1);
              } else {
                hi[z] = pack_f16(e0, e1);
              }
            }
            mx = fmaxf(top[0], top[1]);
            ps += sum.x + sum.y;
            tc_store16(mine + C::cP + b.i % C::NP * NQ * (kPage / 2) + 16 * y, hi);
            if (NQ == 2) tc_store16(mine + C::cP + kPage / 2 + 16 * y, lo);
          }
          mx *= colfac;
          const bool move = mx > m + C::SLACK;
          if (again || !__any_sync(FULL, move)) break;
          if (move) {
            const float g = ex2(m - mx);
            f *= g;
            m = mx;
            l *= g;
          }
        }
        fac[fb.i * kKv4WideRows + row] = f;
        const bool any = __any_sync(FULL, f != 1.0f);
        if (lane == 0) moved[fb.i * kSoftWarps + warp] = any;
        l += ps;
        tc_store_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.p_full[fb.i]);
          if (freed < n + r.pages - p) mbar_arrive(&bar.s_empty[b.i]);
          if (NQ == 2 && p + 1 < r.pages) mbar_arrive(&bar.lo_empty);
        }
        if (freed < n + r.pages - p) ++freed;
      }
      // the run's last products are done before the next run's Q takes the place of this one
      if (!ok || !wait(&bar.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
      tc_after();
      if (row < rows) {
        const size_t at = r.ends ? (size_t)geo.ctas + geo.segments + r.seg : (size_t)blockIdx.x + r.seg;
        ws.ml[at * kKv4WideRows + row] = make_float2(m, l / C::PSCALE);
      }
      x += r.pages;
      ++runs;
    }
  } else {
    // values: quadrant of lanes, half of the columns
    const int quad = warp & 3, half = (warp - kSum0) >> 2, row = quad * 32 + lane;
    constexpr int DH = D / 2;
    const uint32_t mine = tmem + ((uint32_t)(quad * 32) << 16) + C::cO + half * DH;
    Turn<2> b;
    Turn<NO> ob;
    Turn<kFac> fb;
    for (int x = u0; x < u1 && ok;) {
      const Run r = run_at(x);
      const int rows = rows_of(r);
      float O[DH];
#pragma unroll
      for (int d = 0; d < DH; ++d) O[d] = 0.0f;
      for (int p = 0; p < r.pages && ok; ++p, b.next(), ob.next(), fb.next()) {
        if (!wait(&bar.p_full[fb.i], fb.ph) || !wait(&bar.pv_done[b.i], b.ph)) break;
        tc_after();
        if (moved[fb.i * kSoftWarps + quad]) {
          const float f = fac[fb.i * kKv4WideRows + row];
#pragma unroll
          for (int d = 0; d < DH; ++d) O[d] *= f;
        }
#pragma unroll
        for (int d = 0; d < DH; d += 16) {
          uint32_t v[16];
          tc_load16(mine + ob.i * D + d, v);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 o = add2(make_float2(O[d + e], O[d + e + 1]), make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])));
            O[d + e] = o.x, O[d + e + 1] = o.y;
          }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.o_empty[ob.i]);
      }
      if (ok && row < rows) {
        const size_t at = r.ends ? (size_t)geo.ctas + geo.segments + r.seg : (size_t)blockIdx.x + r.seg;
        float4* o = reinterpret_cast<float4*>(ws.o + (at * kKv4WideRows + row) * D + half * DH);
#pragma unroll
        for (int d = 0; d < DH; d += 4)
          o[d / 4] = make_float4(O[d] / C::PSCALE, O[d + 1] / C::PSCALE, O[d + 2] / C::PSCALE, O[d + 3] / C::PSCALE);
      }
      x += r.pages;
    }
  }
  if (!ok && lane == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TIMEOUT);
  tc_before();
  const int cut = __syncthreads_or(!ok);
  tc_after();
  if (cut)  // the CTA's parts are not what they should be: NaN, for the join to pass on
    for (int x = u0; x < u1;) {
      const Run r = run_at(x);
      const size_t at = r.ends ? (size_t)geo.ctas + geo.segments + r.seg : (size_t)blockIdx.x + r.seg;
      if (tid < kKv4WideRows) ws.ml[at * kKv4WideRows + tid] = make_float2(NAN, NAN);
      x += r.pages;
    }
  if (warp == kMmaWarp) {
    // tensor memory is given back and the CTA ends: no product is under way then, also where a wait ran out
    tc_commit(elect_one(), &bar.drained);
    if (!__all_sync(FULL, mbar_wait(&bar.drained, 0, geo.wait_ns)) && lane == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TIMEOUT);
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// The parts of a segment's rows, the CTAs in their order, then the blocks of new rows: RPC rows to a CTA, a warp takes
// every (kJoinWarps / RPC)th part of its row, B loads in flight; then the warps' sums.  No parts: zero.  The
// sum of a part that is not there, where a CTA's wait ran out, is NaN, and so is the row.
constexpr int kJoinWarps = 8;
template <typename T, int D, int RPC>
__global__ void __launch_bounds__(32 * kJoinWarps) k_kv4_join(w4a8_kv4_cache c, w4a8_kv4_attn a, Kv4Geom geo,
                                                              Kv4Scratch ws) {
  constexpr int E = D / 32, WPR = kJoinWarps / RPC;
  using Vec = std::conditional_t<E == 4, float4, float2>;
  __shared__ float2 sm_ml[kJoinWarps];
  __shared__ __align__(16) float sm_o[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = blockIdx.x;
  const int rb = blockIdx.y * RPC + warp / WPR, first = warp % WPR;
  const int cb = seg % geo.CB, h = seg / geo.CB % c.n_kv_heads, s = seg / geo.CB / c.n_kv_heads;
  const int r = cb * geo.RB + rb, i = r / geo.G;
  const int L = kv4_len(c, c.len, s), cnt = kv4_count(c, a.counts, s, a.n);
  const bool mine = L >= 0 && rb < geo.RB && r < geo.R && i < cnt;
  // lengths and counts are older than the wide kernel; its parts are waited for
  griddep_enter();
  float m = -INFINITY, l = 0.0f, o[E] = {};
  if (mine) {
    const int pages = (L + kPage - 1) / kPage;
    int c0 = 0, held = 0, early = 0;  // CTAs that hold parts, and whether the last one went on to another segment
    if (pages > 0) {
      const int U = ws.prefix[c.n_seqs];
      const Kv8Workers wk = kv8_workers(U, geo.ctas, 1);
      const int u0 = ws.prefix[s] + (h * kv4_blocks(geo, cnt) + cb) * pages, u1 = u0 + pages;
      const int w1 = worker_of(u1 - 1, wk.W, U);
      c0 = worker_of(u0, wk.W, U);
      early = worker_begin(w1 + 1, wk.W, U) > u1;
      held = w1 - early - c0 + 1;
    }
    const int blocks = held + early, parts = blocks + (a.k.data ? (cnt + kKv4RowTile - 1) / kKv4RowTile : 0);
    // place of part p: of the CTAs, the early one, the new rows (those beyond the early one: another array)
    auto place = [&](int p) -> int64_t {
      if (p < held) return ((int64_t)c0 + p + seg) * geo.RB + rb;
      if (p < blocks) return ((int64_t)geo.ctas + geo.segments + seg) * geo.RB + rb;
      return ((int64_t)seg * geo.tiles + p - blocks) * geo.RB + rb;
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
          ml[b] = (p < blocks ? ws.ml : ws.rml)[at];
          v[b] = *reinterpret_cast<const Vec*>((p < blocks ? ws.o : ws.ro) + at * D + E * lane);
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
  const int hq = h * geo.G + r % geo.G;
  T* out = static_cast<T*>(a.out.data) + s * a.out.seq + i * a.out.row + hq * a.out.head + E * lane;
#pragma unroll
  for (int e = 0; e < E; ++e) kv8_store(out + e, l == 0.0f ? 0.0f : sum[e] / l);
}

template <typename T, int D>
cudaError_t wide_run(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo, const Kv4Scratch& ws, cudaStream_t st) {
  using C = Wide<T, D>;
  const size_t smem = 1024 + C::sPrefix + 4 * ((size_t)c.n_seqs + 1);
  cudaError_t e = kv8_smem<k_kv4_wide<T, D>>(1024 + C::sPrefix + 4 * (kKv8MaxSeqs + 1));
  if (e != cudaSuccess) return e;
  static_assert(sizeof(RowsSmem<D>) <= C::sPrefix, "new rows");
  e = launch_pdl(k_kv4_wide<T, D>, dim3((unsigned)(geo.ctas + geo.folded)), dim3(kWideThreads), smem, st, c, a, geo, ws);
  if (e != cudaSuccess) return e;
  if (geo.tiles && !geo.folded) {
    e = kv8_smem<k_kv4_rows<T, D>>(sizeof(RowsSmem<D>));
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_kv4_rows<T, D>, dim3((unsigned)kv4_rows_blocks(c, geo)), dim3(kRowsThreads),
                   sizeof(RowsSmem<D>), st, c, a, geo, ws);
    if (e != cudaSuccess) return e;
  }
  // Warps of a row: two where there are many segments of few parts, else all eight of a CTA
  const int rows = geo.R < geo.RB ? geo.R : geo.RB, rpc = geo.segments < kKv4Ctas ? 4 : 8;
  const dim3 grid((unsigned)geo.segments, (unsigned)((rows + rpc - 1) / rpc));
  return launch_pdl(rpc == 4 ? k_kv4_join<T, D, 4> : k_kv4_join<T, D, 8>, grid, dim3(32 * kJoinWarps), 0, st, c, a, geo, ws);
}

}  // namespace

cudaError_t kv4_wide(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo, const Kv4Scratch& ws, cudaStream_t st) {
  if (a.dtype == W4A8_F32) return c.head_dim == 64 ? wide_run<float, 64>(c, a, geo, ws, st) : wide_run<float, 128>(c, a, geo, ws, st);
  return c.head_dim == 64 ? wide_run<__nv_bfloat16, 64>(c, a, geo, ws, st) : wide_run<__nv_bfloat16, 128>(c, a, geo, ws, st);
}

}  // namespace w4a8
