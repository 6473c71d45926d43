// Attention of new rows over the 8-bit key/value cache: the split kernel and its launch.
//
// For query head hq of new row i (KV head h = hq / G), over the tokens t that the row sees
//   l_t = scale q . k_t,  out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x = l log2(e), m = max x
// in one pass: for each half page the running maximum m, sum l and values O of each row become
//   m' = max(m, max x),  c = 2^(m - m'),  O = O c + s_V (P C_V),  l = l c + sum P,  P = 2^(x - m'),
// with m left alone while no x is above m + 8 (P <= 2^8 keeps its f16 range, and most half pages need no
// reduction over the lanes).
//
// Both products run transposed on the tensor cores (m16n8k16, f16): S^T = C_K Q^T and O^T = C_V^T P^T, so the
// 8-bit codes are the 16-row operand and the few query rows of a KV head fill 8-column tiles, half the padding of
// a 16-row query tile.  A page is stored in the operand's own order (the header documents it), so one 16-byte
// shared-memory load gives a lane the bytes of two k-steps, and one byte permute turns two codes into two f16:
// the byte u = code + 128 in the low half of a 16-bit lane is the subnormal u 2^-24, exact, as in the W4A8 matmul.
// bf16 calls start the accumulators at -128 2^-24 sum(q) (or sum(P)), which takes the 128 out again.  fp32 calls
// make whole numbers of the codes (the byte under the exponent of 1024, minus 1152): the tensor core aligns
// products by their exponents and drops what is below, and subnormal operands cost the sums 2^-20 of the
// largest product (outputs 1.9e-6 off in the 2-norm at 4096 tokens; 2.4e-7 with whole numbers).
//
// fp32 operands are split, q = qh + ql and P = Ph + Pl in f16: hi and lo are neighbouring columns of a tile (four
// rows to a tile instead of eight), so the accumulator pair of a thread holds both products of one row and adds
// them there.  Rows of q are scaled by a power of two, to a largest magnitude of at most 2^11; qh is the nearest
// whole number, so the sums of qh with the codes (64 dims to an accumulator) are whole numbers below 2^24 that f32 holds, and
// the tensor core's truncating additions do not touch them.  (With qh the nearest f16 the logits were off by 3e-7 relative.)
// P is scaled by 2^7.  bf16 calls take one f16 term of q (exact: eight bits) and of P (off by 2^-11 at most, in no common
// direction; the sums l are of P before that rounding): over 64 sequences outputs are 0.1658% off in the 2-norm, of which
// their own rounding to bf16 (2^-8) is 0.1652%.  A second term of P would double the products with the values.
// The transposed P fragments are made with movmatrix: no shared memory in the softmax.
//
// Work: every (sequence, KV head, block of rows) is a segment of pages.  The pages of all segments, end to end, are
// cut into equal ranges, one for each worker, so ragged batches balance.  A worker is a group of WC warps that share a
// page and hold different columns; it has its own ring of bulk copies (a page each) and never waits for
// another worker.  The code of half a page is a loop of 500 instructions: unrolled over the page (1000) it outran
// the instruction caches, and twelve warps at different places of it spent a third of their time on fetches.
// The fp32 rows (open page, new rows; at most 63 + 64 of a segment) go to four further warps of each CTA, 16 tokens of
// four query rows at a time, in plain fp32: with the tensor-core form of them inside the page loop their code ran a few
// times per CTA, cold, and one worker's four row tiles took 30 us at the end of a 40 us call.  Each worker's part
// of a segment and each row tile gives (maximum, sum, values); the workers of a CTA add theirs up where they hold the
// same segment, and k_kv8_join puts the rest together.
//
// Bound: the codes once from memory when rows are few, the instructions of the conversion and the softmax when they
// are many.  Measured (join included): one row of 131071 tokens, 8 KV heads of 128, 4 query heads each, bf16, 269 MB:
// 53.7 us, 5.0 TB/s; 64 sequences of up to 8191 tokens, 646 MB: 113 us cold, 5.8 TB/s; a tree of 16 fp32 rows over 4096 tokens:
// 27.7 us, of which 13 remain at 64 tokens (launches, rows, join).
#pragma once
#include <type_traits>

#include "kv8.cuh"
#include "mma16.cuh"

namespace w4a8 {

constexpr int kKv8Ctas = 152;         // one per SM of a GB300
// Warps of a CTA (one CTA per SM, 128 registers): those that take pages and those that take fp32 rows.
constexpr int kKv8Warps = 12, kKv8RowWarps = 4, kKv8Threads = 32 * (kKv8Warps + kKv8RowWarps);
constexpr int kKv8RingBytes = 196608; // ring of pages per SM: 12 of 16 KB or 24 of 8 KB
constexpr float kPScale = 128.0f, kPSlack = 8.0f;  // scale of P; how far (log2) a logit may pass the row's maximum
constexpr int kWideRows = 128;        // query rows of a segment of a wide call (kv8_wide.cu)
constexpr int kRowTile = 16;          // fp32 rows of one part
constexpr int kRowChunk = 4;          // query rows that a row warp takes at a time
constexpr int kRowsApart = 16;        // rows of a KV head above which many parts go to a kernel of their own

struct Kv8Geom {       // of one call, the same for every kernel of it
  int n, G, R;         // new rows; query heads per KV head; query rows of a segment's problem (n G, or G with lists)
  int RB, CB;          // rows of a column block; column blocks
  int ctas, ng;        // of the split kernel, and its workers in each at most
  int tiles;           // row tiles of a segment: four of the open page, those of the new rows
  int segments;
  int apart;           // whether k_kv8_rows takes the fp32 rows, not the split kernel's row warps
  int vec;             // rows may be read 16 bytes at a time: bit 0 q, bit 1 k, bit 2 v
  int withheld;        // CTA whose pages are not copied (w4a8_kv8_attention_inject_timeout), -1: none
  uint64_t wait_ns;    // limit of the kernels' waits
};

struct Kv8Scratch {    // workspace pointers
  int* prefix;         // [n_seqs + 1] pages of the segments before each sequence
  float2* ml;          // [ctas + segments][RB] maximum, sum of the part of a (CTA, segment), at CTA + segment; then
                       // [segments][RB] of the part whose worker went on to another segment
  float* o;            // [..][RB][D] its values
  float2* rml;         // [segments][tiles][RB] maximum, sum of a row tile
  float* ro;           // [segments][tiles][RB][D] its values
  float2* fin;         // [n_seqs][n][n_heads] maximum, sum of each row (with mass)
  float2* page;        // [segments][max_pages][RB] maximum, sum of each page (with mass)
};

// Pages a segment of sequence s reads (L, cnt valid), and its row tiles: of the open page and of the new rows.
struct Kv8Units {
  int pages, open, fresh;
};
__device__ __forceinline__ Kv8Units kv8_units(const w4a8_kv8_attn& a, int L, int cnt) {
  const int whole = L / kPage;
  return {a.pages ? min(a.top_k, whole) : whole, (L % kPage + kRowTile - 1) / kRowTile,
          a.k.data ? (cnt + kRowTile - 1) / kRowTile : 0};
}
// A segment: sequence, KV head, and its column block, or its row with page lists.
struct Kv8Segment {
  int s, h, i, cb;
};
__device__ __forceinline__ Kv8Segment kv8_segment(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& g,
                                                  int seg) {
  const int H = c.n_kv_heads;
  if (a.pages) return {seg / H / a.n, seg % H, seg / H % a.n, 0};
  return {seg / g.CB / H, seg / g.CB % H, 0, seg % g.CB};
}
// Column blocks that hold rows of a sequence of cnt rows: a padded batch reads no pages for the others.
__device__ __forceinline__ int kv8_blocks(const Kv8Geom& g, int cnt) { return (cnt * g.G + g.RB - 1) / g.RB; }
// Segments of a sequence that have rows: (KV head, column block), or (row, KV head) with page lists.
__device__ __forceinline__ int kv8_segments(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& g, int cnt) {
  return c.n_kv_heads * (a.pages ? cnt : kv8_blocks(g, cnt));
}
// Pages of the segments before each sequence, [n_seqs + 1] in shared memory; the block has to be synchronised after it.
__device__ __forceinline__ void kv8_prefix(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, int* prefix) {
  const int S = c.n_seqs;
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    const int L = kv8_len(c, c.len, s), cnt = kv8_count(c, a.counts, s, a.n);
    prefix[s + 1] = L < 0 || cnt < 0 ? 0 : kv8_units(a, L, cnt).pages * kv8_segments(c, a, geo, cnt);
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int b = 0; b < S; b += 32) {
      const int s = b + threadIdx.x;
      int v = s < S ? prefix[s + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)threadIdx.x >= o) v += x;
      }
      if (s < S) prefix[s + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
}
// Two pairs of f16 operands from the four bytes of w: the subnormals u 2^-24, or the whole numbers u - 128 if WHOLE
// (1024 + u is the byte under the exponent of 1024).
template <bool WHOLE>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = __byte_perm(w, WHOLE ? 0x64646464u : 0u, 0x4140);
  hi = __byte_perm(w, WHOLE ? 0x64646464u : 0u, 0x4342);
  if (WHOLE) {
    const __half2 b = __float2half2_rn(1152.0f);
    const __half2 l = __hsub2(*reinterpret_cast<__half2*>(&lo), b), h = __hsub2(*reinterpret_cast<__half2*>(&hi), b);
    lo = *reinterpret_cast<const uint32_t*>(&l);
    hi = *reinterpret_cast<const uint32_t*>(&h);
  }
}
// ---------------------------------------------------------------------------- the split kernel

// Barrier of the page warps (the first of a CTA).
__device__ __forceinline__ void page_warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kKv8Warps) : "memory"); }

template <typename T, int D, int WC>
struct Kv8Split {
  static constexpr bool SPLIT = sizeof(T) == 4;
  static constexpr int RPT = SPLIT ? 4 : 8;        // rows of an 8-column tile
  static constexpr int NC = SPLIT ? 1 : 2;         // rows of a thread in a tile
  static constexpr int RB = WC * RPT;              // rows of a column block
  static constexpr int NG = kKv8Warps / WC;        // workers of a CTA
  static constexpr int PAGE = 2 * kPage * D;       // bytes of a ring entry: keys and values of a page
  static constexpr int NS = kKv8RingBytes / PAGE / NG;  // ring entries of a worker
  static constexpr int KS = D / 16, DT = D / 16;
  static constexpr float UNIT = SPLIT ? 1.0f : 16777216.0f;  // codes enter the products divided by this
};

// What a lane knows of one page of its worker's range.
struct Kv8Unit {
  int src;      // (pair, physical page), or -1: nothing to read
  int seg;      // segment
  int u;        // unit inside the segment
  float sk, sv;
};

// One part in plain fp32: the 16 (or fewer) fp32 rows of tile f of a segment for kRowChunk of its query rows, by one
// warp.  A lane holds its dims of the 16 keys, then of the 16 values, in registers, and its dims of the query rows; the
// 16 dot products of a row are summed over the lanes in 16 exchanges that leave token lane / 2 in each lane.  A
// token that a row does not see is left out of its sums, whatever it holds.  Beside the page warps a load takes
// microseconds, so everything is asked for at once (the values into L2).  
template <typename T, int D>
__device__ void kv8_row_part(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws,
                             int seg, int f, int chunk, float (*pt)[kRowTile]) {
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int E = D / 32;
  using Vec = std::conditional_t<E == 4, float4, float2>;
  const int lane = threadIdx.x & 31;
  const Kv8Segment sg = kv8_segment(c, a, geo, seg);
  const int L = __ldcg(c.len + sg.s), cnt = a.counts ? __ldcg(a.counts + sg.s) : a.n;
  if (L < 0 || L > kPage * c.max_pages + kPage - 1 || cnt <= 0 || cnt > a.n || (a.pages && sg.i >= cnt)) return;
  const int fresh = f - kPage / kRowTile;
  const int nv = min(kRowTile, fresh < 0 ? L % kPage - f * kRowTile : a.k.data ? cnt - fresh * kRowTile : 0);
  const int rows = min(geo.RB, (a.pages ? geo.G : cnt * geo.G) - sg.cb * geo.RB);  // of this column block
  const int r0 = chunk * kRowChunk, nr = min(rows - r0, kRowChunk);
  if (nv <= 0 || nr <= 0) return;
  const float* kt = c.tail + kv8_pair(c, sg.s, sg.h) * 2 * kPage * D + f * kRowTile * D + E * lane;
  const T* kn = static_cast<const T*>(a.k.data) + sg.s * a.k.seq + sg.h * a.k.head + (int64_t)fresh * kRowTile * a.k.row + E * lane;
  const T* vn = static_cast<const T*>(a.v.data) + sg.s * a.v.seq + sg.h * a.v.head + (int64_t)fresh * kRowTile * a.v.row + E * lane;
  float kv[kRowTile][E];
  auto load16 = [&](const float* tail, const T* rows16, int64_t step) {
#pragma unroll
    for (int i = 0; i < kRowTile; ++i) {
      Vec v = {};
      float* ve = reinterpret_cast<float*>(&v);
      if (i < nv) {
        if (fresh < 0) {
          v = __ldcg(reinterpret_cast<const Vec*>(tail + i * D));
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) ve[e] = kv8_float(__ldcg(rows16 + (int64_t)i * step + e));
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) kv[i][e] = ve[e];
    }
  };
  if (lane < nv) {  // the values' lines on their way, a lane a row
    const char* p = fresh < 0 ? reinterpret_cast<const char*>(kt - E * lane + (kPage + lane) * D)
                              : reinterpret_cast<const char*>(vn - E * lane + (int64_t)lane * a.v.row);
#pragma unroll
    for (int x = 0; x < D * (int)sizeof(float); x += 128)
      if (fresh < 0 || x < D * (int)sizeof(T)) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + x));
  }
  // query row r of the chunk: its place in the column block's rows is r0 + r
  auto node_of = [&](int r) { return a.pages ? sg.i : (sg.cb * geo.RB + r0 + r) / geo.G; };
  auto query = [&](int r, float (&q)[E]) {
    const int rr = sg.cb * geo.RB + r0 + r, hq = sg.h * geo.G + (a.pages ? rr : rr % geo.G);
    const T* p = static_cast<const T*>(a.q.data) + sg.s * a.q.seq + node_of(r) * a.q.row + hq * a.q.head + E * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = kv8_float(__ldcg(p + e));
  };
  // two rows at a time, the next two on their way: a row's chain of exchanges leaves room for another's
  float q[2][E], next[2][E];
  query(0, q[0]);
  query(min(1, nr - 1), q[1]);
  load16(kt, kn, a.k.row);
  const float qscale = a.scale * 1.4426950408889634f;
  const int tok = lane >> 1;
  const size_t at = ((size_t)seg * geo.tiles + f) * geo.RB + r0;
#pragma unroll 1
  for (int r = 0; r < nr; r += 2) {
    query(min(r + 2, nr - 1), next[0]);
    query(min(r + 3, nr - 1), next[1]);
    float x[2][kRowTile];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
#pragma unroll
      for (int i = 0; i < kRowTile; ++i) x[y][i] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int i = 0; i < kRowTile; ++i) x[y][i] = fmaf(q[y][e], kv[i][e], x[y][i]);
        q[y][e] = next[y][e];
      }
    }
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
      const bool up = lane & (2 * w);
#pragma unroll
      for (int i = 0; i < w; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float keep = up ? x[y][i + w] : x[y][i], give = up ? x[y][i] : x[y][i + w];
          x[y][i] = keep + __shfl_xor_sync(FULL, give, 2 * w);
        }
    }
    float s[2], m[2], l[2];
    bool see[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      s[y] = (x[y][0] + __shfl_xor_sync(FULL, x[y][0], 1)) * qscale;
      see[y] = tok < nv;
      if (fresh >= 0) {
        const int i = node_of(min(r + y, nr - 1));
        const uint64_t mask = a.mask ? __ldcg(a.mask + (size_t)sg.s * a.n + i) : (i >= 63 ? ~0ull : (1ull << (i + 1)) - 1ull);
        see[y] = see[y] && (mask >> (fresh * kRowTile + tok) & 1ull);
      }
      m[y] = see[y] ? s[y] : -INFINITY;
    }
#pragma unroll
    for (int w = 16; w > 1; w >>= 1)
#pragma unroll
      for (int y = 0; y < 2; ++y) m[y] = fmaxf(m[y], __shfl_xor_sync(FULL, m[y], w));
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const float p = see[y] ? ex2(s[y] - (m[y] == -INFINITY ? 0.0f : m[y])) : 0.0f;
      l[y] = p;
      if (!(lane & 1) && r + y < nr) pt[r + y][tok] = see[y] ? p : -1.0f;
    }
#pragma unroll
    for (int w = 2; w < 32; w <<= 1)
#pragma unroll
      for (int y = 0; y < 2; ++y) l[y] += __shfl_xor_sync(FULL, l[y], w);
    if (lane < 2 && r + lane < nr) ws.rml[at + r + lane] = lane ? make_float2(m[1], l[1]) : make_float2(m[0], l[0]);
  }
  load16(kt + kPage * D, vn, a.v.row);
  __syncwarp();
#pragma unroll 1
  for (int r = 0; r < nr; ++r) {
    float o[E] = {};
#pragma unroll
    for (int i = 0; i < kRowTile; ++i) {
      const float p = pt[r][i];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = p != -1.0f ? fmaf(p, kv[i][e], o[e]) : o[e];
    }
    *reinterpret_cast<Vec*>(ws.ro + (at + r) * D + E * lane) = *reinterpret_cast<Vec*>(o);
  }
  __syncwarp();
}

template <typename T, int D, int WC>
__global__ void __launch_bounds__(kKv8Threads, 1) k_kv8_split(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo,
                                                               Kv8Scratch ws) {
  using C = Kv8Split<T, D, WC>;
  constexpr bool SPLIT = C::SPLIT;
  constexpr int NC = C::NC, KS = C::KS, DT = C::DT;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(16) float row_p[kKv8RowWarps][kRowChunk][kRowTile];
  __shared__ int cut;  // whether a wait of the CTA ran out
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kKv8RingBytes);
  uint64_t* empty = full + C::NG * C::NS;
  int* prefix = reinterpret_cast<int*>(empty + C::NG * C::NS);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp / WC, wg = warp % WC;  // worker of the CTA, warp of the worker
  const int g = lane >> 2, t = lane & 3;
  const int H = c.n_kv_heads, S = c.n_seqs;

  if (tid == 0) cut = 0;
  for (int i = tid; i < C::NG * C::NS; i += kKv8Threads) {
    mbar_init(&full[i], 1);
    mbar_init(&empty[i], WC);
  }
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  griddep_enter();

  kv8_prefix(c, a, geo, prefix);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int s = tid; s <= S; s += kKv8Threads) ws.prefix[s] = prefix[s];

  if (warp >= kKv8Warps) {  // fp32 rows: parts dealt over the row warps of all CTAs
    if (geo.apart) return;
    const int chunks = (min(geo.R, C::RB) + kRowChunk - 1) / kRowChunk;
    const int parts = geo.segments * geo.tiles * chunks;
    for (int x = (warp - kKv8Warps) * gridDim.x + blockIdx.x; x < parts; x += gridDim.x * kKv8RowWarps)
      kv8_row_part<T, D>(c, a, geo, ws, x / chunks / geo.tiles, x / chunks % geo.tiles, x % chunks,
                         row_p[warp - kKv8Warps]);
    return;
  }
  const int U = prefix[S];
  const Kv8Workers wk = kv8_workers(U, geo.ctas, C::NG);
  const int worker = blockIdx.x * wk.ng + grp;
  const bool has = grp < wk.ng && worker < wk.W;
  const int u0 = has ? worker_begin(worker, wk.W, U) : 0, u1 = has ? worker_begin(worker + 1, wk.W, U) : 0;

  // The lane's unit x: its segment, page and scales (32 units in parallel, so the table's latency is paid once).
  auto look = [&](int x) -> Kv8Unit {
    Kv8Unit r{-1, -1, 0, 0.0f, 0.0f};
    if (x >= u1) return r;
    int lo = 0, hi = S - 1;  // the last sequence whose first unit is at or before x and that has units
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    const int s = lo, cnt = a.counts ? a.counts[s] : a.n;
    const Kv8Units un = kv8_units(a, c.len[s], cnt);
    const int per = un.pages, q = (x - prefix[s]) / per, u = (x - prefix[s]) % per;
    const int blocks = kv8_blocks(geo, cnt), h = a.pages ? q % H : q / blocks;
    r.seg = a.pages ? s * a.n * H + q : (s * H + h) * geo.CB + q % blocks;
    r.u = u;
    const size_t pair = kv8_pair(c, s, h);
    int p = u;
    if (a.pages) {
      const int32_t* list = a.pages + (size_t)r.seg * a.top_k;
      p = list[u];
      const int before = u > 0 ? list[u - 1] : -2;
      if (p == -1) return r;
      if (p < 0 || p >= c.len[s] / kPage || (u > 0 && (before < 0 || before >= p))) {
        atomicOr(c.ctl, (unsigned)FLAG_ERR_TREE);
        return r;
      }
    }
    const int phys = kv8_phys(c, pair, p);
    if (phys < 0) return r;
    r.src = (int)kv8_page(c, pair, phys);
    const float2 sc = *reinterpret_cast<const float2*>(c.scales + (size_t)r.src * 2);
    r.sk = sc.x;
    r.sv = sc.y;
    return r;
  };

  uint8_t* ring = sm + (size_t)grp * C::NS * C::PAGE;
  full += grp * C::NS;
  empty += grp * C::NS;
  Kv8Unit cur = look(u0 + lane), nxt = look(u0 + 32 + lane);
  const int nu = u1 - u0;
  int jl = 0;                           // next unit to copy (one warp of the worker copies)
  int is = 0, iph = 0, in_ring = 0;     // its ring entry and that one's phase; entries issued and not consumed
  int cs = 0, cph = 0;                  // entry to consume next
  bool ok = true;

  // ---- state of the segment
  uint32_t qf[KS][2];
  float O[DT][4], m[NC], l[NC], colfac[NC], collow[NC], seed[2];
  int seg = -1, s_cur = 0, h_cur = 0, i_cur = 0, cb_cur = 0, cnt_cur = 0;
  bool act = false;
  // the factor of a column, log2(e) scale UNIT / (power of two of its row), as hi + lo
  const double lscale = (double)a.scale * 1.4426950408889634 * (double)C::UNIT;
  const float lhi = (float)lscale, llo = (float)(lscale - (double)lhi);
  auto row_of = [&](int col) {  // query row (of the segment's R) of column col of the warp's tile
    return cb_cur * C::RB + wg * C::RPT + (SPLIT ? col >> 1 : col);
  };
  auto row_ok = [&](int r) { return r < geo.R && (a.pages || r / geo.G < cnt_cur); };
  auto row_node = [&](int r) { return a.pages ? i_cur : r / geo.G; };
  auto row_head = [&](int r) { return h_cur * geo.G + (a.pages ? r : r % geo.G); };

  auto begin = [&](int sg) {
    const Kv8Segment w = kv8_segment(c, a, geo, sg);
    seg = sg;
    s_cur = w.s, h_cur = w.h, i_cur = w.i, cb_cur = w.cb;
    cnt_cur = a.counts ? a.counts[s_cur] : a.n;
    act = row_ok(cb_cur * C::RB + wg * C::RPT);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[d][e] = 0.0f;
#pragma unroll
    for (int x = 0; x < NC; ++x) m[x] = -INFINITY, l[x] = 0.0f;
    const int r = row_of(g);
    float v[KS * 4];
    if (row_ok(r)) {
      const T* q = static_cast<const T*>(a.q.data) + s_cur * a.q.seq + row_node(r) * a.q.row + row_head(r) * a.q.head;
#pragma unroll
      for (int kp = 0; kp < D / 32; ++kp) {
        const T* p = q + 32 * kp + 8 * t;
        if (geo.vec & 1) {
          uint4 w[sizeof(T) / 2];
#pragma unroll
          for (int x = 0; x < (int)sizeof(T) / 2; ++x) w[x] = reinterpret_cast<const uint4*>(p)[x];
          const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
          for (int x = 0; x < 8; ++x) v[8 * kp + x] = kv8_load(e + x);
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) v[8 * kp + x] = kv8_load(p + x);
        }
      }
    } else {
#pragma unroll
      for (int x = 0; x < KS * 4; ++x) v[x] = 0.0f;
    }
    float am = 0.0f;
#pragma unroll
    for (int x = 0; x < KS * 4; ++x) am = max_nan(am, fabsf(v[x]));
    am = max_nan(am, __shfl_xor_sync(FULL, am, 1));
    am = max_nan(am, __shfl_xor_sync(FULL, am, 2));
    const float up = f16_scale(am);
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = v[4 * x + e] * up;
        if (SPLIT) f[e] = g & 1 ? f[e] - rintf(f[e]) : rintf(f[e]);
        if (!SPLIT) sum += __half2float(__float2half_rn(f[e]));
      }
      qf[x][0] = pack_f16(f[0], f[1]);
      qf[x][1] = pack_f16(f[2], f[3]);
    }
    // per-column values, from the lanes of column g to the lanes of accumulator columns 2t, 2t + 1
    const float down = 1.0f / up;
    if (SPLIT) {
      const float dn = __shfl_sync(FULL, down, 8 * t);
      colfac[0] = lhi * dn;
      collow[0] = llo * dn;
      seed[0] = seed[1] = 0.0f;
    } else {
      sum += __shfl_xor_sync(FULL, sum, 1);
      sum += __shfl_xor_sync(FULL, sum, 2);
      sum *= -128.0f / 16777216.0f;
#pragma unroll
      for (int x = 0; x < NC; ++x) {
        const float dn = __shfl_sync(FULL, down, 4 * (2 * t + x));
        colfac[x] = lhi * dn;
        collow[x] = llo * dn;
        seed[x] = __shfl_sync(FULL, sum, 4 * (2 * t + x));
      }
    }
  };

  // The worker's part of a segment (P carries kPScale, the codes 1 / UNIT) to rows of (ml, o).
  auto flush = [&](float2* ml, float* out) {
    if (!act) return;
#pragma unroll
    for (int x = 0; x < NC; ++x) {
      float sum = l[x];
      sum += __shfl_xor_sync(FULL, sum, 4);
      sum += __shfl_xor_sync(FULL, sum, 8);
      sum += __shfl_xor_sync(FULL, sum, 16);
      const int r = wg * C::RPT + (SPLIT ? t : 2 * t + x);  // of the column block
      if (!row_ok(cb_cur * C::RB + r)) continue;
      if (g == 0) ml[r] = make_float2(m[x], sum / kPScale);
      float* o = out + r * D;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        o[16 * d + g] = (SPLIT ? O[d][0] + O[d][1] : O[d][x]) * (C::UNIT / kPScale);
        o[16 * d + g + 8] = (SPLIT ? O[d][2] + O[d][3] : O[d][x + 2]) * (C::UNIT / kPScale);
      }
    }
  };

  // A page, half of it (32 tokens) at a time: S^T = C_K Q^T, softmax, O^T += C_V^T P^T.  The logit is x (fh + fl), in
  // fp32 calls taken relative to the maximum with one rounding at the size of the difference: a relative error of a
  // factor is one of the softmax's temperature, which large logits multiply.
  auto page = [&](const uint8_t* pg, float sk, float sv, int u) {
    float fh[NC], fl[NC], psum[NC];
#pragma unroll
    for (int y = 0; y < NC; ++y) {
      fh[y] = colfac[y] * sk;
      fl[y] = fmaf(colfac[y], sk, -fh[y]) + collow[y] * sk;
      psum[y] = 0.0f;
    }
#pragma unroll 1
    for (int it = 0; it < 2; ++it) {
      float x[2][4], x1[2][4];  // two 16-token tiles, even and odd k-steps
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = SPLIT ? 0.0f : seed[e & 1], x1[i][e] = 0.0f;
      const uint8_t* kb = pg + (it * (D / 16) * 32 + lane) * 16;
#pragma unroll
      for (int kp = 0; kp < D / 32; ++kp)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(kb + (i * (D / 32) + kp) * 512);
          uint32_t af[4];
          codes_f16<SPLIT>(w.x, af[0], af[2]);
          codes_f16<SPLIT>(w.y, af[1], af[3]);
          mma_f16(x[i], af, qf[2 * kp][0], qf[2 * kp][1]);
          codes_f16<SPLIT>(w.z, af[0], af[2]);
          codes_f16<SPLIT>(w.w, af[1], af[3]);
          mma_f16(x1[i], af, qf[2 * kp + 1][0], qf[2 * kp + 1][1]);
        }
      // logits: entry y + 2 e of tile i is row y of the thread, token g + 8 e of the tile
      bool high = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] += x1[i][e];
        if (SPLIT) x[i][0] += x[i][1], x[i][2] += x[i][3];  // hi + lo
#pragma unroll
        for (int y = 0; y < NC; ++y) high = high || x[i][y] * fh[y] > m[y] + kPSlack || x[i][y + 2] * fh[y] > m[y] + kPSlack;
      }
      if (__any_sync(FULL, high)) {
        float cc[NC];
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          float mx = fmaxf(fmaxf(x[0][y] * fh[y], x[0][y + 2] * fh[y]), fmaxf(x[1][y] * fh[y], x[1][y + 2] * fh[y]));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
          mx = fmaxf(mx, m[y]);
          cc[y] = mx == -INFINITY ? 1.0f : ex2(m[y] - mx);
          m[y] = mx;
          l[y] *= cc[y];
          psum[y] *= cc[y];
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[d][e] *= cc[(e & 1) * (NC - 1)];
      }
      uint32_t pf[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          const float base = m[y] == -INFINITY ? 0.0f : m[y];
#pragma unroll
          for (int e = y; e < 4; e += 2) {
            x[i][e] = SPLIT ? ex2(fmaf(x[i][e], fl[y], fmaf(x[i][e], fh[y], -base))) * kPScale
                            : ex2(fmaf(x[i][e], fh[y], 7.0f - base));
            psum[y] += x[i][e];
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = x[i][2 * e];
          pf[i][e] = movmatrix(SPLIT ? pack_f16(p, p - __half2float(__float2half_rn(p))) : pack_f16(p, x[i][2 * e + 1]));
        }
      }
      // bf16 calls: -128 2^-24 sum(P) of the columns, P as the product uses it, by a row of constants times P
      float ps[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (!SPLIT) {
        const uint32_t k = 0x80808080u;  // f16 -128 2^-24 = 0x8080
        const uint32_t ones[4] = {k, k, k, k};
        mma_f16(ps, ones, pf[0][0], pf[0][1]);
        mma_f16(ps, ones, pf[1][0], pf[1][1]);
      }
      const uint8_t* vb = pg + kPage * D + (it * 32 + lane) * 16;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        float o[4] = {ps[0], ps[1], ps[2], ps[3]};
        const uint4 w = *reinterpret_cast<const uint4*>(vb + d * 1024);
        uint32_t af[4];
        codes_f16<SPLIT>(w.x, af[0], af[2]);
        codes_f16<SPLIT>(w.y, af[1], af[3]);
        mma_f16(o, af, pf[0][0], pf[0][1]);
        codes_f16<SPLIT>(w.z, af[0], af[2]);
        codes_f16<SPLIT>(w.w, af[1], af[3]);
        mma_f16(o, af, pf[1][0], pf[1][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) O[d][e] = fmaf(o[e], sv, O[d][e]);
      }
    }
#pragma unroll
    for (int y = 0; y < NC; ++y) {
      l[y] += psum[y];
      if (ws.page) {
        float v = psum[y];
        v += __shfl_xor_sync(FULL, v, 4);
        v += __shfl_xor_sync(FULL, v, 8);
        v += __shfl_xor_sync(FULL, v, 16);
        if (g == 0)
          ws.page[((size_t)seg * c.max_pages + u) * C::RB + wg * C::RPT + (SPLIT ? t : 2 * t + y)] =
              make_float2(m[y] == -INFINITY ? 0.0f : m[y], v / kPScale);
      }
    }
  };

  // ---- the range
#pragma unroll 1
  for (int j = 0, cbase = 0; j < nu; ++j) {
    if (j - cbase == 32) {
      cbase += 32;
      cur = nxt;
      nxt = look(u0 + cbase + 32 + lane);
    }
    if (wg == 0) {  // copy ahead as far as the ring and the two batches of units allow
      while (in_ring < C::NS && jl < nu && jl < cbase + 64) {
        const int from = __shfl_sync(FULL, jl < cbase + 32 ? cur.src : nxt.src, (jl - cbase) & 31);
        ++jl;
        if (from < 0) continue;
        if (lane == 0) {
          if (WC > 1 && iph > 0) ok = mbar_wait(&empty[is], (iph - 1) & 1, geo.wait_ns);
          if (ok) {
            mbar_expect_tx(&full[is], C::PAGE);
            if (geo.withheld != (int)blockIdx.x)
              bulk_g2s(ring + (size_t)is * C::PAGE, c.codes + (size_t)from * C::PAGE, C::PAGE, &full[is]);
          }
        }
        ok = __shfl_sync(FULL, ok, 0);
        if (!ok) break;
        ++in_ring;
        if (++is == C::NS) is = 0, ++iph;
      }
      if (!ok) break;
    }
    const int src = j - cbase;
    const int from = __shfl_sync(FULL, cur.src, src), sg = __shfl_sync(FULL, cur.seg, src);
    if (sg != seg) {
      if (seg >= 0) {
        const size_t at = ((size_t)geo.ctas + geo.segments + seg) * C::RB;
        flush(ws.ml + at, ws.o + at * D);
      }
      begin(sg);
    }
    const float sk = __shfl_sync(FULL, cur.sk, src), sv = __shfl_sync(FULL, cur.sv, src);
    const int u = __shfl_sync(FULL, cur.u, src);
    if (from < 0) continue;
    ok = __all_sync(FULL, mbar_wait(&full[cs], cph & 1, geo.wait_ns));
    if (!ok) break;
    if (act) page(ring + (size_t)cs * C::PAGE, sk, sv, u);
    __syncwarp();
    if (WC > 1 && lane == 0) mbar_arrive(&empty[cs]);
    if (++cs == C::NS) cs = 0, ++cph;
    --in_ring;
  }
  if (!ok) {  // a bounded wait expired: report it, and wait (again bounded) for the copies still in flight
    if (lane == 0) cut = 1, atomicOr(c.ctl, (unsigned)FLAG_ERR_TIMEOUT);
    if (wg == 0)
      for (; in_ring > 0; --in_ring) {
        (void)mbar_wait(&full[cs], cph & 1, geo.wait_ns);
        if (++cs == C::NS) cs = 0, ++cph;
      }
  }
  // ---- the workers' last parts, in the ring's place, and of each run of workers on one segment the sum
  float2* sml = reinterpret_cast<float2*>(sm);                       // [NG][RB]
  int* sseg = reinterpret_cast<int*>(sml + C::NG * C::RB);           // [NG], -1: none
  float* so = reinterpret_cast<float*>(sm) + ((C::NG * (2 * C::RB + 1) + 31) & ~31);  // [NG][RB][D]
  page_warps_sync();
  if (lane == 0 && wg == 0) sseg[grp] = ok && has ? seg : -1;
  if (ok && has && seg >= 0) flush(sml + grp * C::RB, so + grp * C::RB * D);
  page_warps_sync();
  for (int i0 = 0; i0 < C::NG;) {
    const int sg = sseg[i0];
    int i1 = i0 + 1;
    while (i1 < C::NG && sseg[i1] == sg) ++i1;
    if (sg >= 0) {
      const Kv8Segment w = kv8_segment(c, a, geo, sg);
      const int cnt = a.counts ? a.counts[w.s] : a.n;
      const int rows = min(C::RB, (a.pages ? geo.G : cnt * geo.G) - w.cb * C::RB);
      const size_t at = ((size_t)blockIdx.x + sg) * C::RB;
      for (int x = tid; x < rows * (D / 4); x += 32 * kKv8Warps) {
        const int r = x / (D / 4), d = x % (D / 4);
        float M = -INFINITY, L = 0.0f;
        for (int i = i0; i < i1; ++i) M = fmaxf(M, sml[i * C::RB + r].x);
        const float base = M == -INFINITY ? 0.0f : M;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = i0; i < i1; ++i) {
          const float2 ml = sml[i * C::RB + r];
          const float4 o = reinterpret_cast<const float4*>(so + (i * C::RB + r) * D)[d];
          const float f = ex2(ml.x - base);
          L = fmaf(ml.y, f, L);
          v.x = fmaf(o.x, f, v.x), v.y = fmaf(o.y, f, v.y), v.z = fmaf(o.z, f, v.z), v.w = fmaf(o.w, f, v.w);
        }
        reinterpret_cast<float4*>(ws.o + (at + r) * D)[d] = v;
        if (d == 0) ws.ml[at + r] = make_float2(M, L);
      }
    }
    i0 = i1;
  }
  if (cut) {  // the CTA's parts are not what they should be: NaN, for the join to pass on
    page_warps_sync();
    const int last = u1 > u0 ? look(u1 - 1).seg : -1;
    for (int x = u0 + lane; x < u1; x += 32) {
      const int sg = look(x).seg;
      const size_t at = ((size_t)sg + (sg == last ? blockIdx.x : (size_t)geo.ctas + geo.segments)) * C::RB;
      for (int r = 0; r < C::RB; ++r) ws.ml[at + r] = make_float2(NAN, NAN);
    }
  }
}

// ---------------------------------------------------------------------------- launch

// Warps on a page for R query rows of a problem, a tile each (four rows of fp32, eight of bf16): the number up to four
// that leaves none idle over the column blocks; the largest of them (fewer reads of a page).  With six and
// twelve allowed as well, 96 bf16 rows at 2048 tokens took 28.5 us instead of 18.4 (few workers, each with pages of two
// segments one after the other), and no length gained.  Where only one divides the tiles, the fewer blocks of three or four
// warps, some idle, win as often as they lose; fp32, 8 KV heads of 128, one warp / the best of three and four, us:
//   20 rows: 1024 tokens 13.0 / 13.5, 16384 tokens 25.6 / 26.7; 16 sequences of up to 1024 39.5 / 36.4, of 16384 158 / 155
//   28 rows: 1024 tokens 13.7 / 14.1, 16384 tokens 30.7 / 33.1; 16 sequences of up to 1024 45.4 / 41.3, of 16384 220 / 208
//   44 rows: 1024 tokens 14.0 / 14.4, 4096 tokens 21.5 / 19.5;  16 sequences of up to 1024 53.6 / 49.2, of 4096 99.5 / 99.2
inline int kv8_split_warps(int R, int dtype) {
  const int rpt = dtype == W4A8_F32 ? 4 : 8, tiles = (R + rpt - 1) / rpt;
  int best = 1;
  for (int wc : {2, 3, 4})
    if ((tiles + wc - 1) / wc * wc <= (tiles + best - 1) / best * best) best = wc;
  return best;
}

inline size_t kv8_split_smem(int S, int entries) { return (size_t)kKv8RingBytes + 16 * (size_t)entries + 4 * ((size_t)S + 1); }

template <typename T, int D, int WC>
cudaError_t kv8_split_launch(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws,
                             cudaStream_t st) {
  using C = Kv8Split<T, D, WC>;
  const size_t most = kv8_split_smem(kKv8MaxSeqs, C::NG * C::NS), smem = kv8_split_smem(c.n_seqs, C::NG * C::NS);
  cudaError_t e = kv8_smem<k_kv8_split<T, D, WC>>(most);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_kv8_split<T, D, WC>, dim3((unsigned)geo.ctas), dim3(kKv8Threads), smem, st, c, a,
                    geo, ws);
}
template <typename T, int D>
cudaError_t kv8_split_dispatch(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws,
                               cudaStream_t st) {
  switch (kv8_split_warps(geo.R, a.dtype)) {
    case 1: return kv8_split_launch<T, D, 1>(c, a, geo, ws, st);
    case 2: return kv8_split_launch<T, D, 2>(c, a, geo, ws, st);
    case 3: return kv8_split_launch<T, D, 3>(c, a, geo, ws, st);
    default: return kv8_split_launch<T, D, 4>(c, a, geo, ws, st);
  }
}
// Calls whose KV heads have many query rows run on tcgen05 (kv8_wide.cu): more than 128 rows, or more than 32 and
// 2^21 tile-page-dims of room (the lengths are not known here).  Measured with full caches of 8 KV heads, split / wide
// kernel, us.  Heads of 128, fp32: 32 rows, 32768 tokens 59.6 / 65.0; 64 rows, 4096 tokens 28.2 / 28.4 and 8192 tokens
// 39.1 / 33.6; 128 rows, 2048 tokens 26.6 / 34.7, 4096 tokens 37.9 / 37.6 and 16384 tokens 110 / 55.5; 144 rows, 2048
// tokens 28.9 / 33.1 and 8192 tokens 68.5 / 50.7.  bf16: 96 rows, 8192 tokens 30.6 / 34.7 and 16384 tokens 47.3 / 41.2;
// 128 rows, 8192 tokens 37.4 / 36.7; 144 rows, 512 tokens 29.5 / 25.3 and 8192 tokens 40.1 / 38.6.  Heads of 64, fp32, 64
// rows: 8192 tokens 26.6 / 26.3 and 16384 tokens 40.8 / 36.0.
inline bool kv8_is_wide(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, int R) {
  if (a.pages) return false;
  const int64_t rpt = a.dtype == W4A8_F32 ? 4 : 8, tiles = (R + rpt - 1) / rpt;
  return R > kWideRows || (R > 32 && tiles * c.n_seqs * c.n_kv_heads * c.max_pages * c.head_dim >= 1 << 21);
}
cudaError_t kv8_wide(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
cudaError_t kv8_rows(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
// one translation unit per head size and element type
cudaError_t kv8_split_f32_d64(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
cudaError_t kv8_split_f32_d128(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
cudaError_t kv8_split_bf16_d64(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
cudaError_t kv8_split_bf16_d128(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);

}  // namespace w4a8
