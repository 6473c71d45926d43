// Attention of new rows over the 4-bit key/value cache: the split kernel, its join and its launch.
//
// For query head hq of new row i (KV head h = hq / G), over the tokens t that the row sees
//   l_t = scale q . k_t,  out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x = l log2(e), m = max x
// in one pass: for each half page the running maximum m, sum l and values O of each row become
//   m' = max(m, max x),  c = 2^(m - m'),  O = O c + P V,  l = l c + sum P,  P = 2^(x - m'),
// with m left alone while no x is above m + 8 (P 2^7 keeps its f16 range, and most half pages need no reduction over the lanes).
//
// Both products run transposed on the tensor cores (m16n8k16, f16): S^T = K Q^T and O^T = V^T P^T, so the cache is the 16-row
// operand and the few query rows of a KV head fill 8-column tiles.  A page is stored in the operand's own order (the
// header documents it): one 16-byte shared-memory load gives a lane the codes of four k-steps.  A 4-bit code under the right
// exponent is an f16 number, 256 + u or 16 + u, and one fused multiply-add per two codes makes the cached value of it:
// (256 + u) s - 264 s = (u - 8) s, exact, as 264 s has nine bits, 24 s five and the value seven.  So the scales cost nothing
// behind the products, and a warp's two column tiles share the conversion.
//
// fp32 operands are split, q = qh + ql and P = Ph + Pl in f16: hi and lo are neighbouring columns of a tile (four rows to a
// tile instead of eight), so the accumulator pair of a thread holds both products of one row and adds them there.
// Rows of q are scaled by a power of two, to a largest magnitude of at most 2^11; qh is the nearest whole number, so a sum of
// qh with the codes of one scale (32 dims to an accumulator) is a multiple of the scale's last bit below 2^24 of them: f32
// holds it, and the tensor core's truncating additions do not touch it.  The groups' sums are added in fp32 outside the tensor core.
// bf16 calls take one f16 term of q (exact: eight bits) and of P (2^-11, an eighth of their outputs' own rounding).  In either type the values of a half page are added up
// in fp32 outside the tensor core, whose additions are truncated: left in its accumulator, every 16 tokens took up to 2^-23 of the
// sum (0.6% of the values of a warp that went through 16384 pages; 1 to 2% of a call's time).
//
// Work: every (sequence, KV head, block of rows) is a segment of units: its new rows, then pages (one empty unit where there
// is nothing).  The units of all segments, end to end, are cut into equal ranges, one for each pair of warps, so ragged batches
// balance.  Few units go to few CTAs, a pair each (129 units of one row to 17 CTAs instead of 129: 12 us for 21, the parts that are
// left to join are an eighth).  A pair has its own ring of whole pages, one bulk copy each (four copies to half a page, the
// arithmetic left out, took 105 us of a served batch of 64 sequences, whole pages 88); a warp takes the page's tokens 0..31 or 32..63, and the one that is
// done with a ring entry last refills it, so nobody waits for the other.  The new rows are done in plain fp32, every second
// by either warp.  A segment that lies within one pair's range is finished there; the warps of a CTA add up where they
// hold the same one; and where several CTAs do, each stores its part, and the one that comes last (a ticket, which it sets back
// to zero) joins the parts in their order.  One launch: a second one costs more than the join.
#pragma once
#include <type_traits>

#include "kv4.cuh"
#include "mma16.cuh"

namespace w4a8 {

constexpr int kKv4Ctas = 152;             // one per SM of a GB300
constexpr int kKv4RingBytes = 24 * 8704;  // ring of pages per SM
constexpr int kKv4MaxWarps = 16;
constexpr int kKv4HalfTokens = 32;        // tokens of a page that a warp of a pair takes
constexpr int kKv4Lens = 1024;            // sequences whose lengths are kept in shared memory
constexpr int kKv4WideRows = 128;         // query rows of a segment of a wide call (kv4_wide.cu)
constexpr int kKv4RowTile = 16, kKv4RowsRows = 64;  // new rows and query rows of a CTA of those that do the new rows of a wide call
constexpr float kP4Scale = 128.0f, kP4Slack = 8.0f;  // scale of P; how far (log2) a logit may pass the row's maximum
static_assert(W4A8_KV4_TICKETS >= kKv4Ctas * kKv4MaxWarps * 4, "tickets");

struct Kv4Geom {       // of one call, the same for every kernel of it
  int n, G, R;         // new rows; query heads per KV head; query rows of a KV head
  int RB, CB;          // rows of a column block; column blocks
  int ctas;            // of the kernel over the pages
  int segments;
  int tiles;           // wide calls: blocks of 16 new rows
  int folded;          // CTAs behind the others of the kernel over the pages, for the new rows; 0: those are a kernel of their own
  int vec;             // rows may be read 16 bytes at a time: bit 0 q, bit 1 k, bit 2 v
  int withheld;        // CTA whose pages are not copied (w4a8_kv4_attention_inject_timeout), -1: none
  uint64_t wait_ns;    // limit of the kernels' waits
  float lhi, llo;      // log2(e) scale, as hi + lo
};
struct Kv4Scratch {    // workspace pointers
  int* ticket;         // [workers] parts of the segment that begins in a worker's range and ends in another's
  float2* ml;          // [5 workers][RB] maximum, sum of a part: of the workers of a CTA that hold the same segment, at the first
                       // of them; then, at workers + 2 w, of the two warps of worker w whose range goes on behind the segment
                       // that it began with; then, at 3 workers + 2 w, of those of a segment within the range
  float* o;            // [5 workers][RB][D] its values
  // wide calls: ml and o are [ctas + 2 segments][RB], the part of a (CTA, segment) at CTA + segment, then [segments][RB] of the
  // parts whose CTA went on to another segment
  int* prefix;         // [n_seqs + 1] pages of the segments before each sequence
  float2* rml;         // [segments][tiles][RB] maximum, sum of a block of new rows
  float* ro;           // [segments][tiles][RB][D] its values
};

// CTAs that do the new rows of a wide call.
inline int64_t kv4_rows_blocks(const w4a8_kv4_cache& c, const Kv4Geom& g) {
  return (int64_t)((g.R + kKv4RowsRows - 1) / kKv4RowsRows) * g.tiles * c.n_seqs * c.n_kv_heads;
}
// Column blocks that hold rows of a sequence of cnt rows.
__device__ __forceinline__ int kv4_blocks(const Kv4Geom& g, int cnt) { return (cnt * g.G + g.RB - 1) / g.RB; }
// Units of the segments before each sequence, [n_seqs + 1] in shared memory, units_of(L) to a segment; lens: the first kKv4Lens
// lengths (NULL: not wanted).  The block has to be synchronised after it.
template <typename F>
__device__ __forceinline__ void kv4_prefix(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo, int* prefix,
                                           int* lens, F units_of) {
  const int S = c.n_seqs;
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    const int L = kv4_len(c, c.len, s), cnt = kv4_count(c, a.counts, s, a.n);
    prefix[s + 1] = L < 0 || cnt < 0 ? 0 : units_of(L) * c.n_kv_heads * kv4_blocks(geo, cnt);
    if (lens && s < kKv4Lens) lens[s] = L;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32 && S > 1) {
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
// The sequence that unit x belongs to.
__device__ __forceinline__ int kv4_seq_of(const int* prefix, int S, int x) {
  int lo = 0, hi = S - 1;  // the last sequence whose first unit is at or before x and that has units
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Two f16 numbers of the fields of two words at bits 2..5 (256 + u) or 6..9 (16 + u).
__device__ __forceinline__ uint32_t kv4_f16_low(uint32_t w) { return and_or(w, 0x003c003cu, 0x5c005c00u); }
__device__ __forceinline__ uint32_t kv4_f16_high(uint32_t w) { return and_or(w, 0x03c003c0u, 0x4c004c00u); }
__device__ __forceinline__ uint32_t kv4_swap(uint32_t w) { return __byte_perm(w, 0, 0x2301); }
__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kMinus264 = 0xdc20dc20u, kMinus24 = 0xce00ce00u;  // f16 pairs
// f16 pair of the scale bytes i and j of w
__device__ __forceinline__ uint32_t kv4_scale_pair(uint32_t w, int i, int j) {
  return __byte_perm(w, 0, 0x4040 | i | j << 8) << 7;
}

// A pair of half h of w
__device__ __forceinline__ uint32_t twice(uint32_t w, int h) {
  const __half2 p = *reinterpret_cast<const __half2*>(&w), r = h ? __high2half2(p) : __low2half2(p);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ---------------------------------------------------------------------------- the split kernel

template <typename T, int D, int NT>
struct Kv4Split {
  static constexpr bool SPLIT = sizeof(T) == 4;
  static constexpr int RPT = SPLIT ? 4 : 8;        // rows of an 8-column tile
  static constexpr int NC = SPLIT ? 1 : 2;         // rows of a thread in a tile
  static constexpr int RB = NT * RPT;              // rows of a column block
  static constexpr int NG = NT == 1 ? 16 : 8;      // warps of a CTA: what their registers leave room for
  static constexpr int NP = NG / 2;                // workers: pairs of warps
  static constexpr int PAGE = Kv4Page<D>::BYTES;   // a ring entry
  static constexpr int NS = kKv4RingBytes / PAGE / NP;  // ring entries of a pair
  static constexpr int STEPS = D / 16;  // k-steps of the first product, 16-dim tiles of the second
  static constexpr int THREADS = 32 * NG;
};

// What a lane knows of one unit of its worker's range.
struct Kv4Unit {
  int page;  // number of the (page, head) in the pool, or -1: nothing to read
  int what;  // segment, and in the low seven bits the tokens of the page plus 1; 0 there: the unit of the new rows
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(Kv4Split<T, D, NT>::THREADS, 1)
    k_kv4_split(w4a8_kv4_cache c, w4a8_kv4_attn a, Kv4Geom geo, Kv4Scratch ws) {
  using C = Kv4Split<T, D, NT>;
  constexpr bool SPLIT = C::SPLIT;
  constexpr int NC = C::NC, KS = C::STEPS, DT = C::STEPS, E = D / 32, RB = C::RB, NG = C::NG, NP = C::NP, NS = C::NS;
  constexpr unsigned FULL = 0xffffffffu;
  using Vec = std::conditional_t<E == 4, float4, float2>;
  extern __shared__ __align__(128) uint8_t sm[];
  // a segment's parts: workers of its first and last unit; whether the last goes on behind it (its parts are then stored
  // apart), CTAs that hold the others
  struct Parts {
    int seg, w0, w1, early, held;
  };
  __shared__ Parts sparts[NG + NP];  // of the warps' last segments; of the segments that ended early in the pairs' ranges
  __shared__ int joins[NG + NP], n_joins;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kKv4RingBytes);
  unsigned* used = reinterpret_cast<unsigned*>(full + NP * NS);
  int* prefix = reinterpret_cast<int*>(used + NP * NS);

  const int tid = threadIdx.x, lane = tid & 31, grp = tid >> 5, pair = grp >> 1, side = grp & 1;
  const int g = lane >> 2, t = lane & 3;
  const int H = c.n_kv_heads, S = c.n_seqs;
  int* lens = prefix + S + 1;

  for (int i = tid; i < NP * NS; i += C::THREADS) mbar_init(&full[i], 1), used[i] = 0;
  if (tid < NG + NP) sparts[tid].seg = -1;
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  griddep_enter();
  const int fresh = a.k.data ? 1 : 0;  // units of the new rows
  auto units_of = [&](int L) { return max(1, fresh + (L + kPage - 1) / kPage); };
  kv4_prefix(c, a, geo, prefix, lens, units_of);
  __syncthreads();
  auto len_of = [&](int s) { return s < kKv4Lens ? lens[s] : c.len[s]; };
  auto count_of = [&](int s) { return a.counts ? a.counts[s] : a.n; };

  // equal ranges of the U units: the first `more` of the W workers have one more than `each`
  const int U = prefix[S];
  if (U == 0) return;
  const int W = min(U, geo.ctas * NP), each = U / W, more = U % W;
  auto begin_of = [&](int w) { return w * each + min(w, more); };
  auto worker_at = [&](int u) {
    const int x = more * (each + 1);
    return u < x ? u / (each + 1) : more + (u - x) / each;
  };
  const int worker = blockIdx.x * NP + pair;
  const bool has = worker < W;
  const int u0 = has ? begin_of(worker) : 0, u1 = has ? begin_of(worker + 1) : 0;

  // The lane's unit x (32 units in parallel, so the table's latency is paid once).
  auto look = [&](int x) -> Kv4Unit {
    Kv4Unit r{-1, 0};
    if (x >= u1) return r;
    const int s = kv4_seq_of(prefix, S, x), L = len_of(s), blocks = kv4_blocks(geo, count_of(s));
    const int per = units_of(L), q = (x - prefix[s]) / per, u = (x - prefix[s]) % per - fresh;
    const int tokens = u < 0 ? -1 : max(0, min(kPage, L - u * kPage));
    r.what = ((s * H + q / blocks) * geo.CB + q % blocks) << 7 | (tokens + 1);
    if (tokens <= 0) return r;
    const int phys = kv4_phys(c, s, u);
    if (phys >= 0) r.page = phys * H + q / blocks;
    return r;
  };

  uint8_t* ring = sm + (size_t)pair * NS * C::PAGE;
  full += pair * NS;
  used += pair * NS;
  const int nu = u1 - u0;
  Kv4Unit cur = look(u0 + lane), nxt{-1, 0};
  if (nu > 32) nxt = look(u0 + 32 + lane);
  int jl = 0;                     // next unit to copy
  int is = 0, in_ring = 0;        // its ring entry; entries asked for and not consumed
  int asked = 0;                  // pages asked for
  int cs = 0, cph = 0;            // entry to consume next, and its phase
  bool ok = true;

  // ---- state of the segment
  uint32_t qf[NT][KS][2];
  // m and most: the row's maximum, and the product S that would pass it by the slack (the factors are not negative)
  float O[NT][DT][4], m[NT][NC], most[NT][NC], l[NT][NC], colfac[NT][NC], collow[NT][NC];
  int seg = -1, s_cur = 0, h_cur = 0, cb_cur = 0, rows_cur = 0;
  // the factor of a column, log2(e) |scale| / (power of two of its row), as hi + lo; q takes the scale's sign
  const float lhi = fabsf(geo.lhi), llo = a.scale < 0.0f ? -geo.llo : geo.llo;
  // row (of the column block) of column col of tile x; query rows of the segment's KV head
  auto row_of = [&](int x, int col) { return x * C::RPT + (SPLIT ? col >> 1 : col); };
  auto locate = [&](int sg) {
    seg = sg;
    cb_cur = sg % geo.CB, h_cur = sg / geo.CB % H, s_cur = sg / geo.CB / H;
    rows_cur = min(RB, count_of(s_cur) * geo.G - cb_cur * RB);
  };
  auto query = [&](int row) {  // of the column block
    const int r = cb_cur * RB + row;
    return static_cast<const T*>(a.q.data) + s_cur * a.q.seq + (r / geo.G) * a.q.row + (h_cur * geo.G + r % geo.G) * a.q.head;
  };
  auto output = [&](int sg, int row) {
    const int cb = sg % geo.CB, h = sg / geo.CB % H, s = sg / geo.CB / H, r = cb * RB + row;
    return static_cast<T*>(a.out.data) + s * a.out.seq + (r / geo.G) * a.out.row + (h * geo.G + r % geo.G) * a.out.head;
  };

  auto begin = [&](int sg) {
    locate(sg);
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[x][d][e] = 0.0f;
#pragma unroll
      for (int y = 0; y < NC; ++y) m[x][y] = most[x][y] = -INFINITY, l[x][y] = ok ? 0.0f : NAN;
      const int r = row_of(x, g);
      float v[KS * 4];
      if (r < rows_cur) {
        const T* q = query(r);
#pragma unroll
        for (int kp = 0; kp < D / 32; ++kp) {
          const T* p = q + 32 * kp + 8 * t;
          if (geo.vec & 1) {
            uint4 w[sizeof(T) / 2];
#pragma unroll
            for (int y = 0; y < (int)sizeof(T) / 2; ++y) w[y] = reinterpret_cast<const uint4*>(p)[y];
#pragma unroll
            for (int y = 0; y < 8; ++y) v[8 * kp + y] = kv8_load(reinterpret_cast<const T*>(w) + y);
          } else {
#pragma unroll
            for (int y = 0; y < 8; ++y) v[8 * kp + y] = kv8_load(p + y);
          }
        }
      } else {
#pragma unroll
        for (int y = 0; y < KS * 4; ++y) v[y] = 0.0f;
      }
      float am = 0.0f;
#pragma unroll
      for (int y = 0; y < KS * 4; ++y) am = max_nan(am, fabsf(v[y]));
      am = max_nan(am, __shfl_xor_sync(FULL, am, 1));
      am = max_nan(am, __shfl_xor_sync(FULL, am, 2));
      const float up = f16_scale(am), sup = a.scale < 0.0f ? -up : up;
#pragma unroll
      for (int y = 0; y < KS; ++y) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = v[4 * y + e] * sup;
          if (SPLIT) f[e] = g & 1 ? f[e] - rintf(f[e]) : rintf(f[e]);
        }
        qf[x][y][0] = pack_f16(f[0], f[1]);
        qf[x][y][1] = pack_f16(f[2], f[3]);
      }
      // from the lanes of column g to the lanes of accumulator columns 2 t, 2 t + 1
      const float down = 1.0f / up;
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        const float dn = __shfl_sync(FULL, down, SPLIT ? 8 * t : 4 * (2 * t + y));
        colfac[x][y] = lhi * dn;
        collow[x][y] = llo * dn;
      }
    }
  };
  // The new rows, a warp's every second, one after the other, in plain fp32: a lane has E dims of a key for the dot products, then the values of
  // its accumulators' dims.  A row that does not see the token is left out of everything, whatever the token holds.
  auto new_rows = [&]() {
    const int cnt = count_of(s_cur);
    const T* kn = static_cast<const T*>(a.k.data) + s_cur * a.k.seq + h_cur * a.k.head + E * lane;
    const T* vn = static_cast<const T*>(a.v.data) + s_cur * a.v.seq + h_cur * a.v.head + g;
    const int node0 = cb_cur * RB / geo.G, node1 = (cb_cur * RB + rows_cur - 1) / geo.G;  // the block's nodes
#pragma unroll 1
    for (int j = side; j < cnt; j += 2) {
      if (!a.mask && j > node1) break;
      float k[E], v[2 * DT];
#pragma unroll
      for (int e = 0; e < E; ++e) k[e] = kv8_load(kn + j * a.k.row + e);
#pragma unroll
      for (int d = 0; d < 2 * DT; ++d) v[d] = kv8_load(vn + j * a.v.row + 8 * d);
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float dot[C::RPT];
#pragma unroll
        for (int r = 0; r < C::RPT; ++r) {
          dot[r] = 0.0f;
          if (x * C::RPT + r < rows_cur) {
            const T* q = query(x * C::RPT + r) + E * lane;
#pragma unroll
            for (int e = 0; e < E; ++e) dot[r] = fmaf(kv8_load(q + e), k[e], dot[r]);
          }
        }
        // sums over the lanes; a lane keeps the rows of its half at each step, row lane / (32 / RPT) in the end
        int w = 16;
#pragma unroll
        for (int r = C::RPT / 2; r > 0; r >>= 1, w >>= 1)
#pragma unroll
          for (int y = 0; y < r; ++y) {
            const bool up = lane & w;
            const float keep = up ? dot[y + r] : dot[y], give = up ? dot[y] : dot[y + r];
            dot[y] = keep + __shfl_xor_sync(FULL, give, w);
          }
#pragma unroll
        for (int o = 16 / C::RPT; o > 0; o >>= 1) dot[0] += __shfl_xor_sync(FULL, dot[0], o);
        float s[NC];
        bool see[NC], high = false;
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          const int row = row_of(x, 2 * t + y);
          s[y] = __shfl_sync(FULL, dot[0], (32 / C::RPT) * (SPLIT ? t : 2 * t + y)) * geo.lhi;
          see[y] = row < rows_cur;
          if (see[y]) {
            const int node = node0 == node1 ? node0 : (cb_cur * RB + row) / geo.G;
            see[y] = a.mask ? a.mask[(size_t)s_cur * a.n + node] >> j & 1ull : j <= node;
          }
          high = high || (see[y] && s[y] > m[x][y] + kP4Slack);
        }
        if (__any_sync(FULL, high)) {
          float cc[NC];
#pragma unroll
          for (int y = 0; y < NC; ++y) {
            const float mx = see[y] ? fmaxf(m[x][y], s[y]) : m[x][y];
            cc[y] = mx == -INFINITY ? 1.0f : ex2(m[x][y] - mx);
            m[x][y] = mx;
            most[x][y] = __fdividef(mx + kP4Slack, colfac[x][y]);
            l[x][y] *= cc[y];
          }
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[x][d][e] *= cc[(e & 1) * (NC - 1)];
        }
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          const float p = ex2(s[y] - (m[x][y] == -INFINITY ? 0.0f : m[x][y])) * kP4Scale;
          if (!see[y]) continue;
          if (g == 0) l[x][y] += p;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            O[x][d][y] = fmaf(p, v[2 * d], O[x][d][y]);
            O[x][d][y + 2] = fmaf(p, v[2 * d + 1], O[x][d][y + 2]);
          }
        }
      }
    }
  };

  // The warp's part of its segment.
  auto flush = [&](float2* ml, float* out) {
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        float sum = l[x][y];
        sum += __shfl_xor_sync(FULL, sum, 4);
        sum += __shfl_xor_sync(FULL, sum, 8);
        sum += __shfl_xor_sync(FULL, sum, 16);
        const int r = row_of(x, 2 * t + y);
        if (r >= rows_cur) continue;
        if (g == 0) ml[r] = make_float2(m[x][y], sum);
        float* o = out + r * D;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[16 * d + g] = SPLIT ? O[x][d][0] + O[x][d][1] : O[x][d][y];
          o[16 * d + g + 8] = SPLIT ? O[x][d][2] + O[x][d][3] : O[x][d][y + 2];
        }
      }
  };

  // Half a page: S^T = K Q^T, softmax, O^T += V^T P^T.  The first `left` of its tokens are there.
  auto half = [&](const uint8_t* page, int left) {
    using P = Kv4Page<D>;
    const uint8_t *keys = page + side * (16 * D), *values = keys + P::V;
    const uint8_t *ksc = page + P::KS + side * D, *vsc = page + P::VS + side * D;
    float x[NT][2][4];  // two 16-token tiles
#pragma unroll
    for (int z = 0; z < NT; ++z)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[z][i][e] = 0.0f;
    // scales of tokens g and g + 8 of the tiles as f16 pairs: of groups 0 and 2, of groups 1 and 3 (D = 64: of group 0 of
    // either token, of group 1)
    uint32_t sc[2][2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[2];
      if (D == 128) {
        const uint2 w2 = *reinterpret_cast<const uint2*>(ksc + (i * 8 + g) * 8);
        w[0] = w2.x, w[1] = w2.y;
      } else {
        w[0] = w[1] = *reinterpret_cast<const uint32_t*>(ksc + (i * 8 + g) * 4);
      }
#pragma unroll
      for (int y = 0; y < D / 64; ++y) sc[i][y][0] = w[y] << 7 & 0x7f807f80u, sc[i][y][1] = w[y] >> 1 & 0x7f807f80u;
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint32_t w[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w4 = reinterpret_cast<const uint4*>(keys)[(i * (D / 64) + j) * 32 + lane];
        w[i][0] = w4.x, w[i][1] = w4.y, w[i][2] = w4.z, w[i][3] = w4.w;
      }
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        const int gr = 2 * j + kh;
        float part[NT][2][4];
        uint32_t s0[2], s1[2], b0[2], b1[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s0[i] = D == 128 ? twice(sc[i][0][kh], j) : twice(sc[i][0][kh], 0);
          s1[i] = D == 128 ? twice(sc[i][1][kh], j) : twice(sc[i][0][kh], 1);
          b0[i] = mul_h2(s0[i], kMinus264), b1[i] = mul_h2(s1[i], kMinus24);
#pragma unroll
          for (int z = 0; z < NT; ++z)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[z][i][e] = 0.0f;
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t wa = w[i][2 * kh + p], wb = kv4_swap(wa);
            const uint32_t af[4] = {fma_h2(kv4_f16_low(wa), s0[i], b0[i]), fma_h2(kv4_f16_high(wa), s1[i], b1[i]),
                                    fma_h2(kv4_f16_low(wb), s0[i], b0[i]), fma_h2(kv4_f16_high(wb), s1[i], b1[i])};
#pragma unroll
            for (int z = 0; z < NT; ++z)
              mma_f16(SPLIT ? part[z][i] : x[z][i], af, qf[z][2 * gr + p][0], qf[z][2 * gr + p][1]);
          }
        if (SPLIT)
#pragma unroll
          for (int z = 0; z < NT; ++z)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[z][i][e] += part[z][i][e];
      }
    }
    uint32_t pf[NT][2][2];
#pragma unroll
    for (int z = 0; z < NT; ++z) {
      // logits: entry y + 2 e of tile i is row y of the thread, token g + 8 e of the tile
      if (SPLIT)
#pragma unroll
        for (int i = 0; i < 2; ++i) x[z][i][0] += x[z][i][1], x[z][i][2] += x[z][i][3];  // hi + lo
      if (left < 32) {
        __syncwarp();  // a branch: as predicated instructions it would cost every half page its 16 selects
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * i + g + 8 * (e >> 1) >= left) x[z][i][e] = -INFINITY;
      }
      bool high = false;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int y = 0; y < NC; ++y)
          high = high || x[z][i][y] > most[z][y] || x[z][i][y + 2] > most[z][y];
      if (__any_sync(FULL, high)) {
        float cc[NC];
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          const float f = colfac[z][y];
          float mx = fmaxf(fmaxf(x[z][0][y], x[z][0][y + 2]), fmaxf(x[z][1][y], x[z][1][y + 2])) * f;
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
          mx = fmaxf(mx, m[z][y]);
          cc[y] = mx == -INFINITY ? 1.0f : ex2(m[z][y] - mx);
          m[z][y] = mx;
          most[z][y] = __fdividef(mx + kP4Slack, f);
          l[z][y] *= cc[y];
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[z][d][e] *= cc[(e & 1) * (NC - 1)];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          const float base = m[z][y] == -INFINITY ? 0.0f : m[z][y];
#pragma unroll
          for (int e = y; e < 4; e += 2) {
            x[z][i][e] = SPLIT ? ex2(fmaf(x[z][i][e], collow[z][y], fmaf(x[z][i][e], colfac[z][y], -base))) * kP4Scale
                               : ex2(fmaf(x[z][i][e], colfac[z][y], 7.0f - base));
          }
        }
      }
      if (left < 32) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * i + g + 8 * (e >> 1) >= left) x[z][i][e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int e = y; e < 4; e += 2) l[z][y] += x[z][i][e];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = x[z][i][2 * e];
          pf[z][i][e] = movmatrix(SPLIT ? pack_f16(p, p - __half2float(__float2half_rn(p))) : pack_f16(p, x[z][i][2 * e + 1]));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint32_t w[2][4], vs[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w4 = reinterpret_cast<const uint4*>(values)[(i * (D / 64) + j) * 32 + lane];
        w[i][0] = w4.x, w[i][1] = w4.y, w[i][2] = w4.z, w[i][3] = w4.w;
        const uint2 s2 = *reinterpret_cast<const uint2*>(vsc + (i * 4 + t) * (D / 8) + 8 * j);
        vs[i][0] = s2.x, vs[i][1] = s2.y;
        if (left < 32) {  // tokens that are not there: whatever their bytes hold, scale 0
          __syncwarp();
          uint32_t keep = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (16 * i + 2 * t + (b & 1) + 8 * (b >> 1) < left) keep |= 255u << (8 * b);
          vs[i][0] &= keep, vs[i][1] &= keep;
        }
      }
#pragma unroll
      for (int gh = 0; gh < 2; ++gh) {
        float part[NT][2][4];
#pragma unroll
        for (int z = 0; z < NT; ++z)
#pragma unroll
          for (int dd = 0; dd < 2; ++dd)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[z][dd][e] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t s0 = kv4_scale_pair(vs[i][gh], 0, 1), s1 = kv4_scale_pair(vs[i][gh], 2, 3);
          const uint32_t b0 = mul_h2(s0, kMinus264), b1 = mul_h2(s1, kMinus24);
#pragma unroll
          for (int dd = 0; dd < 2; ++dd) {
            const uint32_t wa = w[i][2 * gh + dd], wb = kv4_swap(wa);
            const uint32_t af[4] = {fma_h2(kv4_f16_low(wa), s0, b0), fma_h2(kv4_f16_low(wb), s0, b0),
                                    fma_h2(kv4_f16_high(wa), s1, b1), fma_h2(kv4_f16_high(wb), s1, b1)};
#pragma unroll
            for (int z = 0; z < NT; ++z) mma_f16(part[z][dd], af, pf[z][i][0], pf[z][i][1]);
          }
        }
#pragma unroll
        for (int z = 0; z < NT; ++z)
#pragma unroll
          for (int dd = 0; dd < 2; ++dd)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[z][4 * j + 2 * gh + dd][e] += part[z][dd][e];
      }
    }
  };

  // ---- a segment's parts
  auto parts_of = [&](int sg) {
    const int cb = sg % geo.CB, h = sg / geo.CB % H, s = sg / geo.CB / H;
    const int per = units_of(len_of(s)), first = prefix[s] + (h * kv4_blocks(geo, count_of(s)) + cb) * per, end = first + per;
    Parts p;
    p.seg = sg;
    p.w0 = worker_at(first), p.w1 = worker_at(end - 1);
    p.early = begin_of(p.w1 + 1) > end;
    p.held = p.w1 - p.early < p.w0 ? 0 : (p.w1 - p.early) / NP - p.w0 / NP + 1;
    return p;
  };
  auto rows_of = [&](int sg) { return min(RB, count_of(sg / geo.CB / H) * geo.G - sg % geo.CB * RB); };
  // The parts first, first + step, .. of a segment's row, of the CTAs in their order, then the early ones: maximum M,
  // sum, and values of the lane's dims; B loads in flight.
  const int slots = geo.ctas * NP;
  constexpr int B = NT == 1 ? 10 : 16;
  auto gather = [&](const Parts& p, int r, int first, int step, float& M, float& sum, float (&o)[E]) {
    const int n = p.held + 2 * p.early, apart = p.held ? slots : 3 * slots;
    M = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    for (int i0 = first; i0 < n; i0 += B * step) {
      float2 ml[B];
      Vec v[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int i = i0 + b * step;
        ml[b] = make_float2(-INFINITY, 0.0f);
        v[b] = {};
        if (i < n) {
          const size_t at = (size_t)(i < p.held ? max(p.w0, (p.w0 / NP + i) * NP) : apart + 2 * p.w1 + i - p.held) * RB + r;
          ml[b] = __ldcg(ws.ml + at);
          v[b] = __ldcg(reinterpret_cast<const Vec*>(ws.o + at * D + E * lane));
        }
      }
      float mx = M;
#pragma unroll
      for (int b = 0; b < B; ++b) mx = fmaxf(mx, ml[b].x);
      const float base = mx == -INFINITY ? 0.0f : mx, f = ex2(M - base);
      M = mx;
      sum *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float w = ex2(ml[b].x - base);
        const float* ve = reinterpret_cast<const float*>(&v[b]);
        sum = fmaf(ml[b].y, w, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(ve[e], w, o[e]);
      }
    }
  };
  auto store = [&](T* to, float sum, const float (&o)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) kv8_store(to + e, sum == 0.0f ? 0.0f : o[e] / sum);
  };
  // The pair's segment ends in front of others of its range.
  auto finish = [&]() {
    const Parts p = parts_of(seg);
    const size_t at = (size_t)((p.held ? slots : 3 * slots) + 2 * worker + side) * RB;
    flush(ws.ml + at, ws.o + at * D);
    if (p.held) {  // joined with the other parts in the end
      if (side == 0 && lane == 0) sparts[NG + pair] = p;
      return;
    }
    auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory"); };
    meet();
    for (int r = side; r < rows_cur; r += 2) {
      float M, sum, o[E];
      gather(p, r, 0, 1, M, sum, o);
      store(output(seg, r) + E * lane, sum, o);
    }
    meet();  // the place is free again
  };

  // ---- the range
  // whether the pair's other warp has been here before, and is done with what this one is done with
  auto second = [&](unsigned* n) {
    unsigned old;
    asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(old) : "r"(smem_u32(n)) : "memory");
    return (old & 1u) != 0;
  };
#pragma unroll 1
  for (int j = 0, cbase = 0; j < nu; ++j) {
    if (j - cbase == 32) {
      cbase += 32;
      cur = nxt;
      nxt = look(u0 + cbase + 32 + lane);
    }
    // copy ahead as far as the ring and the two batches of units allow; the second of the pair to come here fills an entry
    while (ok && in_ring < NS && jl < nu && jl < cbase + 64) {
      const int from = __shfl_sync(FULL, jl < cbase + 32 ? cur.page : nxt.page, (jl - cbase) & 31);
      ++jl;
      if (from < 0) continue;
      if (lane == 0 && (asked < NS ? side == 0 : second(&used[is]))) {
        mbar_expect_tx(&full[is], C::PAGE);
        if (geo.withheld != (int)blockIdx.x) bulk_g2s(ring + is * C::PAGE, c.pages + (size_t)from * C::PAGE, C::PAGE, &full[is]);
      }
      ++asked;
      ++in_ring;
      if (++is == NS) is = 0;
    }
    const int from = __shfl_sync(FULL, cur.page, j - cbase), what = __shfl_sync(FULL, cur.what, j - cbase);
    const int sg = what >> 7, tokens = (what & 127) - 1;
    if (sg != seg) {
      if (seg >= 0) finish();
      begin(sg);
    }
    if (tokens < 0 && ok) new_rows();
    if (from < 0 || !ok) continue;
    ok = __all_sync(FULL, mbar_wait(&full[cs], cph, geo.wait_ns));
    if (ok) {
      const int left = tokens - side * kKv4HalfTokens;
      if (left > 0) half(ring + cs * C::PAGE, left);
      __syncwarp();
      if (++cs == NS) cs = 0, cph ^= 1;
      --in_ring;
      continue;
    }
    // a bounded wait expired: the sums from here on are not what they should be, and NaN says so; no copy stays in flight
    if (lane == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TIMEOUT);
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int y = 0; y < NC; ++y) l[x][y] = NAN;
    const WaitsWithin drain(geo.wait_ns);
    for (; in_ring > 0; --in_ring) {
      (void)drain.wait(&full[cs], cph);
      if (++cs == NS) cs = 0, cph ^= 1;
    }
  }
  // ---- the warps' last parts, in the ring's place, and of each run of warps on one segment the sum
  float2* sml = reinterpret_cast<float2*>(sm);                // [NG][RB]
  float* sfac = reinterpret_cast<float*>(sml + NG * RB);      // [NG][RB] factor of a warp's part in its run
  float* so = sfac + NG * RB;                                 // [NG][RB][D]
  float* jo = so + NG * RB * D;                               // [NG][D], of the join
  float2* jml = reinterpret_cast<float2*>(jo + NG * D);       // [NG]
  static_assert((NG * RB * (3 + D) + NG * D + 2 * NG) * 4 <= kKv4RingBytes, "parts");
  if (seg >= 0) {
    const Parts p = parts_of(seg);
    if (lane == 0) sparts[grp] = p;
  }
  __syncthreads();
  if (seg >= 0) flush(sml + grp * RB, so + grp * RB * D);
  __syncthreads();
  const int mine = lane < NG ? sparts[lane].seg : -1, before = __shfl_up_sync(FULL, mine, 1);
  const unsigned heads = __ballot_sync(FULL, mine >= 0 && (lane == 0 || mine != before));  // first warps of the runs
  const unsigned warps = __ballot_sync(FULL, mine >= 0);  // warps with a part: the first ones
  const int busy = __popc(warps);
  auto run_end = [&](int i) {  // of the run that begins with warp i
    const unsigned later = heads & (0xfffffffeu << i);
    return later ? __ffs(later) - 1 : busy;
  };
  for (int x = tid; x < busy * RB; x += C::THREADS) {
    const int i = x / RB, i0 = 31 - __clz(heads & (0xffffffffu >> (31 - i))), i1 = run_end(i0);
    if (x % RB >= rows_of(sparts[i].seg)) continue;
    float M = -INFINITY;
    for (int y = i0; y < i1; ++y) M = fmaxf(M, sml[y * RB + x % RB].x);
    sfac[x] = ex2(sml[x].x - (M == -INFINITY ? 0.0f : M));
  }
  __syncthreads();
  for (int x = tid; x < __popc(heads) * (RB * D / 4); x += C::THREADS) {
    unsigned rest = heads;
    for (int k = x / (RB * D / 4); k > 0; --k) rest &= rest - 1;
    const int i0 = __ffs(rest) - 1, i1 = run_end(i0), r = x / (D / 4) % RB, d = x % (D / 4);
    const Parts& p = sparts[i0];
    if (r >= rows_of(p.seg)) continue;
    float M = -INFINITY, L = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const float2 ml = sml[i * RB + r];
      const float4 o = reinterpret_cast<const float4*>(so + (i * RB + r) * D)[d];
      const float f = sfac[i * RB + r];
      M = fmaxf(M, ml.x);
      L = fmaf(ml.y, f, L);
      v.x = fmaf(o.x, f, v.x), v.y = fmaf(o.y, f, v.y), v.z = fmaf(o.z, f, v.z), v.w = fmaf(o.w, f, v.w);
    }
    if (p.held + p.early == 1) {  // the only part
      T* out = output(p.seg, r) + 4 * d;
      kv8_store(out, L == 0.0f ? 0.0f : v.x / L), kv8_store(out + 1, L == 0.0f ? 0.0f : v.y / L);
      kv8_store(out + 2, L == 0.0f ? 0.0f : v.z / L), kv8_store(out + 3, L == 0.0f ? 0.0f : v.w / L);
    } else {
      const size_t at = (size_t)(blockIdx.x * NP + i0 / 2) * RB + r;
      reinterpret_cast<float4*>(ws.o + at * D)[d] = v;
      if (d == 0) ws.ml[at] = make_float2(M, L);
    }
  }
  // the parts that other CTAs' are joined with: a ticket each, and the CTA that draws a segment's last joins it
  __syncthreads();
  if (grp == 0) {
    const bool part = lane < NG ? heads >> lane & 1u : lane < NG + NP && sparts[lane].seg >= 0;
    bool last = false;
    if (part) {
      const Parts& p = sparts[lane];
      const int all = p.held + p.early;
      if (all > 1) {
        int old;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(ws.ticket + p.w0) : "memory");
        last = old == all - 1;
        if (last) ws.ticket[p.w0] = 0;  // for the next call
      }
    }
    const unsigned which = __ballot_sync(FULL, last);
    if (last) joins[__popc(which & ((1u << lane) - 1))] = lane;
    if (lane == 0) n_joins = __popc(which);
  }
  __syncthreads();
  // Warps of a row: by the number of its parts, so that the order of a sum does not depend on which CTA draws what.
  const int rows = min(RB, geo.R);
  auto split_of = [&](const Parts& p) {
    int per = 1;
    while (per * B < p.held + 2 * p.early && 2 * per * rows <= NG) per *= 2;
    return per;
  };
  for (int x = grp; x < n_joins * rows; x += NG) {
    const Parts p = sparts[joins[x / rows]];
    const int r = x % rows;
    if (split_of(p) > 1 || r >= rows_of(p.seg)) continue;
    float M, sum, o[E];
    gather(p, r, 0, 1, M, sum, o);
    store(output(p.seg, r) + E * lane, sum, o);
  }
  for (int k = 0; k < n_joins; ++k) {
    const Parts p = sparts[joins[k]];
    const int per = split_of(p), r = grp / per;  // NG / per >= rows
    if (per == 1) continue;
    const bool on = r < rows_of(p.seg);
    float M, sum, o[E];
    if (on) {
      gather(p, r, grp % per, per, M, sum, o);
      if (lane == 0) jml[grp] = make_float2(M, sum);
      *reinterpret_cast<Vec*>(jo + grp * D + E * lane) = *reinterpret_cast<Vec*>(o);
    }
    __syncthreads();
    if (on && grp % per == 0) {
      float top = M;
      for (int y = 1; y < per; ++y) top = fmaxf(top, jml[grp + y].x);
      const float base = top == -INFINITY ? 0.0f : top;
      float f = ex2(M - base);
      sum *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
      for (int y = 1; y < per; ++y) {
        f = ex2(jml[grp + y].x - base);
        sum = fmaf(jml[grp + y].y, f, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(jo[(grp + y) * D + E * lane + e], f, o[e]);
      }
      store(output(p.seg, r) + E * lane, sum, o);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------- launch

inline size_t kv4_split_smem(int S, int entries) {
  return (size_t)kKv4RingBytes + 12 * (size_t)entries + 4 * ((size_t)S + 1 + (S < kKv4Lens ? S : kKv4Lens));
}

template <typename T, int D, int NT>
cudaError_t kv4_split_launch(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo, const Kv4Scratch& ws,
                             cudaStream_t st) {
  using C = Kv4Split<T, D, NT>;
  const size_t most = kv4_split_smem(kKv8MaxSeqs, C::NP * C::NS), smem = kv4_split_smem(c.n_seqs, C::NP * C::NS);
  cudaError_t e = kv8_smem<k_kv4_split<T, D, NT>>(most);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_kv4_split<T, D, NT>, dim3((unsigned)geo.ctas), dim3(C::THREADS), smem, st, c, a, geo, ws);
}
// Column tiles of a warp for R query rows of a KV head: two where one does not hold them (four rows of fp32, eight of bf16).
inline int kv4_split_tiles(int R, int dtype) { return R > (dtype == W4A8_F32 ? 4 : 8) ? 2 : 1; }
inline int kv4_split_warps(int R, int dtype) { return kv4_split_tiles(R, dtype) == 1 ? 16 : 8; }
template <typename T, int D>
cudaError_t kv4_split_dispatch(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo, const Kv4Scratch& ws,
                               cudaStream_t st) {
  return kv4_split_tiles(geo.R, a.dtype) == 1 ? kv4_split_launch<T, D, 1>(c, a, geo, ws, st)
                                              : kv4_split_launch<T, D, 2>(c, a, geo, ws, st);
}
// Calls whose KV heads have many query rows run on tcgen05 (kv4_wide.cu): a tile of it takes 128 rows at one price, the split
// kernel's price goes by blocks of 8 (fp32) or 16 (bf16) rows.  Few pages of few (sequence, KV head) pairs are bound by
// latency, where the wide kernel with the new rows in its own grid is the shorter way; otherwise the blocks count.  The pages are those
// that the cache has room for: the host does not know its lengths.  Measured on full caches (us, split / wide; pairs x tokens,
// heads of 128 unless said), on both sides of the limits: 640 pages for 9 to 16 rows of fp32, 1100 for 17 to 24, 2600 for bf16:
//   fp32, 8 x 4096 (512):  8 rows 18 / 20,  12 rows 21 / 21,  16 rows 23 / 21,  32 rows 31 / 21
//   fp32, 8 x 5000 (632):  12 rows 22.9 / 22.1,  16 rows 23.5 / 22.3;   8 x 6000 (752):  12 rows 23.8 / 24.1,  16 rows 25.8 / 24.4
//   fp32, 8 x 7000 (880):  12 rows 20.2 / 25.6,  16 rows 22.0 / 26.0,  20 rows 28.8 / 26.2;   8 x 8192 (1024):  16 rows 26 / 27,  24 rows 31 / 28
//   fp32, 4 x 12000 (752):  12 rows 22 / 25,  16 rows 25 / 26,  20 rows 28 / 26;   24 x 1500 (576):  12 rows 20 / 22,  16 rows 22 / 23,  20 rows 27 / 23
//   fp32, 24 x 3000 (1128):  20 rows 21 / 23;   8 x 16000 (2000):  16 rows 30 / 39,  24 rows 38 / 40,  32 rows 46 / 40;  8 x 32000:  24 rows 55 / 66,  32 rows 69 / 66
//   fp32, 128 x to 4096:  12 rows 63 / 87,  16 rows 69 / 90,  20 rows 108 / 92
//   bf16, 8 x 4096:  8 rows 15 / 17,  12 rows 26 / 18;  8 x 16000 (2000):  8 rows 23 / 28,  12 rows 34 / 29,  16 rows 38 / 29
//   bf16, 8 x 20000 (2504):  12 rows 35 / 32,  16 rows 39 / 32;   8 x 24000 (3000):  12 rows 37 / 35,  16 rows 40 / 35;   of 64:  16 rows 30 / 33,  24 rows 35 / 34
//   bf16, 16 x 12000 (3008):  12 rows 34 / 35,  16 rows 35 / 35,  20 rows 39 / 36
//   bf16, 8 x 28000 (3500):  12 rows 38 / 40,  16 rows 41 / 40;   8 x 32000 (4000):  12 rows 40 / 45,  16 rows 42 / 45,  20 rows 51 / 45
//   bf16, 128 x to 4096:  16 rows 65 / 78,  20 rows 103 / 79
// fp32 heads of 64, whose split kernel has half the conversions, from 17 rows on up to 128 pages, else as behind the limits:
//   2 x 4096 (128):  14 rows 15 / 15,  21 rows 17 / 16;   2 x 6000 (188):  24 rows 18 / 23;   4 x 4096 (256):  16 rows 16 / 18,  24 rows 20 / 19,  32 rows 20 / 19
//   4 x 8192 (512):  24 rows 21 / 22,  32 rows 21 / 22;   24 x 1500 (576):  24 rows 20 / 21;   8 x 16000 (2000):  24 rows 29 / 35
// Up to about 1000 tokens the wide kernel is the shorter way for 4 to 8 rows too (8 heads: fp32 8 rows over 300 tokens 14.6 / 11.9, over 1000
// 15.1 / 13.4; bf16 13.5 / 11.1 and 14.5 / 12.7, 4 rows 12.1 / 11.0 and 12.6 / 12.5), over 2000 no more (bf16 8 rows 14.7 / 14.7):
// the rule does not go there.
inline bool kv4_is_wide(const w4a8_kv4_cache& c, int R, int dtype) {
  const int64_t pairs = (int64_t)c.n_seqs * c.n_kv_heads, pages = pairs * c.max_pages;
  const bool f32 = dtype == W4A8_F32, d64 = c.head_dim == 64;
  if (pairs <= kKv4Ctas / 6 && pages <= (!f32 ? 2600 : d64 ? 128 : 1100)) return R > (f32 && (d64 || pages > 640) ? 16 : 8);
  return R > (f32 && pairs <= 16 ? 24 : 16);
}
cudaError_t kv4_wide(const w4a8_kv4_cache&, const w4a8_kv4_attn&, const Kv4Geom&, const Kv4Scratch&, cudaStream_t);
// one translation unit per head size and element type
cudaError_t kv4_split_f32_d64(const w4a8_kv4_cache&, const w4a8_kv4_attn&, const Kv4Geom&, const Kv4Scratch&, cudaStream_t);
cudaError_t kv4_split_f32_d128(const w4a8_kv4_cache&, const w4a8_kv4_attn&, const Kv4Geom&, const Kv4Scratch&, cudaStream_t);
cudaError_t kv4_split_bf16_d64(const w4a8_kv4_cache&, const w4a8_kv4_attn&, const Kv4Geom&, const Kv4Scratch&, cudaStream_t);
cudaError_t kv4_split_bf16_d128(const w4a8_kv4_cache&, const w4a8_kv4_attn&, const Kv4Geom&, const Kv4Scratch&, cudaStream_t);

}  // namespace w4a8
