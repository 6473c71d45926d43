// Attention over the 8-bit cache for many query rows of a KV head (draft trees, prompt buckets): tcgen05.
//
// A segment is 128 query rows of one (sequence, KV head); its pages, end to end over the segments, are cut into equal
// ranges, one for each CTA.  Per page, in a pipeline of warps:
//   copy      one bulk copy brings the page's codes (16 KB at D = 128) into a ring of four;
//   convert   codes become f16 whole numbers, keys [64 tokens][D] and values [D][64 tokens], in the 128-byte-swizzled
//             K-major layout of the tensor core's B operand.  A 16-byte group of the page's byte order is two 16-byte
//             chunks of two rows of either tile: one load, eight byte permutes, eight subtractions, two stores;
//   products  S = Q C_K^T and O' = P C_V^T, tcgen05.mma with A (Q, P) in tensor memory, 128 x 64 x D and 128 x D x 64;
//   softmax   a thread holds one query row: no exchange between lanes.  P (scaled by 2^7) returns to tensor memory in the
//             token order of the values' chunks.  A page is tried with the row's old maximum, and done again with
//             its own when a logit passes that by 8 (log2);
//   values    O = O c + s_V O' in registers, a thread half a row: the page's scale needs no common factor with the
//             other pages', and nothing is rescaled in tensor memory.
// fp32 calls split Q and P into f16 hi + lo; the products of P's share an accumulator, those of Q's have one each.  The
// hi terms are the nearest whole numbers at a largest magnitude of 2^11 (P: scaled by 2^10, with the maximum of its own page),
// so their sums with the codes are whole numbers, which the tensor core's truncating additions leave exact up to 2^24: all of
// P's (64 tokens), and Q's but where 128 dims nearly all agree in sign and size (below 2^25: off by 2^-24 relative).
// With hi the nearest f16, and Q's lo product in the accumulator of its hi product, outputs were off by 1.8e-6 in the
// 2-norm at 4096 tokens, against 0.6e-6.
// Why tcgen05 here: the split kernel converts a page once for every eight columns, and mma.sync tops out at a quarter
// of the dense rate; with 128 rows a page is 2 x 256 cycles of tensor core against 700 of memory traffic.
// Measured: 128 rows to each of 8 KV heads of 128, 32768 tokens: 56.7 us bf16, 80.7 us fp32 (0.98 and 1.8 us for a page of a
// CTA, whose products take a quarter of that); 256 rows with the pages' mass, 32000 tokens, bf16: 92.5 us.  Bound by
// the latency of the softmax warps (one to a scheduler; more of them leave too few registers for the values).
#include "kv8_attn.cuh"

namespace w4a8 {
namespace {

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
  static constexpr int PAGE = 2 * kPage * D, TILE = kPage * D * 2;  // bytes of a page of codes, of an f16 tile
  // scale of P, and how far (log2) a logit may pass its row's maximum before that moves
  static constexpr float PSCALE = NQ == 2 ? 1024.0f : kPScale, SLACK = NQ == 2 ? 0.9f : kPSlack;
  // buffers of P
  static constexpr int NP = NQ == 2 ? 1 : 2;
  // tensor memory columns: Q, S twice, the product with the lo term of Q (apart: a sum of whole numbers that
  // fractions are added to is truncated each time), P, O'
  static constexpr int cQ = 0, cS = cQ + NQ * D / 2, cL = cS + 2 * kPage, cP = cL + (NQ - 1) * kPage,
                       cO = cP + NP * NQ * kPage / 2;
  static_assert(cO + NO * D <= 512, "tensor memory");
  // shared memory
  static constexpr int sK = kRing * PAGE, sV = sK + 2 * TILE, sBar = sV + 2 * TILE, sFac = sBar + 256;
  static constexpr int QROW = D * (int)sizeof(T) + 16;  // a staged query row: 16 bytes on, so that lanes of a row each do not collide
  static constexpr int sQ = sFac + kFac * kWideRows * 4 + 64;
  static constexpr int sPrefix = sQ + kWideRows * QROW;
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

__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
// f16 x f16 -> f32, both operands K-major, M = 128
__host__ __device__ constexpr uint32_t tc_idesc(int N) { return 1u << 4 | (uint32_t)(N / 8) << 17 | (128u / 16) << 24; }
// Shared-memory operand, low word: K-major rows of 128 bytes; high word: eight rows 1024 bytes apart, 128-byte swizzle
__device__ __forceinline__ uint32_t tc_desc(uint32_t addr) { return (addr >> 4 & 0x3fffu) | 1u << 16; }
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
// D[128][N] (+)= A (tensor memory) B (shared memory), one k-step of 16, by one thread of a converged warp: the operands
// are uniform values, and no branch around the instruction keeps the compiler from holding them as such
template <int N>
__device__ __forceinline__ void tc_mma(uint32_t leader, uint32_t d, uint32_t a, uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %0, 0;\n mov.b64 b, {%3, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %5, p;\n}\n" ::"r"(leader), "r"(d), "r"(a), "r"(desc),
      "r"((uint32_t)add), "r"(tc_idesc(N)), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %0, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}\n" ::"r"(leader), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
#define W4A8_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define W4A8_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tc_load32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;\n"
      : W4A8_R8(v, 0), W4A8_R8(v, 8), W4A8_R8(v, 16), W4A8_R8(v, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_load16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n tcgen05.wait::ld.sync.aligned;\n"
      : W4A8_R8(v, 0), W4A8_R8(v, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_store16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::W4A8_I8(
                   v, 0),
               W4A8_I8(v, 8), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The nearest whole number of |x| < 2^22 (NaN stays)
__device__ __forceinline__ float whole(float x) { return __fadd_rn(__fadd_rn(x, 12582912.0f), -12582912.0f); }

// Use n of a ring of mbarriers: entry and phase parity.
template <int N>
struct Turn {
  int i, ph;
  __device__ explicit Turn(unsigned n = 0) : i((int)(n % N)), ph((int)(n / N & 1u)) {}
  __device__ void next() {
    if (++i == N) i = 0, ph ^= 1;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWideThreads, 1) k_kv8_wide(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo, Kv8Scratch ws) {
  using C = Wide<T, D>;
  constexpr int NQ = C::NQ, NO = C::NO;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(16) uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);  // swizzle atoms start at multiples of 1024
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + C::sBar + sizeof(Bars));
  Bars& bar = *reinterpret_cast<Bars*>(sm + C::sBar);
  float* fac = reinterpret_cast<float*>(sm + C::sFac);          // [kFac][rows] factor of the old values
  int* moved = reinterpret_cast<int*>(fac + kFac * kWideRows);  // [kFac][softmax warp] whether one is not 1
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
  kv8_prefix(c, a, geo, prefix);
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
    size_t pair;
    Kv8Segment sg;
    int cnt;
  };
  auto run_at = [&](int x) {
    Run r;
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    r.cnt = a.counts ? a.counts[lo] : a.n;
    const int per = c.len[lo] / kPage, q = (x - prefix[lo]) / per;
    r.first = (x - prefix[lo]) % per;
    const int blocks = kv8_blocks(geo, r.cnt);
    r.seg = (lo * c.n_kv_heads + q / blocks) * geo.CB + q % blocks;
    r.pages = min(per - r.first, u1 - x);
    r.ends = x + r.pages < u1;
    r.sg = kv8_segment(c, a, geo, r.seg);
    r.pair = kv8_pair(c, r.sg.s, r.sg.h);
    return r;
  };
  // 32 pages of a run, one for each lane: physical page (-1: left out, as an empty one) and one of its scales
  struct Batch {
    int phys;
    float scale;
  };
  auto batch_at = [&](const Run& r, int p, int which) {
    Batch t{-1, 0.0f};
    if (p + lane < r.pages) {
      const int v = c.table[r.pair * c.max_pages + r.first + p + lane];
      if (v >= 0 && v < c.max_pages) t.phys = v, t.scale = c.scales[kv8_page(c, r.pair, v) * 2 + which];
    }
    return t;
  };
  bool ok = true;
  auto wait = [&](uint64_t* b, int parity) {
    ok = ok && __all_sync(FULL, mbar_wait(b, (unsigned)parity, geo.wait_ns));
    return ok;
  };

  // query row of the run's row `row`
  auto query_row = [&](const Run& r, int row) {
    const int rr = r.sg.cb * kWideRows + row;
    return static_cast<const T*>(a.q.data) + r.sg.s * a.q.seq + (rr / geo.G) * a.q.row + (r.sg.h * geo.G + rr % geo.G) * a.q.head;
  };
  auto rows_of = [&](const Run& r) { return max(0, min(kWideRows, r.cnt * geo.G - r.sg.cb * kWideRows)); };
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
      Batch now{}, then = batch_at(r, 0, 0);
      for (int p = 0; p < r.pages && ok; ++p, ++n, e.next()) {
        if ((p & 31) == 0) now = then, then = batch_at(r, p + 32, 0);
        if (n >= kRing && !wait(&bar.code_empty[e.i], e.ph ^ 1)) break;
        int phys = __shfl_sync(FULL, now.phys, p & 31);
        if (phys < 0) {
          if (lane == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TREE);
          phys = 0;
        }
        if (lane == 0) {
          mbar_expect_tx(&bar.code_full[e.i], C::PAGE);
          if (geo.withheld != (int)blockIdx.x)
            bulk_g2s(sm + e.i * C::PAGE, c.codes + kv8_page(c, r.pair, phys) * C::PAGE, C::PAGE, &bar.code_full[e.i]);
        }
        __syncwarp();
      }
      x += r.pages;
    }
    // no copy in flight when the CTA ends
    for (int i = max(0, n - kRing); i < n; ++i)
      (void)mbar_wait(&bar.code_full[i % kRing], (unsigned)(i / kRing & 1), geo.wait_ns);
    if ((geo.vec & 1) && runs > 0) (void)mbar_wait(&bar.q_full, (unsigned)(runs - 1) & 1, geo.wait_ns);
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
      const uint8_t* from = sm + e.i * C::PAGE + v * kPage * D;
      constexpr int kChunks = D / 32;  // keys: 32-dim chunks of a 16-token tile; values: two 32-token chunks of a 16-dim tile
#pragma unroll 4
      for (int k = 0; k < kPage * D / 16 / (32 * kHalf); ++k) {
        const int gi = k * (32 * kHalf) + ct, t = gi & 3, g = (gi >> 2) & 7;
        // neighbouring rows of a store phase take the other half of a row's 128 bytes: no bank conflict
        const int q = (gi >> 5) ^ (g & 1);
        const uint4 w = *reinterpret_cast<const uint4*>(from + (q * 32 + (gi & 31)) * 16);
        const int tile16 = v ? q >> 1 : q / kChunks, chunk = (v ? q & 1 : q % kChunks) * 4 + t, row = tile16 * 16 + g;
        uint4 lo, hi;
        codes_f16<true>(w.x, lo.x, lo.y);
        codes_f16<true>(w.z, lo.z, lo.w);
        codes_f16<true>(w.y, hi.x, hi.y);
        codes_f16<true>(w.w, hi.z, hi.w);
        // keys of D = 128 are two tiles of 64 dims
        uint8_t* to = tile + (v ? 0 : (chunk >> 3) * (kPage * 128)) + row * 128 + (((chunk & 7) ^ g) << 4);
        *reinterpret_cast<uint4*>(to) = lo;
        *reinterpret_cast<uint4*>(to + 8 * 128) = hi;
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
    const double lscale = fabs((double)a.scale) * 1.4426950408889634;
    const float lhi = (float)lscale, llo = (float)(lscale - (double)lhi);
    for (int x = u0; x < u1 && ok;) {
      const Run r = run_at(x);
      const int rows = rows_of(r);
      Batch now{}, then = batch_at(r, 0, 0);
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
        if ((p & 31) == 0) now = then, then = batch_at(r, p + 32, 0);
        const int phys = __shfl_sync(FULL, now.phys, p & 31);
        const float sk = __shfl_sync(FULL, now.scale, p & 31);
        const float fh = colfac * sk, fl = fmaf(colfac, sk, -fh) + collow * sk;
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
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(v[e]));
          }
          if (phys >= 0 && mx * fh > m) {
            f = ex2(m - mx * fh);
            m = mx * fh;
            l *= f;
          }
        }
        // P's last readers; and the value warps are past page n - 4, whose row factors these replace
        if (n >= C::NP && !wait(&bar.pv_done[(n - C::NP) & 1], (n - C::NP) >> 1 & 1)) break;
#pragma unroll 1
        for (int again = 0;; ++again) {
          // a page that is not there: 2^-inf
          const float base = phys < 0 ? INFINITY : m == -INFINITY ? 0.0f : m;
          ps = 0.0f, mx = -INFINITY;
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
            // register 4 t + 2 ks + h8 holds tokens 16 ks + 8 h8 + 2 t + {0, 1} of the 32: the values' chunk order
            float sum[2] = {0.0f, 0.0f}, top[2] = {mx, mx};
#pragma unroll
            for (int z = 0; z < 16; ++z) {
              const int tok = (z >> 1 & 1) * 16 + (z & 1) * 8 + (z >> 2) * 2;
              float e[2];
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const float s = __uint_as_float(v[tok + w]);
                top[w] = fmaxf(top[w], s);
                e[w] = NQ == 2 ? ex2(fmaf(s, fl, fmaf(s, fh, -base))) * C::PSCALE : ex2(fmaf(s, fh, 7.0f - base));
                sum[w] += e[w];
              }
              if (NQ == 2) {
                const float w0 = whole(e[0]), w1 = whole(e[1]);
                hi[z] = pack_f16(w0, w1);
                lo[z] = pack_f16(e[0] - w0, e[1] - w1);
              } else {
                hi[z] = pack_f16(e[0], e[1]);
              }
            }
            mx = fmaxf(top[0], top[1]);
            ps += sum[0] + sum[1];
            tc_store16(mine + C::cP + b.i % C::NP * NQ * (kPage / 2) + 16 * y, hi);
            if (NQ == 2) tc_store16(mine + C::cP + kPage / 2 + 16 * y, lo);
          }
          mx *= fh;
          const bool move = phys >= 0 && mx > m + C::SLACK;
          if (again || !__any_sync(FULL, move)) break;
          if (move) {
            const float g = ex2(m - mx);
            f *= g;
            m = mx;
            l *= g;
          }
        }
        fac[fb.i * kWideRows + row] = f;
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
        if (ws.page && row < rows)
          ws.page[((size_t)r.seg * c.max_pages + r.first + p) * kWideRows + row] =
              make_float2(m == -INFINITY ? 0.0f : m, ps / C::PSCALE);
      }
      // the run's last products are done before the next run's Q takes the place of this one
      if (!ok || !wait(&bar.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
      tc_after();
      if (row < rows) {
        const size_t at = r.ends ? (size_t)geo.ctas + geo.segments + r.seg : (size_t)blockIdx.x + r.seg;
        ws.ml[at * kWideRows + row] = make_float2(m, l / C::PSCALE);
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
      Batch now{}, then = batch_at(r, 0, 1);
      float O[DH];
#pragma unroll
      for (int d = 0; d < DH; ++d) O[d] = 0.0f;
      for (int p = 0; p < r.pages && ok; ++p, b.next(), ob.next(), fb.next()) {
        if ((p & 31) == 0) now = then, then = batch_at(r, p + 32, 1);
        const float sv = __shfl_sync(FULL, now.scale, p & 31);
        if (!wait(&bar.p_full[fb.i], fb.ph) || !wait(&bar.pv_done[b.i], b.ph)) break;
        tc_after();
        if (moved[fb.i * kSoftWarps + quad]) {
          const float f = fac[fb.i * kWideRows + row];
#pragma unroll
          for (int d = 0; d < DH; ++d) O[d] *= f;
        }
#pragma unroll
        for (int d = 0; d < DH; d += 16) {
          uint32_t v[16];
          tc_load16(mine + ob.i * D + d, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) O[d + e] = fmaf(__uint_as_float(v[e]), sv, O[d + e]);
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.o_empty[ob.i]);
      }
      if (ok && row < rows) {
        const size_t at = r.ends ? (size_t)geo.ctas + geo.segments + r.seg : (size_t)blockIdx.x + r.seg;
        float4* o = reinterpret_cast<float4*>(ws.o + (at * kWideRows + row) * D + half * DH);
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
      if (tid < kWideRows) ws.ml[at * kWideRows + tid] = make_float2(NAN, NAN);
      x += r.pages;
    }
  if (warp == kMmaWarp) {
    // tensor memory is given back and the CTA ends: no product is under way then, also where a wait ran out
    tc_commit(elect_one(), &bar.drained);
    if (!__all_sync(FULL, mbar_wait(&bar.drained, 0, geo.wait_ns)) && lane == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TIMEOUT);
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// The fp32 rows of wide calls, and of others with many: 64 query rows by 16 tokens to a CTA of 256 threads, both products in registers: a thread
// holds the logits of two rows and two tokens, then D / 8 values of the two rows.  Rows 32 apart and tokens 8 apart
// belong to a thread, so that the lanes' 16-byte reads of neighbouring (padded) rows meet no bank twice.  Plain fp32.
// One warp to four rows (the split kernel's form, 16 exchanges between lanes a row) took 49 us for 512 rows of each of 8
// heads and 64 new tokens, with nothing else to do; this takes 25 (whole calls).
// Launched behind the wide or the split kernel and run beside it where an SM has room: it reads (from L2) what that
// kernel waited for before it let this one start, so the wait for that kernel comes last, for the join that follows.
constexpr int kRowsThreads = 256, kRowsRows = 64, kRT = 8 * kRowsRows / kRowsThreads;  // kRT rows of a thread
template <int D>
struct RowsSmem {
  float q[kRowsRows][D + 4], k[kRowTile][D + 4], v[kRowTile][D], p[kRowsRows][kRowTile + 4];
  uint32_t see[kRowsRows];
};
template <typename T, int D>
__global__ void __launch_bounds__(kRowsThreads, 3) k_kv8_rows(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo, Kv8Scratch ws) {
  griddep_launch();
  extern __shared__ __align__(16) uint8_t sm_raw[];
  RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>(sm_raw);
  constexpr int V = D / 8;  // vectors of eight elements in a row
  const int tid = threadIdx.x, rg = tid >> 3, tg = tid & 7;
  // blocks of a KV head's rows (with page lists too: their segments differ in the pages alone)
  const int blocks = (a.n * geo.G + kRowsRows - 1) / kRowsRows, x = blockIdx.x / blocks;
  const int f = x % geo.tiles, fresh = f - kPage / kRowTile, pair = x / geo.tiles;
  const struct { int s, h; } sg = {pair / c.n_kv_heads, pair % c.n_kv_heads};
  const int L = __ldcg(c.len + sg.s), cnt = a.counts ? __ldcg(a.counts + sg.s) : a.n;
  const int first = blockIdx.x % blocks * kRowsRows;
  auto slot = [&](int r) {  // of row first + r of the KV head
    if (a.pages) {
      const size_t seg = ((size_t)sg.s * a.n + (first + r) / geo.G) * c.n_kv_heads + sg.h;
      return (seg * geo.tiles + f) * geo.RB + (first + r) % geo.G;
    }
    return (((size_t)pair * geo.CB + (first + r) / geo.RB) * geo.tiles + f) * geo.RB + (first + r) % geo.RB;
  };
  int nv = 0, rows = 0;
  if (L >= 0 && L <= kPage * c.max_pages + kPage - 1 && cnt > 0 && cnt <= a.n) {
    nv = min(kRowTile, fresh < 0 ? L % kPage - f * kRowTile : a.k.data ? cnt - fresh * kRowTile : 0);
    rows = min(kRowsRows, cnt * geo.G - first);
  }
  if (nv > 0 && rows > 0) {  // the same for the whole block
    const float* tail = c.tail + kv8_pair(c, sg.s, sg.h) * 2 * kPage * D + f * kRowTile * D;
    const T* kn = static_cast<const T*>(a.k.data) + sg.s * a.k.seq + sg.h * a.k.head + (int64_t)fresh * kRowTile * a.k.row;
    const T* vn = static_cast<const T*>(a.v.data) + sg.s * a.v.seq + sg.h * a.v.head + (int64_t)fresh * kRowTile * a.v.row;
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
    for (int y = tid; y < 2 * kRowTile * V; y += kRowsThreads) {
      const int t = y / V % kRowTile, d = y % V * 8;
      const bool val = y >= kRowTile * V;
      float e[8] = {};
      if (t < nv) {
        if (fresh < 0) {
          const float4* p = reinterpret_cast<const float4*>(tail + (val ? kPage * D : 0) + t * D + d);
          *reinterpret_cast<float4*>(e) = __ldcg(p), *reinterpret_cast<float4*>(e + 4) = __ldcg(p + 1);
        } else {
          load8(val ? vn + (int64_t)t * a.v.row + d : kn + (int64_t)t * a.k.row + d, geo.vec & (val ? 4 : 2), e);
        }
      }
      float* to = val ? &sm.v[t][d] : &sm.k[t][d];
      *reinterpret_cast<float4*>(to) = *reinterpret_cast<float4*>(e);
      *reinterpret_cast<float4*>(to + 4) = *reinterpret_cast<float4*>(e + 4);
#pragma unroll
      for (int z = 0; z < 8; ++z) bad = bad || (val && !(fabsf(e[z]) <= 3.402823466e38f));
    }
#pragma unroll 4
    for (int y = tid; y < kRowsRows * V; y += kRowsThreads) {
      const int r = y / V, d = y % V * 8, rr = first + min(r, rows - 1);
      float e[8];
      load8(static_cast<const T*>(a.q.data) + sg.s * a.q.seq + (rr / geo.G) * a.q.row +
                (sg.h * geo.G + rr % geo.G) * a.q.head + d, geo.vec & 1, e);
      *reinterpret_cast<float4*>(&sm.q[r][d]) = *reinterpret_cast<float4*>(e);
      *reinterpret_cast<float4*>(&sm.q[r][d + 4]) = *reinterpret_cast<float4*>(e + 4);
    }
    if (tid < kRowsRows) {  // tokens that a row sees
      const int node = (first + min(tid, rows - 1)) / geo.G;
      uint32_t see = (1u << nv) - 1u;
      if (fresh >= 0) {
        const uint64_t mask = a.mask ? __ldcg(a.mask + (size_t)sg.s * a.n + node) : (node >= 63 ? ~0ull : (1ull << (node + 1)) - 1ull);
        see &= (uint32_t)(mask >> (fresh * kRowTile));
      }
      sm.see[tid] = see;
    }
    bad = __syncthreads_or(bad);
    float s[kRT][2] = {};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 k[2], q[kRT];
#pragma unroll
      for (int j = 0; j < 2; ++j) k[j] = *reinterpret_cast<const float4*>(&sm.k[8 * j + tg][d]);
#pragma unroll
      for (int i = 0; i < kRT; ++i) q[i] = *reinterpret_cast<const float4*>(&sm.q[kRowsRows / kRT * i + rg][d]);
#pragma unroll
      for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          s[i][j] = fmaf(q[i].w, k[j].w, fmaf(q[i].z, k[j].z, fmaf(q[i].y, k[j].y, fmaf(q[i].x, k[j].x, s[i][j]))));
    }
    const float qscale = a.scale * 1.4426950408889634f;
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      const int r = kRowsRows / kRT * i + rg;
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
    for (int t = 0; t < kRowTile; t += 4) {
      float p[kRT][4];
#pragma unroll
      for (int i = 0; i < kRT; ++i) *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(&sm.p[kRowsRows / kRT * i + rg][t]);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float4 v[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) v[e] = *reinterpret_cast<const float4*>(&sm.v[t + y][32 * e + 4 * tg]);
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
          if (bad && !(sm.see[kRowsRows / kRT * i + rg] >> (t + y) & 1u)) continue;  // 0 times it would not be 0
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
      if (kRowsRows / kRT * i + rg < rows)
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
          *reinterpret_cast<float4*>(ws.ro + slot(kRowsRows / kRT * i + rg) * D + 32 * e + 4 * tg) = o[i][e];
  }
  // the grid has not ended before the kernel in front has; only one CTA keeps its place for that
  if (blockIdx.x == 0) griddep_wait();
}

template <typename T, int D>
cudaError_t rows_run(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws, cudaStream_t st) {
  cudaError_t e = kv8_smem<k_kv8_rows<T, D>>(sizeof(RowsSmem<D>));
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.n * geo.G + kRowsRows - 1) / kRowsRows;
  return launch_pdl(k_kv8_rows<T, D>, dim3((unsigned)(blocks * geo.tiles * c.n_seqs * c.n_kv_heads)), dim3(kRowsThreads),
                    sizeof(RowsSmem<D>), st, c, a, geo, ws);
}

template <typename T, int D>
cudaError_t wide_run(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws, cudaStream_t st) {
  using C = Wide<T, D>;
  const size_t smem = 1024 + C::sPrefix + 4 * ((size_t)c.n_seqs + 1);
  cudaError_t e = kv8_smem<k_kv8_wide<T, D>>(1024 + C::sPrefix + 4 * (kKv8MaxSeqs + 1));
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_kv8_wide<T, D>, dim3((unsigned)geo.ctas), dim3(kWideThreads), smem, st, c, a, geo, ws);
  if (e != cudaSuccess) return e;
  return rows_run<T, D>(c, a, geo, ws, st);
}

}  // namespace

cudaError_t kv8_wide(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws, cudaStream_t st) {
  if (a.dtype == W4A8_F32) return c.head_dim == 64 ? wide_run<float, 64>(c, a, geo, ws, st) : wide_run<float, 128>(c, a, geo, ws, st);
  return c.head_dim == 64 ? wide_run<__nv_bfloat16, 64>(c, a, geo, ws, st) : wide_run<__nv_bfloat16, 128>(c, a, geo, ws, st);
}

cudaError_t kv8_rows(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws, cudaStream_t st) {
  if (a.dtype == W4A8_F32) return c.head_dim == 64 ? rows_run<float, 64>(c, a, geo, ws, st) : rows_run<float, 128>(c, a, geo, ws, st);
  return c.head_dim == 64 ? rows_run<__nv_bfloat16, 64>(c, a, geo, ws, st) : rows_run<__nv_bfloat16, 128>(c, a, geo, ws, st);
}

}  // namespace w4a8
