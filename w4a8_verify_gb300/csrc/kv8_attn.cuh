// Attention of new rows over the 8-bit key/value cache: the split kernel and its launch.
//
// For query head hq of new row i (KV head h = hq / G), over the tokens t that the row sees
//   l_t = scale q . k_t,  out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x = l log2(e), m = max x
// in one pass: per page the running maximum m, sum l and values O of each row become
//   m' = max(m, max x),  c = 2^(m - m'),  O = O c + s_V (P C_V),  l = l c + sum P,  P = 2^(x - m').
//
// Both products run transposed on the tensor cores (m16n8k16, f16): S^T = C_K Q^T and O^T = C_V^T P^T, so the
// 8-bit codes are the 16-row operand and the few query rows of a KV head fill 8-column tiles, half the padding of
// a 16-row query tile.  A page is stored in the operand's own order (the header documents it), so one 16-byte
// shared-memory load gives a lane the bytes of two k-steps, and one byte permute turns two codes into two f16:
// the byte u = code + 128 in the low half of a 16-bit lane is the subnormal u 2^-24, exact, as in the W4A8 matmul.
// bf16 calls start the accumulators at -128 2^-24 sum(q) (or sum(P)), which takes the 128 out again; fp32 calls
// subtract it from the operand (exact) so that the sums do not carry it.
//
// fp32 operands are split, q = qh + ql and P = Ph + Pl in f16: hi and lo are neighbouring columns of a tile (four
// rows to a tile instead of eight), so the accumulator pair of a thread holds both products of one row and adds
// them there.  Rows of q are scaled by a power of two to use f16's range; P is scaled by 2^15.
// The transposed P fragments are made with movmatrix: no shared memory in the softmax.
//
// Work: every (sequence, KV head, block of rows) is a segment of units, one per page and one per 16 fp32 rows
// (open page, new rows).  The units of all segments, end to end, are cut into equal ranges, one for each worker,
// so ragged batches balance.  A worker is a group of WC warps that share a page and hold different columns; it
// has its own ring of bulk copies (half a page each) and never waits for another worker.  A worker that
// holds a whole segment writes its output; the parts of a cut segment are joined by k_kv8_join.
#pragma once
#include <type_traits>

#include "kv8.cuh"

namespace w4a8 {

constexpr int kKv8Ctas = 152;         // one per SM of a GB300
constexpr int kKv8Warps = 8;          // warps of a CTA, one CTA per SM (registers: 8 warps x 255)
constexpr int kKv8RingBytes = 196608; // ring of half pages per SM: 24 of 8 KB or 48 of 4 KB
constexpr int kRowTile = 16;          // fp32 rows of one unit

struct Kv8Geom {       // of one call, the same for every kernel of it
  int n, G, R;         // new rows; query heads per KV head; query rows of a segment's problem (n G, or G with lists)
  int RB, CB;          // rows of a column block; column blocks
  int workers;
  int vec;             // bit 0: q rows, bit 1: new key rows may be read 16 bytes at a time
};

struct Kv8Scratch {    // workspace pointers
  int* prefix;         // [n_seqs + 1] units before each sequence
  float2* ml;          // [2 workers][RB] maximum, sum of a part
  float* o;            // [2 workers][RB][D] its values
  float2* fin;         // [n_seqs][n][n_heads] maximum, sum of each row (with mass)
  float2* page;        // [segments][max_pages][RB] maximum, sum of each page (with mass)
};

// Units of a segment of sequence s (L, cnt valid): pages, then 16-row tiles of the open page and the new rows.
struct Kv8Units {
  int pages, open, fresh;  // units of each kind
  __device__ int total() const { return pages + open + fresh; }
};
__device__ __forceinline__ Kv8Units kv8_units(const w4a8_kv8_attn& a, int L, int cnt) {
  const int whole = L / kPage;
  return {a.pages ? min(a.top_k, whole) : whole, (L % kPage + kRowTile - 1) / kRowTile,
          a.k.data ? (cnt + kRowTile - 1) / kRowTile : 0};
}
// Segments of a sequence: (KV head, column block), or (row, KV head) with page lists.
__device__ __forceinline__ int kv8_segments(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& g, int cnt) {
  return a.pages ? cnt * c.n_kv_heads : cnt > 0 ? c.n_kv_heads * g.CB : 0;
}
// First unit of worker w of W <= U over U units, and the worker of unit u.
__device__ __forceinline__ int worker_begin(int w, int W, int U) { return (int)((int64_t)w * U / W); }
__device__ __forceinline__ int worker_of(int u, int W, int U) { return (int)((((int64_t)u + 1) * W - 1) / U); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// two f16 operands from bytes 2 i, 2 i + 1 of w: u 2^-24, or (u - 128) 2^-24 if SIGNED
template <bool SIGNED>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = __byte_perm(w, 0, 0x4140);
  hi = __byte_perm(w, 0, 0x4342);
  if (SIGNED) {
    const uint32_t bias = 0x00800080u;
    const __half2 b = *reinterpret_cast<const __half2*>(&bias);
    const __half2 l = __hsub2(*reinterpret_cast<__half2*>(&lo), b), h = __hsub2(*reinterpret_cast<__half2*>(&hi), b);
    lo = *reinterpret_cast<const uint32_t*>(&l);
    hi = *reinterpret_cast<const uint32_t*>(&h);
  }
}
// power of two that takes a largest magnitude into [2^13, 2^14) (1 where it is not finite)
__device__ __forceinline__ float f16_scale(float amax) {
  const int ex = (int)(__float_as_uint(amax) >> 23) & 255;
  return ex == 255 ? 1.0f : __uint_as_float((uint32_t)min(254, 267 - ex) << 23);
}

// ---------------------------------------------------------------------------- the split kernel

template <typename T, int D, int TW, int WC>
struct Kv8Split {
  static constexpr bool SPLIT = sizeof(T) == 4;
  static constexpr int RPT = SPLIT ? 4 : 8;        // rows of an 8-column tile
  static constexpr int NC = SPLIT ? 1 : 2;         // rows of a thread in a tile
  static constexpr int RB = WC * TW * RPT;         // rows of a column block
  static constexpr int NG = kKv8Warps / WC;        // workers of a CTA
  static constexpr int HALF = kPage * D;           // bytes of a ring entry
  static constexpr int NS = kKv8RingBytes / HALF / NG;  // ring entries of a worker
  static constexpr int BACK = WC == 1 ? 0 : WC;    // entries left unfilled so that the copier does not wait for the slowest warp
  static constexpr int KS = D / 16, DT = D / 16;
};

// What a lane knows of one unit of its worker's range.
struct Kv8Unit {
  int page;     // >= 0: (pair, physical page); -1: nothing; <= -2: row tile -2 - page (tail 0..3, new rows 4..7)
  int seg;      // segment
  int u;        // unit inside the segment
  float sk, sv;
};

template <typename T, int D, int TW, int WC>
__global__ void __launch_bounds__(32 * kKv8Warps, 1) k_kv8_split(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo,
                                                                  Kv8Scratch ws) {
  using C = Kv8Split<T, D, TW, WC>;
  constexpr bool SPLIT = C::SPLIT;
  constexpr int NC = C::NC, KS = C::KS, DT = C::DT;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kKv8RingBytes);
  uint64_t* empty = full + C::NG * C::NS;
  int* prefix = reinterpret_cast<int*>(empty + C::NG * C::NS);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp / WC, wg = warp % WC;  // worker of the CTA, warp of the worker
  const int g = lane >> 2, t = lane & 3;
  const int H = c.n_kv_heads, S = c.n_seqs;

  for (int i = tid; i < C::NG * C::NS; i += 32 * kKv8Warps) {
    mbar_init(&full[i], 1);
    mbar_init(&empty[i], WC);
  }
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  griddep_enter();

  // units before each sequence
  for (int s = tid; s < S; s += 32 * kKv8Warps) {
    const int L = kv8_len(c, c.len, s), cnt = kv8_count(c, a.counts, s, a.n);
    prefix[s + 1] = L < 0 || cnt < 0 ? 0 : kv8_units(a, L, cnt).total() * kv8_segments(c, a, geo, cnt);
  }
  if (tid == 0) prefix[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int b = 0; b < S; b += 32) {
      int v = b + lane < S ? prefix[b + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(FULL, v, o);
        if (lane >= o) v += x;
      }
      if (b + lane < S) prefix[b + lane + 1] = carry + v;
      carry += __shfl_sync(FULL, v, 31);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int s = tid; s <= S; s += 32 * kKv8Warps) ws.prefix[s] = prefix[s];

  const int U = prefix[S];
  const int W = min(geo.workers, U), worker = grp * gridDim.x + blockIdx.x;  // few units spread over the SMs
  if (worker >= W) return;
  const int u0 = worker_begin(worker, W, U), u1 = worker_begin(worker + 1, W, U);

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
    const int per = un.total(), q = (x - prefix[s]) / per, u = (x - prefix[s]) % per;
    const int h = a.pages ? q % H : q / geo.CB;
    r.seg = a.pages ? s * a.n * H + q : s * H * geo.CB + q;
    r.u = u;
    if (u >= un.pages) {
      r.page = -2 - (u < un.pages + un.open ? u - un.pages : 4 + u - un.pages - un.open);
      return r;
    }
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
    const size_t pair = kv8_pair(c, s, h);
    const int phys = kv8_phys(c, pair, p);
    if (phys < 0) return r;
    r.page = (int)kv8_page(c, pair, phys);
    const float2 sc = *reinterpret_cast<const float2*>(c.scales + (size_t)r.page * 2);
    r.sk = sc.x;
    r.sv = sc.y;
    return r;
  };

  uint8_t* ring = sm + (size_t)grp * C::NS * C::HALF;
  full += grp * C::NS;
  empty += grp * C::NS;
  Kv8Unit cur = look(u0 + lane), nxt = look(u0 + 32 + lane);
  const int nu = u1 - u0;
  int jl = 0, half = 0;                 // next unit and half to copy
  int is = 0, iph = 0, in_ring = 0;     // ring entry, its phase, entries issued and not yet consumed
  int cs = 0, cph = 0;                  // entry to consume next
  bool ok = true;
  int cbase = 0;                        // first unit of `cur`

  // Copies ahead as far as the ring and the two batches of units allow (one warp of the worker).
  auto copy_ahead = [&](int room) {
    while (in_ring < room && jl < nu && jl < cbase + 64) {
      const int pg = __shfl_sync(FULL, jl < cbase + 32 ? cur.page : nxt.page, (jl - cbase) & 31);
      if (pg < 0) {
        ++jl;
        continue;
      }
      bool good = true;
      if (lane == 0) {
        if (WC > 1 && iph > 0) good = mbar_wait(&empty[is], (iph - 1) & 1);
        if (good) {
          mbar_expect_tx(&full[is], C::HALF);
          bulk_g2s(ring + (size_t)is * C::HALF, c.codes + ((size_t)pg * 2 + half) * C::HALF, C::HALF, &full[is]);
        }
      }
      good = __shfl_sync(FULL, good, 0);
      if (!good) {
        ok = false;
        return;
      }
      ++in_ring;
      if (++is == C::NS) is = 0, ++iph;
      jl += half;
      half ^= 1;
    }
  };
  auto wait_half = [&]() -> const uint8_t* {
    if (!mbar_wait(&full[cs], cph & 1)) ok = false;
    ok = __all_sync(FULL, ok);
    return ring + (size_t)cs * C::HALF;
  };
  auto release_half = [&]() {
    __syncwarp();
    if (WC > 1 && lane == 0) mbar_arrive(&empty[cs]);
    if (++cs == C::NS) cs = 0, ++cph;
    --in_ring;
    if (wg == 0) copy_ahead(C::NS - C::BACK);
  };
  // in_ring of a warp that does not copy is not used: only warp 0 counts entries
  if (wg == 0) copy_ahead(C::NS);

  // ---- state of the segment
  uint32_t qf[TW][KS][2];
  float O[DT][TW][4], m[TW][NC], l[TW][NC], colfac[TW][NC], seed[TW][2];
  int seg = -1, seg_u = 0, seg_j = 0, s_cur = 0, h_cur = 0, i_cur = 0, cb_cur = 0, cnt_cur = 0, L_cur = 0;
  bool act = false;
  const float lscale = a.scale * 1.4426950408889634f;
  auto row_of = [&](int j, int col) {  // query row (of the segment's R) of column col of the warp's tile j
    return cb_cur * C::RB + (wg * TW + j) * C::RPT + (SPLIT ? col >> 1 : col);
  };
  auto row_ok = [&](int r) { return r < geo.R && (a.pages || r / geo.G < cnt_cur); };
  auto row_node = [&](int r) { return a.pages ? i_cur : r / geo.G; };
  auto row_head = [&](int r) { return h_cur * geo.G + (a.pages ? r : r % geo.G); };

  auto begin = [&](int sg, int u, int j0) {  // the part starts at the segment's unit u, the range's unit j0
    seg = sg;
    seg_u = u;
    seg_j = j0;
    if (a.pages) {
      h_cur = sg % H;
      i_cur = sg / H % a.n;
      s_cur = sg / H / a.n;
      cb_cur = 0;
    } else {
      cb_cur = sg % geo.CB;
      h_cur = sg / geo.CB % H;
      s_cur = sg / geo.CB / H;
    }
    cnt_cur = a.counts ? a.counts[s_cur] : a.n;
    L_cur = c.len[s_cur];
    act = row_ok(cb_cur * C::RB + wg * TW * C::RPT);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[d][j][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < TW; ++j) {
#pragma unroll
      for (int x = 0; x < NC; ++x) m[j][x] = -INFINITY, l[j][x] = 0.0f;
      const int r = row_of(j, g);
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
          if (SPLIT && (g & 1)) f[e] -= __half2float(__float2half_rn(f[e]));
          if (!SPLIT) sum += __half2float(__float2half_rn(f[e]));
        }
        qf[j][x][0] = pack_f16(f[0], f[1]);
        qf[j][x][1] = pack_f16(f[2], f[3]);
      }
      // per-column values, from the lanes of column g to the lanes of accumulator columns 2t, 2t + 1
      const float cf = lscale * 16777216.0f * (1.0f / up);
      if (SPLIT) {
        colfac[j][0] = __shfl_sync(FULL, cf, 8 * t);
        seed[j][0] = seed[j][1] = 0.0f;
      } else {
        sum += __shfl_xor_sync(FULL, sum, 1);
        sum += __shfl_xor_sync(FULL, sum, 2);
        sum *= -128.0f / 16777216.0f;
#pragma unroll
        for (int x = 0; x < NC; ++x) {
          colfac[j][x] = __shfl_sync(FULL, cf, 4 * (2 * t + x));
          seed[j][x] = __shfl_sync(FULL, sum, 4 * (2 * t + x));
        }
      }
    }
  };

  // Ends the worker's part of a segment, its units [seg_u, end): the output of a whole segment, else a part.
  auto flush = [&](int end) {
    const bool whole = seg_u == 0 && end == kv8_units(a, L_cur, cnt_cur).total();
    const size_t slot = (2 * (size_t)worker + (seg_j == 0 ? 0 : 1)) * C::RB;
    if (!act) return;
#pragma unroll
    for (int j = 0; j < TW; ++j)
#pragma unroll
      for (int x = 0; x < NC; ++x) {
        float sum = l[j][x];
        sum += __shfl_xor_sync(FULL, sum, 4);
        sum += __shfl_xor_sync(FULL, sum, 8);
        sum += __shfl_xor_sync(FULL, sum, 16);
        const int r = row_of(j, 2 * t + x);
        if (!row_ok(r)) continue;
        if (whole) {
          const float f = sum == 0.0f ? 0.0f : 16777216.0f / sum;
          T* out = static_cast<T*>(a.out.data) + s_cur * a.out.seq + row_node(r) * a.out.row + row_head(r) * a.out.head;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            kv8_store(out + 16 * d + g, (SPLIT ? O[d][j][0] + O[d][j][1] : O[d][j][x]) * f);
            kv8_store(out + 16 * d + g + 8, (SPLIT ? O[d][j][2] + O[d][j][3] : O[d][j][x + 2]) * f);
          }
          if (ws.fin && g == 0)
            ws.fin[((size_t)s_cur * a.n + row_node(r)) * a.n_heads + row_head(r)] = make_float2(m[j][x], sum);
        } else {
          const size_t at = slot + (r - cb_cur * C::RB);
          if (g == 0) ws.ml[at] = make_float2(m[j][x], sum);
          float* o = ws.o + at * D;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            o[16 * d + g] = (SPLIT ? O[d][j][0] + O[d][j][1] : O[d][j][x]) * 16777216.0f;
            o[16 * d + g + 8] = (SPLIT ? O[d][j][2] + O[d][j][3] : O[d][j][x + 2]) * 16777216.0f;
          }
        }
      }
  };

  // Softmax of MT x 16 tokens: x (log2 units; SPLIT: entries 0 and 2) becomes P 2^15 in place, pf its B fragments,
  // cc the factor of the old sums, psum the sum over the tokens of a lane's own P (as used by the product).
  float cc[TW][NC], psum[TW][NC];
  auto soft = [&](auto mtc, float (&x)[4][TW][4], uint32_t (&pf)[4][TW][2]) {
    constexpr int MT = decltype(mtc)::value;
#pragma unroll
    for (int j = 0; j < TW; ++j) {
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        float mx = x[0][j][y];
#pragma unroll
        for (int i = 0; i < MT; ++i) mx = fmaxf(mx, fmaxf(x[i][j][y], x[i][j][y + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
        const float mn = fmaxf(m[j][y], mx), base = mn == -INFINITY ? 0.0f : mn;
        cc[j][y] = ex2(m[j][y] - base);
        m[j][y] = mn;
        psum[j][y] = 0.0f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = y; e < 4; e += 2) x[i][j][e] = ex2(x[i][j][e] - base) * 32768.0f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t pk;
          if (SPLIT) {
            const float p = x[i][j][2 * e];
            psum[j][0] += p;
            pk = pack_f16(p, p - __half2float(__float2half_rn(p)));
          } else {
            pk = pack_f16(x[i][j][2 * e], x[i][j][2 * e + 1]);
            const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&pk));
            psum[j][0] += r.x;
            psum[j][NC - 1] += r.y;
          }
          pf[i][j][e] = movmatrix(pk);
        }
#pragma unroll
      for (int y = 0; y < NC; ++y) l[j][y] = fmaf(l[j][y], cc[j][y], psum[j][y]);
    }
  };

  // A page: S^T = C_K Q^T, softmax, O^T += C_V^T P^T.
  auto page = [&](float sk, float sv, int u) {
    float x[4][TW][4];
    uint32_t pf[4][TW][2];
    const uint8_t* kb = wait_half();
    if (!ok) return;
    if (act) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TW; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][j][e] = seed[j][e & 1];
#pragma unroll
      for (int kp = 0; kp < D / 32; ++kp)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(kb + ((i * (D / 32) + kp) * 32 + lane) * 16);
          uint32_t af[4];
          codes_f16<SPLIT>(w.x, af[0], af[2]);
          codes_f16<SPLIT>(w.y, af[1], af[3]);
#pragma unroll
          for (int j = 0; j < TW; ++j) mma_f16(x[i][j], af, qf[j][2 * kp][0], qf[j][2 * kp][1]);
          codes_f16<SPLIT>(w.z, af[0], af[2]);
          codes_f16<SPLIT>(w.w, af[1], af[3]);
#pragma unroll
          for (int j = 0; j < TW; ++j) mma_f16(x[i][j], af, qf[j][2 * kp + 1][0], qf[j][2 * kp + 1][1]);
        }
    }
    release_half();
    if (act) {
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (SPLIT) {
            const float f = colfac[j][0] * sk;
            x[i][j][0] = (x[i][j][0] + x[i][j][1]) * f;
            x[i][j][2] = (x[i][j][2] + x[i][j][3]) * f;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][j][e] *= colfac[j][(e & 1) * (NC - 1)] * sk;
          }
        }
      soft(std::integral_constant<int, 4>{}, x, pf);
    }
    const uint8_t* vb = wait_half();
    if (!ok) return;
    if (act) {
      float ps[TW][2];
      if (!SPLIT || ws.page) {
#pragma unroll
        for (int j = 0; j < TW; ++j)
#pragma unroll
          for (int y = 0; y < NC; ++y) {
            float v = psum[j][y];
            v += __shfl_xor_sync(FULL, v, 4);
            v += __shfl_xor_sync(FULL, v, 8);
            v += __shfl_xor_sync(FULL, v, 16);
            if (ws.page && g == 0)
              ws.page[((size_t)seg * c.max_pages + u) * C::RB + (wg * TW + j) * C::RPT + (SPLIT ? t : 2 * t + y)] =
                  make_float2(m[j][y], v);
            ps[j][y] = v * (-128.0f / 16777216.0f);
          }
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        float o[TW][4];
#pragma unroll
        for (int j = 0; j < TW; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = SPLIT ? 0.0f : ps[j][e & 1];
#pragma unroll
        for (int kp = 0; kp < 2; ++kp) {
          const uint4 w = *reinterpret_cast<const uint4*>(vb + ((d * 2 + kp) * 32 + lane) * 16);
          uint32_t af[4];
          codes_f16<SPLIT>(w.x, af[0], af[2]);
          codes_f16<SPLIT>(w.y, af[1], af[3]);
#pragma unroll
          for (int j = 0; j < TW; ++j) mma_f16(o[j], af, pf[2 * kp][j][0], pf[2 * kp][j][1]);
          codes_f16<SPLIT>(w.z, af[0], af[2]);
          codes_f16<SPLIT>(w.w, af[1], af[3]);
#pragma unroll
          for (int j = 0; j < TW; ++j) mma_f16(o[j], af, pf[2 * kp + 1][j][0], pf[2 * kp + 1][j][1]);
        }
#pragma unroll
        for (int j = 0; j < TW; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[d][j][e] = fmaf(o[j][e], sv, O[d][j][e] * cc[j][(e & 1) * (NC - 1)]);
      }
    }
    release_half();
  };

  // Sixteen rows in floating point (open page: fresh = -1; new rows: fresh = their tile), nv of them valid:
  // keys and values as f16 hi (+ lo) of the value times a power of two, from the tile's largest magnitude.
  auto rows = [&](auto* kr, int64_t kstep, auto* vr, int64_t vstep, int nv, int fresh, bool vec) {
    if (!act) return;
    using E = std::remove_cv_t<std::remove_pointer_t<decltype(kr)>>;
    float x[4][TW][4];
    uint32_t pf[4][TW][2];
    auto key8 = [&](int r, int kp, float (&v)[8]) {  // dims 32 kp + 8 t .. + 7 of row r
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
      if (r >= nv) return;
      const E* p = kr + (int64_t)r * kstep + 32 * kp + 8 * t;
      if (vec) {
        uint4 w[sizeof(E) / 2];
#pragma unroll
        for (int e = 0; e < (int)sizeof(E) / 2; ++e) w[e] = reinterpret_cast<const uint4*>(p)[e];
        const E* q = reinterpret_cast<const E*>(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = kv8_load(q + e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = kv8_load(p + e);
      }
    };
    auto value = [&](int r, int d) { return r < nv ? kv8_load(vr + (int64_t)r * vstep + d) : 0.0f; };
    float km = 0.0f, vm = 0.0f;
#pragma unroll
    for (int kp = 0; kp < D / 32; ++kp)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float v[8];
        key8(g + 8 * b, kp, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) km = fabsf(v[e]) <= 3.402823466e38f ? fmaxf(km, fabsf(v[e])) : km;
      }
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 8; ++e) vm = max_nan(vm, fabsf(value(2 * t + (e & 1) + 8 * (e >> 2), 16 * d + g + 8 * ((e >> 1) & 1))));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      km = fmaxf(km, __shfl_xor_sync(FULL, km, o));
      vm = max_nan(vm, __shfl_xor_sync(FULL, vm, o));
    }
    const float kup = f16_scale(km), vup = f16_scale(vm);
    auto split = [&](float v0, float v1, uint32_t& hi, uint32_t& lo) {
      hi = pack_f16(v0, v1);
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      lo = SPLIT ? pack_f16(v0 - h.x, v1 - h.y) : 0u;
    };
#pragma unroll
    for (int j = 0; j < TW; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[0][j][e] = 0.0f;
#pragma unroll
    for (int kp = 0; kp < D / 32; ++kp) {
      float v0[8], v1[8];
      key8(g, kp, v0);
      key8(g + 8, kp, v1);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t hi[4], lo[4];
        split(v0[4 * ks] * kup, v0[4 * ks + 1] * kup, hi[0], lo[0]);
        split(v1[4 * ks] * kup, v1[4 * ks + 1] * kup, hi[1], lo[1]);
        split(v0[4 * ks + 2] * kup, v0[4 * ks + 3] * kup, hi[2], lo[2]);
        split(v1[4 * ks + 2] * kup, v1[4 * ks + 3] * kup, hi[3], lo[3]);
#pragma unroll
        for (int j = 0; j < TW; ++j) {
          mma_f16(x[0][j], hi, qf[j][2 * kp + ks][0], qf[j][2 * kp + ks][1]);
          if (SPLIT) mma_f16(x[0][j], lo, qf[j][2 * kp + ks][0], qf[j][2 * kp + ks][1]);
        }
      }
    }
    uint32_t vis = 0;  // bit (j NC + y) 2 + e: the row of column y sees token g + 8 e
    const float kdown = (1.0f / kup) / 16777216.0f;
#pragma unroll
    for (int j = 0; j < TW; ++j)
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        const int r = row_of(j, 2 * t + y);
        uint32_t bits = (1u << nv) - 1u;
        if (fresh >= 0) {
          const int i = row_node(r);
          const uint64_t mask = !row_ok(r) ? 0ull
                                : a.mask   ? a.mask[(size_t)s_cur * a.n + i]
                                           : (i >= 63 ? ~0ull : (1ull << (i + 1)) - 1ull);
          bits &= (uint32_t)(mask >> (kRowTile * fresh));
        }
        const float f = colfac[j][y] * kdown;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool see = bits >> (g + 8 * e) & 1u;
          vis |= (uint32_t)see << ((j * NC + y) * 2 + e);
          const float v = SPLIT ? x[0][j][2 * e] + x[0][j][2 * e + 1] : x[0][j][2 * e + y];
          x[0][j][2 * e + y] = see ? v * f : -INFINITY;
        }
      }
    soft(std::integral_constant<int, 1>{}, x, pf);
    if (vm <= 3.402823466e38f) {
      const float vdown = (1.0f / vup) / 16777216.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)  // operand register e: dim g + 8 (e & 1), tokens 2t, 2t + 1, + 8 (e >> 1)
          split(value(2 * t + 8 * (e >> 1), 16 * d + g + 8 * (e & 1)) * vup,
                value(2 * t + 1 + 8 * (e >> 1), 16 * d + g + 8 * (e & 1)) * vup, hi[e], lo[e]);
#pragma unroll
        for (int j = 0; j < TW; ++j) {
          float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16(o, hi, pf[0][j][0], pf[0][j][1]);
          if (SPLIT) mma_f16(o, lo, pf[0][j][0], pf[0][j][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) O[d][j][e] = fmaf(o[e], vdown, O[d][j][e] * cc[j][(e & 1) * (NC - 1)]);
        }
      }
      return;
    }
    // A value is not finite: 0 times it would reach rows that do not see it, so each row adds what it sees.
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[d][j][e] *= cc[j][(e & 1) * (NC - 1)];
#pragma unroll 1
    for (int r = 0; r < nv; ++r)
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          const int src = (r & 7) << 2 | t;
          const float p0 = __shfl_sync(FULL, x[0][j][y], src), p1 = __shfl_sync(FULL, x[0][j][y + 2], src);
          const float p = (r < 8 ? p0 : p1) / 16777216.0f;
          const uint32_t see = __shfl_sync(FULL, vis, src) >> ((j * NC + y) * 2 + (r >> 3)) & 1u;
          if (!see) continue;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            O[d][j][y] = fmaf(p, value(r, 16 * d + g), O[d][j][y]);
            O[d][j][y + 2] = fmaf(p, value(r, 16 * d + g + 8), O[d][j][y + 2]);
          }
        }
  };

  // ---- the range
  int last_u = 0;
  for (int j = 0; j < nu && ok; ++j) {
    if (j - cbase == 32) {
      cbase += 32;
      cur = nxt;
      nxt = look(u0 + cbase + 32 + lane);
      if (wg == 0) copy_ahead(C::NS - C::BACK);
    }
    const int src = j - cbase;
    const int pg = __shfl_sync(FULL, cur.page, src), sg = __shfl_sync(FULL, cur.seg, src);
    const int u = __shfl_sync(FULL, cur.u, src);
    if (sg != seg) {
      if (seg >= 0) flush(last_u + 1);
      begin(sg, u, j);
    }
    last_u = u;
    if (pg >= 0) {
      page(__shfl_sync(FULL, cur.sk, src), __shfl_sync(FULL, cur.sv, src), u);
    } else if (pg <= -2) {
      const int tile = -2 - pg;
      if (tile < 4) {
        const float* kt = c.tail + kv8_pair(c, s_cur, h_cur) * 2 * kPage * D + tile * kRowTile * D;
        rows(kt, D, kt + kPage * D, D, min(kRowTile, L_cur % kPage - tile * kRowTile), -1, true);
      } else {
        const int f = tile - 4;
        const T* kn = static_cast<const T*>(a.k.data) + s_cur * a.k.seq + h_cur * a.k.head + f * kRowTile * a.k.row;
        const T* vn = static_cast<const T*>(a.v.data) + s_cur * a.v.seq + h_cur * a.v.head + f * kRowTile * a.v.row;
        rows(kn, a.k.row, vn, a.v.row, min(kRowTile, cnt_cur - f * kRowTile), f, (geo.vec & 2) != 0);
      }
    }
  }
  if (ok) {
    flush(last_u + 1);
    return;
  }
  // A bounded wait expired: report it, and wait (again bounded) for the copies still in flight.
  if (lane == 0) atomicOr(c.ctl, (unsigned)FLAG_ERR_TIMEOUT);
  if (wg == 0)
    for (; in_ring > 0; --in_ring) {
      (void)mbar_wait(&full[cs], cph & 1);
      if (++cs == C::NS) cs = 0, ++cph;
    }
}

// ---------------------------------------------------------------------------- launch

// Warps and tiles for R query rows of a problem (RPT rows to a tile): as few warps on a page as hold its tiles two
// each (one for a single tile), so that narrow calls work on more pages at once.
struct Kv8Shape {
  int TW, WC;
};
inline Kv8Shape kv8_shape(int R, int dtype) {
  const int rpt = dtype == W4A8_F32 ? 4 : 8, tiles = (R + rpt - 1) / rpt;
  if (tiles <= 1) return {1, 1};
  if (tiles <= 2) return {2, 1};
  if (tiles <= 4) return {2, 2};
  if (tiles <= 8) return {2, 4};
  return {2, 8};
}

inline size_t kv8_split_smem(int S, int entries) { return (size_t)kKv8RingBytes + 16 * (size_t)entries + 4 * ((size_t)S + 1); }

template <typename T, int D, int TW, int WC>
cudaError_t kv8_split_launch(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws,
                             cudaStream_t st) {
  using C = Kv8Split<T, D, TW, WC>;
  const size_t most = kv8_split_smem(kKv8MaxSeqs, C::NG * C::NS), smem = kv8_split_smem(c.n_seqs, C::NG * C::NS);
  cudaError_t e = cudaFuncSetAttribute(k_kv8_split<T, D, TW, WC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_kv8_split<T, D, TW, WC>, dim3((unsigned)(geo.workers / C::NG)), dim3(32 * kKv8Warps), smem, st, c, a,
                    geo, ws);
}
template <typename T, int D>
cudaError_t kv8_split_dispatch(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws,
                               cudaStream_t st) {
  const Kv8Shape sh = kv8_shape(geo.R, a.dtype);
  if (sh.WC == 8) return kv8_split_launch<T, D, 2, 8>(c, a, geo, ws, st);
  if (sh.WC == 4) return kv8_split_launch<T, D, 2, 4>(c, a, geo, ws, st);
  if (sh.WC == 2) return kv8_split_launch<T, D, 2, 2>(c, a, geo, ws, st);
  if (sh.TW == 2) return kv8_split_launch<T, D, 2, 1>(c, a, geo, ws, st);
  return kv8_split_launch<T, D, 1, 1>(c, a, geo, ws, st);
}
// one translation unit per head size and element type
cudaError_t kv8_split_f32_d64(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
cudaError_t kv8_split_f32_d128(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
cudaError_t kv8_split_bf16_d64(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);
cudaError_t kv8_split_bf16_d128(const w4a8_kv8_cache&, const w4a8_kv8_attn&, const Kv8Geom&, const Kv8Scratch&, cudaStream_t);

}  // namespace w4a8
