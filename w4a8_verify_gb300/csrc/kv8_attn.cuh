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
// bf16 calls start the accumulators at -128 2^-24 sum(q) (or sum(P)), which takes the 128 out again.  fp32 calls
// make whole numbers of the codes (the byte under the exponent of 1024, minus 1152): the tensor core aligns
// products by their exponents and drops what is below, and subnormal operands cost the sums 2^-20 of the
// largest product (outputs 1.9e-6 off in the 2-norm at 4096 tokens; 2.4e-7 with whole numbers).
//
// fp32 operands are split, q = qh + ql and P = Ph + Pl in f16: hi and lo are neighbouring columns of a tile (four
// rows to a tile instead of eight), so the accumulator pair of a thread holds both products of one row and adds
// them there.  Rows of q are scaled by a power of two, to a largest magnitude of at most 2^11; qh is the nearest
// whole number, so the sums of qh with the codes are whole numbers (times 2^-24) that f32 holds, and the tensor
// core's truncating additions do not touch them.  (With qh the nearest f16 the logits were off by 3e-7 relative.)
// P is scaled by 2^15.
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
// Warps of a CTA (one CTA per SM): twelve where a warp holds one tile (168 registers), eight where it holds two.
__host__ __device__ constexpr int kv8_warps(int TW) { return TW == 1 ? 12 : 8; }
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
// power of two that takes a largest magnitude into [2^10, 2^11) (1 where it is not finite)
__device__ __forceinline__ float f16_scale(float amax) {
  const int ex = (int)(__float_as_uint(amax) >> 23) & 255;
  return ex == 255 ? 1.0f : __uint_as_float((uint32_t)min(254, 264 - ex) << 23);
}

// ---------------------------------------------------------------------------- the split kernel

template <typename T, int D, int TW, int WC>
struct Kv8Split {
  static constexpr bool SPLIT = sizeof(T) == 4;
  static constexpr int RPT = SPLIT ? 4 : 8;        // rows of an 8-column tile
  static constexpr int NC = SPLIT ? 1 : 2;         // rows of a thread in a tile
  static constexpr int RB = WC * TW * RPT;         // rows of a column block
  static constexpr int WARPS = kv8_warps(TW);
  static constexpr int NG = WARPS / WC;            // workers of a CTA
  static constexpr int HALF = kPage * D;           // bytes of a ring entry (kRowTile rows of D floats as well)
  static constexpr int NS = kKv8RingBytes / HALF / NG;  // ring entries of a worker
  static constexpr int BACK = WC == 1 ? 0 : WC;    // entries left unfilled so that the copier does not wait for the slowest warp
  static constexpr int KS = D / 16, DT = D / 16;
  static constexpr float UNIT = SPLIT ? 1.0f : 16777216.0f;  // codes enter the products divided by this
};

// What a lane knows of one unit of its worker's range.
constexpr int kNoUnit = INT_MIN, kNewUnit = INT_MIN + 1, kNewUnits = kKv8MaxRows / kRowTile;
struct Kv8Unit {
  int src;      // >= 0: (pair, physical page); kNoUnit: nothing; kNewUnit + f: tile f of the new rows; else
                // -1 - (4 pair + f): tile f of the open page
  int seg;      // segment
  int u;        // unit inside the segment
  float sk, sv;
};

template <typename T, int D, int TW, int WC>
__global__ void __launch_bounds__(32 * kv8_warps(TW), 1) k_kv8_split(w4a8_kv8_cache c, w4a8_kv8_attn a, Kv8Geom geo,
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

  for (int i = tid; i < C::NG * C::NS; i += 32 * C::WARPS) {
    mbar_init(&full[i], 1);
    mbar_init(&empty[i], WC);
  }
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  griddep_enter();

  // units before each sequence
  for (int s = tid; s < S; s += 32 * C::WARPS) {
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
    for (int s = tid; s <= S; s += 32 * C::WARPS) ws.prefix[s] = prefix[s];

  const int U = prefix[S];
  const int W = min(geo.workers, U), worker = grp * gridDim.x + blockIdx.x;  // few units spread over the SMs
  if (worker >= W) return;
  const int u0 = worker_begin(worker, W, U), u1 = worker_begin(worker + 1, W, U);

  // The lane's unit x: its segment, page and scales (32 units in parallel, so the table's latency is paid once).
  auto look = [&](int x) -> Kv8Unit {
    Kv8Unit r{kNoUnit, -1, 0, 0.0f, 0.0f};
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
    const size_t pair = kv8_pair(c, s, h);
    if (u >= un.pages) {
      const int f = u - un.pages;
      r.src = f < un.open ? -1 - (int)(pair * 4 + f) : kNewUnit + f - un.open;
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
    const int phys = kv8_phys(c, pair, p);
    if (phys < 0) return r;
    r.src = (int)kv8_page(c, pair, phys);
    const float2 sc = *reinterpret_cast<const float2*>(c.scales + (size_t)r.src * 2);
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
      const int from = __shfl_sync(FULL, jl < cbase + 32 ? cur.src : nxt.src, (jl - cbase) & 31);
      if (from < kNewUnit + kNewUnits) {  // new rows do not go through the ring
        ++jl;
        continue;
      }
      bool good = true;
      if (lane == 0) {
        if (WC > 1 && iph > 0) good = mbar_wait(&empty[is], (iph - 1) & 1);
        if (good) {
          mbar_expect_tx(&full[is], C::HALF);
          // half a page of codes, or the keys or values of 16 fp32 rows: as many bytes
          const void* p = from >= 0 ? static_cast<const void*>(c.codes + ((size_t)from * 2 + half) * C::HALF)
                                    : c.tail + ((size_t)((-1 - from) >> 2) * 2 + half) * (kPage * D) +
                                          ((-1 - from) & 3) * (kRowTile * D);
          bulk_g2s(ring + (size_t)is * C::HALF, p, C::HALF, &full[is]);
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
  float O[DT][TW][4], m[TW][NC], l[TW][NC], colfac[TW][NC], collow[TW][NC], seed[TW][2];
  int seg = -1, seg_u = 0, seg_j = 0, s_cur = 0, h_cur = 0, i_cur = 0, cb_cur = 0, cnt_cur = 0, L_cur = 0;
  bool act = false;
  // the factor of a column, log2(e) scale UNIT / (power of two of its row), as hi + lo
  const double lscale = (double)a.scale * 1.4426950408889634 * (double)C::UNIT;
  const float lhi = (float)lscale, llo = (float)(lscale - (double)lhi);
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
          if (SPLIT) f[e] = g & 1 ? f[e] - rintf(f[e]) : rintf(f[e]);
          if (!SPLIT) sum += __half2float(__float2half_rn(f[e]));
        }
        qf[j][x][0] = pack_f16(f[0], f[1]);
        qf[j][x][1] = pack_f16(f[2], f[3]);
      }
      // per-column values, from the lanes of column g to the lanes of accumulator columns 2t, 2t + 1
      const float down = 1.0f / up;
      if (SPLIT) {
        const float dn = __shfl_sync(FULL, down, 8 * t);
        colfac[j][0] = lhi * dn;
        collow[j][0] = llo * dn;
        seed[j][0] = seed[j][1] = 0.0f;
      } else {
        sum += __shfl_xor_sync(FULL, sum, 1);
        sum += __shfl_xor_sync(FULL, sum, 2);
        sum *= -128.0f / 16777216.0f;
#pragma unroll
        for (int x = 0; x < NC; ++x) {
          const float dn = __shfl_sync(FULL, down, 4 * (2 * t + x));
          colfac[j][x] = lhi * dn;
          collow[j][x] = llo * dn;
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
          const float f = sum == 0.0f ? 0.0f : C::UNIT / sum;
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
            o[16 * d + g] = (SPLIT ? O[d][j][0] + O[d][j][1] : O[d][j][x]) * C::UNIT;
            o[16 * d + g + 8] = (SPLIT ? O[d][j][2] + O[d][j][3] : O[d][j][x + 2]) * C::UNIT;
          }
        }
      }
  };

  // Softmax of MT x 16 tokens: x (SPLIT: entries 0 and 2) becomes P 2^15 in place, pf its B fragments, cc the factor
  // of the old sums, psum the sum over the tokens of a lane's own P.  PAGE: x are
  // sums of codes and the logit is x (fh + fl), taken relative to the maximum with one rounding at the size of
  // the difference: a relative error of a factor is one of the softmax's temperature, which large logits multiply.
  float cc[TW][NC], psum[TW][NC];
  auto soft = [&](auto mtc, auto pagec, float (&x)[4][TW][4], uint32_t (&pf)[4][TW][2], const float (&fh)[TW][NC],
                  const float (&fl)[TW][NC]) {
    constexpr int MT = decltype(mtc)::value;
    constexpr bool PAGE = decltype(pagec)::value;
#pragma unroll
    for (int j = 0; j < TW; ++j) {
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = y; e < 4; e += 2) mx = fmaxf(mx, PAGE ? x[i][j][e] * fh[j][y] : x[i][j][e]);
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
          for (int e = y; e < 4; e += 2) {
            if (SPLIT) {
              float v = PAGE ? fmaf(x[i][j][e], fh[j][y], -base) : x[i][j][e] - base;
              if (PAGE) v = fmaf(x[i][j][e], fl[j][y], v);
              x[i][j][e] = ex2(v) * 32768.0f;
            } else {
              x[i][j][e] = ex2(PAGE ? fmaf(x[i][j][e], fh[j][y], 15.0f - base) : x[i][j][e] + (15.0f - base));
            }
            psum[j][y] += x[i][j][e];
          }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t pk;
          if (SPLIT) {
            const float p = x[i][j][2 * e];
            pk = pack_f16(p, p - __half2float(__float2half_rn(p)));
          } else {
            pk = pack_f16(x[i][j][2 * e], x[i][j][2 * e + 1]);
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
          for (int e = 0; e < 4; ++e) x[i][j][e] = SPLIT ? 0.0f : seed[j][e & 1];
#pragma unroll
      for (int kp = 0; kp < D / 32; ++kp)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(kb + ((i * (D / 32) + kp) * 32 + lane) * 16);
          uint32_t a0[4], a1[4];
          codes_f16<SPLIT>(w.x, a0[0], a0[2]);
          codes_f16<SPLIT>(w.y, a0[1], a0[3]);
          codes_f16<SPLIT>(w.z, a1[0], a1[2]);
          codes_f16<SPLIT>(w.w, a1[1], a1[3]);
#pragma unroll
          for (int j = 0; j < TW; ++j) {
            mma_f16(x[i][j], a0, qf[j][2 * kp][0], qf[j][2 * kp][1]);
            mma_f16(x[i][j], a1, qf[j][2 * kp + 1][0], qf[j][2 * kp + 1][1]);
          }
        }
    }
    release_half();
    if (act) {
      if (SPLIT) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < TW; ++j) x[i][j][0] += x[i][j][1], x[i][j][2] += x[i][j][3];  // hi + lo
      }
      float fh[TW][NC], fl[TW][NC];
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          fh[j][y] = colfac[j][y] * sk;
          fl[j][y] = fmaf(colfac[j][y], sk, -fh[j][y]) + collow[j][y] * sk;
        }
      soft(std::integral_constant<int, 4>{}, std::true_type{}, x, pf, fh, fl);
    }
    const uint8_t* vb = wait_half();
    if (!ok) return;
    if (act) {
      // -128 2^-24 sum(P) of the columns, P as the product uses it: a row of constants times P
      float ps[TW][4];
      if (!SPLIT) {
        const uint32_t k = 0x80808080u;  // f16 -128 2^-24 = 0x8080
        const uint32_t ones[4] = {k, k, k, k};
#pragma unroll
        for (int j = 0; j < TW; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) ps[j][e] = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_f16(ps[j], ones, pf[i][j][0], pf[i][j][1]);
        }
      }
      if (ws.page) {
#pragma unroll
        for (int j = 0; j < TW; ++j)
#pragma unroll
          for (int y = 0; y < NC; ++y) {
            float v = psum[j][y];
            v += __shfl_xor_sync(FULL, v, 4);
            v += __shfl_xor_sync(FULL, v, 8);
            v += __shfl_xor_sync(FULL, v, 16);
            if (g == 0)
              ws.page[((size_t)seg * c.max_pages + u) * C::RB + (wg * TW + j) * C::RPT + (SPLIT ? t : 2 * t + y)] =
                  make_float2(m[j][y], v);
          }
      }
      bool same = true;  // no row of the warp has a new maximum
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int y = 0; y < NC; ++y) same = same && cc[j][y] == 1.0f;
      if (!__all_sync(FULL, same)) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int j = 0; j < TW; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[d][j][e] *= cc[j][(e & 1) * (NC - 1)];
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
          for (int e = 0; e < 4; ++e) O[d][j][e] = fmaf(o[j][e], sv, O[d][j][e]);
      }
    }
    release_half();
  };

  // Sixteen rows in floating point, nv of them valid: the open page's from the ring (fresh = -1), or tile `fresh` of
  // the new rows from memory.  Keys and values as f16 hi (+ lo) of the value times a power of two, from the
  // tile's largest magnitude.
  auto rows = [&](int nv, int fresh) {
    float x[4][TW][4];
    uint32_t pf[4][TW][2];
    float kv[D / 32][2][8];  // dims 32 kp + 8 t .. + 7 of rows g, g + 8
    if (fresh < 0) {
      const float* kb = reinterpret_cast<const float*>(wait_half());
      if (!ok) return;
#pragma unroll
      for (int kp = 0; kp < D / 32; ++kp)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float4* p = reinterpret_cast<const float4*>(kb + (g + 8 * b) * D + 32 * kp + 8 * t);
          const float4 v0 = p[0], v1 = p[1];  // rows behind the last one are read and not used
          const float w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) kv[kp][b][e] = g + 8 * b < nv ? w[e] : 0.0f;
        }
      release_half();
    } else if (act) {
      const T* kn = static_cast<const T*>(a.k.data) + s_cur * a.k.seq + h_cur * a.k.head;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = fresh * kRowTile + g + 8 * b;
        const T* p = kn + (int64_t)r * a.k.row + 8 * t;
#pragma unroll
        for (int kp = 0; kp < D / 32; ++kp) {
          if (g + 8 * b >= nv) {
#pragma unroll
            for (int e = 0; e < 8; ++e) kv[kp][b][e] = 0.0f;
          } else if (geo.vec & 2) {
            uint4 w[sizeof(T) / 2];
#pragma unroll
            for (int e = 0; e < (int)sizeof(T) / 2; ++e) w[e] = reinterpret_cast<const uint4*>(p + 32 * kp)[e];
            const T* q = reinterpret_cast<const T*>(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) kv[kp][b][e] = kv8_load(q + e);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) kv[kp][b][e] = kv8_load(p + 32 * kp + e);
          }
        }
      }
    }
    if (!act) {
      if (fresh < 0) {
        wait_half();
        if (ok) release_half();
      }
      return;
    }
    float km = 0.0f, vm = 0.0f;
#pragma unroll
    for (int kp = 0; kp < D / 32; ++kp)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) km = fabsf(kv[kp][b][e]) <= 3.402823466e38f ? fmaxf(km, fabsf(kv[kp][b][e])) : km;
    km = warp_max(km);
    const float kup = f16_scale(km);
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
      const float* v0 = kv[kp][0];
      const float* v1 = kv[kp][1];
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
    const float kdown = (1.0f / kup) / C::UNIT;
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
        const float fh = colfac[j][y] * kdown, fl = collow[j][y] * kdown;  // a power of two: exact
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool see = bits >> (g + 8 * e) & 1u;
          vis |= (uint32_t)see << ((j * NC + y) * 2 + e);
          const float v = SPLIT ? x[0][j][2 * e] + x[0][j][2 * e + 1] : x[0][j][2 * e + y];
          x[0][j][2 * e + y] = see ? fmaf(v, fh, v * fl) : -INFINITY;
        }
      }
    soft(std::integral_constant<int, 1>{}, std::false_type{}, x, pf, colfac, collow);
    // entry (e >> 1, e & 1, d): tokens 2t + (e & 1) + 8 (e >> 2), dims 16 d + g + 8 (e >> 1 & 1)
    float v[DT][8];
    if (fresh < 0) {
      const float* vb = reinterpret_cast<const float*>(wait_half());
      if (!ok) return;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 2 * t + (e & 1) + 8 * (e >> 2);
          v[d][e] = r < nv ? vb[r * D + 16 * d + g + 8 * ((e >> 1) & 1)] : 0.0f;
        }
    } else {
      const T* vn = static_cast<const T*>(a.v.data) + s_cur * a.v.seq + h_cur * a.v.head;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 2 * t + (e & 1) + 8 * (e >> 2);
          v[d][e] = r < nv ? kv8_load(vn + (int64_t)(fresh * kRowTile + r) * a.v.row + 16 * d + g + 8 * ((e >> 1) & 1)) : 0.0f;
        }
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 8; ++e) vm = max_nan(vm, fabsf(v[d][e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) vm = max_nan(vm, __shfl_xor_sync(FULL, vm, o));
    if (vm <= 3.402823466e38f) {
      const float vup = f16_scale(vm), vdown = (1.0f / vup) / C::UNIT;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)  // operand register e: dim g + 8 (e & 1), tokens 2t, 2t + 1, + 8 (e >> 1)
          split(v[d][(e >> 1) * 4 + (e & 1) * 2] * vup, v[d][(e >> 1) * 4 + (e & 1) * 2 + 1] * vup, hi[e], lo[e]);
#pragma unroll
        for (int j = 0; j < TW; ++j) {
          float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16(o, hi, pf[0][j][0], pf[0][j][1]);
          if (SPLIT) mma_f16(o, lo, pf[0][j][0], pf[0][j][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) O[d][j][e] = fmaf(o[e], vdown, O[d][j][e] * cc[j][(e & 1) * (NC - 1)]);
        }
      }
      if (fresh < 0) release_half();
      return;
    }
    // A value is not finite: 0 times it would reach rows that do not see it, so each row adds what it sees.
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[d][j][e] *= cc[j][(e & 1) * (NC - 1)];
    // entry q of a lane's values (token 2t + (q & 1) + 8 (q >> 1)) is handed to the lanes of the same dims
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll 1
      for (int tt = 0; tt < 4; ++tt) {
        const int r = 2 * tt + (q & 1) + 8 * (q >> 1), src = (r & 7) << 2 | t;
#pragma unroll
        for (int j = 0; j < TW; ++j)
#pragma unroll
          for (int y = 0; y < NC; ++y) {
            const float p = __shfl_sync(FULL, x[0][j][2 * (q >> 1) + y], src) / C::UNIT;
            const uint32_t see = __shfl_sync(FULL, vis, src) >> ((j * NC + y) * 2 + (q >> 1)) & 1u;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const float v0 = __shfl_sync(FULL, v[d][(q >> 1) * 4 + (q & 1)], g << 2 | tt);
              const float v1 = __shfl_sync(FULL, v[d][(q >> 1) * 4 + 2 + (q & 1)], g << 2 | tt);
              if (see) O[d][j][y] = fmaf(p, v0, O[d][j][y]);
              if (see) O[d][j][y + 2] = fmaf(p, v1, O[d][j][y + 2]);
            }
          }
      }
    if (fresh < 0) release_half();
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
    const int from = __shfl_sync(FULL, cur.src, src), sg = __shfl_sync(FULL, cur.seg, src);
    const int u = __shfl_sync(FULL, cur.u, src);
    if (sg != seg) {
      if (seg >= 0) flush(last_u + 1);
      begin(sg, u, j);
    }
    last_u = u;
    if (from >= 0) {
      page(__shfl_sync(FULL, cur.sk, src), __shfl_sync(FULL, cur.sv, src), u);
    } else if (from >= kNewUnit + kNewUnits) {
      rows(min(kRowTile, L_cur % kPage - ((-1 - from) & 3) * kRowTile), -1);
    } else if (from != kNoUnit) {
      const int f = from - kNewUnit;
      rows(min(kRowTile, cnt_cur - f * kRowTile), f);
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
  return launch_pdl(k_kv8_split<T, D, TW, WC>, dim3((unsigned)(geo.workers / C::NG)), dim3(32 * C::WARPS), smem, st, c, a,
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
