// Norm and rotary positions of the heads of queries and keys, in one pass.
//
// A head's D dims belong to D / 16 lanes; a lane has the eight first and the eight second dims of its eight pairs, so
// the rotation stays in its registers and the norm is one sum over the head's lanes.  A warp takes one token: its
// lanes keep the cosines and sines of their eight frequencies for all heads that the warp goes through.
//
// The angle of position p at frequency f is the fraction of p f in whole turns.  f is held in units of 2^-64 turns, so p f
// modulo one turn is one wrapping 64-bit product, exact for every 32-bit position; the quarter turn comes from its upper
// bits, and what is left of it, at most an eighth of a turn, goes to the sine and cosine as fp32.  (fp32 angles are off by
// 2^-5 at position 2^19.)
//
// Bound by memory once rows are many: each value is read and written once (32768 tokens of 40 heads of 128 in bf16: 108 us,
// 91% of the copy rate; the rows of a warp's next round are on their way while it works on one, and 32 warps an SM do
// that: two rounds ahead with 16 warps took 164 us, the gains in registers with 24 warps 132).  Few tokens: the heads of a
// token are dealt to several warps, each with the angles once more; 5 us for 256 tokens, bound by latency.
#include "kv8.cuh"

#include <cmath>
#include <type_traits>

using namespace w4a8;

namespace {

constexpr int kRotThreads = 256;
constexpr int kMaxAxes = 4;

struct RotGeom {
  int segs, iters;  // warps of a token, head rounds of each
  float inv_dim;
};

// Cosine and sine of turn 2^-64 turns.
__device__ __forceinline__ void unit(uint64_t turn, float& c, float& s) {
  const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
  // what is left, -1/8 .. 1/8 of a turn, in half turns: the low 62 bits as a signed number
  const float half_turns = (float)(int32_t)((turn << 2) >> 32) * 1.16415321826934814453125e-10f;  // 2^-33
  float a, b;
  sincospif(half_turns, &b, &a);
  c = quarter & 1u ? b : a;
  s = quarter & 1u ? a : b;
  if (quarter == 1u || quarter == 2u) c = -c;
  if (quarter & 2u) s = -s;
}

// LPH lanes to a head (a power of two, D / 16 of them used); vec: 16-byte access to q, k, q_out, k_out, q_gain, k_gain (bits 0 to 5);
// WIDE: to all of them, known at compile time (with the other ways in the code bf16 does not fit 64 registers: 134 us for 108).
template <typename T, int LPH, bool WIDE>
__global__ void __launch_bounds__(kRotThreads, WIDE && sizeof(T) == 2 ? 4 : 3) k_qk_rotary(w4a8_qk_rotary_args a, RotGeom geo, int vec) {
  griddep_enter();
  constexpr int HPW = 32 / LPH;
  const int lane = threadIdx.x & 31, sub = lane % LPH, D = a.head_dim;
  const int64_t task = (int64_t)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5), token = task / geo.segs;
  if (token >= (int64_t)a.n_seqs * a.n) return;
  const int s = (int)(token / a.n), j = (int)(token % a.n), seg = (int)(task % geo.segs);
  if (a.counts && j >= a.counts[s]) return;
  const bool live = sub < D / 16, turned = sub < a.rot_dim / 16, halves = turned && !a.neighbours;
  const int d0 = halves ? 8 * sub : 16 * sub, d1 = halves ? a.rot_dim / 2 + 8 * sub : 16 * sub + 8;
  const int H = a.n_heads + a.n_kv_heads;
  auto place = [&](int it, bool& on, bool& key) -> int64_t {  // of round it: the lane's head, and its offset from q's or k's data
    const int h = (seg * geo.iters + it) * HPW + lane / LPH;
    on = live && h < H && it < geo.iters, key = h >= a.n_heads;
    const w4a8_rows& in = key ? a.k : a.q;
    return s * in.seq + j * in.row + (int64_t)(key ? h - a.n_heads : h) * in.head;
  };
  Eight<T> x0{}, y0{};  // of the round to come
  auto fetch = [&](int it) {
    bool on, key;
    const int64_t at = place(it, on, key);
    if (!on) return;
    const T* p = static_cast<const T*>(key ? a.k.data : a.q.data) + at;
    x0.load(p + d0, WIDE || (vec >> (int)key & 1));
    y0.load(p + d1, WIDE || (vec >> (int)key & 1));
  };
  fetch(0);
  // the lanes of a frequency octet share its angles: PER each, then exchanged
  constexpr int PER = 8 / HPW;
  float c[8], sn[8];
  {
    float mc[PER], ms[PER];
    const int64_t start = a.start ? a.start[s] : 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int i = 8 * sub + lane / LPH * PER + e;
      mc[e] = ms[e] = 0.0f;
      if (!turned) continue;
      int ax = a.axis ? a.axis[i] : 0;
      ax = ax < a.n_axes ? ax : 0;
      const int64_t p = start + (a.pos ? a.pos[((int64_t)ax * a.n_seqs + s) * a.n + j] : j);
      unit((uint64_t)p * a.turns[i], mc[e], ms[e]);
      mc[e] *= a.factor, ms[e] *= a.factor;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = __shfl_sync(0xffffffffu, mc[e % PER], e / PER * LPH + sub);
      sn[e] = __shfl_sync(0xffffffffu, ms[e % PER], e / PER * LPH + sub);
    }
  }
  for (int it = 0; it < geo.iters; ++it) {
    bool on, key;
    (void)place(it, on, key);
    float x[8], y[8];
    x0.get(x), y0.get(y);
    fetch(it + 1);
    if (a.norm) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float r = __frsqrt_rn(fmaf(sum, geo.inv_dim, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= r, y[e] *= r;
      const float* g = key ? a.k_gain : a.q_gain;
      if (g && live) {  // from L1: in registers they would cost a third of the warps
        float u[8], v[8];
        if (WIDE || (vec >> (4 + (int)key) & 1)) {
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            *reinterpret_cast<float4*>(u + e) = *reinterpret_cast<const float4*>(g + d0 + e);
            *reinterpret_cast<float4*>(v + e) = *reinterpret_cast<const float4*>(g + d1 + e);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = g[d0 + e], v[e] = g[d1 + e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= u[e], y[e] *= v[e];
      }
    }
    if (halves) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = x[e], v = y[e];
        x[e] = fmaf(u, c[e], -(v * sn[e]));
        y[e] = fmaf(v, c[e], u * sn[e]);
      }
    } else if (turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float& u = e < 4 ? x[2 * e] : y[2 * e - 8];
        float& v = e < 4 ? x[2 * e + 1] : y[2 * e - 7];
        const float u0 = u, v0 = v;
        u = fmaf(u0, c[e], -(v0 * sn[e]));
        v = fmaf(v0, c[e], u0 * sn[e]);
      }
    }
    if (on) {
      const w4a8_rows& out = key ? a.k_out : a.q_out;
      const int h = (seg * geo.iters + it) * HPW + lane / LPH;
      T* p = static_cast<T*>(out.data) + s * out.seq + j * out.row + (int64_t)(key ? h - a.n_heads : h) * out.head;
      Eight<T> x1, y1;
      x1.set(x), y1.set(y);
      x1.store(p + d0, WIDE || (vec >> (2 + (int)key) & 1));
      y1.store(p + d1, WIDE || (vec >> (2 + (int)key) & 1));
    }
  }
}

bool same_rows(const w4a8_rows& x, const w4a8_rows& y, int S, int n, int heads) {
  return x.data == y.data && (S == 1 || x.seq == y.seq) && (n == 1 || x.row == y.row) && (heads == 1 || x.head == y.head);
}

}  // namespace

W4A8_API w4a8_status w4a8_rotary_turns(const double* inv_freq, int n, uint64_t* turns) {
  if (!inv_freq || !turns || n < 1) return W4A8_ERR_ARG;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return W4A8_ERR_ARG;
  for (int i = 0; i < n; ++i) {
    const double t = inv_freq[i] / 6.283185307179586476925286766559;
    double f = t - std::floor(t);  // 0 <= f, and below 1 but for a t just below a whole number
    if (f >= 1.0) f = 0.0;
    turns[i] = (uint64_t)(f * 18446744073709551616.0);
  }
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_qk_rotary(const w4a8_qk_rotary_args* arg, void* stream) {
  if (!arg) return W4A8_ERR_ARG;
  const w4a8_qk_rotary_args& a = *arg;
  if (a.n_seqs < 1 || a.n < 1 || a.n_heads < 1 || a.n_kv_heads < 0 || a.head_dim < 16 || a.head_dim > 256 ||
      a.head_dim % 16 || a.rot_dim < 0 || a.rot_dim > a.head_dim || a.rot_dim % 16 || a.n_axes < 1 || a.n_axes > kMaxAxes)
    return W4A8_ERR_SHAPE;
  const __int128 rows = (__int128)a.n_seqs * a.n * ((int64_t)a.n_heads + a.n_kv_heads);
  if (rows >= (__int128)1 << 31) return W4A8_ERR_SHAPE;
  const bool keys = a.n_kv_heads > 0;
  const size_t el = kv8_dtype(a.dtype) ? kv8_elem(a.dtype) : 0;
  if (!el || !a.q.data || !a.q_out.data || keys != (a.k.data != nullptr) || keys != (a.k_out.data != nullptr) ||
      (a.rot_dim > 0 && !a.turns) || !(a.eps >= 0.0f) || !(a.eps <= 3.402823466e38f) || !(fabsf(a.factor) <= 3.402823466e38f))
    return W4A8_ERR_ARG;
  if (!aligned(a.q.data, el) || !aligned(a.k.data, el) || !aligned(a.q_out.data, el) || !aligned(a.k_out.data, el) ||
      !aligned(a.turns, 8) || !aligned(a.pos, 4) || !aligned(a.start, 4) || !aligned(a.counts, 4) || !aligned(a.q_gain, 4) ||
      !aligned(a.k_gain, 4))
    return W4A8_ERR_ARG;
  const int S = a.n_seqs, n = a.n, Hq = a.n_heads, Hk = a.n_kv_heads, D = a.head_dim;
  if (rows_overlap(a.q_out, S, n, Hq, D, kMaxDifferences) || (!same_rows(a.q, a.q_out, S, n, Hq) && rows_meet(a.q_out, Hq, a.q, Hq, S, n, D, el)))
    return W4A8_ERR_ARG;
  if (keys && (rows_overlap(a.k_out, S, n, Hk, D, kMaxDifferences) || rows_meet(a.k_out, Hk, a.q_out, Hq, S, n, D, el) ||
               (!same_rows(a.k, a.k_out, S, n, Hk) && rows_meet(a.k_out, Hk, a.k, Hk, S, n, D, el)) ||
               rows_meet(a.k_out, Hk, a.q, Hq, S, n, D, el) || rows_meet(a.q_out, Hq, a.k, Hk, S, n, D, el)))
    return W4A8_ERR_ARG;
  const size_t half = (size_t)a.rot_dim / 2, places = 4 * (size_t)S * n * a.n_axes, gain = 4 * (size_t)D;
  auto on = [&](const w4a8_rows& out, int heads) {  // what other warps of the call still read
    const auto at = [&](const void* p, size_t bytes) { return rows_touch(out, heads, S, n, D, el, p, bytes); };
    return at(a.turns, 8 * half) || at(a.axis, half) || at(a.pos, places) || at(a.start, 4 * (size_t)S) ||
           at(a.counts, 4 * (size_t)S) || at(a.q_gain, gain) || at(a.k_gain, gain);
  };
  if (on(a.q_out, Hq) || (keys && on(a.k_out, Hk))) return W4A8_ERR_ARG;
  auto wide = [&](const w4a8_rows& r) { return !r.data || kv8_vec_rows(r, a.dtype) ? 1 : 0; };
  const int vec = wide(a.q) | wide(a.k) << 1 | wide(a.q_out) << 2 | wide(a.k_out) << 3 |
                  (aligned(a.q_gain, 16) ? 16 : 0) | (aligned(a.k_gain, 16) ? 32 : 0);
  const int lph = D <= 64 ? 4 : D <= 128 ? 8 : 16;
  const int rounds = (Hq + Hk + 32 / lph - 1) / (32 / lph);
  const int64_t tokens = (int64_t)S * n;
  // Head rounds of a warp: all of a token's where there are warps enough for the SMs without splitting, else so many that
  // each of 152 x 16 warps has one task (an SM holds 24, and 32 of the wide bf16 kernel).
  constexpr int64_t kWarps = 152 * 16;
  const int64_t most = (tokens * rounds + kWarps - 1) / kWarps;
  RotGeom geo;
  geo.iters = (int)(most < rounds ? most : rounds);
  geo.segs = (rounds + geo.iters - 1) / geo.iters;
  geo.inv_dim = 1.0f / (float)D;
  const int64_t tasks = tokens * geo.segs;
  const dim3 grid((unsigned)((tasks + kRotThreads / 32 - 1) / (kRotThreads / 32)));
  cudaStream_t st = as_stream(stream);
  auto run = [&](auto four, auto eight, auto sixteen) {
    return launch_pdl(lph == 4 ? four : lph == 8 ? eight : sixteen, grid, dim3(kRotThreads), 0, st, a, geo, vec);
  };
  auto typed = [&](auto t, auto all) {
    using T = decltype(t);
    constexpr bool WIDE = decltype(all)::value;
    return run(k_qk_rotary<T, 4, WIDE>, k_qk_rotary<T, 8, WIDE>, k_qk_rotary<T, 16, WIDE>);
  };
  const std::true_type yes{};
  const std::false_type no{};
  if (a.dtype == W4A8_F32) W4A8_CUDA_TRY(vec == 63 ? typed(float{}, yes) : typed(float{}, no));
  else W4A8_CUDA_TRY(vec == 63 ? typed(__nv_bfloat16{}, yes) : typed(__nv_bfloat16{}, no));
  return W4A8_OK;
}
