// Choosing pages of the 8-bit cache: by score for one query's sparse attention, by accumulated
// attention weight for eviction.  Both keep the k largest of a head's values, ties to the lowest page.
#include "kv8.cuh"

using namespace w4a8;

namespace {

// Order-preserving key of a score; NaN counts as infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = __int_as_float(0x7f800000);
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kInfKey = 0xff800000u;     // the key of infinity
constexpr uint32_t kForcedKey = 0xffffffffu;  // of the first and last pages: above any score's

// The keys of the k largest of P (0 < k < P) are those above *T and *ties of those equal to it.  Forced pages and
// infinities are counted first; the others are looked for by their distance from the smallest, eight bits at a
// time from the highest that differs (the leading bits of scores are much alike: bins of whole bytes would put most keys
// into two or three of them, one atomic after the other).  keys in shared memory; hist: 256 words.
__device__ void kth_largest(const uint32_t* keys, int P, int k, uint32_t* hist, uint32_t* T, int* ties) {
  __shared__ uint32_t s_low, s_high, s_bin;
  __shared__ int s_top, s_left, s_bins;
  if (threadIdx.x == 0) s_low = ~0u, s_high = 0u, s_top = 0;
  __syncthreads();
  uint32_t low = ~0u, high = 0u;
  int top = 0;  // forced pages and infinities, and in the upper half the forced ones (at most 16384 of either)
  for (int i = threadIdx.x; i < P; i += blockDim.x) {
    const uint32_t x = keys[i];
    if (x >= kInfKey) top += x == kForcedKey ? 0x10001 : 1;
    else low = min(low, x), high = max(high, x);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  top = __reduce_add_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) atomicMin(&s_low, low), atomicMax(&s_high, high), atomicAdd(&s_top, top);
  __syncthreads();
  low = s_low, high = s_high, top = s_top & 0xffff;
  const int forced = s_top >> 16;
  if (top >= k) {  // the forced pages, and infinities if they leave room
    *T = forced >= k ? kForcedKey : kInfKey;
    *ties = forced >= k ? k : k - forced;
    return;
  }
  int left = k - top, bits = high > low ? 32 - __clz(high - low) : 0;
  uint32_t prefix = 0;  // of the distance of the key looked for: its bits above `bits`
  while (bits > 0) {
    const int lo = max(bits - 8, 0);
    for (int i = threadIdx.x; i < 256; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += blockDim.x) {
      const uint32_t x = keys[i], d = x - low;
      if (x < kInfKey && (bits == 32 ? 0u : d >> bits) == prefix) atomicAdd(&hist[(d >> lo) & ((1u << (bits - lo)) - 1u)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // lane l: bins 255 - 8l .. 248 - 8l, from the top
      const int lane = threadIdx.x;
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = (int)hist[255 - 8 * lane - i];
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += v;
      }
      above -= sum;
      if (above < left && above + sum >= left) {
        int i = 0;
        while (above + c[i] < left) above += c[i++];
        s_bin = (uint32_t)(255 - 8 * lane - i);
        s_left = left - above;
        s_bins = c[i];
      }
    }
    __syncthreads();
    prefix = prefix << (bits - lo) | s_bin;
    left = s_left;
    bits = lo;
    const int in_bin = s_bins;
    __syncthreads();
    if (in_bin == left) break;  // the whole bin belongs to them: above anything below it
  }
  // bits > 0: every key at or above the bin's first one
  *T = low + (prefix << bits) - (bits > 0 ? 1u : 0u);
  *ties = bits > 0 ? 0 : left;
}

// Calls put(i, kept, rank) for every i in [0, P): kept where key i is among the k largest (ties to the lowest i),
// rank = how many of the same kind come before it.  All threads of the block take part.
template <typename F>
__device__ void split_largest(const uint32_t* keys, int P, int k, uint32_t* hist, F put) {
  __shared__ int s_warp[32];
  uint32_t T = 0;
  int ties = P;  // k >= P: every key is kept
  if (k < P && k > 0) kth_largest(keys, P, k, hist, &T, &ties);
  const bool all = k >= P, none = k <= 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int gt0 = 0, eq0 = 0;  // counts before this round's block of keys
  for (int base = 0; base < P; base += blockDim.x) {
    const int i = base + threadIdx.x;
    const bool in = i < P;
    const bool gt = in && !none && (all || keys[i] > T), eq = in && !none && !all && keys[i] == T;
    const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[warp] = __popc(bg) << 16 | __popc(be);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < warps; ++w) {
      before += w < warp ? s_warp[w] : 0;
      total += s_warp[w];
    }
    __syncthreads();
    const unsigned lt = (1u << lane) - 1u;
    const int ngt = gt0 + (before >> 16) + __popc(bg & lt), neq = eq0 + (before & 0xffff) + __popc(be & lt);
    if (in) {
      const int rank = ngt + min(neq, ties);
      const bool kept = gt || (eq && neq < ties);
      put(i, kept, kept ? rank : i - rank);
    }
    gt0 += total >> 16;
    eq0 += total & 0xffff;
  }
}

// ---------------------------------------------------------------------------- selection

constexpr int kScoreThreads = 256;
constexpr int kScorePages = 128;  // pages of one CTA

// Keys of the scores of one (sequence, new row, KV head) and a range of pages.  Integer dot products of the
// query codes with the pages' code sums (dp2a: two 16-bit sums by two 8-bit codes); eight lanes share a page, whose sums are
// read once for the group's queries.  Bound by instructions where rows are many (53% of the issue slots) and by latency
// where they are few: 16 sequences of 4 rows, 8 heads, up to 511 pages, 14.8 us cold.  Pages are dealt to CTAs by 128, so
// that one row of a long cache fills the GPU.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads) k_kv8_score(w4a8_kv8_cache c, w4a8_rows qr, const int32_t* counts,
                                                             int n, int G, int top_k, int first_pages, int last_pages,
                                                             uint32_t* __restrict__ keys) {
  griddep_enter();
  constexpr int DL = D / 8;  // dims of a lane
  __shared__ float red[kScoreThreads / 32];
  __shared__ __align__(16) int8_t codes[kKv8MaxGroup * D];
  const int h = blockIdx.y, s = blockIdx.x / n, i = blockIdx.x % n;
  const int L = kv8_len(c, c.len, s);
  const int cnt = kv8_count(c, counts, s, n);
  const int whole = L < 0 ? 0 : L / kPage;
  if (i >= cnt || whole <= top_k || (int)blockIdx.z * kScorePages >= whole) return;  // nothing to choose between
  const T* q = static_cast<const T*>(qr.data) + (int64_t)s * qr.seq + (int64_t)i * qr.row + (int64_t)h * G * qr.head;
  float m = 0.0f;
  for (int e = threadIdx.x; e < G * D; e += kScoreThreads) m = max_nan(m, fabsf(kv8_load(q + (e / D) * qr.head + e % D)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int w = 1; w < kScoreThreads / 32; ++w) m = max_nan(m, red[w]);
  const float a = kv8_scale(m);
  for (int e = threadIdx.x; e < G * D; e += kScoreThreads)
    codes[e] = a > 0.0f ? (int8_t)kv8_code(kv8_load(q + (e / D) * qr.head + e % D), a) : (int8_t)0;
  __syncthreads();
  const int lane8 = threadIdx.x & 7;
  const size_t pair = kv8_pair(c, s, h);
  uint32_t* out = keys + ((size_t)blockIdx.x * c.n_kv_heads + h) * c.max_pages;
  const int p1 = min(whole, ((int)blockIdx.z + 1) * kScorePages);
  for (int p0 = blockIdx.z * kScorePages; p0 < p1; p0 += kScoreThreads / 8) {  // uniform: the shuffles need every lane
    const int p = p0 + (threadIdx.x >> 3);
    const int phys = p < p1 ? kv8_phys(c, pair, p) : -1;
    const size_t pg = kv8_page(c, pair, max(phys, 0));
    int2 ks[DL / 4];
    const int4* src = reinterpret_cast<const int4*>(c.sums + pg * D + lane8 * DL);
#pragma unroll
    for (int j = 0; j < DL / 8; ++j) {
      const int4 v = phys >= 0 ? src[j] : make_int4(0, 0, 0, 0);
      ks[2 * j] = make_int2(v.x, v.y);
      ks[2 * j + 1] = make_int2(v.z, v.w);
    }
    const float sk = phys >= 0 ? c.scales[pg * 2] : 0.0f;
    int best = INT_MIN;
    for (int g = 0; g < G; ++g) {
      const int* qc = reinterpret_cast<const int*>(codes + g * D + lane8 * DL);
      int acc = 0;
#pragma unroll
      for (int j = 0; j < DL / 4; ++j) {
        acc = __dp2a_lo(ks[j].x, qc[j], acc);
        acc = __dp2a_hi(ks[j].y, qc[j], acc);
      }
      acc += __shfl_xor_sync(0xffffffffu, acc, 1);
      acc += __shfl_xor_sync(0xffffffffu, acc, 2);
      acc += __shfl_xor_sync(0xffffffffu, acc, 4);
      best = max(best, acc);
    }
    if (lane8 == 0 && p < p1) {
      const bool forced = p < first_pages || p >= whole - last_pages;
      out[p] = forced ? kForcedKey : order_key(__fmul_rn(sk, (float)best));
    }
  }
}

// The top_k pages of the scores, a CTA for each (row, KV head), the keys in shared memory: latency of the selection's
// rounds; 512 lists of 32 of up to 511 pages 11.5 us cold.
__global__ void __launch_bounds__(512) k_kv8_pick(w4a8_kv8_cache c, const int32_t* counts, int n, int top_k,
                                                  const uint32_t* __restrict__ keys, int32_t* __restrict__ pages) {
  griddep_enter();
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t hist[256];
  const int h = blockIdx.y, s = blockIdx.x / n, i = blockIdx.x % n;
  const int L = kv8_len(c, c.len, s);
  const int cnt = kv8_count(c, counts, s, n);
  const int whole = L < 0 || i >= cnt ? 0 : L / kPage;
  const size_t at = (size_t)blockIdx.x * c.n_kv_heads + h;
  int32_t* out = pages + at * top_k;
  const int kept = min(whole, top_k);
  for (int j = kept + threadIdx.x; j < top_k; j += blockDim.x) out[j] = -1;
  if (whole <= top_k) {
    for (int j = threadIdx.x; j < kept; j += blockDim.x) out[j] = j;
    return;
  }
  for (int j = threadIdx.x; j < whole; j += blockDim.x) sm[j] = keys[at * c.max_pages + j];
  __syncthreads();
  split_largest(sm, whole, top_k, hist, [&](int j, bool keep, int rank) {
    if (keep) out[rank] = j;
  });
}

// ---------------------------------------------------------------------------- eviction

// Eviction, a CTA for each head: its table and masses pass through shared memory, 3.8 MB in and out for 32 sequences of 8
// heads of up to 2046 pages: 11 us, the latency of the selection's rounds.
__global__ void __launch_bounds__(512) k_kv8_evict(w4a8_kv8_cache c, const float* mass, int keep, int first_pages,
                                                   int last_pages, int32_t* table_out, float* mass_out, int32_t* len_out,
                                                   bool store_len) {
  griddep_enter();
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t hist[256];
  const int P = c.max_pages, h = blockIdx.x, s = blockIdx.y;
  uint32_t* keys = sm;
  float* ms = reinterpret_cast<float*>(sm + P);
  int32_t* tb = reinterpret_cast<int32_t*>(sm + 2 * (size_t)P);
  const size_t at = kv8_pair(c, s, h) * P;
  const int L = kv8_len(c, c.len, s);
  const int whole = L < 0 ? 0 : L / kPage;
  const int kept = L < 0 ? 0 : min(whole, keep);
  // everything is read before anything is written: the outputs may be the inputs
  for (int j = threadIdx.x; j < P; j += blockDim.x) {
    const float v = mass[at + j];
    ms[j] = v;
    tb[j] = c.table[at + j];
    if (j < whole) keys[j] = j < first_pages || j >= whole - last_pages ? kForcedKey : order_key(v);
  }
  if (store_len && h == 0 && threadIdx.x == 0) len_out[s] = L < 0 ? c.len[s] : L - kPage * (whole - kept);
  __syncthreads();
  split_largest(keys, whole, kept, hist, [&](int j, bool stays, int rank) {
    table_out[at + (stays ? rank : kept + rank)] = tb[j];
    if (stays) mass_out[at + rank] = ms[j];
  });
  for (int j = threadIdx.x; j < P; j += blockDim.x) {
    if (j >= whole) table_out[at + j] = tb[j];
    if (L < 0) mass_out[at + j] = ms[j];
    else if (j >= kept) mass_out[at + j] = 0.0f;
  }
}

// The new lengths of an eviction in place: behind the kernel whose CTAs all read the old ones.
__global__ void k_kv8_evict_len(w4a8_kv8_cache c, int keep) {
  griddep_enter();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= c.n_seqs) return;
  const int L = kv8_len(c, c.len, s);
  if (L >= 0) c.len[s] = L - kPage * max(0, L / kPage - keep);
}

}  // namespace

static w4a8_status select_args(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a) {
  const w4a8_status ok = kv8_dims(c);
  if (ok != W4A8_OK) return ok;
  if (!a || !kv8_dtype(a->dtype)) return W4A8_ERR_ARG;
  if (a->n < 1 || a->n > kKv8MaxRows || a->n_heads < 1 || a->n_heads % c->n_kv_heads ||
      a->n_heads / c->n_kv_heads > kKv8MaxGroup)
    return W4A8_ERR_SHAPE;
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_select_workspace_bytes(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, size_t* bytes) {
  const w4a8_status ok = select_args(c, a);
  if (ok != W4A8_OK) return ok;
  if (!bytes) return W4A8_ERR_ARG;
  *bytes = (size_t)c->n_seqs * a->n * c->n_kv_heads * c->max_pages * 4;
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_select(const w4a8_kv8_cache* c, const w4a8_kv8_attn* a, int top_k, int first_pages,
                                     int last_pages, int32_t* pages_out, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  size_t need = 0;
  w4a8_status ok = w4a8_kv8_select_workspace_bytes(c, a, &need);
  if (ok == W4A8_OK) ok = kv8_valid(c);
  if (ok != W4A8_OK) return ok;
  if (!a->q.data || !aligned(a->q.data, kv8_elem(a->dtype)) || !pages_out || !workspace || !aligned(workspace, 256) ||
      !aligned(pages_out, 4) || !aligned(a->counts, 4) || top_k < 1 || first_pages < 0 || last_pages < 0)
    return W4A8_ERR_ARG;
  if (top_k > kKv8MaxPages) return W4A8_ERR_SHAPE;
  if (workspace_bytes < need) return W4A8_ERR_CAPACITY;
  cudaStream_t st = as_stream(stream);
  uint32_t* keys = static_cast<uint32_t*>(workspace);
  const int G = a->n_heads / c->n_kv_heads, n = a->n;
  if (c->max_pages > top_k) {
    const dim3 grid((unsigned)(c->n_seqs * n), (unsigned)c->n_kv_heads,
                    (unsigned)((c->max_pages + kScorePages - 1) / kScorePages));
    auto run = [&](auto kern) {
      return launch_pdl(kern, grid, dim3(kScoreThreads), 0, st, *c, a->q, a->counts, n, G, top_k, first_pages, last_pages,
                        keys);
    };
    if (a->dtype == W4A8_F32)
      W4A8_CUDA_TRY(c->head_dim == 64 ? run(k_kv8_score<float, 64>) : run(k_kv8_score<float, 128>));
    else
      W4A8_CUDA_TRY(c->head_dim == 64 ? run(k_kv8_score<__nv_bfloat16, 64>) : run(k_kv8_score<__nv_bfloat16, 128>));
  }
  const size_t smem = (size_t)c->max_pages * 4;
  W4A8_CUDA_TRY(kv8_smem<k_kv8_pick>(kKv8MaxPages * 4));
  W4A8_CUDA_TRY(launch_pdl(k_kv8_pick, dim3((unsigned)(c->n_seqs * n), (unsigned)c->n_kv_heads), dim3(512), smem, st, *c,
                           a->counts, n, top_k, (const uint32_t*)keys, pages_out));
  return W4A8_OK;
}

W4A8_API w4a8_status w4a8_kv8_evict(const w4a8_kv8_cache* c, const float* mass, int keep, int first_pages,
                                    int last_pages, int32_t* table_out, float* mass_out, int32_t* len_out,
                                    void* stream) {
  const w4a8_status ok = kv8_valid(c);
  if (ok != W4A8_OK) return ok;
  if (!mass || !table_out || !mass_out || !len_out || keep < 0 || first_pages < 0 || last_pages < 0) return W4A8_ERR_ARG;
  if (!aligned(mass, 4) || !aligned(table_out, 4) || !aligned(mass_out, 4) || !aligned(len_out, 4)) return W4A8_ERR_ARG;
  cudaStream_t st = as_stream(stream);
  const bool own = len_out == c->len;
  W4A8_CUDA_TRY(kv8_smem<k_kv8_evict>(kKv8MaxPages * 12));
  W4A8_CUDA_TRY(launch_pdl(k_kv8_evict, dim3((unsigned)c->n_kv_heads, (unsigned)c->n_seqs), dim3(512),
                           (size_t)c->max_pages * 12, st, *c, mass, keep, first_pages, last_pages, table_out, mass_out,
                           len_out, !own));
  if (own)
    W4A8_CUDA_TRY(launch_pdl(k_kv8_evict_len, dim3((unsigned)((c->n_seqs + 127) / 128)), dim3(128), 0, st, *c, keep));
  return W4A8_OK;
}
