// The split kernels of the 4-bit cache's attention: fp32 rows, head size 64.
#include "kv4_attn.cuh"

namespace w4a8 {
cudaError_t kv4_split_f32_d64(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo, const Kv4Scratch& ws,
                             cudaStream_t st) {
  return kv4_split_dispatch<float, 64>(c, a, geo, ws, st);
}
}  // namespace w4a8
