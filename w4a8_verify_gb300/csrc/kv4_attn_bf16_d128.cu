// The split kernels of the 4-bit cache's attention: bf16 rows, head size 128.
#include "kv4_attn.cuh"

namespace w4a8 {
cudaError_t kv4_split_bf16_d128(const w4a8_kv4_cache& c, const w4a8_kv4_attn& a, const Kv4Geom& geo, const Kv4Scratch& ws,
                             cudaStream_t st) {
  return kv4_split_dispatch<__nv_bfloat16, 128>(c, a, geo, ws, st);
}
}  // namespace w4a8
