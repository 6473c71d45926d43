// The split kernels of the 8-bit cache's attention: bf16 rows, head size 128.
#include "kv8_attn.cuh"

namespace w4a8 {
cudaError_t kv8_split_bf16_d128(const w4a8_kv8_cache& c, const w4a8_kv8_attn& a, const Kv8Geom& geo, const Kv8Scratch& ws,
                             cudaStream_t st) {
  return kv8_split_dispatch<__nv_bfloat16, 128>(c, a, geo, ws, st);
}
}  // namespace w4a8
