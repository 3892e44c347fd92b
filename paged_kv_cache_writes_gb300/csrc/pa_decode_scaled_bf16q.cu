// pa_decode_scaled_bf16q.cu -- decode instantiations for a block-scaled fp8-e4m3
// cache with bf16 queries.
#include "pa_decode_tc.cuh"

namespace pa {
cudaError_t launch_decode_scaled_bf16q(const DecodeTcParams &p, int head_dim, const PoolMaps &m, cudaStream_t s) {
  return launch_decode_scaled<__nv_bfloat16>(p, head_dim, m, s);
}
}  // namespace pa
