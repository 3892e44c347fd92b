// pa_decode_scaled_f16q.cu -- decode instantiations for a block-scaled fp8-e4m3
// cache with f16 queries.
#include "pa_decode_tc.cuh"

namespace pa {
cudaError_t launch_decode_scaled_f16q(const DecodeTcParams &p, int head_dim, const PoolMaps &m, cudaStream_t s) {
  return launch_decode_scaled<__half>(p, head_dim, m, s);
}
}  // namespace pa
