// pa_decode_ext_fp8_bf16q.cu -- bounded-cache decode instantiations for an
// fp8-e4m3 cache with bf16 queries.
#include "pa_decode_tc.cuh"

namespace pa {
cudaError_t launch_decode_ext_fp8_bf16q(const DecodeTcParams &p, int head_dim, const PoolMaps &m, cudaStream_t s) {
  return launch_decode_ext<uint8_t, __nv_bfloat16>(p, head_dim, m, s);
}
}  // namespace pa
