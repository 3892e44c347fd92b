// pa_decode_ext_fp8_f16q.cu -- bounded-cache decode instantiations for an
// fp8-e4m3 cache with f16 queries.
#include "pa_decode_tc.cuh"

namespace pa {
cudaError_t launch_decode_ext_fp8_f16q(const DecodeTcParams &p, int head_dim, const PoolMaps &m, cudaStream_t s) {
  return launch_decode_ext<uint8_t, __half>(p, head_dim, m, s);
}
}  // namespace pa
