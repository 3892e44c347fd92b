// pa_decode_ext_f16.cu -- bounded-cache decode instantiations for a f16 cache.
#include "pa_decode_tc.cuh"

namespace pa {
cudaError_t launch_decode_ext_f16(const DecodeTcParams &p, int head_dim, const PoolMaps &m, cudaStream_t s) {
  return launch_decode_ext<__half, __half>(p, head_dim, m, s);
}
}  // namespace pa
