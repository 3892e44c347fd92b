// pa_prefill_scaled_f16q.cu -- chunked-prefill instantiations for a block-scaled
// fp8-e4m3 cache with f16 queries.
#include "pa_prefill_tc.cuh"

namespace pa {
cudaError_t launch_prefill_scaled_f16q(const PrefillTcParams &p, const PoolMaps &m, int head_dim, int num_chunks,
                                      cudaStream_t s) {
  return launch_prefill_scaled<__half>(p, m, head_dim, num_chunks, s);
}
}  // namespace pa
