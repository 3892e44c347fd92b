// pa_prefill_scaled_f16q.cu -- chunked-prefill instantiations for a block-scaled
// fp8-e4m3 cache with f16 queries.
#include "pa_prefill_scaled.cuh"

namespace pa {
cudaError_t launch_prefill_scaled_f16q(const PrefillTcParams &p, const CUtensorMap &k, int head_dim, int num_chunks,
                                        cudaStream_t s) {
  return launch_prefill_scaled<__half>(p, k, head_dim, num_chunks, s);
}
}  // namespace pa
