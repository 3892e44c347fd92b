// pa_prefill_window_fp8_f16q.cu -- sliding-window chunked-prefill instantiations
// for an fp8-e4m3 cache with f16 queries.
#include "pa_prefill_tc.cuh"

namespace pa {
cudaError_t launch_prefill_window_fp8_f16q(const PrefillTcParams &p, const PoolMaps &m, int head_dim, int num_chunks,
                                          cudaStream_t s) {
  return launch_prefill_window<uint8_t, __half>(p, m, head_dim, num_chunks, s);
}
}  // namespace pa
