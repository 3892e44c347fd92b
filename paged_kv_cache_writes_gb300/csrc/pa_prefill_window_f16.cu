// pa_prefill_window_f16.cu -- sliding-window chunked-prefill instantiations for a f16 cache.
#include "pa_prefill_tc.cuh"

namespace pa {
cudaError_t launch_prefill_window_f16(const PrefillTcParams &p, const PoolMaps &m, int head_dim, int num_chunks,
                                      cudaStream_t s) {
  return launch_prefill_window<__half, __half>(p, m, head_dim, num_chunks, s);
}
}  // namespace pa
