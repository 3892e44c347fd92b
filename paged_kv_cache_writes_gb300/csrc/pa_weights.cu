// pa_weights.cu -- the weights half of pa_decode_weights: from the scores that
// the decode left in the workspace, each cached token's softmax weight summed
// over the query heads of its KV head, added to its running sum.
//
//   w[g][p] = sum over the heads h of KV head g of 2^(t[h][p] - M[h]) / l[h]
//   weights[g][p] = (p < fresh_from ? decay * weights[g][p] : 0) + w[g][p]
//
// with t the scores in log2 units, M and l the row's softmax maximum and sum.
// One pass over the scores (4 bytes per head and token) and the weights (read
// and written); the sum runs over the heads in order, in one thread, so the
// result does not depend on scheduling.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 1024;   // tokens per CTA

template <int G>
__global__ void __launch_bounds__(kThreads) decode_weights_kernel(const WeightsParams p, int chunks) {
  extern __shared__ float2 ml[];   // [num_q_heads / num_kv_heads]
  const int chunk = blockIdx.x % chunks;
  const int64_t rg = blockIdx.x / chunks;
  const int g = (int)(rg % p.num_kv_heads), row = (int)(rg / p.num_kv_heads);
  const int L = min(max(__ldg(p.seq_lens + row), 0), p.max_len);   // a bad length was reported by the decode
  const int first = chunk * kChunk;
  if (first >= L) return;
  const int at = p.weight_rows ? __ldg(p.weight_rows + row) : row;
  if (at < 0 || at >= p.num_weight_rows) {
    if (threadIdx.x == 0) record_error(p.err, PA_ERR_DEVICE_CHECK);
    return;
  }
  const int fresh = p.fresh_from ? __ldg(p.fresh_from + row) : L - 1;
  const int gqa = p.num_q_heads / p.num_kv_heads;
  for (int h = threadIdx.x; h < gqa; h += kThreads)
    ml[h] = __ldg(p.row_ml + (int64_t)row * p.num_q_heads + (int64_t)g * gqa + h);
  __syncthreads();
  float *weights = p.weights + ((int64_t)at * p.num_kv_heads + g) * p.weights_stride;
  for (int t = first + threadIdx.x; t < min(L, first + kChunk); t += kThreads) {
    float w = 0.f;
    for (int s = 0; s < p.shares; ++s) {
      const float4 *src = reinterpret_cast<const float4 *>(
          p.scores + (((rg * p.shares) + s) * p.score_stride + t) * G);
      const int h0 = s * p.share_heads, n = min(p.share_heads, gqa - h0);
      float v[G];
#pragma unroll
      for (int i = 0; i < G / 4; ++i) {
        const float4 x = __ldcs(src + i);
        v[4 * i] = x.x;
        v[4 * i + 1] = x.y;
        v[4 * i + 2] = x.z;
        v[4 * i + 3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (i < n) w = fmaf(fast_exp2(v[i] - ml[h0 + i].x), ml[h0 + i].y, w);
    }
    weights[t] = t < fresh ? fmaf(p.decay, weights[t], w) : w;
  }
}

}  // namespace

cudaError_t launch_decode_weights(const WeightsParams &p, cudaStream_t s) {
  const int chunks = (p.max_len + kChunk - 1) / kChunk;
  const int64_t grid = (int64_t)p.num_seqs * p.num_kv_heads * chunks;
  if (chunks == 0) return cudaSuccess;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  const size_t smem = (size_t)(p.num_q_heads / p.num_kv_heads) * sizeof(float2);
  switch (p.score_rows) {
    case 4: decode_weights_kernel<4><<<(unsigned)grid, kThreads, smem, s>>>(p, chunks); break;
    case 8: decode_weights_kernel<8><<<(unsigned)grid, kThreads, smem, s>>>(p, chunks); break;
    default: decode_weights_kernel<16><<<(unsigned)grid, kThreads, smem, s>>>(p, chunks); break;
  }
  return cudaGetLastError();
}

}  // namespace pa
