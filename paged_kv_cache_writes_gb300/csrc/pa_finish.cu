// pa_finish.cu -- the second launch of the bounded-cache decodes.
//
// Two kinds of CTA in one grid:
//  * merging (direct launches, whose decode kernel leaves split rows in
//    partitions): one CTA per (row, query head), its warps sharing the row's
//    partitions p,
//      out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p.
//    Every partition's sums are read by themselves, so a row of 19 partitions
//    costs three dependent round trips to the L2 (lengths, then everything
//    else, up to three partitions a warp), where one warp walking the row took a
//    round trip for each pair of them.
//  * weights (pa_decode_weights): from the scores that the decode left in the
//    workspace, each cached token's softmax weight summed over the query heads
//    of its KV head, added to its running sum,
//      w[g][p] = sum over the heads h of KV head g of 2^(t[h][p] - M[h]) / l[h]
//      weights[g][p] = (p < fresh_from ? decay * weights[g][p] : 0) + w[g][p]
//    with t the scores in log2 units, M and l the row's softmax maximum and sum.
//    One pass over the scores (4 bytes per head and token) and the weights; the
//    sum runs over the heads in order, in one thread, so that the result does
//    not depend on scheduling.
#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_window.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTokens = 4;                   // tokens per thread of a weights CTA, their scores in flight together
constexpr int kChunk = kTokens * kThreads;   // tokens per weights CTA
#define kNegInfF (-__int_as_float(0x7f800000))

// The row's packed tokens, cut as the decode cut them (which reported what was out of range).
__device__ __forceinline__ int packed_len(const FinishParams &p, int row) {
  int64_t L = max(__ldg(p.seq_lens + row), 0);
  L = min(L, (int64_t)p.max_blocks_per_seq << p.bs_log2);
  const WindowSpan w = window_span(window_low((int)L, p.window), p.num_sinks, p.bs_log2);
  return (int)min(L - ((int64_t)w.skip_blocks << p.bs_log2), (int64_t)p.max_partitions * p.partition_size);
}

// Maximum and sum of the softmax of (row, head) over its partitions, by one warp.
__device__ __forceinline__ float2 merge_ml(const FinishParams &p, int64_t row_head, int nparts) {
  const int lane = threadIdx.x & 31;
  const float2 *ml = p.ws_ml + row_head * p.max_partitions;
  float M = kNegInfF, l = 0.f;
  for (int q = lane; q < nparts; q += 32) {
    const float2 x = __ldcg(ml + q);
    const float m = fmaxf(M, x.x), ref = m == kNegInfF ? 0.f : m;
    l = l * fast_exp2(M - ref) + x.y * fast_exp2(x.x - ref);
    M = m;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, M, off), ol = __shfl_xor_sync(0xffffffffu, l, off);
    const float m = fmaxf(M, om), ref = m == kNegInfF ? 0.f : m;
    l = l * fast_exp2(M - ref) + ol * fast_exp2(om - ref);
    M = m;
  }
  return make_float2(M, l);
}

template <int D>
__device__ __forceinline__ void merge_cta(const FinishParams &p, int64_t row_head, float4 (*part)[32], float *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = (int)(row_head / p.num_q_heads), head = (int)(row_head - (int64_t)row * p.num_q_heads);
  const int nparts = (packed_len(p, row) + p.partition_size - 1) / p.partition_size;
  if (nparts <= 1) return;   // the decode wrote the row's output
  constexpr int kPer = D / 32;   // elements per lane
  const float *acc = p.ws_acc + row_head * p.max_partitions * D + lane * kPer;
  const float2 *ml = p.ws_ml + row_head * p.max_partitions;
  // this warp's partitions warp, warp + kWarps, ...: a running maximum of its own
  float M = kNegInfF, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  auto load = [&](int q) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (kPer == 4) {
      x = __ldcg(reinterpret_cast<const float4 *>(acc + (int64_t)q * D));
    } else {
      const float2 y = __ldcg(reinterpret_cast<const float2 *>(acc + (int64_t)q * D));
      x.x = y.x;
      x.y = y.y;
    }
    return x;
  };
  constexpr int kDeep = 4;   // partitions in flight
  for (int q0 = warp; q0 < nparts; q0 += kDeep * kWarps) {
    float4 x[kDeep];
    float2 y[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int q = q0 + k * kWarps;
      y[k] = q < nparts ? __ldcg(ml + q) : make_float2(kNegInfF, 0.f);
      x[k] = load(min(q, nparts - 1));
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const float m = fmaxf(M, y[k].x), ref = m == kNegInfF ? 0.f : m;
      const float so = fast_exp2(M - ref), sn = q0 + k * kWarps < nparts ? fast_exp2(y[k].x - ref) : 0.f;
      M = m;
      l = l * so + y[k].y * sn;
      a = make_float4(a.x * so + x[k].x * sn, a.y * so + x[k].y * sn, a.z * so + x[k].z * sn, a.w * so + x[k].w * sn);
    }
  }
  part[warp][lane] = a;
  if (lane == 0) {
    red[2 * warp] = M;
    red[2 * warp + 1] = l;
  }
  __syncthreads();
  if (warp != 0) return;
  float m = kNegInfF;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) m = fmaxf(m, red[2 * k]);
  const float ref = m == kNegInfF ? 0.f : m;
  a = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const float sc = fast_exp2(red[2 * k] - ref);
    const float4 x = part[k][lane];
    l += red[2 * k + 1] * sc;
    a = make_float4(a.x + x.x * sc, a.y + x.y * sc, a.z + x.z * sc, a.w + x.w * sc);
  }
  const float om = p.v_hs ? p.out_mult * __ldg(p.v_hs + head / (p.num_q_heads / p.num_kv_heads)) : p.out_mult;
  const float inv = l > 0.f ? om / l : 0.f;
  const int64_t o = row_head * D + lane * kPer;
  const float v[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (p.out_dtype == PA_F32) static_cast<float *>(p.out)[o + i] = v[i];
    else if (p.out_dtype == PA_BF16) static_cast<__nv_bfloat16 *>(p.out)[o + i] = __float2bfloat16_rn(v[i]);
    else static_cast<__half *>(p.out)[o + i] = __float2half_rn(v[i]);
  }
}

template <int G>
__device__ __forceinline__ void weights_cta(const FinishParams &p, int64_t block, float2 *ml) {
  const int chunk = (int)(block % p.chunks);
  const int64_t rg = block / p.chunks;
  const int g = (int)(rg % p.num_kv_heads), row = (int)(rg / p.num_kv_heads);
  const int packed = packed_len(p, row), L = min(packed, p.max_len);   // no window: the row's tokens
  const int first = chunk * kChunk;
  if (first >= L) return;
  const int at = p.weight_rows ? __ldg(p.weight_rows + row) : row;
  if (at < 0 || at >= p.num_weight_rows) {
    if (threadIdx.x == 0) record_error(p.err, PA_ERR_DEVICE_CHECK);
    return;
  }
  const int gqa = p.num_q_heads / p.num_kv_heads;
  float *weights = p.weights + ((int64_t)at * p.num_kv_heads + g) * p.weights_stride;
  // the first share's scores, and the running weights, are loaded before the rows' maxima arrive
  float4 v[kTokens][G / 4];
  float old[kTokens];
  auto load = [&](int s) {
    const float4 *src = reinterpret_cast<const float4 *>(p.scores + (rg * p.shares + s) * p.score_stride * G);
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const int t = first + k * kThreads + threadIdx.x;
      if (t < L) {
#pragma unroll
        for (int i = 0; i < G / 4; ++i) v[k][i] = __ldcs(src + (int64_t)t * (G / 4) + i);
      }
    }
  };
  load(0);
  // (a decay of 0 reads no running weight: whatever it is, NaN included, nothing of it is kept)
  const int fresh = p.decay == 0.f ? 0 : p.fresh_from ? __ldg(p.fresh_from + row) : L - 1;
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    const int t = first + k * kThreads + threadIdx.x;
    old[k] = t < L && t < fresh ? p.decay * weights[t] : 0.f;
  }
  const int64_t head0 = (int64_t)row * p.num_q_heads + (int64_t)g * gqa;
  const int nparts = (packed + p.partition_size - 1) / p.partition_size;
  if (p.direct && nparts > 1) {
    for (int h = threadIdx.x >> 5; h < gqa; h += kWarps) {
      const float2 x = merge_ml(p, head0 + h, nparts);
      if ((threadIdx.x & 31) == 0) ml[h] = make_float2(x.x, x.y > 0.f ? 1.f / x.y : 0.f);
    }
  } else {
    for (int h = threadIdx.x; h < gqa; h += kThreads) ml[h] = __ldcg(p.row_ml + head0 + h);
  }
  __syncthreads();
  float w[kTokens];
#pragma unroll
  for (int k = 0; k < kTokens; ++k) w[k] = 0.f;
  for (int s = 0; s < p.shares; ++s) {
    if (s > 0) load(s);
    const int h0 = s * p.share_heads, n = min(p.share_heads, gqa - h0);
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (i < n) {
        const float2 x = ml[h0 + i];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
          const float4 y = v[k][i / 4];
          w[k] = fmaf(fast_exp2((i % 4 == 0 ? y.x : i % 4 == 1 ? y.y : i % 4 == 2 ? y.z : y.w) - x.x), x.y, w[k]);
        }
      }
  }
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    const int t = first + k * kThreads + threadIdx.x;
    if (t < L) weights[t] = old[k] + w[k];
  }
}

// CTAs per SM that the registers allow.  A weights CTA is bound by its loads: more CTAs help a batch while the scores that
// a thread holds (kTokens * G) fit.  Both launches, at 4 against 2 per SM: 64 sequences of 100 to 8192 tokens G = 4 204 /
// 212 us, G = 8 230 / 234, G = 16 319 (it spills 376 bytes) / 299; 2 sequences of 8000 18.4 / 17.5, 22.3 / 20.2, 38 / 28.
constexpr int finish_ctas(int g) { return g == 16 ? 2 : 4; }

template <int G, int D>
__global__ void __launch_bounds__(kThreads, finish_ctas(G)) decode_finish_kernel(const FinishParams p) {
  extern __shared__ __align__(16) float smem[];
  // launched as the decode's programmatic dependent
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x < p.merge_blocks) {
    float4(*part)[32] = reinterpret_cast<float4(*)[32]>(smem);
    merge_cta<D>(p, blockIdx.x, part, smem + kWarps * 32 * 4);
  } else {
    weights_cta<G>(p, blockIdx.x - p.merge_blocks, reinterpret_cast<float2 *>(smem));
  }
}

template <int G, int D>
cudaError_t launch_one(const FinishParams &p, unsigned grid, cudaStream_t s) {
  const size_t merge = (kWarps * 32 * 4 + 2 * kWarps) * 4, ml = (size_t)(p.num_q_heads / p.num_kv_heads) * 8;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = merge > ml ? merge : ml;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_finish_kernel<G, D>, p);
}

}  // namespace

cudaError_t launch_decode_finish(const FinishParams &p0, int head_dim, cudaStream_t s) {
  FinishParams p = p0;
  p.chunks = p.weights ? (p.max_len + kChunk - 1) / kChunk : 0;
  const bool merge = p.direct && p.max_partitions > 1;
  const int64_t grid = (merge ? (int64_t)p.num_seqs * p.num_q_heads : 0) + (int64_t)p.num_seqs * p.num_kv_heads * p.chunks;
  if (grid == 0) return cudaSuccess;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  p.merge_blocks = merge ? (uint32_t)((int64_t)p.num_seqs * p.num_q_heads) : 0;
  switch (p.score_rows) {
    case 4: return head_dim == 64 ? launch_one<4, 64>(p, (unsigned)grid, s) : launch_one<4, 128>(p, (unsigned)grid, s);
    case 8: return head_dim == 64 ? launch_one<8, 64>(p, (unsigned)grid, s) : launch_one<8, 128>(p, (unsigned)grid, s);
    default: return launch_one<16, 128>(p, (unsigned)grid, s);
  }
}

}  // namespace pa
