// pa_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, KV head) of L cached tokens and a budget B < L: the protected
// tokens (position < num_sinks or >= T - num_recent, T tokens seen so far)
// and, of the others, those with the largest weights stay, B in all (ties: the
// lowest slot).  The kept tokens of slots >= B move into the slots < B whose
// tokens go: the i-th of them, in slot order, into the i-th such slot.  Sources
// and destinations are disjoint, so the moves run in place and in parallel,
// and a token that is kept in a slot < B costs nothing: only what has to move
// is read and written.
//
// Selection: the B-th largest of L 32-bit keys (a weight's bits in an order-
// preserving form; a protected token the largest key of all) by four passes
// of 8 bits over a 256-bin histogram, then one pass that ranks equal keys and
// lists the moves in slot order.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;

// Order-preserving bits of a weight: larger weight, larger key; -0 equals +0,
// and a NaN counts as less than every number.  At most 0xff800000 (+inf).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
constexpr uint32_t kProtected = 0xffffffffu;

// Exclusive scan over the CTA's threads of a small count; *total: the sum.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int before = warp ? warp_sums[warp - 1] : 0;
  *total = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

// One CTA per (sequence, KV head): choose, write the metadata of the tokens
// that stay in place, list the moves.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int g = blockIdx.x % p.num_kv_heads, row = blockIdx.x / p.num_kv_heads, tid = threadIdx.x;
  int32_t *list = p.lists + (int64_t)blockIdx.x * p.list_stride;
  const int raw = __ldg(p.seq_lens + row);
  const int at = p.weight_rows ? __ldg(p.weight_rows + row) : row;
  int seen = __ldg(p.num_tokens + row), old = __ldg(p.ordered_from + row);
  const bool bad_row = raw < 0 || raw > p.max_seq_len || raw > (int64_t)p.max_blocks_per_seq * p.block_size || at < 0 ||
                       at >= p.num_weight_rows;
  if (tid == 0) {
    if (bad_row || seen < raw || old < 0 || old > raw) record_error(p.err, PA_ERR_DEVICE_CHECK);
    if (g == 0) p.lens[row] = bad_row ? raw : min(raw, p.budget);
  }
  if (bad_row) {   // left as it is
    if (tid == 0) list[0] = 0;
    return;
  }
  const int L = raw, B = min(p.budget, L);
  seen = max(seen, L);
  old = min(max(old, 0), L);
  const int64_t base = ((int64_t)at * p.num_kv_heads + g) * p.stride;
  const float *w = p.weights + base;
  const int32_t *pos = p.positions + base;
  auto position = [&](int s) { return s < old ? pos[s] : seen - L + s; };
  auto key = [&](int s) {
    const int t = position(s);
    return t < p.num_sinks || t >= seen - p.num_recent ? kProtected : weight_key(w[s]);
  };
  // the B-th largest key: 8 bits a pass, from the top
  uint32_t prefix = 0;   // the digits found so far
  int need = B;          // how many of the keys with this prefix stay
  if (L > B) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int s = tid; s < L; s += kSelThreads) {
        const uint32_t k = key(s);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = need, d = 255;
        for (; d > 0 && hist[d] < left; --d) left -= hist[d];
        s_prefix = prefix | ((uint32_t)d << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      __syncthreads();
    }
  }
  // in slot order: keys above the threshold stay, and the first `need` equal to it
  int ties = 0, holes = 0, movers = 0;
  int32_t *hole_list = list + 4, *mover_list = hole_list + p.list_cap, *mover_pos = mover_list + p.list_cap;
  for (int s0 = 0; s0 < L; s0 += kSelThreads) {
    const int s = s0 + tid;
    const bool in = s < L;
    const uint32_t k = in && L > B ? key(s) : kProtected;
    bool kept = in;
    if (L > B) {
      int n;
      const int rank = ties + block_scan(in && k == prefix, warp_sums, &n);
      ties += n;
      kept = in && (k > prefix || (k == prefix && rank < need));
    }
    const bool hole = in && !kept && s < B, mover = kept && s >= B;
    int nh, nm;
    const int hi = holes + block_scan(hole, warp_sums, &nh), mi = movers + block_scan(mover, warp_sums, &nm);
    holes += nh;
    movers += nm;
    if (hole) hole_list[hi] = s;
    if (mover) {
      mover_list[mi] = s;
      mover_pos[mi] = position(s);
    }
    if (kept && s < B) {
      const int t = position(s);
      const float x = w[s];
      p.new_weights[base + s] = x;
      p.new_positions[base + s] = t;
    }
  }
  if (tid == 0) list[0] = holes;   // as many as movers
}

// One warp per move: the K row, the V row and the metadata of one token.
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictParams p, int chunks) {
  const int64_t rg = blockIdx.x / chunks;
  const int g = (int)(rg % p.num_kv_heads), row = (int)(rg / p.num_kv_heads);
  const int lane = threadIdx.x & 31;
  if (g == 0 && blockIdx.x % chunks == 0 && threadIdx.x == 0) p.new_seq_lens[row] = p.lens[row];
  const int32_t *list = p.lists + rg * p.list_stride;
  const int n = list[0];
  const int32_t *hole_list = list + 4, *mover_list = hole_list + p.list_cap, *mover_pos = mover_list + p.list_cap;
  const int at = p.weight_rows ? __ldg(p.weight_rows + row) : row;
  const int64_t base = ((int64_t)at * p.num_kv_heads + g) * p.stride;
  const int32_t *table = p.block_tables + (int64_t)row * p.max_blocks_per_seq;
  const int words = p.row_bytes / 16;
  for (int i = (blockIdx.x % chunks) * 8 + (threadIdx.x >> 5); i < n; i += chunks * 8) {
    const int to = hole_list[i], from = mover_list[i];
    if (lane == 0) {
      p.new_weights[base + to] = p.weights[base + from];
      p.new_positions[base + to] = mover_pos[i];
    }
    const int bf = table[from / p.block_size], bt = table[to / p.block_size];
    if (bf < 0 || bt < 0 || bf >= p.num_blocks || bt >= p.num_blocks) {
      if (lane == 0) record_error(p.err, PA_ERR_DEVICE_CHECK);
      continue;
    }
    const int64_t src = (((int64_t)bf * p.num_kv_heads + g) * p.block_size + from % p.block_size) * p.row_bytes;
    const int64_t dst = (((int64_t)bt * p.num_kv_heads + g) * p.block_size + to % p.block_size) * p.row_bytes;
    for (int e = lane; e < 2 * words; e += 32) {
      char *pool = e < words ? p.k_cache : p.v_cache;
      const int o = (e < words ? e : e - words) * 16;
      *reinterpret_cast<uint4 *>(pool + dst + o) = *reinterpret_cast<const uint4 *>(pool + src + o);
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s) {
  const int64_t heads = (int64_t)p.num_seqs * p.num_kv_heads;
  const int most = p.max_seq_len - p.budget;   // moves per head
  const int chunks = most <= 0 ? 1 : (most < p.budget ? most : p.budget) / 64 + 1;
  if (heads * chunks > 2147483647ll) return cudaErrorInvalidValue;
  evict_select_kernel<<<(unsigned)heads, kSelThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_move_kernel<<<(unsigned)(heads * chunks), 256, 0, s>>>(p, chunks);
  return cudaGetLastError();
}

}  // namespace pa
