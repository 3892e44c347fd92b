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
// One launch; a cluster of 1 to 8 CTAs per (sequence, KV head), the slots cut
// into one range per CTA:
//  * every CTA computes its slots' 32-bit keys once (a weight's bits in an
//    order-preserving form; a protected token the largest key of all) and keeps
//    them in shared memory;
//  * the B-th largest key by three passes of 11, 11 and 10 bits: a histogram
//    per CTA (equal digits within a warp are added by one lane, since weights
//    crowd into few exponents), read by all CTAs of the cluster through
//    distributed shared memory, each then finding the same digit;
//  * each warp owns a contiguous run of slots, so that one count per warp, one
//    scan over the warps and one over the cluster rank the equal keys, the
//    freed slots and the moving tokens in slot order;
//  * the list of moves goes through the workspace, and the cluster's warps
//    share it: a lane looks up one move's blocks and moves its metadata, then the
//    warp copies the K and V rows of 32 moves, several rows in flight.
// The cluster's barriers order the reads of weights and positions before the
// writes of the new ones, which may be the same arrays.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;              // 11 bits
constexpr int kBinsPerThread = kBins / kThreads;
constexpr int kMaxCluster = 8;
constexpr int kCachedKeys = 40960;       // keys a CTA holds in shared memory at most (160 KB)

// Order-preserving bits of a weight: larger weight, larger key; -0 equals +0,
// and a NaN counts as less than every number.  At most 0xff800000 (+inf).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
constexpr uint32_t kProtected = 0xffffffffu;

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of `p` (this CTA's shared memory) in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ int4 remote_int4(uint32_t a) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ int remote_int(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ int warp_inclusive(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

struct Shared {
  int hist[3][kBins];          // one per pass, so that a pass may be read while the next one counts
  int warp_sum[kWarps];
  int ties[kWarps], holes[kWarps], movers[kWarps];   // per warp, then their exclusive sums
  int digit, left, tie_total;
  int counts[2];               // this CTA's holes and movers, for the cluster
};

// kLanes: lanes that copy one token's K and V rows of a head, 16 bytes each.
template <int kLanes>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p, int cluster, int cached) {
  __shared__ __align__(16) Shared sh;
  extern __shared__ uint32_t keys[];   // this CTA's slots (cached)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
  const int64_t rg = blockIdx.x / cluster;
  const int g = (int)(rg % p.num_kv_heads), row = (int)(rg / p.num_kv_heads);
  auto barrier = [&]() {
    if (cluster > 1) cluster_barrier();
    else __syncthreads();
  };

  const int L = __ldg(p.seq_lens + row);
  const int at = p.weight_rows ? __ldg(p.weight_rows + row) : row;
  int seen = __ldg(p.num_tokens + row), old = __ldg(p.ordered_from + row);
  const bool bad_row = L < 0 || L > p.max_seq_len || L > (int64_t)p.max_blocks_per_seq * p.block_size || at < 0 ||
                       at >= p.num_weight_rows || seen < L || old < 0 || old > L;
  if (tid == 0 && rank == 0) {
    if (bad_row) record_error(p.err, PA_ERR_DEVICE_CHECK);
    if (g == 0) p.new_seq_lens[row] = bad_row ? L : min(L, p.budget);
  }
  if (bad_row) return;   // left as it is (the same for every CTA of the cluster)
  const int64_t base = ((int64_t)at * p.num_kv_heads + g) * p.stride;
  const float *w = p.weights + base;
  const int32_t *pos = p.positions + base;
  auto position = [&](int s) { return s < old ? pos[s] : seen - L + s; };
  const int B = p.budget;

  if (L <= B) {   // everything stays: only the metadata is written
    for (int s = rank * kThreads + tid; s < L; s += cluster * kThreads) {
      const float x = w[s];
      const int t = position(s);
      p.new_weights[base + s] = x;
      p.new_positions[base + s] = t;
    }
    return;
  }

  // this CTA's slots [lo, hi), a multiple of 32 per warp
  const int per_warp = ((L + cluster * kWarps - 1) / (cluster * kWarps) + 31) & ~31;
  const int lo = min((int64_t)L, (int64_t)rank * kWarps * per_warp), hi = min((int64_t)L, lo + (int64_t)kWarps * per_warp);
  const int wlo = min(hi, lo + warp * per_warp), whi = min(hi, wlo + per_warp);
  auto make_key = [&](int s) {
    const int t = position(s);
    return t < p.num_sinks || t >= seen - p.num_recent ? kProtected : weight_key(w[s]);
  };
  auto key = [&](int s) { return cached ? keys[s - lo] : make_key(s); };

  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();

  // ------------------------------------------------ the B-th largest key
  uint32_t prefix = 0, mask = 0;   // the digits found so far
  int need = B;                    // how many of the keys with this prefix stay
  int ties_before = 0, tie_total = 0;   // equal keys in the cluster's CTAs before this one, and in all
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    int *hist = sh.hist[pass];
    for (int s0 = wlo; s0 < whi; s0 += 32) {
      const int s = s0 + lane;
      bool in = s < whi;
      uint32_t k = 0;
      if (in) {
        if (pass == 0) {
          k = make_key(s);
          if (cached) keys[s - lo] = k;
        } else {
          k = key(s);
        }
        in = (k & mask) == prefix;
      }
      const uint32_t d = in ? (k >> shift) & digits : 0xffffffffu;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (in && lane == __ffs(same) - 1) atomicAdd(&hist[d], __popc(same));
    }
    barrier();
    // thread t: bins 4t .. 4t+3 counted from the largest digit down, over the cluster
    const int b0 = kBins - kBinsPerThread * (tid + 1);
    int v[kBinsPerThread] = {0, 0, 0, 0};
    int sum = 0;
    for (int c = 0; c < cluster; ++c) {
      const int4 x = cluster > 1 ? remote_int4(remote(&hist[b0], c)) : *reinterpret_cast<const int4 *>(&hist[b0]);
      v[0] += x.w;
      v[1] += x.z;
      v[2] += x.y;
      v[3] += x.x;
    }
#pragma unroll
    for (int i = 0; i < kBinsPerThread; ++i) sum += v[i];
    const int inc = warp_inclusive(sum);
    if (lane == 31) sh.warp_sum[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    {
      const int t = warp_inclusive(lane < kWarps ? sh.warp_sum[lane] : 0);
      before += warp ? __shfl_sync(0xffffffffu, t, warp - 1) : 0;
    }
    if (before < need && before + sum >= need) {   // exactly one thread
#pragma unroll
      for (int i = 0; i < kBinsPerThread; ++i) {
        if (before < need && before + v[i] >= need) {
          sh.digit = b0 + kBinsPerThread - 1 - i;
          sh.left = need - before;
          sh.tie_total = v[i];
          before = need;   // no later bin
        } else if (before < need) {
          before += v[i];
        }
      }
    }
    __syncthreads();
    const int d = sh.digit;
    prefix |= (uint32_t)d << shift;
    mask |= digits << shift;
    need = sh.left;
    tie_total = sh.tie_total;
    // as many keys with this prefix as stay: they all do, whatever their other digits
    if (need == tie_total) break;
    if (pass == 2)
      for (int c = 0; c < (int)rank; ++c) ties_before += remote_int(remote(&hist[d], c));
  }
  // a key stays if its digits found so far are larger, or equal and among the first `need`
  auto above = [&](uint32_t k) { return (k & mask) > prefix; };
  const bool rank_ties = need < tie_total;

  // ------------------------------------------------ ranks in slot order
  if (rank_ties) {
    int n = 0;
    for (int s0 = wlo; s0 < whi; s0 += 32)
      n += __popc(__ballot_sync(0xffffffffu, s0 + lane < whi && (key(s0 + lane) & mask) == prefix));
    if (lane == 0) sh.ties[warp] = n;
    __syncthreads();
  }
  int tie0 = ties_before;   // equal keys before this warp
  if (rank_ties)
    for (int i = 0; i < warp; ++i) tie0 += sh.ties[i];
  // kept slots of this warp, 32 at a time; f(s0, kept ballot) in slot order
  auto sweep = [&](auto &&f) {
    int ties = tie0;
    for (int s0 = wlo; s0 < whi; s0 += 32) {
      const int s = s0 + lane;
      const uint32_t k = s < whi ? key(s) : 0u;
      const bool tie = s < whi && (k & mask) == prefix;
      bool kept = s < whi && (above(k) || (tie && !rank_ties));
      if (rank_ties) {
        const uint32_t t = __ballot_sync(0xffffffffu, tie);
        kept |= tie && ties + __popc(t & ((1u << lane) - 1)) < need;
        ties += __popc(t);
      }
      f(s, kept);
    }
  };
  {
    int nh = 0, nm = 0;
    sweep([&](int s, bool kept) {
      nh += __popc(__ballot_sync(0xffffffffu, s < whi && s < B && !kept));
      nm += __popc(__ballot_sync(0xffffffffu, kept && s >= B));
    });
    if (lane == 0) {
      sh.holes[warp] = nh;
      sh.movers[warp] = nm;
    }
  }
  __syncthreads();
  int hole0 = 0, mover0 = 0;   // before this warp, in the CTA
  {
    const int h = warp_inclusive(lane < kWarps ? sh.holes[lane] : 0), m = warp_inclusive(lane < kWarps ? sh.movers[lane] : 0);
    if (warp) {
      hole0 = __shfl_sync(0xffffffffu, h, warp - 1);
      mover0 = __shfl_sync(0xffffffffu, m, warp - 1);
    }
    if (tid == 31) {
      sh.counts[0] = h;
      sh.counts[1] = m;
    }
  }
  barrier();   // also: every read of weights and positions for the selection is done
  int moves = 0;
  if (cluster > 1) {
    for (int c = 0; c < cluster; ++c) {
      const int h = remote_int(remote(&sh.counts[0], c)), m = remote_int(remote(&sh.counts[1], c));
      moves += h;
      if (c < (int)rank) {
        hole0 += h;
        mover0 += m;
      }
    }
  } else {
    moves = sh.counts[0];
  }
  int32_t *hole_list = p.lists + rg * p.list_stride, *mover_list = hole_list + p.list_cap;
  sweep([&](int s, bool kept) {
    const bool hole = s < whi && s < B && !kept, mover = kept && s >= B;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    const uint32_t below = (1u << lane) - 1;
    if (hole) hole_list[hole0 + __popc(hb & below)] = s;
    if (mover) mover_list[mover0 + __popc(mb & below)] = s;
    hole0 += __popc(hb);
    mover0 += __popc(mb);
    if (kept && s < B) {   // stays where it is
      const float x = w[s];
      const int t = position(s);
      p.new_weights[base + s] = x;
      p.new_positions[base + s] = t;
    }
  });
  barrier();   // the lists (this cluster's global writes) are complete

  // ------------------------------------------------ the moves
  const int32_t *table = p.block_tables + (int64_t)row * p.max_blocks_per_seq;
  const int bs = p.block_size;
  constexpr int kPer = 32 / kLanes;        // moves one warp instruction copies
  constexpr int kDeep = 8;                 // such instructions in flight
  const int sub = lane / kLanes, word = lane % kLanes;
  char *pool = word < kLanes / 2 ? p.k_cache : p.v_cache;
  const int64_t o = (word % (kLanes / 2)) * 16;
  constexpr int kRow = kLanes / 2 * 16;    // bytes of a row
  for (int i0 = (rank * kWarps + warp) * 32; i0 < moves; i0 += cluster * kWarps * 32) {
    const int i = i0 + lane;
    int64_t src = -1, dst = -1;            // row indexes
    if (i < moves) {
      const int to = hole_list[i], from = mover_list[i];
      const float x = w[from];
      const int t = position(from);
      p.new_weights[base + to] = x;
      p.new_positions[base + to] = t;
      const int bf = __ldg(table + from / bs), bt = __ldg(table + to / bs);
      if (bf < 0 || bt < 0 || bf >= p.num_blocks || bt >= p.num_blocks) {
        record_error(p.err, PA_ERR_DEVICE_CHECK);
      } else {
        src = ((int64_t)bf * p.num_kv_heads + g) * bs + from % bs;
        dst = ((int64_t)bt * p.num_kv_heads + g) * bs + to % bs;
      }
    }
    const int n = min(32, moves - i0);
    for (int j0 = 0; j0 < n; j0 += kPer * kDeep) {
      uint4 x[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int64_t r = __shfl_sync(0xffffffffu, src, (j0 + u * kPer + sub) & 31);
        if (j0 + u * kPer + sub < n && r >= 0) x[u] = *reinterpret_cast<const uint4 *>(pool + r * kRow + o);
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int64_t r = __shfl_sync(0xffffffffu, dst, (j0 + u * kPer + sub) & 31);
        if (j0 + u * kPer + sub < n && r >= 0) *reinterpret_cast<uint4 *>(pool + r * kRow + o) = x[u];
      }
    }
  }
}

template <int kLanes>
cudaError_t launch_one(const EvictParams &p, cudaStream_t s) {
  const int64_t heads = (int64_t)p.num_seqs * p.num_kv_heads;
  // CTAs per head: more while they fit on the GPU together and have a warp's worth of slots each
  int sms = 0;
  cudaError_t e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  int cluster = 1;
  while (cluster < kMaxCluster && heads * cluster * 2 <= 2 * sms && p.max_seq_len / (2 * cluster) >= kThreads) cluster *= 2;
  while (cluster < kMaxCluster && p.max_seq_len / cluster > kCachedKeys) cluster *= 2;
  // a CTA's slots: per_warp rounded up to 32, times the warps
  const int64_t slots = (((int64_t)p.max_seq_len + cluster * kWarps - 1) / (cluster * kWarps) + 31) / 32 * 32 * kWarps;
  const int cached = slots <= kCachedKeys;
  const int smem = cached ? (int)slots * 4 : 0;
  if (heads * cluster > 2147483647ll) return cudaErrorInvalidValue;
  if ((e = ensure_smem_limit<evict_kernel<kLanes>>(kCachedKeys * 4)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(heads * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<kLanes>, p, cluster, cached);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s) {
  switch (p.row_bytes) {
    case 64: return launch_one<8>(p, s);
    case 128: return launch_one<16>(p, s);
    case 256: return launch_one<32>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
