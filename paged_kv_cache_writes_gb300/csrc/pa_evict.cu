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
// A cluster of 1 to 8 CTAs per (sequence, KV head), the slots cut into one
// range per CTA:
//  * every CTA computes its slots' 32-bit keys once (a weight's bits in an
//    order-preserving form; a protected token the largest key of all) and keeps
//    them in shared memory;
//  * the B-th largest key by at most three passes of 11, 11 and 10 bits: a
//    histogram per CTA (a warp adds its protected tokens at once), whose non-zero
//    bins are added to the cluster's in its first CTA, through distributed shared
//    memory; that CTA finds the digit and the others read it (all of them reading
//    a histogram of 8 KB took 2.5 us a pass: distributed shared memory gives an SM
//    some 10 bytes a clock).  When all keys with the digits so far stay, the rest
//    is not looked at;
//  * each warp owns a contiguous run of slots, a lane four in a row of every 128,
//    so that one count per warp, one scan over the warps and one over the cluster
//    rank the equal keys, the freed slots and the moving tokens in slot order;
//  * a lane looks up one move's blocks and moves its metadata, then its warp
//    copies the K and V rows of up to 32 moves, several rows in flight.  With few
//    moves the cluster's warps share them, at the end of the same launch (the list
//    goes through shared memory where the head has one CTA); with many a second
//    launch deals all heads' moves evenly to the SMs.
// A head's selection is short and every phase of it runs once: fetching the
// instructions costs more than running them, so its loops stay loops (with the
// keys in registers and the loops unrolled it took as long as the simple form).
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
constexpr int kSmemMoves = 2048;         // moves a CTA lists in shared memory at most
// Moves of all heads (at most) that the first launch does itself.  Measured, one launch against two: 8 heads of 8192
// slots to 2048 (16384 moves at most) 13.6 / 15.3 us, 64 of 4096 to 2048 (131072) 21.1 / 24.6, 256 of 2048 to 1024
// (262144) 44.7 / 39.4, 512 of 3000 to 4096 to 1777 (909824) 122 / 113.
constexpr int64_t kFusedMoves = 196608;

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
__device__ __forceinline__ void remote_add(uint32_t a, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
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
  int own[kBins];              // cluster > 1: this CTA's part (hist: the cluster's, in its first CTA)
  int warp_sum[kWarps];
  int ties[kWarps], holes[kWarps], movers[kWarps];   // per warp, then their exclusive sums
  int4 found;                  // of a pass: the digit, how many keys with it stay, how many have it
  int counts[3];               // this CTA's holes, movers and equal keys, for the cluster
};

// What a head's moves need.
struct Head {
  int g, row, L, seen, old;
  int64_t base;   // of its weights and positions
};

// Moves i0 .. i0 + n - 1 (n <= 32) of a head, by one warp.
// kLanes: lanes that copy one token's K and V rows of a head, 16 bytes each.
template <int kLanes>
__device__ __forceinline__ void move_tokens(const EvictParams &p, const Head &h, const int32_t *hole_list,
                                            const int32_t *mover_list, int i0, int n) {
  constexpr int kPer = 32 / kLanes;        // moves one warp instruction copies
  constexpr int kDeep = 8;                 // such instructions in flight
  constexpr int kRow = kLanes / 2 * 16;    // bytes of a row
  const int lane = threadIdx.x & 31, bs = p.block_size;
  const int sub = lane / kLanes, word = lane % kLanes;
  char *pool = word < kLanes / 2 ? p.k_cache : p.v_cache;
  const int64_t o = (word % (kLanes / 2)) * 16;
  int64_t src = -1, dst = -1;              // row indexes
  if (lane < n) {
    // (within the sequence in any case: see where the lists are written)
    const int to = min((uint32_t)hole_list[i0 + lane], h.L - 1u), from = min((uint32_t)mover_list[i0 + lane], h.L - 1u);
    const int32_t *table = p.block_tables + (int64_t)h.row * p.max_blocks_per_seq;
    const int bf = __ldg(table + from / bs), bt = __ldg(table + to / bs);
    float x = p.weights[h.base + from];
    auto position = [&](int s) { return s < h.old ? p.positions[h.base + s] : h.seen - h.L + s; };
    int t = position(from);
    if (bf < 0 || bt < 0 || bf >= p.num_blocks || bt >= p.num_blocks) {
      // refused: the slot keeps its own token, and so that token's weight and position (in a slot that nothing else writes)
      record_error(p.err, PA_ERR_DEVICE_CHECK);
      x = p.weights[h.base + to];
      t = position(to);
    } else {
      src = ((int64_t)bf * p.num_kv_heads + h.g) * bs + from % bs;
      dst = ((int64_t)bt * p.num_kv_heads + h.g) * bs + to % bs;
    }
    p.new_weights[h.base + to] = x;
    p.new_positions[h.base + to] = t;
  }
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

// kCached: the keys fit in shared memory; else they are computed again in each phase.
template <int kLanes, bool kCached>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictParams p, int cluster, int smem_list, int split) {
  __shared__ __align__(16) Shared sh;
  extern __shared__ __align__(16) uint32_t dynamic[];   // kCached: this CTA's keys; smem_list: its list of moves
  // launched as a programmatic dependent: nothing is read before what precedes it is complete
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  const int seen = __ldg(p.num_tokens + row), old = __ldg(p.ordered_from + row);
  for (int i = tid; i < (cluster > 1 ? 4 : 3) * kBins / 4; i += kThreads)
    reinterpret_cast<int4 *>(&sh.hist[0][0])[i] = make_int4(0, 0, 0, 0);
  const bool bad_row = L < 0 || L > p.max_seq_len || L > (int64_t)p.max_blocks_per_seq * p.block_size || at < 0 ||
                       at >= p.num_weight_rows || seen < L || old < 0 || old > L;
  if (tid == 0 && rank == 0) {
    if (bad_row) record_error(p.err, PA_ERR_DEVICE_CHECK);
    if (g == 0) p.new_seq_lens[row] = bad_row ? L : min(L, p.budget);
  }
  int32_t *list = p.lists + rg * p.list_stride;   // the number of moves, padded to 16 bytes, destinations, sources
  if (split && tid == 0 && rank == 0) list[0] = 0;
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

  // this CTA's slots [lo, hi), a multiple of 128 per warp
  const int per_warp = ((L + cluster * kWarps - 1) / (cluster * kWarps) + 127) & ~127;
  const int lo = min((int64_t)L, (int64_t)rank * kWarps * per_warp), hi = min((int64_t)L, lo + (int64_t)kWarps * per_warp);
  const int wlo = min(hi, lo + warp * per_warp), whi = min(hi, wlo + per_warp);
  auto key_of = [&](float x, int t) { return t < p.num_sinks || t >= seen - p.num_recent ? kProtected : weight_key(x); };
  if constexpr (kCached) {
#pragma unroll 1
    for (int s0 = wlo + lane; s0 < whi; s0 += 4 * 32) {   // four slots' loads in flight
      float x[4];
      int t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = min(s0 + 32 * i, whi - 1);
        x[i] = w[s];
        t[i] = s < old ? pos[s] : seen - L + s;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s0 + 32 * i < whi) dynamic[s0 + 32 * i - lo] = key_of(x[i], t[i]);
    }
    __syncwarp();   // a warp reads its own keys only
  }
  // the keys of slots s .. s + 3 (s from lo on in steps of 4; slots past the warp's: 0, which `own` tells apart)
  auto four_keys = [&](int s, uint32_t (&k)[4]) {
    if constexpr (kCached) {
      const uint4 x = *reinterpret_cast<const uint4 *>(dynamic + (s - lo));   // (past the warp's: unused)
      k[0] = x.x;
      k[1] = x.y;
      k[2] = x.z;
      k[3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = s + j < whi ? key_of(w[s + j], position(s + j)) : 0u;
    }
  };
  const int mine = wlo + 4 * lane;   // the lane's first four slots
  barrier();   // the histograms are zeroed

  // ------------------------------------------------ the B-th largest key
  uint32_t prefix = 0, mask = 0;   // the digits found so far
  int need = B;                    // how many of the keys with this prefix stay
  int tie_total = 0;               // and how many have it
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    int *hist = cluster > 1 ? sh.own : sh.hist[pass];
    int safe = 0;   // protected tokens of the lane, of which there are many
#pragma unroll 1
    for (int s = mine; s < whi; s += 128) {
      uint32_t k[4];
      four_keys(s, k);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (s + j < whi && (k[j] & mask) == prefix) {
          if (k[j] == kProtected) ++safe;
          else atomicAdd(&hist[(k[j] >> shift) & digits], 1);
        }
    }
    safe = __reduce_add_sync(0xffffffffu, safe);
    if (safe && lane == 0) atomicAdd(&hist[digits], safe);
    // thread t: kBinsPerThread bins counted from the largest digit down, over the cluster
    const int b0 = kBins - kBinsPerThread * (tid + 1);
    if (cluster > 1) {
      __syncthreads();
      const uint32_t first = remote(&sh.hist[pass][b0], 0);
#pragma unroll
      for (int i = 0; i < kBinsPerThread; ++i) {
        const int n = sh.own[b0 + i];
        if (n) remote_add(first + 4 * i, n);
        sh.own[b0 + i] = 0;   // for the next pass
      }
    }
    barrier();
    if (rank == 0) {
      int v[kBinsPerThread];
      int sum = 0;
#pragma unroll
      for (int i = 0; i < kBinsPerThread; i += 4) {
        const int4 x = *reinterpret_cast<const int4 *>(&sh.hist[pass][b0 + i]);
        v[kBinsPerThread - 1 - i] = x.x;
        v[kBinsPerThread - 2 - i] = x.y;
        v[kBinsPerThread - 3 - i] = x.z;
        v[kBinsPerThread - 4 - i] = x.w;
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
            sh.found = make_int4(b0 + kBinsPerThread - 1 - i, need - before, v[i], 0);
            before = need;   // no later bin
          } else if (before < need) {
            before += v[i];
          }
        }
      }
    }
    barrier();
    const int4 found = cluster > 1 ? remote_int4(remote(&sh.found, 0)) : sh.found;
    prefix |= (uint32_t)found.x << shift;
    mask |= digits << shift;
    need = found.y;
    tie_total = found.z;
    // as many keys with this prefix as stay: they all do, whatever their other digits
    if (need == tie_total) break;
  }
  // a key stays if its digits found so far are larger, or equal and among the first `need`
  const bool rank_ties = need < tie_total;

  // ------------------------------------------------ ranks in slot order
  int tie0 = 0;   // equal keys before this warp
  if (rank_ties) {
    int n = 0;
#pragma unroll 1
    for (int s = mine; s < whi; s += 128) {
      uint32_t k[4];
      four_keys(s, k);
#pragma unroll
      for (int j = 0; j < 4; ++j) n += s + j < whi && (k[j] & mask) == prefix;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sh.ties[warp] = n;
    __syncthreads();
    tie0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.ties[lane] : 0);
    if (cluster > 1) {
      n = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.ties[lane] : 0);
      if (tid == 0) sh.counts[2] = n;
      barrier();
      n = remote_int(remote(&sh.counts[2], lane < cluster ? lane : 0));   // lane c: CTA c's
      tie0 += __reduce_add_sync(0xffffffffu, lane < (int)rank ? n : 0);
    }
  }
  // Which of the lane's four slots from s on stay, as bits; every lane calls it, `ties` equal keys before the warp's 128
  auto kept_of = [&](int s, int &ties) {
    uint32_t k[4], kept = 0, tie = 0;
    if (s < whi) four_keys(s, k);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (s + j < whi) {
        kept |= (uint32_t)((k[j] & mask) > prefix) << j;
        tie |= (uint32_t)((k[j] & mask) == prefix) << j;
      }
    if (!rank_ties) return kept | tie;
    const int end = warp_inclusive(__popc(tie));
    int left = need - ties - (end - __popc(tie));   // how many of the lane's equal keys may stay
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (tie >> j & 1u) kept |= (uint32_t)(left-- > 0) << j;
    ties += __shfl_sync(0xffffffffu, end, 31);
    return kept;
  };
  // the slots s .. s + 3 that are the warp's, and those of them below B, as bits
  auto first_bits = [](int n) { return n >= 4 ? 15u : n <= 0 ? 0u : (1u << n) - 1u; };
  {
    int nh = 0, nm = 0, ties = tie0;
#pragma unroll 1
    for (int s0 = wlo; s0 < whi; s0 += 128) {
      const int s = s0 + 4 * lane;
      const uint32_t kept = kept_of(s, ties), low = first_bits(B - s);
      nh += __popc(first_bits(whi - s) & low & ~kept);
      nm += __popc(kept & ~low);
    }
    nh = __reduce_add_sync(0xffffffffu, nh);
    nm = __reduce_add_sync(0xffffffffu, nm);
    if (lane == 0) {
      sh.holes[warp] = nh;
      sh.movers[warp] = nm;
    }
  }
  __syncthreads();
  int hole0 = 0, mover0 = 0;   // before this warp, in the CTA
  int moves = 0;
  {
    const int h = warp_inclusive(lane < kWarps ? sh.holes[lane] : 0), m = warp_inclusive(lane < kWarps ? sh.movers[lane] : 0);
    if (warp) {
      hole0 = __shfl_sync(0xffffffffu, h, warp - 1);
      mover0 = __shfl_sync(0xffffffffu, m, warp - 1);
    }
    moves = __shfl_sync(0xffffffffu, h, 31);
    if (cluster > 1 && tid == 31) {
      sh.counts[0] = h;
      sh.counts[1] = m;
    }
  }
  if (cluster > 1) {
    barrier();   // also: every read of weights and positions for the selection is done
    const int c = lane < cluster ? lane : 0;   // lane c: CTA c's
    const int h = remote_int(remote(&sh.counts[0], c)), m = remote_int(remote(&sh.counts[1], c));
    moves = __reduce_add_sync(0xffffffffu, lane < cluster ? h : 0);
    hole0 += __reduce_add_sync(0xffffffffu, lane < (int)rank ? h : 0);
    mover0 += __reduce_add_sync(0xffffffffu, lane < (int)rank ? m : 0);
  }   // one CTA: the barrier before the counts did
  int32_t *hole_list = smem_list ? reinterpret_cast<int32_t *>(dynamic) + smem_list : list + 4;
  int32_t *mover_list = hole_list + p.list_cap;
  // As many tokens move as slots are freed, at most list_cap.  Where keys are computed again that holds only while nobody
  // changes the weights under the kernel (two sequences of one weights row, in place), and the lists are not left even then.
  if constexpr (!kCached) moves = min(moves, (int)p.list_cap);
  auto listed = [&](int i) { return kCached ? i : min(i, (int)p.list_cap - 1); };
  {
    int ties = tie0;
#pragma unroll 1
    for (int s0 = wlo; s0 < whi; s0 += 128) {
      const int s = s0 + 4 * lane;
      const uint32_t kept = kept_of(s, ties), low = first_bits(B - s);
      const uint32_t hole = first_bits(whi - s) & low & ~kept, mover = kept & ~low;
      const int own = __popc(hole) | __popc(mover) << 16;
      const int end = warp_inclusive(own);   // both ranks in one scan: at most 128 each
      int hi0 = hole0 + ((end - own) & 0xffff), mi0 = mover0 + ((end - own) >> 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (hole >> j & 1u) hole_list[listed(hi0++)] = s + j;
        if (mover >> j & 1u) mover_list[listed(mi0++)] = s + j;
      }
      const int all = __shfl_sync(0xffffffffu, end, 31);
      hole0 += all & 0xffff;
      mover0 += all >> 16;
      // the tokens that stay where they are, 32 consecutive slots at a time
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t bits = __shfl_sync(0xffffffffu, kept & low, 8 * c + (lane >> 2));
        const int t = s0 + 32 * c + lane;
        if (bits >> (lane & 3) & 1u) {
          const float x = w[t];
          const int at_pos = position(t);
          p.new_weights[base + t] = x;
          p.new_positions[base + t] = at_pos;
        }
      }
    }
  }
  if (split && tid == 0 && rank == 0) list[0] = moves;
  // the lists (this cluster's global writes, or shared memory) are complete, and no CTA of the cluster ends while
  // another still reads its counts
  barrier();
  if (split) return;

  // up to 32 moves a turn, fewer where every warp then has some
  const Head head{g, row, L, seen, old, base};
  const int per_turn = min(32, max(8, (moves + cluster * kWarps - 1) / (cluster * kWarps)));
  for (int i0 = (rank * kWarps + warp) * per_turn; i0 < moves; i0 += cluster * kWarps * per_turn)
    move_tokens<kLanes>(p, head, hole_list, mover_list, i0, min(per_turn, moves - i0));
}

// The second launch: CTA b does kMoveWarps turns of 32 moves of head b / chunks.
constexpr int kMoveWarps = 8;
template <int kLanes>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p, int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t rg = blockIdx.x / chunks;
  const int32_t *list = p.lists + rg * p.list_stride;
  const int moves = __ldcg(list);
  const int i0 = ((int)(blockIdx.x - rg * chunks) * kMoveWarps + (threadIdx.x >> 5)) * 32;
  if (i0 >= moves) return;
  const int row = (int)(rg / p.num_kv_heads), g = (int)(rg - (int64_t)row * p.num_kv_heads);
  const int at = p.weight_rows ? __ldg(p.weight_rows + row) : row;
  const Head head{g, row, __ldg(p.seq_lens + row), __ldg(p.num_tokens + row), __ldg(p.ordered_from + row),
                  ((int64_t)at * p.num_kv_heads + g) * p.stride};
  move_tokens<kLanes>(p, head, list + 4, list + 4 + p.list_cap, i0, min(32, moves - i0));
}

template <int kLanes, bool kCached>
cudaError_t launch_one(const EvictParams &p, int cluster, int smem, int smem_list, bool split, cudaStream_t s) {
  cudaError_t e = ensure_smem_limit<evict_kernel<kLanes, kCached>>(kCachedKeys * 4 + kSmemMoves * 8);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)p.num_seqs * p.num_kv_heads * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((e = cudaLaunchKernelEx(&cfg, evict_kernel<kLanes, kCached>, p, cluster, smem_list, (int)split)) != cudaSuccess || !split)
    return e;
  const int chunks = (int)((p.list_cap + kMoveWarps * 32 - 1) / (kMoveWarps * 32));
  const int64_t grid = (int64_t)p.num_seqs * p.num_kv_heads * chunks;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kMoveWarps * 32);
  cfg.dynamicSmemBytes = 0;
  attr[0] = attr[1];
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<kLanes>, p, chunks);
}

template <int kLanes>
cudaError_t launch_lanes(const EvictParams &p, cudaStream_t s) {
  const int64_t heads = (int64_t)p.num_seqs * p.num_kv_heads;
  int sms = 0;
  cudaError_t e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  // CTAs per head: more while they fit on the GPU together and have a slot per thread, or while the keys do not fit
  int cluster = 1;
  while (cluster < kMaxCluster && heads * cluster * 2 <= 2 * sms && p.max_seq_len / (2 * cluster) >= kThreads) cluster *= 2;
  while (cluster < kMaxCluster && p.max_seq_len / cluster > kCachedKeys) cluster *= 2;
  if (heads * cluster > 2147483647ll) return cudaErrorInvalidValue;
  // a CTA's slots: per_warp rounded up to 128, times the warps
  const int64_t slots = (((int64_t)p.max_seq_len + cluster * kWarps - 1) / (cluster * kWarps) + 127) / 128 * 128 * kWarps;
  const bool cached = slots <= kCachedKeys;
  // the list of moves: behind the keys, 16 words in (an offset of 0 stands for the workspace)
  const int keys = cached ? (int)slots : 16;
  const bool split = heads * p.list_cap > kFusedMoves;
  const int smem_list = !split && cluster == 1 && p.list_cap <= kSmemMoves ? keys : 0;
  const int smem = smem_list ? (keys + 2 * (int)p.list_cap) * 4 : cached ? keys * 4 : 0;
  return cached ? launch_one<kLanes, true>(p, cluster, smem, smem_list, split, s)
                : launch_one<kLanes, false>(p, cluster, smem, smem_list, split, s);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s) {
  switch (p.row_bytes) {
    case 64: return launch_lanes<8>(p, s);
    case 128: return launch_lanes<16>(p, s);
    case 256: return launch_lanes<32>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
