// pa_decode_scaled.cu -- paged decode over a block-scaled fp8 cache
// (pa_decode_scaled).
//
// For a row's query head h of KV head g, over the row's L tokens:
//   out = sum_p w_p v_p / sum_p w_p / sv_p,   w_p = 2^(a_p + log2 sv_p - m),
//   a_p = scale log2(e) (q . k_p) sk_p,
// k_p, v_p the codes' values, sk_p, sv_p the scales of their block and head, m a
// running maximum.  V's scale is an addend of the exponent, so that the second
// product takes the codes as they are; the sum takes 1 / sv_p, in fp32, from
// unrounded w: a token whose values are tiny may hold most of the softmax.
//
// Bound by HBM: 2 head_dim bytes per token and KV head.  Everything between the load and the products therefore stays in the
// registers of one warp: no shared memory, no barrier, no hand-over between roles.  A warp takes 32 keys at a time, in two
// halves, and all (up to 8 or 16) query heads of the KV head:
//   S (16 keys x 8 heads)     = K (16 x D) . Q^T       mma.sync m16n8k16, f16
//   O^T (16 d x 8 heads) +=     V^T (16 d x 16 keys) . P^T
// The next tile's K is loaded as soon as S is done with this one's, V's likewise after the second product.
// The codes are widened to f16 in registers, exactly.  Any order of the D products
// will do, so the fragments are loaded as memory has them: a thread's K codes are
// 16 consecutive ones of a row per 64, and Q's fragments are laid out once to
// match.  V^T needs pairs of keys: a thread has the same 16 (head_dim 64: 8) codes
// of keys 2t, 2t+1, 2t+8, 2t+9, whose bytes are interleaved before they are widened.
// P goes from the first product's layout to the second's by a transposing move of 8
// x 8 matrices.  The queries are f16 as they are, or bf16 times a power of two that
// puts a row's largest element in [2^14, 2^15) (exact for every element above 2^-28
// of it).  P (the weights w) is rounded once to f16 for a 16-bit output, else taken as hi + lo.  From a piece's first tile on
// that has a V scale under 2^-8 of the largest that the warp has met, P is two bf16 terms for either, within 2^-17, and V's codes are
// widened to bf16: f16 would lose the tokens of small values (pa_internal.h).  (That loop apart costs the other one 1 % of the
// batch of 64, a branch within one loop 2 %.)
// (The tensor-memory decode of pa_decode_tc.cuh, given block scales, was bound by the hand-overs between its roles: 64
// sequences of 300-16000, 64/8 heads 279 us against 175; 33 of 1-5000, 40/8 heads of 64, f16 72 against 27.  Tiles of 16 keys
// left each warp one chain of dependent steps: 222 us.  With the codes copied to shared memory two tiles ahead: 248; an
// SM's loads in flight are not what it is short of.)  The batch of 64 runs at 6.0 TB/s, 89 % of a plain copy's rate (178 us; 193 with V
// scales 2^12 apart, 184 with an fp32 output).  Few tokens cost 7.6 us whatever they are: two launches and the chain lengths,
// block ids, codes, join; one sequence of 31999 tokens takes 22.8 us, 26 tiles to each CTA.
//
// Work.  The tiles of 32 keys of all (row, KV head share) in order are cut into equal ranges, one per CTA (six or eight
// warps, two CTAs per SM; fewer CTAs where a range would fall under kMinTiles): whatever the lengths, all finish together.  Every CTA
// finds its range from the lengths alone.  Within a range each (row, share) is a piece, its tiles dealt to the warps in turn
// and joined through shared memory.  A piece that is a whole row is final; others leave their sums in the workspace, at most
// two per CTA, and a second launch joins them.
#include <algorithm>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kTile = 32, kHalf = 16;     // keys per step of a warp, and per MMA
constexpr int kMinTiles = 8;              // tiles per CTA at least, while there are enough: about one per warp
// What a piece costs beside its tiles (its queries, the first codes' latency, the join of the warps), in tiles: some 3 us,
// which is 8 (head_dim 64: 15) tiles at an SM's share of the copy rate.  Chosen by time: with 1, 8, 12 and 16 tiles 64 sequences of
// 300-16000 take 195, 181, 177 and 177 us; at head_dim 64, with 1, 8, 16 and 24, 126, 114, 108 and 109, and 33 of 1-5000 44, 31,
// 27 and 28.
template <int D>
constexpr int kPieceCost = D == 128 ? 12 : 16;
constexpr int kChunk = 1024;              // rows whose tile counts a CTA has at hand
// A weight times V's scale is 2^kTopLog2 where the reference was taken, and O is rescaled before one exceeds 2^kRescaleLog2: as high as
// f16 allows, so that a small one keeps what bits it can.
constexpr float kTopLog2 = 7.f, kRescaleLog2 = 15.f;
#define kNegInfF (-__int_as_float(0x7f800000))

// Codes once read are not read again by this launch.
__device__ __forceinline__ uint4 ld16(const void *p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}
__device__ __forceinline__ uint2 ld8(const void *p, uint64_t policy) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v2.u32 {%0, %1}, [%2], %3;" : "=r"(v.x), "=r"(v.y) : "l"(p), "l"(policy));
  return v;
}

// Two e4m3 codes (the low 16 bits) -> f16x2, exactly.
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// The same -> bf16x2, exactly (the upper halves of the fp32 patterns).
__device__ __forceinline__ uint32_t widen2_bf16(uint32_t w) {
  const float2 f = unpack2_e4m3(w);
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}

// c (16 x 8) += a (16 x 16) . b (16 x 8), f16 operands (or bf16 ones).  (volatile: the whole warp has to execute it
// together, so that it must not be moved into a branch)
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements, rows by lane / 4 and pairs of columns by lane % 4, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A row's tokens, checked, and what a share of it costs, in tiles (an empty row has one, without keys).
__device__ __forceinline__ int row_len(const DecodeScaledParams &p, int row, bool report) {
  const int raw = __ldg(p.seq_lens + row);
  const int most = (int)min((int64_t)p.max_seq_len, (int64_t)p.max_blocks_per_seq * p.block_size);
  if (report && (raw < 0 || raw > most)) record_error(p.err, PA_ERR_DEVICE_CHECK);
  return min(max(raw, 0), most);
}
template <int D>
__device__ __forceinline__ int row_cost(int len) {
  return kPieceCost<D> + max(1, (len + kTile - 1) / kTile);
}

// a / b for a >= 0, b > 0: numbers of 32 bits, the usual ones, take a fifth of the time.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The cut of `total` tiles into `workers` ranges, the first `rem` one tile longer.
struct Cut {
  int64_t base, rem;
  int workers;
  __device__ Cut(int64_t total, int ctas) {
    workers = (int)max((int64_t)1, min((int64_t)ctas, total / kMinTiles));
    base = quotient(total, workers);
    rem = total - base * workers;
  }
  __device__ int64_t begin(int w) const { return w * base + min((int64_t)w, rem); }
  __device__ int worker(int64_t tile) const {
    const int64_t longer = rem * (base + 1);
    return (int)(tile < longer ? quotient(tile, base + 1) : rem + quotient(tile - longer, base));
  }
};

// Warps per CTA, and CTAs per SM: by the registers of a thread, 168 for 8 heads of 128 elements or 16 of 64 (12 warps), 255
// for 16 of 128, 128 for 8 of 64
template <int D, int NT>
constexpr int warps_of() {
  return (D == 128) == (NT == 1) ? 6 : 8;
}
template <int D, int NT>
constexpr int ctas_per_sm() {
  return D == 128 && NT == 2 ? 1 : 2;
}

template <typename QT, int D, int NT, bool kLo>
__global__ void __launch_bounds__(32 * warps_of<D, NT>(), ctas_per_sm<D, NT>()) decode_scaled_kernel(const DecodeScaledParams p) {
  constexpr int kHeads = 8 * NT, kSteps = D / 16, kHalves = D / 64, kRows = NT * kSteps * 4;
  constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;
  constexpr int kWarps = warps_of<D, NT>(), kThreads = 32 * kWarps;
  extern __shared__ __align__(16) float part[];   // [warp][kRows][lane]: the warps' sums
  __shared__ float2 part_ml[kWarps][kHeads];
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int64_t tiles_end[kChunk];    // of the present chunk of rows: tiles up to and including row i
  __shared__ int row_lens[kChunk];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // (each launch waits for what precedes it; the joining one is launched while this one runs)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint64_t policy = tc::l2_evict_first();
  const int units = p.num_kv_heads * p.shares, gqa = p.num_q_heads / p.num_kv_heads;

  // ---- this CTA's range of tiles
  auto block_sum = [&](int64_t x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    __syncthreads();
    if (lane == 0) warp_sum[warp] = x;
    __syncthreads();
    int64_t s = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += warp_sum[i];
    return s;
  };
  // rows [first, first + kChunk): their lengths and tiles_end, and the sum of their tiles
  auto scan_chunk = [&](int first, bool report) {
    constexpr int kPer = (kChunk + kThreads - 1) / kThreads;
    int mine[kPer];
    int64_t sum = 0;
    const int r0 = first + tid * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      mine[i] = tid * kPer + i < kChunk && r0 + i < p.num_seqs ? row_len(p, r0 + i, report) : -1;
    }
    __syncthreads();                       // (the lengths in use so far are no longer)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (mine[i] >= 0) row_lens[tid * kPer + i] = mine[i];
      mine[i] = mine[i] >= 0 ? row_cost<D>(mine[i]) : 0;
      sum += mine[i];
    }
    int64_t x = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int64_t before = x - sum, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += warp_sum[i];
      total += warp_sum[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      before += mine[i];
      if (tid * kPer + i < kChunk) tiles_end[tid * kPer + i] = before;
    }
    __syncthreads();
    return total;
  };
  int chunk = 0;
  int64_t chunk_total = scan_chunk(0, blockIdx.x == 0), total = chunk_total;
  if (p.num_seqs > kChunk) {
    int64_t x = 0;
    for (int r = kChunk + tid; r < p.num_seqs; r += kThreads) x += row_cost<D>(row_len(p, r, blockIdx.x == 0));
    total += block_sum(x);
  }
  const Cut cut(total * units, gridDim.x);
  const int worker = blockIdx.x;
  if (worker >= cut.workers) {
    if (tid == 0) p.joins[worker] = make_int4(0, 0, 0, 0);
    return;
  }
  int64_t pos = cut.begin(worker);
  const int64_t end = cut.begin(worker + 1);
  int64_t chunk_first = 0;                 // tiles (of one share) before the chunk
  bool joined = false;                     // a piece of this CTA goes on in the next one

  // the first piece: the chunk's first row with tiles_end above the range's first tile, by two ballots
  while (pos >= (chunk_first + chunk_total) * units) {
    chunk_first += chunk_total;
    chunk += kChunk;
    chunk_total = scan_chunk(chunk, false);
  }
  const int64_t in_chunk = quotient(pos, units) - chunk_first;   // (rows are whole multiples of `units` tiles)
  static_assert(kChunk == 1024, "a ballot of ballots");
  const int some = __ffs(__ballot_sync(0xffffffffu, tiles_end[32 * lane + 31] > in_chunk)) - 1;
  int at = 32 * some + __ffs(__ballot_sync(0xffffffffu, tiles_end[32 * some + lane] > in_chunk)) - 1;   // row, in the chunk
  int64_t before = at ? tiles_end[at - 1] : 0;
  constexpr int kCost = kPieceCost<D>;     // a share is kCost places, then its n tiles
  int n = (int)(tiles_end[at] - before) - kCost;
  int share = (int)quotient(pos - (chunk_first + before) * units, n + kCost);
  int place = (int)(pos - (chunk_first + before) * units - (int64_t)share * (n + kCost));

  while (pos < end) {
    // ---- the piece at pos: row, share, tiles [tile0, tile0 + count) of n
    const int places = (int)min((int64_t)(n + kCost - place), end - pos);
    const int tile0 = max(place - kCost, 0), count = max(place + places - kCost, 0) - tile0;
    if (count == 0) break;                 // the range ends before the share's first tile
    const int row = chunk + at, len = row_lens[at];
    const int kvh = share / p.shares, h_first = (share - kvh * p.shares) * p.share_heads;
    const int heads = min(p.share_heads, gqa - h_first), h0 = kvh * gqa + h_first;

    // ---- the piece's tiles, every kWarps-th to this warp: codes and scales a tile ahead, block ids two
    const int32_t *table = p.block_tables + (int64_t)row * p.max_blocks_per_seq;
    const int bs_log2 = p.block_size == 32 ? 5 : 4;
    const char *kpool = static_cast<const char *>(p.k_cache) + g * D + t * 16;
    const char *vpool = static_cast<const char *>(p.v_cache) + 2 * t * D + g * (D / 8);
    const int last = tile0 + count;
    struct Blocks {
      int32_t half[2];                     // block ids of the tile's halves; -1: past the piece, no token, or out of range
    };
    auto read_blocks = [&](int tile) {     // as the table has them
      Blocks b;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = tile * kTile + h * kHalf;
        b.half[h] = tile < last && key < len ? __ldg(table + (key >> bs_log2)) : -1;
      }
      return b;
    };
    // (checked when they are used: a check at once would wait for the table)
    auto check_blocks = [&](Blocks b, int tile) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (b.half[h] < 0 || b.half[h] >= p.num_blocks) {
          if (tile < last && tile * kTile + h * kHalf < len) record_error(p.err, PA_ERR_DEVICE_CHECK);
          b.half[h] = -1;
        }
      return b;
    };
    uint32_t kw[2][2][4 * kHalves];        // [half][row g or g + 8]: 16 codes of each 64
    uint32_t vw[2][4][D / 32];             // [half][keys 2t, 2t + 1, 2t + 8, 2t + 9]: D / 8 codes from g D / 8 on
    float sk[2], sv[2];
    // bytes before a half's first row in the pools (a half without a block reads the pools' first rows, unused)
    auto at_of = [&](int32_t b, int h) {
      const int off = h * (p.block_size - kHalf);   // blocks of 16: each half its own; of 32: its upper half
      return b < 0 ? (int64_t)0 : (((int64_t)b * p.num_kv_heads + kvh) * p.block_size + off) * D;
    };
    auto load_k = [&](const Blocks &b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const char *src = kpool + at_of(b.half[h], h);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < kHalves; ++j) {
            const uint4 x = ld16(src + r * 8 * D + j * 64, policy);
            kw[h][r][4 * j] = x.x, kw[h][r][4 * j + 1] = x.y, kw[h][r][4 * j + 2] = x.z, kw[h][r][4 * j + 3] = x.w;
          }
      }
    };
    auto load_v = [&](const Blocks &b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const char *src = vpool + at_of(b.half[h], h);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const char *at = src + ((r & 1) + (r >> 1) * 8) * D;
          if constexpr (D == 128) {
            const uint4 x = ld16(at, policy);
            vw[h][r][0] = x.x, vw[h][r][1] = x.y, vw[h][r][2] = x.z, vw[h][r][3] = x.w;
          } else {
            const uint2 x = ld8(at, policy);
            vw[h][r][0] = x.x, vw[h][r][1] = x.y;
          }
        }
      }
    };
    auto load_scales = [&](const Blocks &b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = b.half[h] < 0 ? 0 : (int64_t)b.half[h] * p.num_kv_heads + kvh;
        sk[h] = __ldg(p.k_scales + at);
        sv[h] = __ldg(p.v_scales + at);
      }
    };
    int tile = tile0 + warp;
    Blocks now = read_blocks(tile), next = read_blocks(tile + kWarps);
    // ---- Q's fragments: element pairs 4m, 4m + 1 and 4m + 2, 4m + 3 of this thread's codes, m = 0 .. kSteps - 1 (loaded
    // beside the block ids, laid out while the first codes are in flight)
    uint32_t qb[NT][kSteps][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < kHalves; ++j) {
        const int h = nt * 8 + g;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (h < heads) {
          const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const QT *>(p.q) + ((int64_t)row * p.num_q_heads + h0 + h) * D + j * 64 + t * 16);
          a = __ldg(src);
          b = __ldg(src + 1);
        }
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) qb[nt][4 * j + (i >> 1)][i & 1] = w[i];
      }
    now = check_blocks(now, tile);
    if (tile < last) {
      load_k(now);
      load_scales(now);
      load_v(now);
    }
    float factor[NT][2];                   // of heads 2t, 2t + 1: scale log2(e), over the row's power of two
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float back = 1.f;
      if constexpr (kBf16) {
        float amax = 0.f;
#pragma unroll
        for (int m = 0; m < kSteps; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            amax = fmaxf(amax, fmaxf(__uint_as_float((qb[nt][m][i] << 16) & 0x7fffffffu), __uint_as_float(qb[nt][m][i] & 0x7fff0000u)));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int eb = max(1, (int)((__float_as_uint(amax) >> 23) & 0xff));
        const int e = amax > 0.f ? max(-126, min(126, 141 - eb)) : 0;
        const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
        back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int m = 0; m < kSteps; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = unpack2(qb[nt][m][i], __nv_bfloat16{});
            const __half2 x = __floats2half2_rn(f.x * sc, f.y * sc);
            qb[nt][m][i] = *reinterpret_cast<const uint32_t *>(&x);
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) factor[nt][i] = p.s_mult * __shfl_sync(0xffffffffu, back, (2 * t + i) * 4);
    }

    float o[NT][kSteps][4];                // O^T: step i's rows g, g + 8 are elements g (D / 8) + 2 i, + 1; heads 2t, 2t + 1
    float m_ref[NT][2], l[NT][2], v_top = 0.f;   // v_top: the largest of V's scales in this warp's tiles so far
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m_ref[nt][i] = kNegInfF;
        l[nt][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

    // this warp's tiles, until one needs P and V in bf16; then (kWide) the rest of them
    auto walk = [&](auto in_bf16) {
      constexpr bool kWide = decltype(in_bf16)::value;
      for (; tile < last; tile += kWarps) {
        const bool more = tile + kWarps < last;
        float ks[2], lv[2], iv[2], v_low = -kNegInfF;   // this tile's scales (the next one's come in flight), the smallest of V's
        bool full = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool good = block_scale_ok(sk[h]) && block_scale_ok(sv[h]);
          if (!good && now.half[h] >= 0) record_error(p.err, PA_ERR_DEVICE_CHECK);
          ks[h] = good ? sk[h] : 1.f;
          lv[h] = good ? __log2f(sv[h]) : 0.f;
          iv[h] = good ? __fdividef(1.f, sv[h]) : 1.f;
          full = full && now.half[h] >= 0;
          if (now.half[h] >= 0) {
            v_low = fminf(v_low, good ? sv[h] : 1.f);
            v_top = fmaxf(v_top, good ? sv[h] : 1.f);
          }
        }
        // (every lane has the same scales; the vote makes it sure that they take one branch)
        if (!kWide && __any_sync(0xffffffffu, v_low * kNarrowScales < v_top)) return;
        // scores of each half's keys g, g + 8 and heads 2t, 2t + 1
        float s[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][nt][e] = 0.f;
#pragma unroll
        for (int m = 0; m < kSteps; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = widen2(kw[h][0][m]), a1 = widen2(kw[h][1][m]);
            const uint32_t a2 = widen2(kw[h][0][m] >> 16), a3 = widen2(kw[h][1][m] >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(s[h][nt], a0, a1, a2, a3, qb[nt][m][0], qb[nt][m][1]);
          }
        next = check_blocks(next, tile + kWarps);
        if (more) load_k(next);
        if (more) load_scales(next);
        const int nvis = len - tile * kTile; // keys of the tile that exist
        full = full && nvis >= kTile;
        // x: how far a score times V's scale is above the reference, log2 units
        float x[2][NT][4], top = kNegInfF;
        auto relative = [&]() {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[h][nt][e] = fmaf(s[h][nt][e], factor[nt][e & 1] * ks[h], lv[h] - m_ref[nt][e & 1]);
          if (!full)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (now.half[h] < 0 || h * kHalf + (e < 2 ? g : g + 8) >= nvis) x[h][nt][e] = kNegInfF;
        };
        relative();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; e += 2) top = tc::fmax3(top, x[h][nt][e], x[h][nt][e + 1]);
        if (__any_sync(0xffffffffu, top > kRescaleLog2)) {
          // new references, the maxima (before the first, the reference is -inf, and x is +inf or -inf)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float m = kNegInfF;
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = i; e < 4; e += 2)
                  if (x[h][nt][e] != kNegInfF) m = fmaxf(m, fmaf(s[h][nt][e], factor[nt][i] * ks[h], lv[h]));
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
              m = fmaxf(m - kTopLog2, m_ref[nt][i]);
              const float alpha = m == kNegInfF ? 1.f : fast_exp2(m_ref[nt][i] - m);
              m_ref[nt][i] = m;
              l[nt][i] *= alpha;
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                o[nt][k][i] *= alpha;
                o[nt][k][2 + i] *= alpha;
              }
            }
          relative();
        }
        // the weights times V's scale, in the place of the scores, and the sum without it
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[h][nt][e] = fast_exp2(x[h][nt][e]);
#pragma unroll
            for (int i = 0; i < 2; ++i) l[nt][i] = fmaf(x[h][nt][i] + x[h][nt][2 + i], iv[h], l[nt][i]);
          }
        if (!full) {   // V of keys that do not exist may hold anything, and P is 0 there
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (now.half[h] < 0 || h * kHalf + 2 * t + (r & 1) + (r >> 1) * 8 >= nvis)
#pragma unroll
                for (int k = 0; k < D / 32; ++k) vw[h][r][k] = 0;
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pb[NT][2], pl[NT][2];   // P's fragments, and (two terms) those of the rest, exact in fp32, rounded too
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // keys g, g + 8
              const float wa = x[h][nt][2 * r], wb = x[h][nt][2 * r + 1];
              if constexpr (kWide) {
                const uint32_t hi = tc::pack2(wa, wb, __nv_bfloat16{});
                pb[nt][r] = transpose8(hi);
                pl[nt][r] = transpose8(tc::pack2(wa - __uint_as_float(hi << 16), wb - __uint_as_float(hi & 0xffff0000u), __nv_bfloat16{}));
              } else {
                const __half2 hi = __floats2half2_rn(wa, wb);
                pb[nt][r] = transpose8(*reinterpret_cast<const uint32_t *>(&hi));
                if constexpr (kLo) {
                  const float2 f = __half22float2(hi);
                  pl[nt][r] = transpose8(tc::pack2(wa - f.x, wb - f.y, __half{}));
                }
              }
            }
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {   // four elements of each key at a time
            uint32_t a[2][2];              // [keys 2t.., 2t + 8..][elements 0 and 1, 2 and 3]: bytes of the two keys in turn
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              a[r][0] = __byte_perm(vw[h][2 * r][k], vw[h][2 * r + 1][k], 0x5140);
              a[r][1] = __byte_perm(vw[h][2 * r][k], vw[h][2 * r + 1][k], 0x7362);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              auto w2 = [](uint32_t c) { return kWide ? widen2_bf16(c) : widen2(c); };
              const uint32_t a0 = w2(a[0][i]), a1 = w2(a[0][i] >> 16), a2 = w2(a[1][i]), a3 = w2(a[1][i] >> 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float (&c)[4] = o[nt][2 * k + i];
                if constexpr (kWide) mma_bf16(c, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                else mma(c, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                if constexpr (kWide) mma_bf16(c, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                else if constexpr (kLo) mma(c, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
              }
            }
          }
        }
        if (more) load_v(next);
        now = next;
        next = read_blocks(tile + 2 * kWarps);
      }
    };
    walk(std::false_type{});
    walk(std::true_type{});

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[nt][i];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const int h = nt * 8 + 2 * t + i;
        if (g == 0) part_ml[warp][h] = make_float2(m_ref[nt][i], sum);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[(warp * kRows + 4 * (nt * kSteps + k) + e) * 32 + lane] = o[nt][k][e];
    __syncthreads();
    const bool whole = count == n, starts = tile0 == 0;
    const int64_t slot = 2 * (int64_t)worker + (starts ? 1 : 0);
    // a step's accumulators (elements d, d + 1 of heads 2t, 2t + 1) per warp and turn
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int ha = nt * 8 + 2 * t;
      float2 ml[kWarps][2];
      float M[2] = {kNegInfF, kNegInfF}, sum[2] = {0.f, 0.f}, sc[kWarps][2], inv[2];
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ml[w][i] = part_ml[w][ha + i];
          M[i] = fmaxf(M[i], ml[w][i].x);
        }
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sc[w][i] = ml[w][i].x == kNegInfF ? 0.f : fast_exp2(ml[w][i].x - M[i]);
          sum[i] = fmaf(ml[w][i].y, sc[w][i], sum[i]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) inv[i] = sum[i] == 0.f ? 0.f : 1.f / sum[i];
      for (int k = warp; k < kSteps; k += kWarps) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = fmaf(part[(w * kRows + 4 * (nt * kSteps + k) + e) * 32 + lane], sc[w][e & 1], x[e]);
        if (whole) {
          const int64_t to = ((int64_t)row * p.num_q_heads + h0 + ha) * D + g * (D / 8) + 2 * k;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (ha + i >= heads) continue;
            if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + to + i * D) = make_float2(x[i] * inv[i], x[2 + i] * inv[i]);
            else *reinterpret_cast<uint32_t *>(static_cast<QT *>(p.out) + to + i * D) = tc::pack2(x[i] * inv[i], x[2 + i] * inv[i], QT{});
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) p.ws_acc[(slot * kRows + 4 * (nt * kSteps + k) + e) * 32 + lane] = x[e];
          if (g == 0 && k == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i) p.ws_ml[slot * kHeads + ha + i] = make_float2(M[i], sum[i]);
        }
      }
    }
    __syncthreads();                       // part and part_ml are free
    if (starts && !whole) {                // it goes on in the CTAs up to that of its last tile
      joined = true;
      if (tid == 0) p.joins[worker] = make_int4(row, share, cut.worker(pos - place + n + kCost - 1) - worker + 1, 0);
    }
    // the next piece begins a share: of this row, of the next one
    pos += places;
    place = 0;
    if (++share == units && pos < end) {
      share = 0;
      if (++at == kChunk) {
        chunk_first += chunk_total;
        chunk += kChunk;
        chunk_total = scan_chunk(chunk, false);
        at = 0;
      }
      before = at ? tiles_end[at - 1] : 0;
      n = (int)(tiles_end[at] - before) - kCost;
    }
  }
  if (!joined && tid == 0) p.joins[worker] = make_int4(0, 0, 0, 0);
}

// The second launch: CTA (w, step) joins the pieces of the (row, share) that CTA w began and did not end, one step's
// accumulators (elements d, d + 1 of heads 2t, 2t + 1): slot 2w + 1, then slots 2(w + 1), 2(w + 2), ...; its warps share
// the pieces.
constexpr int kJoinWarps = 4;
template <typename QT, int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) decode_scaled_join_kernel(const DecodeScaledParams p) {
  constexpr int kHeads = 8 * NT, kSteps = D / 16, kRows = NT * kSteps * 4;
  __shared__ float part[kJoinWarps][4][32];
  __shared__ float2 part_ml[kJoinWarps][2][4];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w0 = blockIdx.x, step = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int4 j = __ldcg(p.joins + w0);
  if (j.z == 0) return;
  const int gqa = p.num_q_heads / p.num_kv_heads, kvh = j.y / p.shares, h_first = (j.y - kvh * p.shares) * p.share_heads;
  const int heads = min(p.share_heads, gqa - h_first), ha = step / kSteps * 8 + 2 * t;
  constexpr int kDeep = 8;                 // pieces in flight
  float M[2] = {kNegInfF, kNegInfF}, l[2] = {0.f, 0.f}, x[4] = {0.f, 0.f, 0.f, 0.f};
  for (int q0 = warp; q0 < j.z; q0 += kDeep * kJoinWarps) {
    float2 ml[kDeep][2];
    float y[kDeep][4];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int q = q0 + k * kJoinWarps;
      const int64_t slot = 2 * ((int64_t)w0 + min(q, j.z - 1)) + (q == 0 ? 1 : 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) ml[k][i] = __ldcg(p.ws_ml + slot * kHeads + ha + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[k][e] = __ldcg(p.ws_acc + (slot * kRows + 4 * step + e) * 32 + lane);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float m = M[i];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) m = fmaxf(m, ml[k][i].x);   // (the last piece may be there twice)
      const float ref = m == kNegInfF ? 0.f : m, so = fast_exp2(M[i] - ref);
      M[i] = m;
      l[i] *= so;
      x[i] *= so;
      x[2 + i] *= so;
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const float sn = q0 + k * kJoinWarps < j.z ? fast_exp2(ml[k][i].x - ref) : 0.f;
        l[i] = fmaf(ml[k][i].y, sn, l[i]);
        x[i] = fmaf(y[k][i], sn, x[i]);
        x[2 + i] = fmaf(y[k][2 + i], sn, x[2 + i]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) part[warp][e][lane] = x[e];
  if (g == 0)
#pragma unroll
    for (int i = 0; i < 2; ++i) part_ml[warp][i][t] = make_float2(M[i], l[i]);
  __syncthreads();
  if (warp >= 2 || ha + warp >= heads) return;   // warp i: head 2t + i
  float top = kNegInfF, sum = 0.f, a = 0.f, b = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, part_ml[w][warp][t].x);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float2 ml = part_ml[w][warp][t];
    const float sc = ml.x == kNegInfF ? 0.f : fast_exp2(ml.x - top);
    sum = fmaf(ml.y, sc, sum);
    a = fmaf(part[w][warp][lane], sc, a);
    b = fmaf(part[w][2 + warp][lane], sc, b);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t to = ((int64_t)j.x * p.num_q_heads + kvh * gqa + h_first + ha + warp) * D + g * (D / 8) + 2 * (step % kSteps);
  if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + to) = make_float2(a * inv, b * inv);
  else *reinterpret_cast<uint32_t *>(static_cast<QT *>(p.out) + to) = tc::pack2(a * inv, b * inv, QT{});
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, int warps, int smem, const DecodeScaledParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename QT, int D, int NT, bool kLo>
cudaError_t launch_heads(const DecodeScaledParams &p, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = current_sm_count(&sms);
  constexpr int warps = warps_of<D, NT>(), smem = warps * 8 * NT * D * 4;
  if (e == cudaSuccess) e = ensure_smem_limit<decode_scaled_kernel<QT, D, NT, kLo>>(smem);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)(std::min(sms, kPlanSms) * ctas_per_sm<D, NT>());
  if ((e = launch(decode_scaled_kernel<QT, D, NT, kLo>, dim3(ctas), warps, smem, p, s)) != cudaSuccess) return e;
  return launch(decode_scaled_join_kernel<QT, D, NT>, dim3(ctas, NT * (D / 16)), kJoinWarps, 0, p, s);
}

template <typename QT, int D>
cudaError_t launch_dim(const DecodeScaledParams &p, cudaStream_t s) {
  if (p.share_heads <= 8) return p.out_f32 ? launch_heads<QT, D, 1, true>(p, s) : launch_heads<QT, D, 1, false>(p, s);
  return p.out_f32 ? launch_heads<QT, D, 2, true>(p, s) : launch_heads<QT, D, 2, false>(p, s);
}

template <typename QT>
cudaError_t launch_type(const DecodeScaledParams &p, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? launch_dim<QT, 64>(p, s) : launch_dim<QT, 128>(p, s);
}

}  // namespace

cudaError_t launch_decode_scaled(const DecodeScaledParams &p, pa_dtype q_dtype, int head_dim, cudaStream_t s) {
  return q_dtype == PA_BF16 ? launch_type<__nv_bfloat16>(p, head_dim, s) : launch_type<__half>(p, head_dim, s);
}

}  // namespace pa
