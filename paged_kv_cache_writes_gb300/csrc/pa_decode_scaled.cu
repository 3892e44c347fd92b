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
// Bound by HBM: 2 head_dim bytes per token and KV head.  Everything between the load and the products therefore stays in
// one warp: no barrier, no hand-over between roles.  A warp takes 16 keys at a time and all (up to 8 or 16) query heads of
// the KV head:
//   S (16 keys x 8 heads)     = K (16 x D) . Q^T       mma.sync m16n8k16, f16
//   O^T (16 d x 8 heads) +=     V^T (16 d x 16 keys) . P^T
// Each lane copies the codes that it will itself need, two tiles ahead, into places of its own in shared memory
// (cp.async): the bytes in flight cost no registers, and no lane waits for another.
// The codes are widened to f16 in registers, exactly.  Any order of the D products
// will do, so the fragments are loaded as memory has them: a thread's K codes are
// 16 consecutive ones of a row per 64, and Q's fragments are laid out once to
// match.  V^T needs pairs of keys: a thread has the same 16 (head_dim 64: 8) codes
// of keys 2t, 2t+1, 2t+8, 2t+9, whose bytes are interleaved before they are widened.
// P goes from the first product's layout to the second's by a transposing move of 8
// x 8 matrices.  The queries are f16 as they are, or bf16 times a power of two that
// puts a row's largest element in [2^14, 2^15) (exact for every element above 2^-28
// of it).  P is rounded once to f16 for a 16-bit output, else taken as hi + lo.
// Per 16 keys with D = 128 a warp issues about 190 instructions, 16 of them MMAs, for
// 4 KB of codes: a quarter of what an SM could issue at the copy rate.  (The
// tensor-memory decode of pa_decode_tc.cuh, given block scales, was bound by the
// hand-overs between its roles: 64 sequences of 300-16000, 64/8 heads 279 us against
// XXX; 33 of 1-5000, head_dim 64, f16 72 against XXX.)
//
// Work.  The tiles of 16 keys of all (row, KV head share) in order are cut into equal ranges, one per CTA (eight warps, two
// CTAs per SM; fewer CTAs where a range would fall under kMinTiles): whatever the lengths, all finish together.  Every CTA
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

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 3;                // tiles of a warp in shared memory
constexpr int kTile = 16;                 // keys per step of a warp
constexpr int kMinTiles = 32;             // tiles per CTA at least (while there are enough)
constexpr int kChunk = 1024;              // rows whose tile counts a CTA has at hand
constexpr float kRescaleLog2 = 8.f;       // O is rescaled when a score exceeds the reference maximum by 2^8
#define kNegInfF (-__int_as_float(0x7f800000))

// Copies of codes to shared memory.  (Without an L2 policy: the same copies with an evict-first one, the addresses checked
// to be in bounds and aligned, ended in an SM exception; plain loads with it had not.)
__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Two e4m3 codes (the low 16 bits) -> f16x2, exactly.
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// c (16 x 8) += a (16 x 16) . b (16 x 8), f16 operands.  (volatile: the whole warp has to execute it together, so that it
// must not be moved into a branch)
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements, rows by lane / 4 and pairs of columns by lane % 4, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A row's tokens, checked, and its tiles (an empty row has one, without keys).
__device__ __forceinline__ int row_len(const DecodeScaledParams &p, int row, bool report) {
  const int raw = __ldg(p.seq_lens + row);
  const int most = (int)min((int64_t)p.max_seq_len, (int64_t)p.max_blocks_per_seq * p.block_size);
  if (report && (raw < 0 || raw > most)) record_error(p.err, PA_ERR_DEVICE_CHECK);
  return min(max(raw, 0), most);
}
__device__ __forceinline__ int row_tiles(int len) { return max(1, (len + kTile - 1) / kTile); }

// The cut of `total` tiles into `workers` ranges, the first `rem` one tile longer.
struct Cut {
  int64_t base, rem;
  int workers;
  __device__ Cut(int64_t total, int ctas) {
    workers = (int)max((int64_t)1, min((int64_t)ctas, total / kMinTiles));
    base = total / workers;
    rem = total - base * workers;
  }
  __device__ int64_t begin(int w) const { return w * base + min((int64_t)w, rem); }
  __device__ int worker(int64_t tile) const {
    const int64_t longer = rem * (base + 1);
    return (int)(tile < longer ? tile / (base + 1) : rem + (tile - longer) / base);
  }
};

// CTAs per SM: the O of 16 query heads of 128 elements takes 64 registers more
template <int D, int NT>
constexpr int ctas_per_sm() {
  return D == 128 && NT == 2 ? 1 : 2;
}
template <int D>
constexpr int kRingBytes = kWarps *kStages * 2 * kTile * D;

template <typename QT, int D, int NT, bool kLo>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<D, NT>()) decode_scaled_kernel(const DecodeScaledParams p) {
  constexpr int kHeads = 8 * NT, kSteps = D / 16, kHalves = D / 64, kRows = NT * kSteps * 4;
  constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;
  // [warp][stage]: K as [row 0 or 1][half][lane] of 16 bytes, V as [key 0 .. 3][lane] of D / 8; between pieces the warps'
  // sums, float [warp][kRows][lane]
  extern __shared__ __align__(16) uint8_t ring[];
  static_assert(kRows * 128 <= kStages * 2 * kTile * D, "a warp's sums fit in its part of the ring");
  float *part = reinterpret_cast<float *>(ring);
  __shared__ float2 part_ml[kWarps][kHeads];
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int64_t tiles_end[kChunk];    // of the present chunk of rows: tiles up to and including row i

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // (each launch waits for what precedes it; the joining one is launched while this one runs)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  // rows [first, first + kChunk): tiles_end, and their sum
  auto scan_chunk = [&](int first) {
    constexpr int kPer = kChunk / kThreads;
    int mine[kPer];
    int64_t sum = 0;
    const int r0 = first + tid * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      mine[i] = r0 + i < p.num_seqs ? row_tiles(row_len(p, r0 + i, false)) : 0;
      sum += mine[i];
    }
    int64_t x = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    __syncthreads();
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
      tiles_end[tid * kPer + i] = before;
    }
    __syncthreads();
    return total;
  };
  int chunk = 0;
  int64_t chunk_total = scan_chunk(0), total = chunk_total;
  if (p.num_seqs > kChunk) {
    int64_t x = 0;
    for (int r = kChunk + tid; r < p.num_seqs; r += kThreads) x += row_tiles(row_len(p, r, false));
    total += block_sum(x);
  }
  if (blockIdx.x == 0)
    for (int r = tid; r < p.num_seqs; r += kThreads) (void)row_len(p, r, true);
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

  while (pos < end) {
    // ---- the piece at pos: row, share, tiles [tile0, tile0 + count) of n
    while (pos >= (chunk_first + chunk_total) * units) {
      chunk_first += chunk_total;
      chunk += kChunk;
      chunk_total = scan_chunk(chunk);
    }
    const int64_t in_chunk = pos / units - chunk_first;   // (rows are whole multiples of `units` tiles)
    int lo = 0, hi = kChunk - 1;           // the first row of the chunk with tiles_end > in_chunk
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tiles_end[mid] > in_chunk) hi = mid;
      else lo = mid + 1;
    }
    const int row = chunk + lo;
    const int64_t before = lo ? tiles_end[lo - 1] : 0;
    const int n = (int)(tiles_end[lo] - before);
    const int64_t row_first = (chunk_first + before) * units;
    const int share = (int)((pos - row_first) / n), tile0 = (int)(pos - row_first - (int64_t)share * n);
    const int count = (int)min((int64_t)(n - tile0), end - pos);
    const int kvh = share / p.shares, h_first = (share - kvh * p.shares) * p.share_heads;
    const int heads = min(p.share_heads, gqa - h_first), h0 = kvh * gqa + h_first;
    const int len = row_len(p, row, false);

    // ---- Q's fragments: element pairs 4m, 4m + 1 and 4m + 2, 4m + 3 of this thread's codes, m = 0 .. kSteps - 1
    uint32_t qb[NT][kSteps][2];
    float factor[NT][2];                   // of heads 2t, 2t + 1: scale log2(e), over the row's power of two
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + g;
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < kHalves; ++j) {
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (h < heads) {
          const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const QT *>(p.q) + ((int64_t)row * p.num_q_heads + h0 + h) * D + j * 64 + t * 16);
          a = __ldg(src);
          b = __ldg(src + 1);
        }
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          qb[nt][4 * j + (i >> 1)][i & 1] = w[i];
          if constexpr (kBf16)
            amax = fmaxf(amax, fmaxf(__uint_as_float((w[i] << 16) & 0x7fffffffu), __uint_as_float(w[i] & 0x7fff0000u)));
        }
      }
      float back = 1.f;
      if constexpr (kBf16) {
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
    float m_ref[NT][2], l[NT][2];
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

    // ---- the piece's tiles, every kWarps-th to this warp: lane i has the block id and the scales of the warp's tile 32 w + i
    // (w the present window), and those of the next window; codes two tiles ahead
    const int32_t *table = p.block_tables + (int64_t)row * p.max_blocks_per_seq;
    const int bs_log2 = p.block_size == 32 ? 5 : 4;
    const char *kpool = static_cast<const char *>(p.k_cache), *vpool = static_cast<const char *>(p.v_cache);
    const int mine = (count - warp + kWarps - 1) / kWarps;   // this warp's tiles
    struct Window {
      int32_t blk;                         // -1: past the piece, no token, or out of range
      float k, log2_v, inv_v;
    };
    auto window = [&](int first) {
      Window w{-1, 1.f, 0.f, 1.f};
      const int i = first + lane, key = (tile0 + warp + kWarps * i) * kTile;
      if (i < mine && key < len) {
        const int32_t bi = __ldg(table + (key >> bs_log2));
        if (bi >= 0 && bi < p.num_blocks) {
          w.blk = bi;
          const int64_t at = (int64_t)bi * p.num_kv_heads + kvh;
          const float sk = __ldg(p.k_scales + at), sv = __ldg(p.v_scales + at);
          if (block_scale_ok(sk) && block_scale_ok(sv)) w = {bi, sk, __log2f(sv), __fdividef(1.f, sv)};
          else record_error(p.err, PA_ERR_DEVICE_CHECK);
        } else {
          record_error(p.err, PA_ERR_DEVICE_CHECK);
        }
      }
      return w;
    };
    uint8_t *stage0 = ring + warp * (kStages * 2 * kTile * D);
    // the codes of a tile in block b (-1: the pool's first rows, unused); always a group, so that they count in order
    auto copy_tile = [&](int i, int32_t b) {
      if (i < mine) {
        const int off = ((tile0 + warp + kWarps * i) * kTile) & (p.block_size - 1);
        const int64_t at = b < 0 ? (int64_t)0 : (((int64_t)b * p.num_kv_heads + kvh) * p.block_size + off) * D;
        uint8_t *dst = stage0 + i % kStages * (2 * kTile * D);
        const char *ks = kpool + at + g * D + t * 16;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < kHalves; ++j) copy16(dst + ((r * kHalves + j) * 32 + lane) * 16, ks + r * 8 * D + j * 64);
        const char *vs = vpool + at + 2 * t * D + g * (D / 8);
        dst += kTile * D;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const char *src = vs + ((r & 1) + (r >> 1) * 8) * D;
          if constexpr (D == 128) copy16(dst + (r * 32 + lane) * 16, src);
          else copy8(dst + (r * 32 + lane) * 8, src);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Window now = window(0), next = window(32);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy_tile(i, __shfl_sync(0xffffffffu, now.blk, i));
    for (int i = 0; i < mine; ++i) {
      const int32_t blk = __shfl_sync(0xffffffffu, now.blk, i & 31);
      const float ks = __shfl_sync(0xffffffffu, now.k, i & 31), lv = __shfl_sync(0xffffffffu, now.log2_v, i & 31);
      const float iv = __shfl_sync(0xffffffffu, now.inv_v, i & 31);
      const int ahead = (i & 31) + kStages - 1;
      const int32_t ahead_blk = __shfl_sync(0xffffffffu, ahead < 32 ? now.blk : next.blk, ahead & 31);
      const uint8_t *src = stage0 + i % kStages * (2 * kTile * D);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      // scores of keys g, g + 8 and heads 2t, 2t + 1
      float s[NT][4], s2[NT][4];           // two chains of MMAs
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
      for (int j = 0; j < kHalves; ++j) {
        const uint4 x = *reinterpret_cast<const uint4 *>(src + (j * 32 + lane) * 16);
        const uint4 y = *reinterpret_cast<const uint4 *>(src + ((kHalves + j) * 32 + lane) * 16);
        const uint32_t r0[4] = {x.x, x.y, x.z, x.w}, r1[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t a0 = widen2(r0[q]), a1 = widen2(r1[q]), a2 = widen2(r0[q] >> 16), a3 = widen2(r1[q] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(q & 1 ? s2[nt] : s[nt], a0, a1, a2, a3, qb[nt][4 * j + q][0], qb[nt][4 * j + q][1]);
        }
      }
      uint32_t vw[4][D / 32];              // V codes of keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint8_t *at = src + kTile * D + (r * 32 + lane) * (D / 8);
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4 *>(at);
          vw[r][0] = x.x, vw[r][1] = x.y, vw[r][2] = x.z, vw[r][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2 *>(at);
          vw[r][0] = x.x, vw[r][1] = x.y;
        }
      }
      copy_tile(i + kStages - 1, ahead_blk);   // (the place of tile i - 1, which this lane has read)
      if ((i & 31) == 31) {
        now = next;
        next = window(i + 33);
      }
      const int nvis = blk < 0 ? 0 : len - (tile0 + warp + kWarps * i) * kTile;   // keys of the tile that exist
      float top = kNegInfF;                                                      // how far a score is above its reference
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = fmaf(s[nt][e] + s2[nt][e], factor[nt][e & 1] * ks, lv);
          s[nt][e] = (e < 2 ? g : g + 8) < nvis ? x : kNegInfF;
          top = fmaxf(top, s[nt][e] - m_ref[nt][e & 1]);   // (NaN, -inf less -inf, is ignored)
        }
      if (__any_sync(0xffffffffu, top > kRescaleLog2)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = fmaxf(s[nt][i], s[nt][2 + i]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            m = fmaxf(m, m_ref[nt][i]);
            const float alpha = m == kNegInfF ? 1.f : fast_exp2(m_ref[nt][i] - m);
            m_ref[nt][i] = m;
            l[nt][i] *= alpha;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              o[nt][k][i] *= alpha;
              o[nt][k][2 + i] *= alpha;
            }
          }
      }
      // P, its sum, and its fragments
      uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = s[nt][e] == kNegInfF ? 0.f : fast_exp2(s[nt][e] - m_ref[nt][e & 1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) l[nt][i] = fmaf(w[i] + w[2 + i], iv, l[nt][i]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {   // keys g, g + 8
          const __half2 hi = __floats2half2_rn(w[2 * r], w[2 * r + 1]);
          pb[nt][r] = transpose8(*reinterpret_cast<const uint32_t *>(&hi));
          if constexpr (kLo) {          // the rest, exact in fp32, rounded too
            const float2 h = __half22float2(hi);
            const __half2 low = __floats2half2_rn(w[2 * r] - h.x, w[2 * r + 1] - h.y);
            pl[nt][r] = transpose8(*reinterpret_cast<const uint32_t *>(&low));
          }
        }
      }
      if (nvis < kTile) {   // V of keys that do not exist may hold anything, and P is 0 there
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (2 * t + (r & 1) + (r >> 1) * 8 >= nvis)
#pragma unroll
            for (int k = 0; k < D / 32; ++k) vw[r][k] = 0;
      }
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {   // four elements of each key at a time
        uint32_t a[2][2];                  // [keys 2t.., 2t + 8..][elements 0 and 1, 2 and 3]: bytes of the two keys in turn
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          a[r][0] = __byte_perm(vw[2 * r][k], vw[2 * r + 1][k], 0x5140);
          a[r][1] = __byte_perm(vw[2 * r][k], vw[2 * r + 1][k], 0x7362);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a0 = widen2(a[0][i]), a1 = widen2(a[0][i] >> 16), a2 = widen2(a[1][i]), a3 = widen2(a[1][i] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(o[nt][2 * k + i], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            if constexpr (kLo) mma(o[nt][2 * k + i], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }

    // ---- join the warps, each of whose sums goes to its own part of the ring
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    float *mine_part = part + warp * (kStages * 2 * kTile * D / 4);
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
        for (int e = 0; e < 4; ++e) mine_part[(4 * (nt * kSteps + k) + e) * 32 + lane] = o[nt][k][e];
    __syncthreads();
    const bool whole = count == n, starts = tile0 == 0;
    const int64_t slot = 2 * (int64_t)worker + (starts ? 1 : 0);
    // a step's accumulators (elements d, d + 1 of heads 2t, 2t + 1) per warp and turn
    for (int k = warp; k < NT * kSteps; k += kWarps) {
      const int ha = k / kSteps * 8 + 2 * t, d = g * (D / 8) + 2 * (k % kSteps);
      float M[2] = {kNegInfF, kNegInfF}, sum[2] = {0.f, 0.f}, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) M[i] = fmaxf(M[i], part_ml[w][ha + i].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        float sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 ml = part_ml[w][ha + i];
          sc[i] = ml.x == kNegInfF ? 0.f : fast_exp2(ml.x - M[i]);
          sum[i] = fmaf(ml.y, sc[i], sum[i]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fmaf(part[w * (kStages * 2 * kTile * D / 4) + (4 * k + e) * 32 + lane], sc[e & 1], x[e]);
      }
      if (whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (ha + i >= heads) continue;
          const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
          const int64_t at = ((int64_t)row * p.num_q_heads + h0 + ha + i) * D + d;
          if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at) = make_float2(x[i] * inv, x[2 + i] * inv);
          else *reinterpret_cast<uint32_t *>(static_cast<QT *>(p.out) + at) = tc::pack2(x[i] * inv, x[2 + i] * inv, QT{});
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) p.ws_acc[(slot * kRows + 4 * k + e) * 32 + lane] = x[e];
        if (g == 0 && k % kSteps == 0)
#pragma unroll
          for (int i = 0; i < 2; ++i) p.ws_ml[slot * kHeads + ha + i] = make_float2(M[i], sum[i]);
      }
    }
    __syncthreads();                       // the ring and part_ml are free
    if (starts && !whole) {                // it goes on in the CTAs up to that of its last tile
      joined = true;
      if (tid == 0) p.joins[worker] = make_int4(row, share, cut.worker(pos - tile0 + n - 1) - worker + 1, 0);
    }
    pos += count;
  }
  if (!joined && tid == 0) p.joins[worker] = make_int4(0, 0, 0, 0);
}

// The second launch: CTA (w, k) joins the pieces of the (row, share) that CTA w began and did not end, accumulators of step
// k: slot 2w + 1, then slots 2(w + 1), 2(w + 2), ...; its warps share the pieces.
template <typename QT, int D, int NT>
__global__ void __launch_bounds__(kThreads) decode_scaled_join_kernel(const DecodeScaledParams p) {
  constexpr int kHeads = 8 * NT, kSteps = D / 16, kRows = NT * kSteps * 4;
  __shared__ float part[kWarps][4][32];
  __shared__ float2 part_ml[kWarps][2][4];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w0 = blockIdx.x, step = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int4 j = __ldcg(p.joins + w0);
  if (j.z == 0) return;
  const int gqa = p.num_q_heads / p.num_kv_heads, kvh = j.y / p.shares, h_first = (j.y - kvh * p.shares) * p.share_heads;
  const int heads = min(p.share_heads, gqa - h_first), ha = step / kSteps * 8 + 2 * t;
  constexpr int kDeep = 4;                 // pieces in flight
  float M[2] = {kNegInfF, kNegInfF}, l[2] = {0.f, 0.f}, x[4] = {0.f, 0.f, 0.f, 0.f};
  for (int q0 = warp; q0 < j.z; q0 += kDeep * kWarps) {
    float2 ml[kDeep][2];
    float y[kDeep][4];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int q = min(q0 + k * kWarps, j.z - 1);
      const int64_t slot = q == 0 ? 2 * (int64_t)w0 + 1 : 2 * ((int64_t)w0 + q);
#pragma unroll
      for (int i = 0; i < 2; ++i) ml[k][i] = __ldcg(p.ws_ml + slot * kHeads + ha + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[k][e] = __ldcg(p.ws_acc + (slot * kRows + 4 * step + e) * 32 + lane);
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      if (q0 + k * kWarps >= j.z) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float m = fmaxf(M[i], ml[k][i].x), ref = m == kNegInfF ? 0.f : m;
        const float so = fast_exp2(M[i] - ref), sn = fast_exp2(ml[k][i].x - ref);
        M[i] = m;
        l[i] = l[i] * so + ml[k][i].y * sn;
        x[i] = x[i] * so + y[k][i] * sn;
        x[2 + i] = x[2 + i] * so + y[k][2 + i] * sn;
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
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_ml[w][warp][t].x);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float2 ml = part_ml[w][warp][t];
    const float sc = ml.x == kNegInfF ? 0.f : fast_exp2(ml.x - top);
    sum = fmaf(ml.y, sc, sum);
    a = fmaf(part[w][warp][lane], sc, a);
    b = fmaf(part[w][2 + warp][lane], sc, b);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t at = ((int64_t)j.x * p.num_q_heads + kvh * gqa + h_first + ha + warp) * D + g * (D / 8) + 2 * (step % kSteps);
  if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at) = make_float2(a * inv, b * inv);
  else *reinterpret_cast<uint32_t *>(static_cast<QT *>(p.out) + at) = tc::pack2(a * inv, b * inv, QT{});
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, int smem, const DecodeScaledParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
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
  if (e == cudaSuccess) e = ensure_smem_limit<decode_scaled_kernel<QT, D, NT, kLo>>(kRingBytes<D>);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)(std::min(sms, kPlanSms) * ctas_per_sm<D, NT>());
  if ((e = launch(decode_scaled_kernel<QT, D, NT, kLo>, dim3(ctas), kRingBytes<D>, p, s)) != cudaSuccess) return e;
  return launch(decode_scaled_join_kernel<QT, D, NT>, dim3(ctas, NT * (D / 16)), 0, p, s);
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
