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
// Bound by HBM: 2 head_dim bytes per token and KV head.  Everything between the
// load and the products therefore stays in the registers of one warp: no shared
// memory, no barrier, no hand-over between roles.  A warp takes 16 keys at a time
// and all (up to 8 or 16) query heads of the KV head:
//   S (16 keys x 8 heads)     = K (16 x D) . Q^T       mma.sync m16n8k16, f16
//   O^T (16 d x 8 heads) +=     V^T (16 d x 16 keys) . P^T
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
// Work.  The tiles of 16 keys of all (row, KV head share) in order are cut into equal
// ranges, one per CTA (four warps, four CTAs per SM; fewer CTAs where a range would
// fall under kMinTiles): whatever the lengths, all finish together.  Every CTA finds
// its range from the lengths alone.  Within a range each (row, share) is a piece,
// its tiles dealt to the warps in turn and joined through shared memory.  A piece
// that is a whole row is final; others leave their sums in the workspace, at most
// two per CTA, and a second launch joins them.
#include <algorithm>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;                 // keys per step of a warp
constexpr int kMinTiles = 16;             // tiles per CTA at least (while there are enough)
constexpr int kChunk = 1024;              // rows whose tile counts a CTA has at hand
constexpr float kRescaleLog2 = 8.f;       // O is rescaled when a score exceeds the reference maximum by 2^8
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

// c (16 x 8) += a (16 x 16) . b (16 x 8), f16 operands.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
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

template <typename QT, int D, int NT, bool kLo>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3) decode_scaled_kernel(const DecodeScaledParams p) {
  constexpr int kHeads = 8 * NT, kSteps = D / 16, kHalves = D / 64;
  constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;
  __shared__ float part[kWarps][kHeads][D];
  __shared__ float2 part_ml[kWarps][kHeads];
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int64_t tiles_end[kChunk];    // of the present chunk of rows: tiles up to and including row i

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

    // ---- the piece's tiles, every kWarps-th to this warp: codes and scales a tile ahead, block ids two
    const int32_t *table = p.block_tables + (int64_t)row * p.max_blocks_per_seq;
    const int bs_log2 = p.block_size == 32 ? 5 : 4;
    const char *kpool = static_cast<const char *>(p.k_cache), *vpool = static_cast<const char *>(p.v_cache);
    const int last = tile0 + count;
    auto block_of = [&](int tile) -> int32_t {   // -1: past the piece, no token, or out of range
      const int key = tile * kTile;
      if (tile >= last || key >= len) return -1;
      const int32_t bi = __ldg(table + (key >> bs_log2));
      if (bi >= 0 && bi < p.num_blocks) return bi;
      record_error(p.err, PA_ERR_DEVICE_CHECK);
      return -1;
    };
    using KWords = uint32_t[2][4 * kHalves];     // rows g, g + 8: 16 codes of each 64
    using VWords = uint32_t[4][D / 32];          // keys 2t, 2t + 1, 2t + 8, 2t + 9: D / 8 codes from g D / 8 on
    KWords kw;
    VWords vw;
    float sk, sv;
    // the tile's first row in the pool (a tile without a block reads the pool's first rows, unused)
    auto row_of = [&](int32_t b, int tile) {
      return b < 0 ? (int64_t)0 : ((int64_t)b * p.num_kv_heads + kvh) * p.block_size + ((tile * kTile) & (p.block_size - 1));
    };
    auto load_k = [&](int32_t b, int tile) {
      const char *src = kpool + (row_of(b, tile) + g) * D + t * 16;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < kHalves; ++j) {
          const uint4 x = ld16(src + r * 8 * D + j * 64, policy);
          kw[r][4 * j] = x.x, kw[r][4 * j + 1] = x.y, kw[r][4 * j + 2] = x.z, kw[r][4 * j + 3] = x.w;
        }
    };
    auto load_v = [&](int32_t b, int tile) {
      const char *src = vpool + (row_of(b, tile) + 2 * t) * D + g * (D / 8);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const char *at = src + ((r & 1) + (r >> 1) * 8) * D;
        if constexpr (D == 128) {
          const uint4 x = ld16(at, policy);
          vw[r][0] = x.x, vw[r][1] = x.y, vw[r][2] = x.z, vw[r][3] = x.w;
        } else {
          const uint2 x = ld8(at, policy);
          vw[r][0] = x.x, vw[r][1] = x.y;
        }
      }
    };
    auto load_scales = [&](int32_t b) {
      const int64_t at = b < 0 ? 0 : (int64_t)b * p.num_kv_heads + kvh;
      sk = __ldg(p.k_scales + at);
      sv = __ldg(p.v_scales + at);
    };
    int tile = tile0 + warp;
    int32_t blk = block_of(tile), next_blk = block_of(tile + kWarps);
    load_k(blk, tile);
    load_scales(blk);
    load_v(blk, tile);
    for (; tile < last; tile += kWarps) {
      // scores of keys g, g + 8 and heads 2t, 2t + 1
      float s[NT][4], s2[NT][4];           // two chains of MMAs
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
      for (int m = 0; m < kSteps; ++m) {
        const uint32_t a0 = widen2(kw[0][m]), a1 = widen2(kw[1][m]), a2 = widen2(kw[0][m] >> 16), a3 = widen2(kw[1][m] >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(m & 1 ? s2[nt] : s[nt], a0, a1, a2, a3, qb[nt][m][0], qb[nt][m][1]);
      }
      load_k(next_blk, tile + kWarps);
      // scales of this tile; the next one's in flight
      float ks = sk, lv = 0.f, iv = 1.f;
      if (blk >= 0) {
        if (block_scale_ok(sk) && block_scale_ok(sv)) {
          lv = __log2f(sv);
          iv = __fdividef(1.f, sv);
        } else {
          record_error(p.err, PA_ERR_DEVICE_CHECK);
          ks = 1.f;
        }
      }
      load_scales(next_blk);
      const int nvis = blk < 0 ? 0 : len - tile * kTile;   // keys of the tile that exist
      float top = kNegInfF;                                // how far a score is above its reference
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
      load_v(next_blk, tile + kWarps);
      blk = next_blk;
      next_blk = block_of(tile + 2 * kWarps);
    }

    // ---- join the warps
    __syncthreads();                       // the last piece's join is done
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[nt][i];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const int h = nt * 8 + 2 * t + i;
        if (g == 0) part_ml[warp][h] = make_float2(m_ref[nt][i], sum);
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          *reinterpret_cast<float2 *>(&part[warp][h][g * (D / 8) + 2 * k]) = make_float2(o[nt][k][i], o[nt][k][2 + i]);
      }
    __syncthreads();
    const bool whole = count == n, starts = tile0 == 0;
    const int64_t slot = 2 * (int64_t)worker + (starts ? 1 : 0);
    // 8 elements of a head per thread
    for (int e = tid; e < heads * (D / 8); e += kThreads) {
      const int h = e / (D / 8), d = e % (D / 8) * 8;
      float M = kNegInfF, sum = 0.f, x[8];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_ml[w][h].x);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = part_ml[w][h];
        const float sc = ml.x == kNegInfF ? 0.f : fast_exp2(ml.x - M);
        sum = fmaf(ml.y, sc, sum);
        const float4 a = *reinterpret_cast<const float4 *>(&part[w][h][d]), b = *reinterpret_cast<const float4 *>(&part[w][h][d + 4]);
        x[0] = fmaf(a.x, sc, x[0]), x[1] = fmaf(a.y, sc, x[1]), x[2] = fmaf(a.z, sc, x[2]), x[3] = fmaf(a.w, sc, x[3]);
        x[4] = fmaf(b.x, sc, x[4]), x[5] = fmaf(b.y, sc, x[5]), x[6] = fmaf(b.z, sc, x[6]), x[7] = fmaf(b.w, sc, x[7]);
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t at = ((int64_t)row * p.num_q_heads + h0 + h) * D + d;
        if (p.out_f32) {
          float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
          dst[0] = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
          dst[1] = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
        } else {
          *reinterpret_cast<uint4 *>(static_cast<QT *>(p.out) + at) =
              make_uint4(tc::pack2(x[0] * inv, x[1] * inv, QT{}), tc::pack2(x[2] * inv, x[3] * inv, QT{}),
                         tc::pack2(x[4] * inv, x[5] * inv, QT{}), tc::pack2(x[6] * inv, x[7] * inv, QT{}));
        }
      } else {
        float4 *dst = reinterpret_cast<float4 *>(p.ws_acc + (slot * p.share_heads + h) * D + d);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (d == 0) p.ws_ml[slot * p.share_heads + h] = make_float2(M, sum);
      }
    }
    if (starts && !whole) {                // it goes on in the CTAs up to that of its last tile
      joined = true;
      if (tid == 0) p.joins[worker] = make_int4(row, share, cut.worker(pos - tile0 + n - 1) - worker + 1, 0);
    }
    pos += count;
  }
  if (!joined && tid == 0) p.joins[worker] = make_int4(0, 0, 0, 0);
}

// The second launch: CTA (w, h) joins the pieces of the (row, share) that CTA w began and did not end, query head h:
// slot 2w + 1, then slots 2(w + 1), 2(w + 2), ...; its warps share the pieces.
template <typename QT, int D>
__global__ void __launch_bounds__(kThreads) decode_scaled_join_kernel(const DecodeScaledParams p) {
  __shared__ float part[kWarps][D];
  __shared__ float2 part_ml[kWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w0 = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 j = __ldcg(p.joins + w0);
  if (j.z == 0) return;
  const int gqa = p.num_q_heads / p.num_kv_heads, kvh = j.y / p.shares, h_first = (j.y - kvh * p.shares) * p.share_heads;
  if (h >= min(p.share_heads, gqa - h_first)) return;
  constexpr int kPer = D / 32, kDeep = 4;  // elements per lane, pieces in flight
  float M = kNegInfF, l = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int q0 = warp; q0 < j.z; q0 += kDeep * kWarps) {
    float2 ml[kDeep];
    float x[kDeep][kPer];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int q = min(q0 + k * kWarps, j.z - 1);
      const int64_t at = (q == 0 ? 2 * (int64_t)w0 + 1 : 2 * ((int64_t)w0 + q)) * p.share_heads + h;
      ml[k] = __ldcg(p.ws_ml + at);
      if constexpr (kPer == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4 *>(p.ws_acc + at * D) + lane);
        x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
      } else {
        const float2 y = __ldcg(reinterpret_cast<const float2 *>(p.ws_acc + at * D) + lane);
        x[k][0] = y.x, x[k][1] = y.y;
      }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      if (q0 + k * kWarps >= j.z) break;
      const float m = fmaxf(M, ml[k].x), ref = m == kNegInfF ? 0.f : m;
      const float so = fast_exp2(M - ref), sn = fast_exp2(ml[k].x - ref);
      M = m;
      l = l * so + ml[k].y * sn;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * so + x[k][e] * sn;
    }
  }
  if (lane == 0) part_ml[warp] = make_float2(M, l);
#pragma unroll
  for (int e = 0; e < kPer; ++e) part[warp][lane * kPer + e] = acc[e];
  __syncthreads();
  const int64_t out = ((int64_t)j.x * p.num_q_heads + kvh * gqa + h_first + h) * D;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float top = kNegInfF, sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_ml[w].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float sc = part_ml[w].x == kNegInfF ? 0.f : fast_exp2(part_ml[w].x - top);
      sum = fmaf(part_ml[w].y, sc, sum);
      x = fmaf(part[w][d], sc, x);
    }
    x = sum == 0.f ? 0.f : x / sum;
    if (p.out_f32) static_cast<float *>(p.out)[out + d] = x;
    else static_cast<QT *>(p.out)[out + d] = Elem<QT>::from_f32(x);
  }
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, const DecodeScaledParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename QT, int D, int NT>
cudaError_t launch_heads(const DecodeScaledParams &p, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)std::min(sms, kPlanSms) * (NT == 1 ? 4 : 3);
  e = p.out_f32 ? launch(decode_scaled_kernel<QT, D, NT, true>, dim3(ctas), p, s)
                : launch(decode_scaled_kernel<QT, D, NT, false>, dim3(ctas), p, s);
  return e != cudaSuccess ? e : launch(decode_scaled_join_kernel<QT, D>, dim3(ctas, (unsigned)p.share_heads), p, s);
}

template <typename QT>
cudaError_t launch_type(const DecodeScaledParams &p, int head_dim, cudaStream_t s) {
  if (head_dim == 64) return p.share_heads <= 8 ? launch_heads<QT, 64, 1>(p, s) : launch_heads<QT, 64, 2>(p, s);
  return p.share_heads <= 8 ? launch_heads<QT, 128, 1>(p, s) : launch_heads<QT, 128, 2>(p, s);
}

}  // namespace

cudaError_t launch_decode_scaled(const DecodeScaledParams &p, pa_dtype q_dtype, int head_dim, cudaStream_t s) {
  return q_dtype == PA_BF16 ? launch_type<__nv_bfloat16>(p, head_dim, s) : launch_type<__half>(p, head_dim, s);
}

}  // namespace pa
