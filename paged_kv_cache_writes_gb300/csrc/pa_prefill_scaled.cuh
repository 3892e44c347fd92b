// pa_prefill_scaled.cuh -- chunked-prefill attention over a block-scaled fp8
// cache (pa_prefill_chunk_scaled) on the 5th-generation tensor cores.
//
// Row r of chunk c, at position t = q_start[c] + r, query head h of KV head g:
//   out = sum_p w_p v_p / sum_p w_p / sv_p  over p <= t,
//   w_p = 2^(a_p + log2 sv_p - m),  a_p = scale log2(e) (q . k_p) sk_p,
// k_p, v_p the codes' values, sk_p, sv_p the scales of their block and head, m a
// running maximum of a_p + log2 sv_p.  K's scale multiplies the scores and V's is
// an addend of the exponent, so that both products take the codes as they are;
// the sum takes 1 / sv_p, in fp32, from unrounded w: a token whose values are
// tiny may hold most of the softmax.  A run of 16 keys lies in one block.
//
// Operands.  V's codes are widened to f16, exactly, on their way into shared memory, and w is rounded once to f16 for a
// 16-bit output (kLo false), else taken as hi + lo.  In a CTA whose keys' V scales lie more than 2^8 apart (the loaders look
// first) both are bf16 instead, w in two terms, within 2^-17: f16 would lose the tokens of small values (pa_internal.h).
// K, for bf16 queries and a bf16 output (raw_k): the codes as stored (kind::f8f6f4), a query row being two e4m3 terms of its elements times a power of two that puts the largest in [128,
// 256): elements down to 2^-9 of it are exact, smaller ones off by 2^-17 of it at most.  Otherwise K is widened too, and
// bf16 query rows are multiplied by a power of two that puts their largest element in [2^14, 2^15) and rounded to f16,
// exact for every element above 2^-28 of it.  (Raw K tiles come by bulk copies and cost no warp anything; widening takes
// a warp some 200 instructions per tile.)
//
// One CTA per SM, two teams.  A team is 128 softmax threads (thread m owns packed
// row m: token m / heads, head m % heads), a score buffer and an O accumulator in
// tensor memory (2 x 128 + 2 x head_dim columns): while one team's softmax works,
// the tensor cores have the other team's P.V and Q.K^T.
//  * kSplitKeys false: the teams have two Q tiles of 128 packed rows and walk the
//    same key tiles (128 keys), each of which is widened once for both.
//  * kSplitKeys true (few rows: two Q tiles per CTA would leave SMs idle): both
//    teams have the same Q tile, team 0 the even key tiles and team 1 the odd
//    ones; their results are joined by their maxima through shared memory.
//
// A team's score buffer is two halves of 64 keys, each with its own softmax step: while a team's threads work on one half,
// the tensor cores compute the other half's scores and the P.V of the one before.  P (f16 pairs; hi + lo) goes over its own
// half.  (With one buffer of 128 keys a team waited for P.V and the next Q.K^T in turn: 821 us against 721 for 4 chunks of
// 2048 at 2048, 64/8 heads; 688 now, 959 with V scales 2^12 apart, 923 with an fp32 output.)
//
// Bound by the softmax warps, two per scheduler, one step's chain after another: scores, maximum, weights, hand-over.  At 688
// us the tensor pipe is busy 51 % of the time, the issue slots 51 %, the special functions 26 %.  (Scales published for four key
// tiles at once, so that a team waits for them every eighth step: 682 against 694.)  What was tried on that chain
// at 695 and cost more than it gave: scores and P in buffers of their own, so that Q.K^T waits for no P.V (one more wait per step:
// 752), the next step's scores loaded under this one's exponentials (814), the two teams' exponentials in turn by a barrier
// (726), one arrival per warp instead of per thread (706), a rolled loop for the queries' terms (710).
//
// Loaders: four warps, 32 keys of a tile each, a key tile ahead in registers (8-byte loads, a row of codes per 8 lanes),
// widened into the MMAs' 128-byte-swizzled panels.  Codes staged by bulk copies instead would cost shared memory's
// bandwidth twice more, and that is what the MMAs are short of: an SS MMA of 128 x 128 x 16 reads 8 KB in 64 clocks.
// Raw K tiles: one bulk-tensor box per cache block, by a warp of its own.
//
// Every mbarrier wait is bounded (PA_ERR_TIMEOUT, then the CTA abandons its work).
#pragma once

#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_prefill_tc.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace psc {

constexpr int kM = 128, kN = 128;              // packed rows per Q tile, keys per tile
constexpr int kTeams = 2, kSoftmax = kTeams * 128;
constexpr int kLoadWarp0 = kSoftmax / 32, kLoaders = 128, kMmaWarp = kLoadWarp0 + 4, kKWarp = kMmaWarp + kTeams;
constexpr int kThreads = (kKWarp + 1) * 32;
constexpr int kHalf = 64;                      // keys per softmax step
constexpr int kGroup = 4;                      // key tiles whose scales are published together: a warp's 32 runs
constexpr int kPanel = kN * 128;               // 64 elements of 128 rows
constexpr int32_t kNoKeys = -1, kLost = -2;    // in a block id's place: behind the sequence's end, or an id out of range
constexpr float kRescaleLog2 = 8.f;            // O is rescaled when the maximum exceeds its reference by 2^8
constexpr float kTopLog2 = 7.f;                // w at the reference, 2^15 at most: as high as f16 allows, for the small ones' sake

// K as stored for bf16 queries and outputs.
template <typename QT, bool kLo>
constexpr bool raw_k() {
  return std::is_same<QT, __nv_bfloat16>::value && !kLo;
}

template <int D, bool kSplitKeys, bool kRaw>
struct Layout {
  static constexpr int kTile = kN * D * 2;                     // a Q or V tile (Q: f16, or two terms of codes)
  static constexpr int kKTile = kRaw ? kN * D : kTile;
  static constexpr int kStages = 2, kKStages = kRaw ? 3 : 2;   // V, K tiles in flight
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + (kSplitKeys ? 1 : 2) * kTile;
  static constexpr int kOffV = kOffK + kKStages * kKTile;
  static constexpr int kOffBar = kOffV + kStages * kTile;
  static constexpr int kNumBars = 2 * kStages + 2 * kKStages + 3 * 2 * kTeams + 2 + 2 + kTeams;   // (even: 16-byte alignment behind them)
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffRow = kOffMisc + 16;                // float2 [kTeams][128]
  static constexpr int kOffRuns = (kOffRow + kTeams * 128 * 8 + 15) / 16 * 16;  // float4 [2 groups][kGroup tiles][8 runs]
  static constexpr int kOffRange = kOffRuns + 2 * kGroup * 8 * 16;       // float2 [loader warps]
  static constexpr int kBytes = kOffRange + kLoaders / 32 * 8 + 1024;    // + alignment slack
  static_assert(kBytes <= 227 * 1024 && kOffRow % 8 == 0 && kOffRuns % 16 == 0, "shared memory");
  static constexpr int kStage = kOffBar - kSoftmax / 32 * 4096;   // kSplitKeys: 4 KB per softmax warp for the output's way
  static_assert(kOffV % 1024 == 0 && (!kSplitKeys || kStage >= 128 * D * 4), "room for the teams' halves of O before it");
};

__device__ __forceinline__ uint2 ld_nc8(const void *p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
// 8 e4m3 codes -> 8 f16 values, exactly.
__device__ __forceinline__ uint4 widen8(uint2 w) {
  auto two = [](uint32_t x) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3);
    return *reinterpret_cast<const uint32_t *>(&h);
  };
  return make_uint4(two(w.x), two(w.x >> 16), two(w.y), two(w.y >> 16));
}
// The same -> bf16 values, exactly (the upper halves of the fp32 patterns).
__device__ __forceinline__ uint4 widen8_bf16(uint2 w) {
  auto two = [](uint32_t x) {
    const float2 f = unpack2_e4m3(x);
    return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
  };
  return make_uint4(two(w.x), two(w.x >> 16), two(w.y), two(w.y >> 16));
}
// Two f16 values, an infinity made NaN: x + 0 x.
__device__ __forceinline__ uint32_t nan_for_inf(uint32_t x) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %1;" : "=r"(y) : "r"(x), "r"(0u));
  return y;
}

template <typename QT, int D, bool kSplitKeys, bool kLo>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_scaled_kernel(const PrefillTcParams p, int num_chunks, const __grid_constant__ CUtensorMap tmap_k) {
  using namespace tc;
  constexpr bool kRaw = raw_k<QT, kLo>();
  using L = Layout<D, kSplitKeys, kRaw>;
  constexpr int kStages = L::kStages, kKStages = L::kKStages, kTile = L::kTile, kKTile = L::kKTile;
  constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;
  const float kNegInf = -__int_as_float(0x7f800000);

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *v_full = bars;                       // [kStages] a tile is widened (128 loader arrivals)
  uint64_t *v_free = v_full + kStages;           // [kStages] the MMAs that read it are complete (every team's that walks the tile)
  uint64_t *k_full = v_free + kStages;           // [kKStages] the same of K (raw: one expect-tx arrival)
  uint64_t *k_free = k_full + kKStages;
  uint64_t *s_full = k_free + kKStages;          // [team][half] scores of its step h (half h & 1, phase h >> 1)
  uint64_t *p_full = s_full + 2 * kTeams;        // [team][half] P written over them (128 arrivals)
  uint64_t *o_done = p_full + 2 * kTeams;        // [team][half] P.V complete
  uint64_t *sc_full = o_done + 2 * kTeams;       // [2] the scales of tiles kGroup G .. + kGroup - 1 (G & 1)
  uint64_t *q_ready = sc_full + 2;
  uint64_t *fin = q_ready + 1;                   // [team] every MMA of the team complete
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 8);
  volatile int *wide_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 12);   // V and w in bf16; set when sc_full[0] is
  float2 *row_info = reinterpret_cast<float2 *>(smem + L::kOffRow);
  // of each run of 16 keys of tile j, at [j % (2 kGroup)]: K's scale, log2 of V's, 1 / V's
  float4 *runs = reinterpret_cast<float4 *>(smem + L::kOffRuns);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // work item: KV head share fastest, then chunk, then row block from the last (longest) one down
  const int gy = p.num_kv_heads * p.shares, by = blockIdx.x % gy, rest = blockIdx.x / gy;
  const int c = rest % num_chunks, rb = p.row_blocks - 1 - rest / num_chunks;
  const int g = by / p.shares, gr = p.share_heads, h_first = (by - g * p.shares) * gr;
  const int gqa = p.num_q_heads / p.num_kv_heads;
  const int BR = kM / gr;                        // token rows per Q tile
  const int cu0 = __ldg(p.cu_q_lens + c), nrows = __ldg(p.cu_q_lens + c + 1) - cu0, qs = __ldg(p.q_start + c);
  if (tid == 0 && by == 0 && rb == 0) {
    const int64_t len = (int64_t)qs + nrows;
    if (nrows < 0 || nrows > p.max_q_len || qs < 0 || __ldg(p.seq_lens + c) != len ||
        len > (int64_t)p.max_blocks_per_seq * p.block_size)
      record_error(p.err, PA_ERR_DEVICE_CHECK);
  }
  const int r0 = rb * BR * (kSplitKeys ? 1 : kTeams);
  if (r0 >= nrows) return;   // whole CTA, before any barrier or tensor memory
  const int64_t cap = (int64_t)p.max_blocks_per_seq * p.block_size, len64 = (int64_t)qs + nrows;
  const int seq_eff = len64 <= 0 ? 0 : (int)(len64 < cap ? len64 : cap);
  const int bs_log2 = p.block_size == 32 ? 5 : 4;
  const int32_t *table = p.block_tables + (int64_t)c * p.max_blocks_per_seq;
  // keys that a team's Q tile sees, the CTA's key tiles, and a team's steps of 64 keys: step h of team t is half h & 1 of key
  // tile tile_of(t, h)
  auto keys_of = [&](int t) {
    const int first = r0 + (kSplitKeys ? 0 : t * BR);
    return first >= nrows ? 0 : min(seq_eff, max(0, qs + min(first + BR, nrows)));
  };
  const int keys0 = keys_of(0), keys1 = keys_of(1), nkt = (max(keys0, keys1) + kN - 1) / kN;
  auto steps = [&](int t) {
    if (!kSplitKeys) return ((t ? keys1 : keys0) + kHalf - 1) / kHalf;
    const int tiles = (nkt + 1 - t) / 2, last = keys0 - (nkt - 1) * kN;   // last: keys of the last tile
    return 2 * tiles - (tiles > 0 && ((nkt - 1) & 1) == t && last <= kHalf ? 1 : 0);
  };
  auto tile_of = [&](int t, int h) { return kSplitKeys ? (h & ~1) + t : h >> 1; };

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&v_full[s], kLoaders);
      mbar_init(&v_free[s], kSplitKeys ? 1 : kTeams);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&k_full[s], kRaw ? 1 : kLoaders);
      mbar_init(&k_free[s], kSplitKeys ? 1 : kTeams);
    }
    for (int t = 0; t < 2 * kTeams; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(q_ready, kSplitKeys ? 128 : kSoftmax);
    for (int i = 0; i < 2; ++i) mbar_init(&sc_full[i], 1);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto sbuf = [&](int t) { return tmem + (uint32_t)(t * kN); };
  auto obuf = [&](int t) { return tmem + (uint32_t)(kTeams * kN + t * D); };
  auto wait_all = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_or_abort(bar, parity, p.err, abort_flag));
  };

  if (warp < kLoadWarp0) {
    // ===================================================== softmax
    const int team = warp >> 2, quad = warp & 3, m = tid & 127;
    const int tile0 = r0 + (kSplitKeys ? 0 : team * BR);         // the Q tile's first token row
    const int rl = m / gr, hq = m - rl * gr;
    const bool row_ok = tile0 + rl < nrows && rl < BR && h_first + hq < gqa;
    const int64_t row_elem = row_ok ? ((int64_t)(cu0 + tile0 + rl) * p.num_q_heads + g * gqa + h_first + hq) * D : -1;
    // the row sees keys < lim (idle rows, with q = 0, all of them: they are not stored)
    const int lim = row_ok ? min(seq_eff, max(0, qs + tile0 + rl + 1)) : 1 << 30;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    // scores are scaled by |s_mult| in the exponent; a negative scale flips q's sign instead.  A masked score of
    // -inf has to stay -inf whatever the scale (a scale of 0 gives scores of about 0).
    float cmul = fmaxf(fabsf(p.s_mult), 1e-30f);
    const uint32_t qflip = p.s_mult < 0.f ? 0x80008000u : 0u;
    auto both_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory"); };
    {
      // Stage Q: a warp brings its own 32 rows, kC lanes of 16 bytes per row (kSplitKeys: team 0 for both)
      constexpr int kC = D / 8, kRI = 32 / kC;
      if (!kSplitKeys || team == 0) {
        uint4 v[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const int64_t e = __shfl_sync(0xffffffffu, row_elem, i * kRI + lane / kC);
          // (idle rows read row 0, and are zeroed: a branch around each load would wait for it)
          v[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const QT *>(p.q) + max(e, (int64_t)0)) + lane % kC);
        }
#pragma unroll
        for (int i = 0; i < kC; ++i)
          if (__shfl_sync(0xffffffffu, (int)row_ok, i * kRI + lane / kC) == 0) v[i] = make_uint4(0, 0, 0, 0);
        uint8_t *qt = smem + L::kOffQ + (kSplitKeys ? 0 : team * kTile);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const int mr = quad * 32 + i * kRI + lane / kC, ch = lane % kC;
          uint32_t ws[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          float back = 1.f;
          if constexpr (kBf16) {
            // the row times 2^e: its largest element in [128, 256), or [2^14, 2^15)
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = fmaxf(amax, fmaxf(__uint_as_float((ws[k] << 16) & 0x7fffffffu), __uint_as_float(ws[k] & 0x7fff0000u)));
#pragma unroll
            for (int off = kC / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const int eb = max(1, (int)((__float_as_uint(amax) >> 23) & 0xff));
            const int e = amax > 0.f ? max(-126, min(126, (kRaw ? 134 : 141) - eb)) : 0;
            // (an infinity makes the whole row NaN, as every score of the row is infinite or NaN: e4m3 has no infinity, and a row
            // of scores that are all -inf would pass for one that sees no key)
            const float sc = __uint_as_float(amax == -kNegInf ? 0x7fc00000u : (uint32_t)(e + 127) << 23);
            back = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e
            if constexpr (kRaw) {
              const float sign = p.s_mult < 0.f ? -sc : sc;
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = unpack2(ws[k], __nv_bfloat16{});
                const float2 x = make_float2(f.x * sign, f.y * sign);
                hi[k] = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
                const float2 h = unpack2_e4m3(hi[k]);
                lo[k] = __nv_cvt_float2_to_fp8x2(make_float2(x.x - h.x, x.y - h.y), __NV_SATFINITE, __NV_E4M3);
              }
              // 8 bytes of a D-byte row, in the 128- or 64-byte swizzle
              const int at = mr * D + (((ch >> 1) ^ (D == 128 ? mr & 7 : (mr >> 1) & 3)) << 4) + (ch & 1) * 8;
              *reinterpret_cast<uint2 *>(qt + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
              *reinterpret_cast<uint2 *>(qt + kM * D + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = unpack2(ws[k], __nv_bfloat16{});
                const __half2 h = __floats2half2_rn(f.x * sc, f.y * sc);
                ws[k] = *reinterpret_cast<const uint32_t *>(&h);
              }
            }
          }
          if (ch == 0) {
            row_info[(kSplitKeys ? 0 : team * 128) + mr].x = back;
            if (kSplitKeys) row_info[128 + mr].x = back;
          }
          if constexpr (!kBf16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) ws[k] = nan_for_inf(ws[k]);
          }
          if constexpr (!kRaw)
            *reinterpret_cast<uint4 *>(qt + (ch >> 3) * kPanel + mr * 128 + (((ch & 7) ^ (mr & 7)) << 4)) =
                make_uint4(ws[0] ^ qflip, ws[1] ^ qflip, ws[2] ^ qflip, ws[3] ^ qflip);
        }
        fence_async_smem();
        mbar_arrive(q_ready);
      }
      if (kSplitKeys) both_sync();
      else __syncwarp();   // a warp's rows are staged by itself
      cmul = fmaxf(cmul * row_info[team * 128 + m].x, 1e-30f);
    }

    const int n = steps(team);
    float m_ref = kNegInf, msub = 0.f;           // reference maximum, log2 units, and what exponents are less of
    float2 lacc = make_float2(0.f, 0.f);         // row sum in two parts
    const float2 ones = make_float2(1.f, 1.f);
    bool ok = true;
    const uint32_t sb = sbuf(team) + lane_base, ob = obuf(team) + lane_base;
    auto softmax = [&](auto in_bf16) {
      constexpr bool kWide = decltype(in_bf16)::value;
      for (int h = 0; h < n; ++h) {
        const int b = h & 1, tb = team * 2 + b;
        const int j = tile_of(team, h);
        if ((h & (kGroup * (kSplitKeys ? 1 : 2) - 1)) == 0) ok = wait_all(&sc_full[(j / kGroup) & 1], (j / (2 * kGroup)) & 1);
        const float4 *run = runs + 8 * (j % (2 * kGroup)) + 4 * b;   // the half's four runs
        ok = ok && wait_all(&s_full[tb], (h >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sh = sb + kHalf * b;
        float v[2][32];
        tmem_ld32_start(sh, v[0]);
        tmem_ld32_start(sh + 32, v[1]);
        // run r's score factor, log2 units (not 0: a masked score stays -inf), and log2 of V's scale
        float factor[4], add[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 x = run[r];
          factor[r] = fmaxf(cmul * x.x, 1e-37f);
          add[r] = x.y;
        }
        tmem_ld32_finish(v[0]);
        tmem_ld32_finish(v[1]);
        const int nvis = lim - j * kN - kHalf * b;
        if (!__all_sync(0xffffffffu, nvis >= kHalf)) {
#pragma unroll
          for (int e = 0; e < kHalf; ++e)
            if (e >= nvis) v[e >> 5][e & 31] = kNegInf;
        }
        // maximum of a + log2 sv
        float mt = kNegInf;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float *x = &v[r >> 1][16 * (r & 1)];
          float c0 = fmax3(x[0], x[1], x[2]), c1 = fmax3(x[3], x[4], x[5]);
          c0 = fmax3(c0, x[6], x[7]), c1 = fmax3(c1, x[8], x[9]);
          c0 = fmax3(c0, x[10], x[11]), c1 = fmax3(c1, x[12], x[13]);
          mt = fmaxf(mt, fmaf(fmax3(fmaxf(c0, c1), x[14], x[15]), factor[r], add[r]));
        }
        const bool rescale = mt > m_ref + kRescaleLog2;
        if (__any_sync(0xffffffffu, rescale)) {
          const float alpha = rescale ? fast_exp2(m_ref - mt) : 1.f;
          if (h > 0) {   // O holds the P.V of steps 0 .. h - 1: the last of them has to be complete
            ok = wait_all(&o_done[tb ^ 1], ((h - 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              float o[16];
              uint32_t ow[16];
              tmem_ld16(ob + c0, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e] * alpha);
              tmem_st16(ob + c0, ow);
            }
          }
          if (rescale) {
            lacc = make_float2(lacc.x * alpha, lacc.y * alpha);
            m_ref = mt;
            msub = mt - kTopLog2;
          }
        }
        // w = 2^(a + log2 sv - msub), rounded to f16 (or in two terms), and the sum of w / sv
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float *x = &v[r >> 1][16 * (r & 1)];
          const float nr = add[r] - msub, iv = run[r].z;
          const float2 cc = make_float2(factor[r], factor[r]), nm = make_float2(nr, nr);
          float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
          uint32_t w[8], wl[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 a = ffma2(make_float2(x[2 * k], x[2 * k + 1]), cc, nm);
            const float2 pk = make_float2(fast_exp2(a.x), fast_exp2(a.y));
            if constexpr (kWide) {
              w[k] = pack2(pk.x, pk.y, __nv_bfloat16{});
              wl[k] = pack2(pk.x - __uint_as_float(w[k] << 16), pk.y - __uint_as_float(w[k] & 0xffff0000u), __nv_bfloat16{});
            } else if constexpr (kLo) {
              w[k] = f16x2_split(pk.x, pk.y, wl[k]);
            } else {
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(pk.y), "f"(pk.x));
            }
            sum[k & 1] = ffma2(pk, ones, sum[k & 1]);
          }
          lacc = ffma2(make_float2(sum[0].x + sum[1].x, sum[0].y + sum[1].y), make_float2(iv, iv), lacc);
          if constexpr (kLo || kWide) {   // hi, lo of 16 keys over their own 16 columns
            tmem_st8(sh + 16 * r, w);
            tmem_st8(sh + 16 * r + 8, wl);
          } else {
            tmem_st8(sh + 8 * r, w);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[tb]);
      }
    };
    if (n > 0) {
      ok = wait_all(&sc_full[0], 0);
      // (the vote: a branch that the whole warp is known to take)
      if (ok) __any_sync(0xffffffffu, *wide_flag) ? softmax(std::true_type{}) : softmax(std::false_type{});
    }
    float l = lacc.x + lacc.y;
    if (ok && n > 0) ok = wait_all(&o_done[team * 2 + ((n - 1) & 1)], ((n - 1) >> 1) & 1);
    tc_fence_after();
    // Columns [c0, c1) of the row, kCols at a time through `value`, normalised by inv and stored by 8 (or 4) lanes per
    // row: the threads write 128 bytes of their rows into the warp's 4 KB (16-byte chunk c of row r at chunk c ^ (r & 7))
    auto emit = [&](auto f32, uint8_t *stage, int c0, int c1, float inv, auto &&value) {
      constexpr bool kF32 = decltype(f32)::value;
      constexpr int kCols = 32, kCh = kCols * (kF32 ? 4 : 2) / 16, kRI = 32 / kCh;
      int64_t e[kCh];
#pragma unroll
      for (int i = 0; i < kCh; ++i) e[i] = __shfl_sync(0xffffffffu, row_elem, i * kRI + lane / kCh);
#pragma unroll 1
      for (int at = c0; at < c1; at += kCols) {
        float o[32];
        value(at, o);
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          uint4 x;
          if constexpr (kF32) {
            x = make_uint4(__float_as_uint(o[4 * i] * inv), __float_as_uint(o[4 * i + 1] * inv),
                           __float_as_uint(o[4 * i + 2] * inv), __float_as_uint(o[4 * i + 3] * inv));
          } else {
            const float *v = o + 8 * i;
            x = make_uint4(pack2(v[0] * inv, v[1] * inv, QT{}), pack2(v[2] * inv, v[3] * inv, QT{}),
                           pack2(v[4] * inv, v[5] * inv, QT{}), pack2(v[6] * inv, v[7] * inv, QT{}));
          }
          *reinterpret_cast<uint4 *>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = x;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          const int r = i * kRI + lane / kCh, ch = lane % kCh;
          const uint4 x = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((ch ^ (r & 7)) << 4));
          if (e[i] >= 0)
            *reinterpret_cast<uint4 *>(static_cast<char *>(p.out) + (e[i] + at) * (kF32 ? 4 : 2) + ch * 16) = x;
        }
        __syncwarp();
      }
    };
    auto load_o = [&](int at, float (&o)[32]) {
      if (n > 0) {
        tmem_ld32_start(ob + at, o);
        tmem_ld32_finish(o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
      }
    };
    if constexpr (!kSplitKeys) {
      if (ok) {
        // every MMA of this Q tile is complete: its place takes the output on its way
        uint8_t *stage = smem + L::kOffQ + team * kTile + quad * 4096;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        if (p.out_f32) emit(std::true_type{}, stage, 0, D, inv, load_o);
        else emit(std::false_type{}, stage, 0, D, inv, load_o);
      }
    } else {
      // Join the teams: each takes half of the columns and hands the other half to the other one, through the place of the
      // Q, K and V tiles (every MMA is complete for both)
      ok = __all_sync(0xffffffffu, ok);
      row_info[team * 128 + m] = make_float2(m_ref, l);
      both_sync();
      const float2 other = row_info[(team ^ 1) * 128 + m];
      const bool live = !*abort_flag;
      const float top = fmaxf(m_ref, other.x), ref = top == kNegInf ? 0.f : top;
      const float mine = fast_exp2(m_ref - ref), theirs = fast_exp2(other.x - ref);
      l = l * mine + other.y * theirs;
      float4 *box = reinterpret_cast<float4 *>(smem);   // [team][column / 4 of the half][row]
      constexpr int kCols = D / 2;
      if (live && ok) {
#pragma unroll 1
        for (int at = 0; at < kCols; at += 32) {
          float o[32];
          load_o((team ^ 1) * kCols + at, o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            box[(team * (kCols / 4) + at / 4 + k) * 128 + m] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      both_sync();
      if (live && ok) {
        auto joined = [&](int at, float (&o)[32]) {
          load_o(at, o);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 x = box[((team ^ 1) * (kCols / 4) + (at - team * kCols) / 4 + k) * 128 + m];
            o[4 * k] = o[4 * k] * mine + x.x * theirs;
            o[4 * k + 1] = o[4 * k + 1] * mine + x.y * theirs;
            o[4 * k + 2] = o[4 * k + 2] * mine + x.z * theirs;
            o[4 * k + 3] = o[4 * k + 3] * mine + x.w * theirs;
          }
        };
        uint8_t *stage = smem + L::kStage + warp * 4096;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        if (p.out_f32) emit(std::true_type{}, stage, team * kCols, (team + 1) * kCols, inv, joined);
        else emit(std::false_type{}, stage, team * kCols, (team + 1) * kCols, inv, joined);
      }
    }
  } else if (warp < kMmaWarp) {
    // ===================================================== loaders
    const int lw = warp - kLoadWarp0;
    constexpr int kPanels = D / 64;
    const char *kpool = static_cast<const char *>(p.k_cache), *vpool = static_cast<const char *>(p.v_cache);
    const int q = lane & 7, rr0 = lane >> 3;     // 8 bytes q of each 64-byte half of rows rr0, rr0 + 4, ...
    int32_t win = -1;                            // lane l: block id of run (l & 1) of tile win_base + (l >> 1)
    int win_base = -16;
    auto block_of = [&](int j, int r) -> int32_t {
      if (j - win_base >= 16) {
        win_base = j;
        const int jt = j + (lane >> 1), key = jt * kN + 32 * lw + 16 * (lane & 1);
        win = -1;
        if (jt < nkt && key < seq_eff) {
          const int32_t bi = __ldg(table + (key >> bs_log2));
          if (bi < 0 || bi >= p.num_blocks) record_error(p.err, PA_ERR_DEVICE_CHECK);
          else win = bi;
        }
      }
      return __shfl_sync(0xffffffffu, win, 2 * (j - win_base) + r);
    };
    // Where this lane's words of the warp's two runs of tile j begin, and how many rows of each hold tokens.  A run without
    // any (past the sequence's end, or in a bad block) is read from the pool's first rows; what is read of rows past the
    // end is replaced by zeros.
    struct Rows {
      int64_t at[2];
      int n[2];
    };
    auto rows_of = [&](int j) {
      Rows x;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key0 = j * kN + 32 * lw + 16 * r;
        const int32_t b = block_of(j, r);
        x.n[r] = b < 0 ? 0 : min(16, seq_eff - key0);
        x.at[r] = (((int64_t)max(b, 0) * p.num_kv_heads + (b < 0 ? 0 : g)) * p.block_size + (b < 0 ? 0 : key0 & (p.block_size - 1)) + rr0) * D + q * 8;
      }
      return x;
    };
    using Words = uint2[kPanels][8];
    auto load = [&](const Rows &x, const char *pool, Words &w) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int pn = 0; pn < kPanels; ++pn) w[pn][i] = ld_nc8(pool + x.at[i >> 2] + ((4 * i) & 15) * D + pn * 64);
    };
    const uint32_t to0 = (32 * lw + rr0) * 128 + ((q ^ rr0) << 4), to1 = to0 ^ 64;   // row 4 i + rr0: its chunk q ^ (row & 7)
    auto widen = [&](Words &w, const Rows &x, uint8_t *tile, auto wider) {
      if (x.n[0] + x.n[1] < 32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (((4 * i) & 15) + rr0 >= x.n[i >> 2])
#pragma unroll
            for (int pn = 0; pn < kPanels; ++pn) w[pn][i] = make_uint2(0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int pn = 0; pn < kPanels; ++pn)
          *reinterpret_cast<uint4 *>(tile + (i & 1 ? to1 : to0) + i * 512 + pn * kPanel) = wider(w[pn][i]);
      fence_async_smem();
    };
    // Scales, by loader warp 0, a run to each lane (1 for a run without tokens; -inf as log2 of V's, which leaves its keys out of
    // the softmax, for one whose block is lost, its K and V being zeros, or has a scale out of range): those of tiles kGroup G
    // .. + kGroup - 1 are published when the P.V of tile kGroup (G - 2) + kGroup - 1, the last that used their place, is
    // complete; the next group's are in flight then, and the block ids of the one after it
    auto run_block = [&](int group) -> int32_t {
      const int j = kGroup * group + (lane >> 3), key = j * kN + 16 * (lane & 7);
      if (j >= nkt || key >= seq_eff) return kNoKeys;
      const int32_t bi = __ldg(table + (key >> bs_log2));
      return bi >= 0 && bi < p.num_blocks ? bi : kLost;
    };
    static_assert(kGroup * 8 == 32, "a warp's runs");
    float sk = 1.f, sv = 1.f;
    auto read_scales = [&](int32_t b) {
      sk = 1.f;
      sv = b == kLost ? 0.f : 1.f;           // (out of range)
      if (b >= 0) {
        const int64_t at = (int64_t)b * p.num_kv_heads + g;
        sk = __ldg(p.k_scales + at);
        sv = __ldg(p.v_scales + at);
      }
    };
    auto put_scales = [&](int group) {
      const bool good = block_scale_ok(sk) && block_scale_ok(sv);
      if (!good) record_error(p.err, PA_ERR_DEVICE_CHECK);
      runs[32 * (group & 1) + lane] = good ? make_float4(sk, __log2f(sv), __fdividef(1.f, sv), 0.f) : make_float4(1.f, kNegInf, 1.f, 0.f);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc_full[group & 1]);
    };
    Words kw, vw;
    Rows now = rows_of(0), next = now;
    if (nkt > 0) {
      if constexpr (!kRaw) load(now, kpool, kw);
      load(now, vpool, vw);
    }
    int32_t scale_blk = kNoKeys, second = kNoKeys;
    if (lw == 0) {
      scale_blk = run_block(0);
      second = run_block(1);
      read_scales(scale_blk);
      scale_blk = run_block(2);
    }
    // The least and the largest of V's scales of all the CTA's keys (bad ones are reported where they are published).  Its loads
    // run beside those of the first scales: 4 chunks of 2048 take 685 us with the scan and without it, 699 with the scan first.
    bool wide;
    {
      float low = -kNegInf, top = 0.f;
      const int blocks = (max(keys0, keys1) + p.block_size - 1) >> bs_log2;
#pragma unroll 4
      for (int i = lw * 32 + lane; i < blocks; i += kLoaders) {
        const int32_t bi = __ldg(table + i);
        const bool in = bi >= 0 && bi < p.num_blocks;
        const float s = __ldg(p.v_scales + (in ? (int64_t)bi * p.num_kv_heads + g : 0));
        if (in && block_scale_ok(s)) low = fminf(low, s), top = fmaxf(top, s);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      }
      float2 *range = reinterpret_cast<float2 *>(smem + L::kOffRange);
      if (lane == 0) range[lw] = make_float2(low, top);
      asm volatile("bar.sync 2, %0;" ::"n"(kLoaders) : "memory");
      const float2 x = range[lane % (kLoaders / 32)];
      low = x.x, top = x.y;
#pragma unroll
      for (int off = kLoaders / 64; off > 0; off >>= 1) {
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      }
      wide = __any_sync(0xffffffffu, low * kNarrowScales < top);
      if (lw == 0 && lane == 0) *wide_flag = wide;
    }
    if (lw == 0) {
      put_scales(0);
      read_scales(second);
      put_scales(1);
      read_scales(scale_blk);
      scale_blk = run_block(3);
    }
    auto walk = [&](auto wider) {
      for (int j = 0; j < nkt; ++j) {
        const int s = j % kStages;
        if (j + 1 < nkt) next = rows_of(j + 1);
        if constexpr (!kRaw) {
          const int ks = j % kKStages;
          if (j >= kKStages && !wait_all(&k_free[ks], ((j / kKStages) - 1) & 1)) break;
          widen(kw, now, smem + L::kOffK + ks * kKTile, [](uint2 c) { return widen8(c); });
          mbar_arrive(&k_full[ks]);
          if (j + 1 < nkt) load(next, kpool, kw);
        }
        if (j >= kStages && !wait_all(&v_free[s], ((j / kStages) - 1) & 1)) break;
        widen(vw, now, smem + L::kOffV + s * kTile, wider);
        mbar_arrive(&v_full[s]);
        if (j + 1 < nkt) load(next, vpool, vw);
        now = next;
        if (lw == 0 && j % kGroup == kStages - 1 && j > kGroup) {
          const int group = j / kGroup + 1;
          put_scales(group);
          read_scales(scale_blk);
          scale_blk = run_block(group + 2);
        }
      }
    };
    if (wide) walk([](uint2 c) { return widen8_bf16(c); });
    else walk([](uint2 c) { return widen8(c); });
  } else if (kRaw && warp == kKWarp) {
    // ===================================================== K tiles as stored
    // one box per cache block that holds a key; what the rows behind the end hold is masked in the scores
    const int bs = p.block_size, per_tile = kN / bs;
    // lane i: the id of block i of tile j; for one out of range (the loaders report it) that of the block behind the pool, whose
    // box the copy fills with zeros
    auto block = [&](int j) -> int32_t {
      const int key = j * kN + lane * bs;
      if (lane >= per_tile || j >= nkt || key >= seq_eff) return kNoKeys;
      const int32_t bi = __ldg(table + (key >> bs_log2));
      return bi >= 0 && bi < p.num_blocks ? bi : (int32_t)p.num_blocks;
    };
    int32_t next = block(0);
    int issued = 0;
    for (int j = 0; j < nkt; ++j) {
      const int s = j % kKStages;
      const int32_t bi = next;
      next = block(j + 1);
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, bi >= 0));
      if (j >= kKStages && !wait_all(&k_free[s], ((j / kKStages) - 1) & 1)) break;
      if (lane == 0) mbar_arrive_expect_tx(&k_full[s], boxes * bs * D);
      __syncwarp();
      if (bi >= 0)
        tma_load_2d(smem + L::kOffK + s * kKTile + lane * bs * D, &tmap_k, &k_full[s], 0,
                    (int32_t)(((int64_t)bi * p.num_kv_heads + g) * bs));
      ++issued;
    }
    // no box in flight at exit
    for (int j = max(0, issued - kKStages); j < issued; ++j) mbar_wait(&k_full[j % kKStages], (j / kKStages) & 1, p.err);
  } else if (warp >= kMmaWarp && warp < kMmaWarp + kTeams) {
    // ===================================================== MMA issue, a warp per team
    // (one warp for both had its own instructions as the bound: 16 waits per key tile at some 100 clocks.  The whole warp
    // runs the schedule, the elected lane's predicate issues: operands stay in uniform registers)
    const bool leader = elect_one();
    const int team = warp - kMmaWarp, n = steps(team);
    const uint32_t idesc_s = umma_idesc(0, kHalf, false);
    constexpr bool kSw64 = kRaw && D == 64;     // rows of 64 bytes
    const uint32_t q_at = smem_u32(smem + L::kOffQ) + (kSplitKeys ? 0 : team * kTile), k_at = smem_u32(smem + L::kOffK);
    const uint64_t qdesc = kSw64 ? umma_desc_sw64(q_at, 16, 512) : umma_desc(q_at, 16);
    const uint64_t kdesc0 = kSw64 ? umma_desc_sw64(k_at, 16, 512) : umma_desc(k_at, 16);
    const uint64_t vdesc0 = umma_desc(smem_u32(smem + L::kOffV), kPanel);
    const uint32_t s_at = sbuf(team), o_at = obuf(team);
    uint64_t *s_bar = s_full + 2 * team, *p_bar = p_full + 2 * team, *o_bar = o_done + 2 * team;
    bool ok = nkt == 0 || wait_all(q_ready, 0);
    // S of step h, its buffer's last P.V (step h - 2) complete
    auto issue_s = [&](int h) {
      const int j = tile_of(team, h), b = h & 1, slot = j % kKStages;
      if (b == 0) ok = wait_all(&k_full[slot], (j / kKStages) & 1);
      if (h >= 2) ok = ok && wait_all(&o_bar[b], ((h >> 1) - 1) & 1);
      if (!ok) return;
      tc_fence_after();
      const uint32_t d = s_at + kHalf * b;
      const uint64_t kd = kdesc0 + ((slot * kKTile + b * (kRaw ? kHalf * D : kHalf * 128)) >> 4);
      if constexpr (kRaw) {
#pragma unroll
        for (int k = 0; k < 2 * (D / 32); ++k)
          umma_f8_if(leader, d, qdesc + (k / (D / 32)) * ((kM * D) >> 4) + (k % (D / 32)) * 2, kd + (k % (D / 32)) * 2, idesc_s, k > 0 ? 1u : 0u);
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_if(leader, d, qdesc + (k >> 2) * (kPanel >> 4) + (k & 3) * 2, kd + (k >> 2) * (kPanel >> 4) + (k & 3) * 2, idesc_s, k > 0 ? 1u : 0u);
      }
      umma_commit_if(leader, &s_bar[b]);
      if (b || h + 1 == n) umma_commit_if(leader, &k_free[slot]);
    };
    if (n > 0) issue_s(0);
    if (n > 1 && ok) issue_s(1);
    auto walk = [&](auto in_bf16) {
      constexpr bool kWide = decltype(in_bf16)::value;
      const uint32_t idesc_o = umma_idesc(kWide ? 1 : 0, D, true);
      for (int h = 0; h < n && ok; ++h) {
        const int j = tile_of(team, h), b = h & 1, slot = j % kStages;
        if (b == 0) ok = wait_all(&v_full[slot], (j / kStages) & 1);
        ok = ok && wait_all(&p_bar[b], (h >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vdesc0 + ((slot * kTile + b * kHalf * 128) >> 4);
        const uint32_t pa = s_at + kHalf * b;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          constexpr int kStep = (16 * 128) >> 4;
          const uint32_t acc = h + kk > 0 ? 1u : 0u;
          if constexpr (kLo || kWide) {
            umma_ts_if(leader, o_at, pa + 16 * kk, vd + kk * kStep, idesc_o, acc);
            umma_ts_if(leader, o_at, pa + 16 * kk + 8, vd + kk * kStep, idesc_o, 1u);
          } else {
            umma_ts_if(leader, o_at, pa + 8 * kk, vd + kk * kStep, idesc_o, acc);
          }
        }
        umma_commit_if(leader, &o_bar[b]);
        if (b || h + 1 == n) umma_commit_if(leader, &v_free[slot]);
        if (h + 2 < n) issue_s(h + 2);
      }
    };
    if (n > 0 && ok) ok = wait_all(&sc_full[0], 0);
    if (n > 0 && ok) __any_sync(0xffffffffu, *wide_flag) ? walk(std::true_type{}) : walk(std::false_type{});
    // key tiles that only the other team walks
    if constexpr (!kSplitKeys)
      for (int j = (n + 1) / 2; j < nkt && ok; ++j) {
        ok = wait_all(&k_full[j % kKStages], (j / kKStages) & 1);
        if (ok && leader) mbar_arrive(&k_free[j % kKStages]);
        ok = ok && wait_all(&v_full[j % kStages], (j / kStages) & 1);
        if (ok && leader) mbar_arrive(&v_free[j % kStages]);
        __syncwarp();
      }
    // every MMA issued above is complete before tensor memory is freed
    if (n > 0) {
      umma_commit_if(leader, &fin[team]);
      __syncwarp();
      mbar_wait(&fin[team], 0, p.err);
    }
  }

  // ===================================================== teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <typename QT, int D, bool kSplitKeys, bool kLo>
cudaError_t launch_tiles(const PrefillTcParams &p0, const CUtensorMap &k, int num_chunks, cudaStream_t s) {
  PrefillTcParams p = p0;
  const int rows = kM / p.share_heads * (kSplitKeys ? 1 : kTeams);
  p.row_blocks = (p.max_q_len + rows - 1) / rows;
  const int64_t grid = (int64_t)num_chunks * p.row_blocks * p.num_kv_heads * p.shares;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  constexpr int smem = Layout<D, kSplitKeys, raw_k<QT, kLo>()>::kBytes;
  cudaError_t e = ensure_smem_limit<prefill_scaled_kernel<QT, D, kSplitKeys, kLo>>(smem);
  if (e != cudaSuccess) return e;
  prefill_scaled_kernel<QT, D, kSplitKeys, kLo><<<(unsigned)grid, kThreads, smem, s>>>(p, num_chunks, k);
  return cudaGetLastError();
}

template <typename QT, int D>
cudaError_t launch_dim(const PrefillTcParams &p, const CUtensorMap &k, int num_chunks, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int rows = kTeams * (kM / p.share_heads);
  const int64_t pairs = (int64_t)num_chunks * ((p.max_q_len + rows - 1) / rows) * p.num_kv_heads * p.shares;
  const bool split = pairs < sms;
  if (p.out_f32) return split ? launch_tiles<QT, D, true, true>(p, k, num_chunks, s) : launch_tiles<QT, D, false, true>(p, k, num_chunks, s);
  return split ? launch_tiles<QT, D, true, false>(p, k, num_chunks, s) : launch_tiles<QT, D, false, false>(p, k, num_chunks, s);
}

}  // namespace psc

// k: K's pool as [rows][head_dim codes], one cache block per box.
template <typename QT>
cudaError_t launch_prefill_scaled(const PrefillTcParams &p, const CUtensorMap &k, int head_dim, int num_chunks, cudaStream_t s) {
  if (head_dim == 64) return psc::launch_dim<QT, 64>(p, k, num_chunks, s);
  if (head_dim == 128) return psc::launch_dim<QT, 128>(p, k, num_chunks, s);
  return cudaErrorInvalidValue;
}

}  // namespace pa
