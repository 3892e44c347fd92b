// pa_prefill_tc.cuh -- chunked-prefill attention on the 5th-generation tensor
// cores (tcgen05.mma, accumulators in tensor memory), head_dim 128.
//
// What it computes ("Inside vLLM v0.7 ...", section "Architectural Blueprint
// 3: Chunked Prefill"; "High-Throughput LLM Serving with vLLM &
// PagedAttention", section "5. Chunked Prefill & Latency SLA Management"):
// row r of chunk c sits at position q_start[c] + r and attends causally to
// positions 0 .. q_start[c] + r of its paged context:
//   out[row][h] = sum_p softmax_p(scale * q[row][h] . K[p][g]) V[p][g].
// Prefill is compute-bound ("High-Throughput LLM Serving ...", section "1. The
// KV Cache Bottleneck in LLM Serving"), so Q.K^T and P.V run as dense tiles on
// the tensor pipe; the softmax stays in fp32 on the CUDA cores.
//
// Tiling.  One CTA = one or two Q tiles of 128 GQA-packed query rows (128/G
// token rows per tile x the G query heads of one KV head; packed row m =
// token m / G, head m % G; tile m / 128) x every key tile of 128 keys up to
// its causal limit.  Each K/V tile feeds every Q tile and all G heads.
//
// Roles (416 threads with two Q tiles, 288 with one):
//  * warps 0-3 / 4-7, softmax of Q tile 0 / 1: thread m owns packed row m
//    (tensor-memory lane m % 128).  It reads its 128 scores with tcgen05.ld
//    twice (maximum, then probabilities), masks them on tiles that reach its
//    causal limit, keeps a lazy reference maximum (its O row in tensor memory
//    is rescaled only when a tile maximum exceeds the reference by more than
//    2^8), and writes P (16-bit pairs) back over the scores with tcgen05.st,
//    each 16 keys' P into those keys' own 16 columns (hi pairs, then lo
//    pairs for a bf16 cache): the P.V MMA reads P straight from tensor
//    memory.
//  * the next 4 warps load: each warp gathers 32 rows (two runs of 16 keys,
//    each inside one block of the block table) of every K and V tile into a
//    ring of kStages tiles, 512 contiguous bytes per warp instruction.
//    16-bit caches: 16-byte cp.async straight into the 128-byte-swizzled MMA
//    layout; fp8 caches, one Q tile per CTA: each warp brings its rows'
//    cache blocks (one bulk-tensor box per block) into a ring of code tiles
//    two tiles ahead, then widens them exactly to f16 from shared memory
//    into the MMA layout; with two Q tiles (no shared memory to spare):
//    register loads half a tile ahead, widened on the way to shared memory.
//    Rows past the end of the sequence are
//    zero-filled so a zero probability never meets a stale (possibly NaN)
//    value in the MMA.
//  * last warp, MMA (one elected lane issues): for each Q tile t in turn,
//    O_t += P_t(j) V_j as soon as P_t(j) is written, then S_t(j+1) = Q_t
//    K_{j+1}^T into the same buffer once that P.V has completed; with two Q
//    tiles, one tile's MMAs run while the other tile's softmax works.
//
// Precision.  K and V are exact in the MMA; accumulation is fp32.  With a
// 16-bit cache the MMAs take the cache's type and Q is exact.  With an fp8
// cache they take f16 operands: the codes widen to f16 exactly (one
// conversion per pair, where bf16 would take three), and bf16 query rows are
// each multiplied by a power of two 2^e that puts the row's largest element
// in [2^14, 2^15) and rounded to f16, exact for every element above 2^-28 of
// that largest one (bf16 has 8 significant bits, f16 11); the scores are
// multiplied back by 2^-e in the softmax.  P must be 16-bit in the MMA: with
// a bf16 cache P is split into hi + lo bf16 parts (two P.V MMAs) that sum to
// P within 2^-16 relative; otherwise P is rounded once to f16 (to nearest
// even) and the softmax denominator sums the rounded P, so the output
// remains a convex combination of V rows.
//
// pa_prefill_chunk_window (kWin) shares the set-up, the loaders of an fp8 cache
// and the teardown, with softmax and MMA roles of its own, further down.
//
// Every mbarrier wait is bounded (PA_ERR_TIMEOUT, then the CTA abandons its
// work); before tensor memory is freed the CTA waits for its outstanding MMAs
// and copies.
#pragma once

#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"
#include "pa_window.cuh"

namespace pa {

struct PrefillTcParams {
  const void *q;               // [total_q][Hq][128]
  const void *k_cache;         // [num_blocks][Hkv][block_size][128]
  const void *v_cache;
  void *out;                   // [total_q][Hq][128]
  int32_t out_f32;
  const int32_t *cu_q_lens;
  const int32_t *q_start;
  const int32_t *seq_lens;
  const int32_t *block_tables;
  int32_t max_blocks_per_seq;
  int32_t max_q_len;
  int32_t row_blocks;          // CTAs per chunk along the query rows
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t block_size;
  int64_t num_blocks;
  float s_mult;                // scale * log2(e) (* k_scale for fp8); a negative value flips q's sign
  float out_mult;              // v_scale for fp8, else 1
  const float *k_hs;           // fp8, optional: [Hkv] per-head scales multiplying s_mult / out_mult
  const float *v_hs;
  int32_t *err;
  // kernels built with kWin: a sliding window with first tokens that stay
  // visible, and query groups of any size, each cut into `shares` of
  // share_heads heads (the last may have fewer) that a CTA row packs
  int32_t window;
  int32_t num_sinks;
  int32_t shares, share_heads;
};

namespace tc {

// p0, p1 -> one f16x2 word (p0 in the low half), each rounded to nearest
// even by the conversion pipe; the two rounded values, widened exactly, are
// added to acc on the FMA pipe (mixed-precision fma with f16 sources).  The
// integer pipe, which the masks, maxima and addressing keep busy, is left
// alone.
__device__ __forceinline__ uint32_t f16x2_rn_add(float p0, float p1, float2 &acc) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(p1), "f"(p0));
  unsigned short lo, hi;
  asm("mov.b32 {%0, %1}, %2;" : "=h"(lo), "=h"(hi) : "r"(w));
  const unsigned short one = 0x3c00;   // f16 1.0
  asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(acc.x) : "h"(lo), "h"(one));
  asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(acc.y) : "h"(hi), "h"(one));
  return w;
}

// The two as f16x2 hi + lo: hi rounded to nearest, lo the rest (exact in fp32), rounded to nearest.
__device__ __forceinline__ uint32_t f16x2_split(float p0, float p1, uint32_t &lo) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(p1), "f"(p0));
  unsigned short h0, h1;
  asm("mov.b32 {%0, %1}, %2;" : "=h"(h0), "=h"(h1) : "r"(w));
  const unsigned short minus = 0xbc00;   // f16 -1.0
  asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(p0) : "h"(h0), "h"(minus));
  asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(p1) : "h"(h1), "h"(minus));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(p1), "f"(p0));
  return w;
}

// f16x2_rn_add in bf16 (8 chunks of 2048 at a window of 1024 + 4: 617 us with the halves widened by shifts, 608 so).
__device__ __forceinline__ uint32_t bf16x2_rn_add(float p0, float p1, float2 &acc) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(p1), "f"(p0));
  unsigned short lo, hi;
  asm("mov.b32 {%0, %1}, %2;" : "=h"(lo), "=h"(hi) : "r"(w));
  const unsigned short one = 0x3f80;   // bf16 1.0
  asm("fma.rn.f32.bf16 %0, %1, %2, %0;" : "+f"(acc.x) : "h"(lo), "h"(one));
  asm("fma.rn.f32.bf16 %0, %1, %2, %0;" : "+f"(acc.y) : "h"(hi), "h"(one));
  return w;
}

constexpr int kD = 128;         // head_dim
constexpr int kM = 128;         // packed query rows per Q tile (MMA M, tensor-memory lanes)
constexpr int kN = 128;         // keys per tile
constexpr int kStages = 2;      // K/V tiles in flight

// Warp roles and tensor-memory size for a CTA of QT Q tiles (1 or 2).
template <int QT>
struct Roles {
  static constexpr int kStages = tc::kStages;
  static constexpr int kSoftmax = QT * 128;           // softmax threads (warps 0 .. 4*QT-1)
  static constexpr int kLoadWarp0 = kSoftmax / 32;    // the next 4 warps load
  static constexpr int kMmaWarp = kLoadWarp0 + 4;     // the last warp issues the MMAs
  static constexpr int kThreads = (kMmaWarp + 1) * 32;
  // score/P buffers of 128 columns per Q tile: two with one Q tile (the next
  // scores are computed while the softmax works), one with two Q tiles
  static constexpr int kBufs = QT == 1 ? 2 : 1;
  static constexpr int kTmemCols = 512;               // QT*kBufs*128 score/P columns, then QT*128 of O
};
// The windowed kernel (kWin): one Q tile per CTA.  kPair: two CTAs share an SM,
// each with one K/V stage, one score/P buffer and half of tensor memory, so that
// one CTA's set-up, softmax and epilogue run under the other's MMAs; else one CTA
// has the SM, with two stages, two score buffers and two softmax threads per row.
// One warp loads a 16-bit cache's tiles (bulk-tensor boxes), four an fp8 one's.
template <bool kPair, bool kFp8>
struct WinRoles {
  static constexpr int kSoftmax = kPair ? 128 : 256;
  static constexpr int kLoadWarp0 = kSoftmax / 32;
  static constexpr int kMmaWarp = kLoadWarp0 + (kFp8 ? 4 : 1);
  static constexpr int kThreads = (4 + kLoadWarp0 + (kFp8 ? 1 : 0)) * 32;
  // Role of a warp: the MMAs are issued by warp 0 and the loads by the next ones, the softmax by warps 4 on
  __device__ static int role(int w) {
    if (w >= 4 && w < 4 + kLoadWarp0) return w - 4;
    if (w == 0) return kMmaWarp;
    const int l = w < 4 ? w - 1 : 3;   // loader
    return l < (kFp8 ? 4 : 1) ? kLoadWarp0 + l : kMmaWarp + 1;
  }
  static constexpr int kBufs = kPair ? 1 : 2;
  static constexpr int kStages = kPair ? 1 : 2;
  static constexpr int kTmemCols = kPair ? 256 : 512;
};
constexpr float kRescaleLog2 = 8.f;

// a Q tile, and a K or V tile: D / 64 panels of [128 rows x 128 B] (Layout::kQBytes, kTileBytes)
constexpr int kTilePanel = kN * 128;        // 16 KB
constexpr int kLoaders = 128;               // threads of the load warps
constexpr int kCodeTile = kN * kD;          // fp8 codes of one K or V tile (128 rows x 128 B)
constexpr int kMaxCodeStages = 2;
constexpr int kNumBars = 4 * kStages + 3 * 4 + 2 + 4 * kMaxCodeStages;

// Shared-memory map, bytes from a 1024-aligned base (128-byte swizzle atoms).
// fp8 caches with one Q tile: kCStages tiles of codes (K then V) after the
// 16-bit K/V stages.
// kWin: the softmax warps' exchange (floats [2][128] and [128]) behind the barriers.
template <int QT, bool kFp8 = false, int D = 128, int kStages = tc::kStages, bool kWin = false>
struct Layout {
  static constexpr int kQBytes = kM * D * 2, kTileBytes = kN * D * 2;
  static constexpr int kCStages = (kFp8 && QT == 1 && D == 128 && kStages == tc::kStages) ? kMaxCodeStages : 0;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + QT * kQBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffCode = kOffV + kStages * kTileBytes;
  static constexpr int kOffBar = kOffCode + kCStages * 2 * kCodeTile;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffExch = kOffMisc + 64;
  static constexpr int kSmemBytes = kOffExch + (kWin ? 3 * 128 * 4 : 0) + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static_assert(kOffExch % 4 == 0, "aligned floats");
  static_assert(kOffCode % 1024 == 0 && kCodeTile % 1024 == 0, "1024-byte swizzle atoms for the code boxes");
};

}  // namespace tc

// The prefill CTA (chunk x row block bx, KV head by), for prefill_tc_kernel and
// for the prefill CTAs of the mixed kernel (pa_mixed_tc.cuh).
// G: query heads per KV head; with kWin 0, the group then being p.share_heads
// heads, rows past the last whole token of the CTA's tiles left idle.
template <typename KV, typename QT, int G, int kQTiles, int D = 128, bool kWin = false, bool kPair = false,
          bool kLo = true>
__device__ __forceinline__ void prefill_tc_body(const PrefillTcParams &p, int bx, int by, const CUtensorMap *tmap_k,
                                                const CUtensorMap *tmap_v) {
  using namespace tc;
  static_assert(D == 64 || D == 128, "head_dim 64 or 128");
  static_assert(kWin == (G == 0) && (kWin || D == 128), "any group and head_dim 64 with kWin only");
  constexpr int kD = D;                       // head_dim (hides tc::kD)
  static_assert(!kWin || kQTiles == 1, "the windowed kernel has one Q tile per CTA");
  using R = std::conditional_t<kWin, WinRoles<kPair, std::is_same<KV, uint8_t>::value>, Roles<kQTiles>>;
  constexpr int kStages = R::kStages;         // (hides tc::kStages)
  using L = Layout<kQTiles, std::is_same<KV, uint8_t>::value, D, kStages, kWin>;
  constexpr int kQBytes = L::kQBytes, kTileBytes = L::kTileBytes;
  constexpr int kSoftmax = R::kSoftmax, kLoadWarp0 = R::kLoadWarp0, kMmaWarp = R::kMmaWarp;
  constexpr int kTmemCols = R::kTmemCols;
  constexpr int kBufs = R::kBufs;
  constexpr bool kFp8 = std::is_same<KV, uint8_t>::value;
  constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;
  constexpr bool kSplit = kWin ? kLo : kBf16 && !kFp8;   // P as hi + lo (kWin: for an fp32 output, else a bf16 cache)
  // K and V tiles come as bulk-tensor boxes of whole cache blocks, in atoms of 8 keys (all panels) of kAtom
  // bytes; else the loaders write panels of 128 keys
  constexpr bool kBoxes = kWin && !kFp8;
  constexpr int kAtom = 8 * 2 * kD;
  constexpr int kGroup = kWin ? 1 : G;
  const int gr = kWin ? p.share_heads : G;
  const int BR = kQTiles * kM / (kWin ? gr : kGroup);      // token rows per CTA
  constexpr bool kF16Ops = kFp8 || !kBf16;   // f16 MMA operands (f16 cache, or any fp8 cache)
  constexpr uint32_t kAB = kF16Ops ? 0u : 1u;
  const float kNegInf = -__int_as_float(0x7f800000);

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *k_full = bars;                       // [kStages] K tile in shared memory (128 loader arrivals)
  uint64_t *v_full = k_full + kStages;           // [kStages] V tile (128)
  uint64_t *k_free = v_full + kStages;           // [kStages] MMAs finished reading the K tile
  uint64_t *v_free = k_free + kStages;           // [kStages] MMAs finished reading the V tile
  uint64_t *s_full = v_free + kStages;           // [tile][buf] scores of key tile j in buffer j % kBufs
  uint64_t *p_full = s_full + 4;                 // [tile][buf] P of key tile j written over them (128 arrivals)
  uint64_t *o_done = p_full + 4;                 // [tile] P.V of key tile j complete (phase j)
  uint64_t *q_ready = o_done + 4;                // Q staged (every softmax thread)
  uint64_t *fin = q_ready + 1;                   // every MMA of the CTA complete
  uint64_t *code_full = fin + 1;                 // [load warp][code stage] the warp's fp8 boxes landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 8);

  const int tid = threadIdx.x, lane = tid & 31;
  int warp = tid >> 5;
  if constexpr (kWin) warp = R::role(warp);
  const int c = bx / p.row_blocks, rb = bx % p.row_blocks;
  const int g = kWin ? by / p.shares : by;   // KV head
  const int h_first = kWin ? (by - g * p.shares) * gr : 0;             // the share's first head of the group
  const int gqa = kWin ? p.num_q_heads / p.num_kv_heads : G;
  const int cu0 = __ldg(p.cu_q_lens + c), nrows = __ldg(p.cu_q_lens + c + 1) - cu0;
  const int qs = __ldg(p.q_start + c);
  if (tid == 0 && by == 0 && rb == 0) {
    const int64_t len = (int64_t)qs + nrows;
    if (nrows < 0 || nrows > p.max_q_len || qs < 0 || __ldg(p.seq_lens + c) != len ||
        len > (int64_t)p.max_blocks_per_seq * p.block_size)
      record_error(p.err, PA_ERR_DEVICE_CHECK);
  }
  const int r0 = rb * BR;
  if (r0 >= nrows) return;  // whole CTA, before any barrier or tensor memory
  // keys this chunk may read: its sequence, clamped to the block table
  const int64_t cap = (int64_t)p.max_blocks_per_seq * p.block_size;
  const int64_t len64 = (int64_t)qs + nrows;
  int seq_eff = len64 <= 0 ? 0 : (int)(len64 < cap ? len64 : cap);
  const int r_last = min(r0 + BR, nrows) - 1;
  int kv_end = min(seq_eff, max(0, qs + r_last + 1));   // keys this CTA needs
  // kWin: from here on keys are packed positions (pa_window.cuh) of the keys that
  // some row of the CTA may see, its first row reaching back furthest; keys of
  // [gap_lo, gap_hi) are seen by none of its rows.
  const int bs_log2 = p.block_size == 32 ? 5 : 4;
  WindowSpan span{0, 0, 0, 0};
  int skip = 0;   // tokens left out between the two parts
  if constexpr (kWin) {
    span = window_span(min(window_low(max(0, qs + r0 + 1), p.window), seq_eff), p.num_sinks, bs_log2);
    skip = span.skip_blocks << bs_log2;
    seq_eff -= skip;
    kv_end = max(0, kv_end - skip);
  }
  const int nkt = (kv_end + kN - 1) / kN;                      // key tiles (may be 0)
  const int32_t *table = p.block_tables + (int64_t)c * p.max_blocks_per_seq;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], kBoxes ? 1 : kLoaders);   // boxes: one expect-tx arrival
      mbar_init(&v_full[s], kBoxes ? 1 : kLoaders);
      mbar_init(&k_free[s], 1);
      mbar_init(&v_free[s], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_ready, kSoftmax);
    mbar_init(fin, 1);
    for (int i = 0; i < 4 * kMaxCodeStages; ++i) mbar_init(&code_full[i], 1);   // one expect-tx arrival
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "n"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // columns: tile t's score/P buffer b at (t*kBufs + b)*128; tile t's O after all of them
  auto sbuf = [&](int t, int b) { return tmem + (uint32_t)((t * kBufs + b) * kN); };
  auto obuf = [&](int t) { return tmem + (uint32_t)(kQTiles * kBufs * kN + t * kD); };

  if (kWin && warp < kLoadWarp0) {
    if constexpr (kWin) {
      // ===================================================== softmax warps, windowed kernel
      // Thread m of each of the kGroups groups owns packed row m.  With two groups (one CTA per SM, few CTAs)
      // they share a row: 64 keys of every tile each, half of the row's elements of Q and O each; what they
      // tell each other (maxima, sums) goes through shared memory between barriers of 64 threads, two warps.
      constexpr int kGroups = R::kSoftmax / 128;
      constexpr int kOwn = kN / kGroups;           // keys per thread and tile
      const int grp = warp >> 2, m = tid & 127, quad = warp & 3;
      const int rl = m / gr, hq = m % gr;
      const bool row_ok = r0 + rl < nrows && rl < BR && h_first + hq < gqa;
      const int64_t row_elem = row_ok ? ((int64_t)(cu0 + r0 + rl) * p.num_q_heads + g * gqa + h_first + hq) * kD : -1;
      // the row sees keys < lim but for those in [num_sinks, row_low), packed positions
      // (idle rows, with q = 0, see everything: they are not stored, and need no masking)
      const int lim = row_ok ? min(seq_eff, max(0, qs + r0 + rl + 1) - skip) : 1 << 30;
      const int row_low = row_ok ? window_low(max(0, qs + r0 + rl + 1), p.window) - skip : 0;
      const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
      // scores are scaled by |s_mult| in the exponent; a negative scale flips q's sign instead.  A masked score of
      // -inf has to stay -inf whatever the scale (a scale of 0 gives scores of about 0).
      float cmul = fmaxf(fabsf(p.s_mult) * (p.k_hs ? __ldg(p.k_hs + g) : 1.f), 1e-30f);
      const uint32_t qflip = p.s_mult < 0.f ? 0x80008000u : 0u;
      float *exch = reinterpret_cast<float *>(smem + L::kOffExch);   // [2][128], then the rows' score factors [128]
      auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory"); };
      auto all_sync = [&]() { asm volatile("bar.sync 5, %0;" ::"n"(R::kSoftmax) : "memory"); };
      {
        // Stage Q: a warp brings its own 32 rows, kC lanes of 16 bytes per row (each group its part of the row;
        // fp8 caches, whose rows are scaled by their largest element: group 0 the whole row)
        constexpr bool kScaled = kFp8 && kBf16;
        constexpr int kC = kD / 8 / (kScaled ? 1 : kGroups), kRI = 32 / kC;   // chunks per row, rows per instruction
        if (!kScaled || grp == 0) {
          uint4 v[kC];
#pragma unroll
          for (int i = 0; i < kC; ++i) {
            const int64_t e = __shfl_sync(0xffffffffu, row_elem, i * kRI + lane / kC);
            // (idle rows read row 0, and are zeroed: a branch around each load would wait for it)
            v[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const QT *>(p.q) + max(e, (int64_t)0)) +
                         (kScaled ? 0 : grp * kC) + lane % kC);
          }
#pragma unroll
          for (int i = 0; i < kC; ++i)
            if (__shfl_sync(0xffffffffu, (int)row_ok, i * kRI + lane / kC) == 0) v[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kC; ++i) {
            const int mr = quad * 32 + i * kRI + lane / kC, ch = (kScaled ? 0 : grp * kC) + lane % kC;
            uint32_t ws[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            if constexpr (kScaled) {
              // f16 operands: the row times 2^e (its largest element in [2^14, 2^15)), rounded to f16
              float amax = 0.f;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                amax = fmaxf(amax, fmaxf(__uint_as_float((ws[k] << 16) & 0x7fffffffu),
                                         __uint_as_float(ws[k] & 0x7fff0000u)));   // NaN ignored
#pragma unroll
              for (int off = kC / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
              const int eb = max(1, (int)((__float_as_uint(amax) >> 23) & 0xff));
              const int e = amax > 0.f ? max(-126, min(126, 141 - eb)) : 0;
              const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
              if (lane % kC == 0) exch[256 + mr] = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = unpack2(ws[k], __nv_bfloat16{});
                const __half2 h = __floats2half2_rn(f.x * sc, f.y * sc);
                ws[k] = *reinterpret_cast<const uint32_t *>(&h);
              }
            }
            *reinterpret_cast<uint4 *>(smem + L::kOffQ + (ch >> 3) * (kM * 128) + mr * 128 + (((ch & 7) ^ (mr & 7)) << 4)) =
                make_uint4(ws[0] ^ qflip, ws[1] ^ qflip, ws[2] ^ qflip, ws[3] ^ qflip);
          }
        }
        fence_async_smem();
        mbar_arrive(q_ready);
        if constexpr (kScaled) {
          all_sync();
          cmul = fmaxf(cmul * exch[256 + m], 1e-30f);
        }
      }

      float m_ref = kNegInf;                     // reference maximum, log2 units
      float2 lacc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};   // partial row sums
      const float2 ones = make_float2(1.f, 1.f);
      bool ok = true;
      auto wait_all = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_or_abort(bar, parity, p.err, abort_flag));
      };
      // The scores are read from tensor memory once into registers, but for fp8 caches with two CTAs per SM (whose four
      // loader warps leave 96 registers per thread): those in chunks of 32, twice (maximum, then probabilities), each
      // read while the one before is worked on.
      constexpr bool kTwice = kGroups == 1;
      constexpr int kChunks = kOwn / 32, kHeld = kTwice ? 2 : kChunks;   // chunks of 32 scores, and how many in registers
      for (int j = 0; j < nkt; ++j) {
        const int b = j % kBufs;
        ok = wait_all(&s_full[b], (j / kBufs) & 1) && ok;
        if (kGroups == 1 && !ok) break;   // two groups: the partner may be at a barrier; go through them without work to do
        const uint32_t sb = sbuf(0, b) + lane_base + grp * kOwn;
        tc_fence_after();
        // of the tile's keys (this group's: from 0 on) the row sees those below nvis but for the glen from g0 on;
        // most tiles are seen whole by every row of the warp
        const int key0 = j * kN + grp * kOwn;
        const int nvis = lim - key0, g0 = p.num_sinks - key0, g1 = row_low - key0;
        const bool full_tile = __all_sync(0xffffffffu, nvis >= kOwn && (g0 >= g1 || g0 >= kOwn || g1 <= 0));
        // The last tile may hold fewer chunks of keys: what the others' columns hold is never a score.  (8 chunks of
        // 2048, whose rows see eight tiles and 32 keys: 699 -> 619 us, with S of the last tile cut short likewise.  The
        // second pass of fp8 caches, two CTAs per SM, has no register for the test: the kernel spills 130 to 190 bytes
        // without it, and with it 5 ragged chunks take 48.1 us instead of 44.5.)
        const int nch = kTwice && kFp8 ? kChunks : min(kChunks, (kv_end - key0 + 31) >> 5);
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = kNegInf;
        float sv[kHeld][32];
        auto take_max = [&](float (&v)[32]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) mx[i & 7] = fmax3(mx[i & 7], v[2 * i], v[2 * i + 1]);
        };
        // bits [0, n) of a word
        auto below = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; };
        auto mask = [&](int ck, float (&v)[32]) {   // hidden scores of chunk ck to -inf
          const uint32_t seen = below(nvis - 32 * ck) & ~(below(g1 - 32 * ck) & ~below(g0 - 32 * ck));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(seen >> i & 1u)) v[i] = kNegInf;
        };
        if constexpr (!kTwice) {
#pragma unroll
          for (int ck = 0; ck < kChunks; ++ck) tmem_ld32_start(sb + 32 * ck, sv[ck]);
#pragma unroll
          for (int ck = 0; ck < kChunks; ++ck) {
            tmem_ld32_finish(sv[ck]);   // (the first one waits for all)
            if (!full_tile) mask(ck, sv[ck]);
            take_max(sv[ck]);
          }
        } else {
          if (!full_tile) {   // mask in place: the second pass then finds -inf
#pragma unroll 1
            for (int ck = 0; ck < nch; ++ck) {
              tmem_ld32_start(sb + 32 * ck, sv[0]);
              tmem_ld32_finish(sv[0]);
              mask(ck, sv[0]);
              take_max(sv[0]);
              tmem_st32(sb + 32 * ck, sv[0]);
            }
          } else {
            tmem_ld32_start(sb, sv[0]);
#pragma unroll
            for (int ck = 0; ck < kChunks; ++ck) {
              tmem_ld32_finish(sv[ck & 1]);
              if (ck + 1 < kChunks) tmem_ld32_start(sb + 32 * (ck + 1), sv[(ck + 1) & 1]);
              take_max(sv[ck & 1]);
            }
          }
          tmem_ld32_start(sb, sv[0]);   // for the second pass
        }
        float mr = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                         fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        if constexpr (kGroups == 2) {
          exch[grp * 128 + m] = mr;
          pair_sync();
          mr = fmaxf(mr, exch[(grp ^ 1) * 128 + m]);
          pair_sync();
        }
        const float mt = mr == kNegInf ? kNegInf : mr * cmul;   // tile maximum, log2 units
        const bool rescale = mt > m_ref + tc::kRescaleLog2;
        if (__any_sync(0xffffffffu, rescale)) {
          const float alpha = rescale ? fast_exp2(m_ref - mt) : 1.f;
          if constexpr (kTwice) tmem_ld32_finish(sv[0]);
          if (j > 0) {
            // O holds the P.V of tiles 0 .. j-1: wait for the last of them, then rescale (this group's part) in place
            ok = wait_all(&o_done[0], (j - 1) & 1) && ok;
            if (kGroups == 1 && !ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = grp * (kD / kGroups); c0 < (grp + 1) * (kD / kGroups); c0 += 16) {
              float o[16];
              uint32_t ow[16];
              tmem_ld16(obuf(0) + lane_base + c0, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) ow[i] = __float_as_uint(o[i] * alpha);
              tmem_st16(obuf(0) + lane_base + c0, ow);
            }
            if constexpr (kGroups == 2) {   // the other group's half of P must not meet this group's O before it is rescaled
              tmem_wait_st();
              tc_fence_before();
              pair_sync();
              tc_fence_after();
            }
          }
          if (rescale) {
#pragma unroll
            for (int i = 0; i < 4; ++i) lacc[i] = make_float2(lacc[i].x * alpha, lacc[i].y * alpha);
            m_ref = mt;
          }
        }
        // p = 2^(s * |s_mult| - m_ref), 16 keys at a time, written over those keys' own 16 score columns; the P.V MMAs
        // of a half of the tile (64 keys) start when it is written
        const float msub = m_ref == kNegInf ? 0.f : m_ref;
        const float2 cc = make_float2(cmul, cmul), nm = make_float2(-msub, -msub);
#pragma unroll
        for (int ck = 0; ck < kChunks; ++ck) {
          float (&v)[32] = sv[ck % kHeld];
          if (ck < nch) {
            if constexpr (kTwice) {
              tmem_ld32_finish(v);
              if (ck + 1 < nch) tmem_ld32_start(sb + 32 * (ck + 1), sv[(ck + 1) & 1]);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {   // keys 32ck + 16hh .. +15
              uint32_t w[8], wl[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int i0 = 16 * hh + 2 * k;
                const float2 a = ffma2(make_float2(v[i0], v[i0 + 1]), cc, nm);
                const float2 pk = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                if constexpr (!kSplit) {   // rounded to the MMA's type, the sum that of the rounded P
                  if constexpr (kF16Ops) w[k] = f16x2_rn_add(pk.x, pk.y, lacc[k & 3]);
                  else w[k] = bf16x2_rn_add(pk.x, pk.y, lacc[k & 3]);
                } else if constexpr (kF16Ops) {   // hi + lo: hi rounded to f16, lo = p - hi, exact in fp32, rounded too
                  w[k] = f16x2_split(pk.x, pk.y, wl[k]);
                  lacc[k & 3] = ffma2(pk, ones, lacc[k & 3]);
                } else {   // the same in bf16, as in the other kernel
                  uint32_t hw, lw2;
                  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hw) : "f"(pk.y), "f"(pk.x));
                  w[k] = hw;
                  const float2 lo = ffma2(make_float2(__uint_as_float(hw << 16), __uint_as_float(hw & 0xffff0000u)),
                                          make_float2(-1.f, -1.f), pk);
                  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lw2) : "f"(lo.y), "f"(lo.x));
                  wl[k] = lw2;
                  lacc[k & 3] = ffma2(pk, ones, lacc[k & 3]);
                }
              }
              tmem_st8(sb + 32 * ck + 16 * hh, w);
              if constexpr (kSplit) tmem_st8(sb + 32 * ck + 16 * hh + 8, wl);
            }
          }
          if (ck == kChunks - 1 || (kGroups == 1 && ck == 1)) {   // a half of the tile is written
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[2 * b + (kGroups == 2 ? grp : ck >> 1)]);
          }
        }
      }
      float l = ((lacc[0].x + lacc[0].y) + (lacc[1].x + lacc[1].y)) + ((lacc[2].x + lacc[2].y) + (lacc[3].x + lacc[3].y));
      // O is complete once the last tile's P.V has finished; with two score buffers, the scores of that tile came when
      // the P.V before the previous one was complete, so the previous one is waited for first
      if (ok && kBufs == 2 && nkt > 1) ok = wait_all(&o_done[0], (nkt - 2) & 1);
      if (ok && nkt > 0) ok = wait_all(&o_done[0], (nkt - 1) & 1);
      all_sync();   // Q is staged and no longer read: its place (and K's behind it) takes the output on its way
      if constexpr (kGroups == 2) {
        exch[grp * 128 + m] = l;
        pair_sync();
        l += exch[(grp ^ 1) * 128 + m];
      }
      if (ok) {
        tc_fence_after();
        const float inv = l > 0.f ? p.out_mult * (p.v_hs ? __ldg(p.v_hs + g) : 1.f) / l : 0.f;
        // Up to 128 bytes of each of the warp's 32 rows at a time: written by the rows' threads (16-byte chunk c of row
        // r at chunk c ^ (r & 7)), then stored by 8 (or 4) lanes per row
        uint8_t *stage = smem + L::kOffQ + warp * 4096;
        auto emit = [&](auto f32) {
          constexpr bool kF32 = decltype(f32)::value;
          constexpr int kPart = kD / kGroups;                            // this thread's elements of its row
          constexpr int kCols = 32;                                      // elements at a time
          constexpr int kCh = kCols * (kF32 ? 4 : 2) / 16, kRI = 32 / kCh;   // chunks per row, rows per instruction
          int64_t e[kCh];
#pragma unroll
          for (int i = 0; i < kCh; ++i) e[i] = __shfl_sync(0xffffffffu, row_elem, i * kRI + lane / kCh);
          // (a loop, not unrolled: this code runs once per CTA, and fetching it costs more than running it)
#pragma unroll 1
          for (int c0 = grp * kPart; c0 < (grp + 1) * kPart; c0 += kCols) {
            float o[kCols / 32][32];
#pragma unroll
            for (int k = 0; k < kCols / 32; ++k)
              if (nkt > 0) tmem_ld32_start(obuf(0) + lane_base + c0 + 32 * k, o[k]);
#pragma unroll
            for (int k = 0; k < kCols / 32; ++k) {
              if (nkt > 0) {
                tmem_ld32_finish(o[k]);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[k][i] = 0.f;
              }
            }
#pragma unroll
            for (int i = 0; i < kCh; ++i) {
              uint4 x;
              if constexpr (kF32) {
                x = make_uint4(__float_as_uint(o[0][4 * i] * inv), __float_as_uint(o[0][4 * i + 1] * inv),
                               __float_as_uint(o[0][4 * i + 2] * inv), __float_as_uint(o[0][4 * i + 3] * inv));
              } else {
                const float *v = &o[i >> 2][8 * (i & 3)];
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
                *reinterpret_cast<uint4 *>(static_cast<char *>(p.out) + (e[i] + c0) * (kF32 ? 4 : 2) + ch * 16) = x;
            }
            __syncwarp();
          }
        };
        if (p.out_f32) emit(std::true_type{});
        else emit(std::false_type{});
      }
    }
  } else if (warp < kLoadWarp0) {
    // ===================================================== softmax warps (Q tile t = warp / 4)
    const int m = tid;                         // packed row
    const int t = m / kM;
    const int rl = m / kGroup, hq = m % kGroup;
    const bool row_ok = r0 + rl < nrows;
    const int head = g * kGroup + hq;
    // keys this row attends to: positions < lim
    const int lim = row_ok ? min(seq_eff, max(0, qs + r0 + rl + 1)) : 0;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // scores are scaled by |s_mult| in the exponent; a negative scale flips q's sign instead
    float cmul = fabsf(p.s_mult) * (p.k_hs ? __ldg(p.k_hs + g) : 1.f);
    const uint32_t qflip = p.s_mult < 0.f ? 0x80008000u : 0u;
    {  // stage row m of Q (16-bit, 128-byte-swizzled K-major, 2 panels per tile)
      const QT *src = static_cast<const QT *>(p.q) + ((int64_t)(cu0 + r0 + rl) * p.num_q_heads + head) * kD;
      const int mr = m % kM;
      uint8_t *qt = smem + L::kOffQ + t * kQBytes;
      if constexpr (kFp8 && kBf16) {
        // f16 operands: the row times 2^e (its largest element in [2^14, 2^15)), rounded to f16;
        // the scores are multiplied back by 2^-e
        uint4 v[16];
        float amax = 0.f;
#pragma unroll
        for (int ch = 0; ch < 16; ++ch) {
          v[ch] = row_ok ? __ldg(reinterpret_cast<const uint4 *>(src) + ch) : make_uint4(0, 0, 0, 0);
          const uint32_t ws[4] = {v[ch].x, v[ch].y, v[ch].z, v[ch].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            amax = fmaxf(amax, fmaxf(__uint_as_float((ws[i] << 16) & 0x7fffffffu),
                                     __uint_as_float(ws[i] & 0x7fff0000u)));   // NaN ignored
        }
        const int eb = max(1, (int)((__float_as_uint(amax) >> 23) & 0xff));
        const int e = amax > 0.f ? max(-126, min(126, 141 - eb)) : 0;
        const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
        cmul *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int ch = 0; ch < 16; ++ch) {
          const uint32_t ws[4] = {v[ch].x, v[ch].y, v[ch].z, v[ch].w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(ws[i], __nv_bfloat16{});
            const __half2 h = __floats2half2_rn(f.x * sc, f.y * sc);
            o[i] = *reinterpret_cast<const uint32_t *>(&h) ^ qflip;
          }
          *reinterpret_cast<uint4 *>(qt + (ch >> 3) * (kM * 128) + mr * 128 + (((ch & 7) ^ (mr & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < 16; ++ch) {
          uint4 v = row_ok ? __ldg(reinterpret_cast<const uint4 *>(src) + ch) : make_uint4(0, 0, 0, 0);
          v.x ^= qflip; v.y ^= qflip; v.z ^= qflip; v.w ^= qflip;
          *reinterpret_cast<uint4 *>(qt + (ch >> 3) * (kM * 128) + mr * 128 + (((ch & 7) ^ (mr & 7)) << 4)) = v;
        }
      }
    }
    fence_async_smem();
    mbar_arrive(q_ready);

    float m_ref = kNegInf;                     // reference maximum, log2 units
    float2 lacc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};   // partial row sums
    const float2 ones = make_float2(1.f, 1.f);
    bool ok = true;
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_or_abort(bar, parity, p.err, abort_flag));
    };
    for (int j = 0; j < nkt; ++j) {
      const int b = j % kBufs;
      ok = wait_all(&s_full[t * kBufs + b], (j / kBufs) & 1);
      if (!ok) break;
      const uint32_t sb = sbuf(t, b) + lane_base;
      tc_fence_after();
      // keys at or past this row's limit are masked, but only tiles that reach
      // some row's limit (the causal diagonal, the sequence end) need the test
      const int nvis = lim - j * kN;
      const bool full_tile = __all_sync(0xffffffffu, nvis >= kN);
      // pass 1: the tile maximum
      float mx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) mx[i] = kNegInf;
#pragma unroll
      for (int ck = 0; ck < kN / 32; ++ck) {
        float sv[32];
        tmem_ld32(sb + 32 * ck, sv);
        if (!full_tile) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * ck + i >= nvis) sv[i] = kNegInf;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) mx[i & 7] = fmax3(mx[i & 7], sv[2 * i], sv[2 * i + 1]);
      }
      const float mr = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                             fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
      const float mt = mr == kNegInf ? kNegInf : mr * cmul;   // tile maximum, log2 units
      const bool rescale = mt > m_ref + tc::kRescaleLog2;
      if (__any_sync(0xffffffffu, rescale)) {
        const float alpha = rescale ? fast_exp2(m_ref - mt) : 1.f;
        if (j > 0) {
          // O holds the P.V of tiles 0 .. j-1: wait for the last of them, then rescale in place
          ok = wait_all(&o_done[t], (j - 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < kD; c0 += 32) {
            float o[32];
            tmem_ld32(obuf(t) + lane_base + c0, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tmem_st32(obuf(t) + lane_base + c0, o);
          }
        }
        if (rescale) {
#pragma unroll
          for (int i = 0; i < 4; ++i) lacc[i] = make_float2(lacc[i].x * alpha, lacc[i].y * alpha);
          m_ref = mt;
        }
      }
      // pass 2: p = 2^(s * |s_mult| - m_ref), 16 keys at a time, written over
      // those keys' own 16 score columns.  A row with nothing visible yet keeps
      // m_ref = -inf.
      const float msub = m_ref == kNegInf ? 0.f : m_ref;
      const float2 cc = make_float2(cmul, cmul), nm = make_float2(-msub, -msub);
#pragma unroll 1
      for (int ck = 0; ck < kN / 32; ++ck) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {   // keys 32ck + 16hh .. +15
          float sv[16];
          tmem_ld16(sb + 32 * ck + 16 * hh, sv);
          uint32_t w[8], wl[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int i0 = 32 * ck + 16 * hh + 2 * k;
            const float2 a = ffma2(make_float2(sv[2 * k], sv[2 * k + 1]), cc, nm);
            float2 pk = make_float2(fast_exp2(a.x), fast_exp2(a.y));
            if (!full_tile) {
              if (i0 >= nvis) pk.x = 0.f;
              if (i0 + 1 >= nvis) pk.y = 0.f;
            }
            if constexpr (kSplit) {
              // bf16 cache: hi = p rounded to bf16, lo = p - hi (exact in fp32) rounded to
              // bf16, both by the conversion pipe; hi + lo is within 2^-16 of p, and the
              // denominator sums p itself
              uint32_t hw, lw2;
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hw) : "f"(pk.y), "f"(pk.x));
              w[k] = hw;
              const float2 lo = ffma2(make_float2(__uint_as_float(hw << 16), __uint_as_float(hw & 0xffff0000u)),
                                      make_float2(-1.f, -1.f), pk);
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lw2) : "f"(lo.y), "f"(lo.x));
              wl[k] = lw2;
              lacc[k & 3] = ffma2(pk, ones, lacc[k & 3]);
            } else {
              // f16 P (p <= 2^8), rounded to nearest even; the denominator sums the rounded P
              w[k] = f16x2_rn_add(pk.x, pk.y, lacc[k & 3]);
            }
          }
          // P of these 16 keys goes over their own 16 score columns (read just
          // above): hi words in the first 8, lo words (bf16 cache) in the next 8
          tmem_st8(sb + 32 * ck + 16 * hh, w);
          if constexpr (kSplit) tmem_st8(sb + 32 * ck + 16 * hh + 8, wl);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[t * kBufs + b]);
    }
    const float l = ((lacc[0].x + lacc[0].y) + (lacc[1].x + lacc[1].y)) +
                    ((lacc[2].x + lacc[2].y) + (lacc[3].x + lacc[3].y));
    // O is complete once the tile's last P.V has finished; with two score buffers, the last tile's scores came when the
    // P.V before the previous one was complete, so the previous one is waited for first (phases of the same parity)
    if (ok && kBufs == 2 && nkt > 1) ok = wait_all(&o_done[t], (nkt - 2) & 1);
    if (ok && nkt > 0) ok = wait_all(&o_done[t], (nkt - 1) & 1);
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.f ? p.out_mult * (p.v_hs ? __ldg(p.v_hs + g) : 1.f) / l : 0.f;
      const int64_t obase = ((int64_t)(cu0 + r0 + rl) * p.num_q_heads + head) * kD;
#pragma unroll 1
      for (int c0 = 0; c0 < kD; c0 += 32) {
        float o[32];
        if (nkt > 0) {
          tmem_ld32(obuf(t) + lane_base + c0, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (!row_ok) continue;
        if (p.out_f32) {
          float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + obase + c0);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
        } else {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<QT *>(p.out) + obase + c0);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack2(o[8 * i] * inv, o[8 * i + 1] * inv, QT{}),
                                pack2(o[8 * i + 2] * inv, o[8 * i + 3] * inv, QT{}),
                                pack2(o[8 * i + 4] * inv, o[8 * i + 5] * inv, QT{}),
                                pack2(o[8 * i + 6] * inv, o[8 * i + 7] * inv, QT{}));
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ===================================================== loaders (4 warps)
    // Warp lw fills rows 32*lw .. 32*lw+31 of every K and V tile: two runs of
    // 16 keys, each inside one block of the block table (tiles start at
    // multiples of 128, blocks hold 16 or 32 keys).
    const int lw = warp - kLoadWarp0;
    constexpr int kRowBytes = kFp8 ? kD : 2 * kD;
    const char *kpool = static_cast<const char *>(p.k_cache);
    const char *vpool = static_cast<const char *>(p.v_cache);
    int32_t win = -1;                 // lane l: block id of run (l & 1) of tile win_base + (l >> 1)
    int win_base = -16;
    // block id of this warp's run r (0/1) of tile j (warp-uniform); -1 past the sequence
    auto block_of = [&](int j, int r) -> int32_t {
      if (j - win_base >= 16) {
        win_base = j;
        const int jt = j + (lane >> 1);
        const int key = jt * kN + 32 * lw + 16 * (lane & 1);
        win = -1;
        if (jt < nkt && key < seq_eff) {
          int lb = key / p.block_size;
          if (kWin && lb >= span.head_blocks) lb += span.skip_blocks;
          const int32_t bi = __ldg(table + lb);
          if (bi < 0 || bi >= p.num_blocks) record_error(p.err, PA_ERR_DEVICE_CHECK);
          else win = bi;
        }
      }
      return __shfl_sync(0xffffffffu, win, 2 * (j - win_base) + r);
    };
    // first cache row of run r's 16 keys in tile j, and how many of them hold data
    auto rows_of = [&](int j, int r, int64_t &row0) -> int {
      const int key0 = j * kN + 32 * lw + 16 * r;
      const int32_t blk = block_of(j, r);
      row0 = ((int64_t)max(blk, 0) * p.num_kv_heads + g) * p.block_size + (key0 % p.block_size);
      return blk < 0 ? 0 : min(16, seq_eff - key0);
    };
    // whether row rr of run r of tile j holds a key that some row of the CTA may see
    // (nval: the run's rows that hold data); the others are zero-filled
    auto seen = [&](int j, int r, int rr, int nval) {
      if (!kWin) return rr < nval;
      const int key = j * kN + 32 * lw + 16 * r + rr;
      return rr < nval && !(key >= span.gap_lo && key < span.gap_hi);
    };
    bool ok = true;
    auto wait_slot = [&](uint64_t *bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, wait_or_abort(bar, parity, p.err, abort_flag));
      return ok;
    };
    if constexpr (kBoxes) {
      // one box per cache block that holds a key < kv_end, straight into the tile
      const int bs = p.block_size, atoms = bs >> 3, per_tile = kN / bs;
      auto block = [&](int j) -> int32_t {   // lane i: the id of block i of tile j, -1: none, or out of range
        const int key = j * kN + lane * bs;
        if (lane >= per_tile || j >= nkt || key >= kv_end) return -1;
        int lb = key / bs;
        if (lb >= span.head_blocks) lb += span.skip_blocks;
        const int32_t bi = __ldg(table + lb);
        if (bi >= 0 && bi < p.num_blocks) return bi;
        record_error(p.err, PA_ERR_DEVICE_CHECK);
        return -1;
      };
      int32_t next = block(0);
      int filled[2] = {0, 0};   // K and V tiles whose boxes are issued
      for (int j = 0; j < nkt && ok; ++j) {
        const int s = j % kStages;
        const int32_t bi = next;
        next = block(j + 1);
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, bi >= 0));
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          if (j >= kStages && !wait_slot(which ? &v_free[s] : &k_free[s], ((j / kStages) - 1) & 1)) break;
          uint64_t *full = which ? &v_full[s] : &k_full[s];
          if (lane == 0) mbar_arrive_expect_tx(full, boxes * atoms * kAtom);
          __syncwarp();
          if (bi >= 0) {
            uint8_t *dst = smem + (which ? L::kOffV : L::kOffK) + s * kTileBytes + lane * atoms * kAtom;
            const CUtensorMap *map = which ? tmap_v : tmap_k;
            const int32_t at = (int32_t)(((int64_t)bi * p.num_kv_heads + g) * atoms);
            if constexpr (kD == 128) tma_load_4d(dst, map, full, 0, 0, 0, at);
            else tma_load_3d(dst, map, full, 0, 0, at);
          }
          ++filled[which];
        }
      }
      // given up: no box in flight at exit (bounded waits)
      if (!ok)
        for (int which = 0; which < 2; ++which)
          for (int t = max(0, filled[which] - kStages); t < filled[which]; ++t)
            mbar_wait(which ? &v_full[t % kStages] : &k_full[t % kStages], (t / kStages) & 1, p.err);
    } else if constexpr (!kFp8) {
      // 16-bit rows (256 B): per instruction 2 rows x 16 chunks of 16 B
      const int q = lane & 15, pn = q >> 3, cq = q & 7;
      for (int j = 0; j < nkt && ok; ++j) {
        const int s = j % kStages;
        const uint32_t ph_prev = ((j / kStages) - 1) & 1;
        int64_t row0[2];
        int nval[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) nval[r] = rows_of(j, r, row0[r]);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          if (j >= kStages && !wait_slot(which ? &v_free[s] : &k_free[s], ph_prev)) break;
          const char *pool = which ? vpool : kpool;
          uint8_t *tile = smem + (which ? L::kOffV : L::kOffK) + s * kTileBytes + pn * kTilePanel;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 2 * i + (lane >> 4);             // row among the run's 16
              const int row = 32 * lw + 16 * r + rr;           // row of the tile
              const bool v = rr < nval[r];
              const char *src = v ? pool + (row0[r] + rr) * kRowBytes + q * 16 : pool;
              cp_async16(tile + row * 128 + ((cq ^ (row & 7)) << 4), src, v ? 16u : 0u);
            }
          }
          cp_async_arrive_noinc(which ? &v_full[s] : &k_full[s]);
        }
      }
    } else if constexpr (L::kCStages > 0) {
      // fp8, one Q tile: warp lw's rows of tile j are one or two whole cache
      // blocks (block_size 32 or 16) of K and of V; it copies them with one
      // bulk-tensor box each into code stage j % kCS (128-byte swizzle, as in
      // the pool map) kCS tiles ahead, then widens them to f16 into the K/V
      // stage.  Each warp waits only for its own boxes.
      constexpr int kCS = L::kCStages;
      const int q = lane & 7, pn = q >> 2, c0 = (2 * q) & 7;
      const int bs = p.block_size;
      uint64_t *cbar = code_full + lw * kCS;
      int issued = 0;      // tiles whose boxes this warp has issued
      uint32_t nvs = 0;    // byte 2 * stage + run: rows of that run holding keys (the block-id window only moves forward)
      auto issue_codes = [&](int j) {
        const int cs = j % kCS;
        int64_t row0;
        const uint32_t n0 = (uint32_t)rows_of(j, 0, row0), n1 = (uint32_t)rows_of(j, 1, row0);
        nvs = (nvs & ~(0xffffu << (16 * cs))) | ((n0 | (n1 << 8)) << (16 * cs));
        const int32_t b0 = block_of(j, 0), b1 = bs == 16 ? block_of(j, 1) : -1;
        const uint32_t n = (b0 >= 0 ? 1u : 0u) + (b1 >= 0 ? 1u : 0u);
        if (lane == 0) mbar_arrive_expect_tx(&cbar[cs], n * 2u * (uint32_t)(bs * kD));
        __syncwarp();
        if (lane < 4) {   // lane = 2 * which + run
          const int which = lane >> 1, r = lane & 1;
          const int32_t blk = r ? b1 : b0;
          if (blk >= 0)
            tma_load_2d(smem + L::kOffCode + cs * 2 * kCodeTile + which * kCodeTile + (32 * lw + 16 * r) * 128,
                        which ? tmap_v : tmap_k, &cbar[cs], 0, (int32_t)(((int64_t)blk * p.num_kv_heads + g) * bs));
        }
        ++issued;
      };
      for (int j = 0; j < kCS && j < nkt; ++j) issue_codes(j);
      for (int j = 0; j < nkt && ok; ++j) {
        const int s = j % kStages, cs = j % kCS;
        const uint32_t ph_prev = ((j / kStages) - 1) & 1;
        if (!wait_slot(&cbar[cs], (j / kCS) & 1)) break;
        const uint8_t *cst = smem + L::kOffCode + cs * 2 * kCodeTile;
#pragma unroll
        for (int qi = 0; qi < 4; ++qi) {
          const int which = qi >> 1, r = qi & 1;
          if (r == 0 && j >= kStages && !wait_slot(which ? &v_free[s] : &k_free[s], ph_prev)) break;
          const int nval = (int)((nvs >> (16 * cs + 8 * r)) & 0xffu);   // rows past the sequence end: zeros
          uint8_t *tile = smem + (which ? L::kOffV : L::kOffK) + s * kTileBytes + pn * kTilePanel;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 4 * i + (lane >> 3), row = 32 * lw + 16 * r + rr;
            const uint4 cw = seen(j, r, rr, nval) ? *reinterpret_cast<const uint4 *>(cst + which * kCodeTile + row * 128 +
                                                                            ((q ^ (row & 7)) << 4))
                                       : make_uint4(0, 0, 0, 0);
            uint32_t o[8];
            widen16<__half>(cw, o);   // the MMAs take f16 operands with an fp8 cache
            uint8_t *dst = tile + row * 128;
            *reinterpret_cast<uint4 *>(dst + ((c0 ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(dst + (((c0 + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          if (r == 1) {
            fence_async_smem();
            mbar_arrive(which ? &v_full[s] : &k_full[s]);
          }
        }
        if (!ok) break;
        // code stage cs is read: its next boxes (generic reads before the async-proxy writes)
        fence_async_smem();
        if (j + kCS < nkt) issue_codes(j + kCS);
      }
      // no box of this warp in flight at exit (bounded waits)
      for (int jj = max(0, issued - kCS); jj < issued; ++jj)
        wait_or_abort(&cbar[jj % kCS], (jj / kCS) & 1, p.err, abort_flag);
    } else {
      // fp8 rows (128 B), two Q tiles: per instruction 4 rows x 8 words of 16
      // codes; the windowed kernel, two CTAs per SM or head_dim 64 (8 rows x 4 words).
      // A tile is four quarters (K run 0, K run 1, V run 0, V run 1).
      // The loads run kPf quarters (half a tile) ahead of the widening into
      // shared memory.
      constexpr int kPf = 2;
      constexpr int kC = kD / 16, kRI = 32 / kC, kIt = 16 / kRI;   // words per row, rows per instruction, instructions
      const int q = lane % kC, pn = q >> 2, c0 = (2 * q) & 7;
      auto load = [&](int j, int qi, uint4 (&w)[kIt]) {
        int64_t row0;
        const int nval = rows_of(j, qi & 1, row0);
        const char *pool = (qi >> 1) ? vpool : kpool;
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          const int rr = kRI * i + lane / kC;
          w[i] = seen(j, qi & 1, rr, nval) ? ld_nc16(pool + (row0 + rr) * kRowBytes + q * 16) : make_uint4(0, 0, 0, 0);
        }
      };
      uint4 buf[kPf][kIt];   // quarter g of the load order in buf[g % kPf]
#pragma unroll
      for (int g = 0; g < kPf; ++g)
        if (g / 4 < nkt) load(g / 4, g % 4, buf[g]);
      for (int j = 0; j < nkt && ok; ++j) {
        const int s = j % kStages;
        const uint32_t ph_prev = ((j / kStages) - 1) & 1;
#pragma unroll
        for (int qi = 0; qi < 4; ++qi) {
          const int which = qi >> 1, r = qi & 1;
          if (r == 0 && j >= kStages && !wait_slot(which ? &v_free[s] : &k_free[s], ph_prev)) break;
          uint8_t *tile = smem + (which ? L::kOffV : L::kOffK) + s * kTileBytes + pn * kTilePanel;
          uint4 (&cur)[kIt] = buf[qi % kPf];
#pragma unroll
          for (int i = 0; i < kIt; ++i) {
            const int row = 32 * lw + 16 * r + kRI * i + lane / kC;
            uint32_t o[8];
            widen16<__half>(cur[i], o);   // the MMAs take f16 operands with an fp8 cache
            uint8_t *dst = tile + row * 128;
            *reinterpret_cast<uint4 *>(dst + ((c0 ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(dst + (((c0 + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          // refill the buffer with the quarter kPf ahead in the load order
          const int g = 4 * j + qi + kPf;
          if (g / 4 < nkt) load(g / 4, g % 4, cur);
          if (r == 1) {
            fence_async_smem();
            mbar_arrive(which ? &v_full[s] : &k_full[s]);
          }
        }
      }
    }
    // before exit: the MMAs' releases of the last tiles have arrived, and no copy is in flight
    if (ok) {
      for (int tt = max(0, nkt - kStages); tt < nkt; ++tt) {
        wait_or_abort(&k_free[tt % kStages], (tt / kStages) & 1, p.err, abort_flag);
        wait_or_abort(&v_free[tt % kStages], (tt / kStages) & 1, p.err, abort_flag);
      }
    }
    if constexpr (!kFp8) cp_async_wait_all();
  } else if (kWin && warp == kMmaWarp) {
    if constexpr (kWin) {
      // ===================================================== MMA issue, windowed kernel
      // Per key tile j: O += P(j) V_j, half a tile of P at a time, then S(j + kBufs) = Q K^T over the buffer P(j) was
      // in, once that P.V is complete.  Keys past kv_end take part up to the end of their group of 16.
      const bool leader = elect_one();
      const uint32_t idesc_s = umma_idesc(kAB, kN, false);
      const uint32_t idesc_last = umma_idesc(kAB, (kv_end - (nkt - 1) * kN + 15) & ~15, false);   // the last tile's keys
      const uint32_t idesc_o = umma_idesc(kAB, kD, true);
      const uint32_t kv_k = smem_u32(smem + L::kOffK), kv_v = smem_u32(smem + L::kOffV);
      const uint64_t qdesc = umma_desc(smem_u32(smem + L::kOffQ), 16);
      const uint64_t kdesc0 = kBoxes ? umma_desc_sbo(kv_k, 16, kAtom) : umma_desc(kv_k, 16);
      const uint64_t vdesc0 = kBoxes ? umma_desc_sbo(kv_v, 1024, kAtom) : umma_desc(kv_v, kTilePanel);
      constexpr uint32_t kKPanel = kBoxes ? 1024 : kTilePanel, kVStep = kBoxes ? 2 * kAtom : 16 * 128;
      auto wait_all = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_or_abort(bar, parity, p.err, abort_flag));
      };
      bool ok = nkt == 0 || wait_all(q_ready, 0);
      bool issued = false;
      auto issue_s = [&](int j) {   // S(j), its K tile waited for
        const uint64_t kd = kdesc0 + (((j % kStages) * kTileBytes) >> 4);
        const uint32_t idesc = j == nkt - 1 ? idesc_last : idesc_s;
        if (leader) {
#pragma unroll 1
          for (int k = 0; k < kD / 16; ++k)
            umma(sbuf(0, j % kBufs), qdesc + (((k >> 2) * (kM * 128) + (k & 3) * 32) >> 4),
                 kd + (((k >> 2) * kKPanel + (k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
          umma_commit(&s_full[j % kBufs]);
          umma_commit(&k_free[j % kStages]);
        }
        __syncwarp();
        issued = true;
      };
      for (int j = 0; j < kBufs && j < nkt && ok; ++j) {
        ok = wait_all(&k_full[j % kStages], (j / kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        issue_s(j);
      }
      for (int j = 0; j < nkt && ok; ++j) {
        const int s = j % kStages, b = j % kBufs, jn = j + kBufs;
        ok = wait_all(&v_full[s], (j / kStages) & 1);
        if (!ok) break;
        const int nvalid = min(kN, kv_end - j * kN), groups = (nvalid + 15) >> 4;
        if constexpr (kBoxes) {
          // rows of V that no row of the CTA sees, in the groups that take part: they may hold anything, and P is 0
          // there, so they are zeroed (fp8 caches: the loaders wrote zeros)
          uint8_t *vt = smem + L::kOffV + s * kTileBytes;
          auto zero_rows = [&](int r0, int r1) {
            constexpr int kRowC = kD / 8;
            for (int e = lane; e < (r1 - r0) * kRowC; e += 32) {
              const int r = r0 + e / kRowC, c = e % kRowC;
              *reinterpret_cast<uint4 *>(vt + (r >> 3) * kAtom + (c >> 3) * 1024 + (r & 7) * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
          };
          const int z0 = max(span.gap_lo - j * kN, 0), z1 = min(span.gap_hi - j * kN, nvalid);
          if (nvalid < 16 * groups || z0 < z1) {
            zero_rows(nvalid, 16 * groups);
            if (z0 < z1) zero_rows(z0, z1);
            fence_async_smem();   // generic stores -> the MMAs' reads
            __syncwarp();
          }
        }
        const uint64_t vd = vdesc0 + ((s * kTileBytes) >> 4);
        for (int h = 0; h < 2 && ok; ++h) {
          ok = wait_all(&p_full[2 * b + h], (j / kBufs) & 1);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            // keys 16kk..16kk+15: P hi at column 16kk, lo at 16kk+8.  A loop, not unrolled: between its turns the warp's
            // code is pushed out of the instruction cache by the softmax's (unrolled, its first 8 MMAs took 1600 clocks
            // to issue, the next 8 530)
            const int k1 = min(groups, (h + 1) * (kN / 32));
#pragma unroll 1
            for (int kk = h * (kN / 32); kk < k1; ++kk) {
              umma_ts(obuf(0), sbuf(0, b) + 16 * kk, vd + ((kk * kVStep) >> 4), idesc_o, j > 0 || kk > 0 ? 1u : 0u);
              if constexpr (kSplit) umma_ts(obuf(0), sbuf(0, b) + 16 * kk + 8, vd + ((kk * kVStep) >> 4), idesc_o, 1u);
            }
            if (h == 1) {
              umma_commit(&o_done[0]);
              umma_commit(&v_free[s]);
            }
          }
          __syncwarp();
          issued = true;
        }
        if (ok && jn < nkt) {
          ok = wait_all(&k_full[jn % kStages], (jn / kStages) & 1) && wait_all(&o_done[0], j & 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(jn);
        }
      }
      // every MMA issued above is complete before tensor memory is freed
      if (issued) {
        if (leader) umma_commit(fin);
        __syncwarp();
        mbar_wait(fin, 0, p.err);
      }
    }
  } else if (warp == kMmaWarp) {
    // ===================================================== MMA issue (warp kMmaWarp; warps
    // past it, in a larger block such as the mixed launch's, have no role)
    // The whole warp runs the schedule (so descriptors stay warp-uniform); one
    // elected lane issues the MMAs and their commits.  Per key tile j and Q
    // tile t: O_t += P_t(j) V_j, then -- once that P.V is complete, because
    // the scores of tile j+1 go where P_t(j) is -- S_t(j+1) = Q_t K_{j+1}^T.
    const bool leader = elect_one();
    const uint32_t idesc_s = umma_idesc(kAB, kN, false);
    const uint32_t idesc_o = umma_idesc(kAB, kD, true);
    const uint64_t qdesc = umma_desc(smem_u32(smem + L::kOffQ), 16);
    const uint64_t kdesc0 = umma_desc(smem_u32(smem + L::kOffK), 16);
    const uint64_t vdesc0 = umma_desc(smem_u32(smem + L::kOffV), kTilePanel);
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_or_abort(bar, parity, p.err, abort_flag));
    };
    bool ok = nkt == 0 || wait_all(q_ready, 0);
    bool issued = false;
    auto issue_s = [&](int t, int j) {  // S_t(j) = Q_t K_j^T into buffer j % kBufs (K tile j waited for)
      const uint64_t kd = kdesc0 + (((j % kStages) * kTileBytes) >> 4);
      const uint64_t qd = qdesc + ((t * kQBytes) >> 4);
      const int bb = j % kBufs;
      if (leader) {
#pragma unroll
        for (int k = 0; k < kD / 16; ++k)
          umma(sbuf(t, bb), qd + (((k >> 2) * (kM * 128) + (k & 3) * 32) >> 4),
               kd + (((k >> 2) * kTilePanel + (k & 3) * 32) >> 4), idesc_s, k > 0 ? 1u : 0u);
        umma_commit(&s_full[t * kBufs + bb]);
      }
      __syncwarp();
      issued = true;
    };
    // the first kBufs score tiles
    for (int jj = 0; jj < kBufs && jj < nkt && ok; ++jj) {
      ok = wait_all(&k_full[jj % kStages], (jj / kStages) & 1);
      if (!ok) break;
      fence_async_smem();
      tc_fence_after();
      for (int t = 0; t < kQTiles; ++t) issue_s(t, jj);
      if (leader) umma_commit(&k_free[jj % kStages]);
      __syncwarp();
    }
    for (int j = 0; j < nkt && ok; ++j) {
      const int s = j % kStages, b = j % kBufs;
      ok = wait_all(&v_full[s], (j / kStages) & 1);
      if (!ok) break;
      const int jn = j + kBufs;                 // the score tile that reuses buffer b
      const bool more = jn < nkt;
      const int sn = jn % kStages;
      const uint64_t vd = vdesc0 + ((s * kTileBytes) >> 4);
      for (int t = 0; t < kQTiles && ok; ++t) {
        ok = wait_all(&p_full[t * kBufs + b], (j / kBufs) & 1);
        if (!ok) break;
        fence_async_smem();   // V tile written through the generic proxy (cp.async / st.shared)
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int half = 0; half < (kSplit ? 2 : 1); ++half) {
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)   // keys 16kk..16kk+15: P hi at column 16kk, lo at 16kk+8
              umma_ts(obuf(t), sbuf(t, b) + 16 * kk + 8 * half, vd + ((kk * 16 * 128) >> 4), idesc_o,
                      (j > 0 || half > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&o_done[t]);
          if (t == kQTiles - 1) umma_commit(&v_free[s]);
        }
        __syncwarp();
        if (more) {
          if (t == 0) {
            ok = wait_all(&k_full[sn], (jn / kStages) & 1);
            if (!ok) break;
          }
          // S_t(jn) overwrites P_t(j): wait for its P.V
          ok = wait_all(&o_done[t], j & 1);
          if (!ok) break;
          fence_async_smem();
          tc_fence_after();
          issue_s(t, jn);
          if (t == kQTiles - 1 && leader) umma_commit(&k_free[sn]);
          __syncwarp();
        }
      }
    }
    // every MMA issued above is complete before tensor memory is freed
    if (issued) {
      if (leader) umma_commit(fin);
      __syncwarp();
      mbar_wait(fin, 0, p.err);
    }
  }

  // ===================================================== teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
  }
}

template <typename KV, typename QT, int G, int kQTiles>
__global__ void __launch_bounds__(tc::Roles<kQTiles>::kThreads, 1)
    prefill_tc_kernel(const PrefillTcParams p, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v) {
  prefill_tc_body<KV, QT, G, kQTiles>(p, blockIdx.x, blockIdx.y, &tmap_k, &tmap_v);
}

// Host launcher: grid (chunks x row blocks, KV heads), one CTA per SM.  Two Q
// tiles per CTA share every K/V tile, unless that leaves SMs idle (few rows):
// then one Q tile per CTA doubles the grid.
template <typename KV, typename QT, int G, int kQTiles>
cudaError_t launch_prefill_tc_tiles(const PrefillTcParams &p0, const PoolMaps &m, int num_chunks, cudaStream_t s) {
  constexpr int smem = tc::Layout<kQTiles, std::is_same<KV, uint8_t>::value>::kSmemBytes;
  constexpr int BR = kQTiles * tc::kM / G;
  PrefillTcParams p = p0;
  p.row_blocks = (p.max_q_len + BR - 1) / BR;
  auto kern = prefill_tc_kernel<KV, QT, G, kQTiles>;
  cudaError_t e = ensure_smem_limit<prefill_tc_kernel<KV, QT, G, kQTiles>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t gx = (int64_t)num_chunks * p.row_blocks;
  if (gx > 2147483647ll || p.num_kv_heads > 65535) return cudaErrorInvalidValue;
  dim3 grid((unsigned)gx, (unsigned)p.num_kv_heads);
  kern<<<grid, tc::Roles<kQTiles>::kThreads, smem, s>>>(p, m.k, m.v);
  return cudaGetLastError();
}

template <typename KV, typename QT, int G>
cudaError_t launch_prefill_tc_one(const PrefillTcParams &p, const PoolMaps &m, int num_chunks, int num_sms,
                                  cudaStream_t s) {
  const int64_t two = (int64_t)num_chunks * ((p.max_q_len + 2 * tc::kM / G - 1) / (2 * tc::kM / G)) * p.num_kv_heads;
  if (two >= num_sms) return launch_prefill_tc_tiles<KV, QT, G, 2>(p, m, num_chunks, s);
  return launch_prefill_tc_tiles<KV, QT, G, 1>(p, m, num_chunks, s);
}

// m: with an fp8 cache, each pool as [rows][128 codes] with one cache block per
// box (encode_pool_map_fp8_blocks); unused with a 16-bit cache.
template <typename KV, typename QT>
cudaError_t launch_prefill_tc(const PrefillTcParams &p, const PoolMaps &m, int gqa, int num_chunks, cudaStream_t s) {
  int num_sms = 0;
  if (current_sm_count(&num_sms) != cudaSuccess) return cudaErrorUnknown;
  switch (gqa) {
    case 1: return launch_prefill_tc_one<KV, QT, 1>(p, m, num_chunks, num_sms, s);
    case 2: return launch_prefill_tc_one<KV, QT, 2>(p, m, num_chunks, num_sms, s);
    case 4: return launch_prefill_tc_one<KV, QT, 4>(p, m, num_chunks, num_sms, s);
    case 8: return launch_prefill_tc_one<KV, QT, 8>(p, m, num_chunks, num_sms, s);
    case 16: return launch_prefill_tc_one<KV, QT, 16>(p, m, num_chunks, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// pa_prefill_chunk_window: the same tiles over the packed keys of a sliding
// window with first tokens that stay visible (pa_window.cuh).  A CTA of BR
// token rows walks window + BR + sinks keys instead of the whole context.
// One kernel for every group size (the group is a run-time number: one
// division per thread) and for head_dim 64 and 128.
//
// P for an fp32 output: hi + lo in the MMA's type (kLo; bf16 for a bf16 cache,
// f16 for the others), within 2^-16 or 2^-22 of it.  For a 16-bit output it is
// rounded once to that type (to nearest, the softmax sum that of the rounded P,
// so that the output stays a convex combination of V rows), about as much as
// the output's own rounding.  Measured for a bf16 cache: the error against 64 bits
// goes from 1.7e-3 (the output's rounding alone) to 2.3e-3 of the output's
// norm, and a third of the MMAs go away: 8 chunks of 2048, 64/8 heads 701 ->
// 607 us, one of 512, 32/8 heads 19.3 -> 17.0, 4 of 1024, head_dim 64 54.8 -> 51.0,
// 3 of 700, 40/8 heads 36.9 -> 33.2.  A caller that wants all bits of P asks for
// an fp32 output.
template <typename KV, typename QT, int D, bool kPair, bool kLo>
__global__ void __launch_bounds__((tc::WinRoles<kPair, std::is_same<KV, uint8_t>::value>::kThreads), kPair ? 2 : 1)
    prefill_window_kernel(const PrefillTcParams p, const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v) {
  prefill_tc_body<KV, QT, 0, 1, D, true, kPair, kLo>(p, blockIdx.x, blockIdx.y, &tmap_k, &tmap_v);
}

template <typename KV, typename QT, int D, bool kPair, bool kLo>
cudaError_t launch_prefill_window_tiles(const PrefillTcParams &p, const PoolMaps &m, dim3 grid, cudaStream_t s) {
  using R = tc::WinRoles<kPair, std::is_same<KV, uint8_t>::value>;
  constexpr int smem = tc::Layout<1, std::is_same<KV, uint8_t>::value, D, R::kStages, true>::kSmemBytes;
  static_assert(!kPair || 2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
  cudaError_t e = ensure_smem_limit<prefill_window_kernel<KV, QT, D, kPair, kLo>>(smem);
  if (e != cudaSuccess) return e;
  prefill_window_kernel<KV, QT, D, kPair, kLo><<<grid, R::kThreads, smem, s>>>(p, m.k, m.v);
  return cudaGetLastError();
}

template <typename KV, typename QT, int D>
cudaError_t launch_prefill_window_one(const PrefillTcParams &p0, const PoolMaps &m, int num_chunks, cudaStream_t s) {
  int num_sms = 0;
  if (current_sm_count(&num_sms) != cudaSuccess) return cudaErrorUnknown;
  PrefillTcParams p = p0;
  const int BR = tc::kM / p.share_heads;   // token rows per CTA
  p.row_blocks = (p.max_q_len + BR - 1) / BR;
  const int64_t gx = (int64_t)num_chunks * p.row_blocks, gy = (int64_t)p.num_kv_heads * p.shares;
  if (gx > 2147483647ll || gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  // One CTA per SM while that is all there is: a 512-token chunk of 32/8 heads (128 CTAs) 17.2 us, as pairs 20.1;
  // beyond that pairs: 8 chunks of 2048, 64/8 heads (8192 CTAs), 0.61 ms, one CTA per SM 0.86.
  const bool pair = gx * gy > num_sms;
  if (!p.out_f32)
    return pair ? launch_prefill_window_tiles<KV, QT, D, true, false>(p, m, grid, s)
                : launch_prefill_window_tiles<KV, QT, D, false, false>(p, m, grid, s);
  return pair ? launch_prefill_window_tiles<KV, QT, D, true, true>(p, m, grid, s)
              : launch_prefill_window_tiles<KV, QT, D, false, true>(p, m, grid, s);
}

template <typename KV, typename QT>
cudaError_t launch_prefill_window(const PrefillTcParams &p, const PoolMaps &m, int head_dim, int num_chunks,
                                  cudaStream_t s) {
  if (head_dim == 64) return launch_prefill_window_one<KV, QT, 64>(p, m, num_chunks, s);
  if (head_dim == 128) return launch_prefill_window_one<KV, QT, 128>(p, m, num_chunks, s);
  return cudaErrorInvalidValue;
}

}  // namespace pa
