// pa_rope.cu -- a step's new tokens: queries and keys rotated by their
// positions, keys and values stored in the paged cache (pa_rope_and_cache).
//
// Rotation: pairs (a, b) -> (a c - b s, b c + a s) with the cosines and sines of
// a table row; products and sum rounded to fp32 one by one (no fused
// multiply-add), so that the largest element of a block, which decides its
// scale, is the same number however it is computed.
//
// All of it is data movement.  A thread's unit is 16 elements of a row: two
// 16-byte vectors, chosen so that both halves of every pair are in one thread
// (halves: the vectors i and i + r/16 elements-of-8 apart; neighbours: two
// consecutive ones), with 8 cosines and 8 sines.
//
// 16-bit caches and fp8 ones with fixed scales: one CTA per token, thread =
// (row, unit of it), rows being the token's q, k and v heads.
//
// Block-scaled caches: a scale belongs to all new tokens of a block, so a warp
// takes one (block, KV head, K or V) as a whole: its new rows, up to block_size of
// them, wait in registers (every load in flight at once), the largest element
// comes from a warp reduction, the scale from its exponent, then the rows go out
// as codes.  Rows the block held before are read only if its scale grows.  There
// are no atomics: the warp of a block's first new token does the block.
//
// Bounds and times, bf16 rows, head_dim 128: 4 x 2048 tokens of 64 + 2 x 8 heads take 52.4 us into a bf16 cache (6.5 TB/s,
// 95 % of a plain copy's rate) and 62.9 us into a block-scaled one (5.1 TB/s: the blocks' chain of slots, rows, largest
// element, codes runs with 16 warps per SM).  64 tokens take 2.5 and 4.1 us: a launch and its chain of loads (position,
// table row, row; slots first for blocks), not bytes.
#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;   // block-scaled launches
constexpr float kMaxCode = 448.f;

// 16 elements of a row: 8 consecutive ones from a and 8 from b.
struct Item {
  uint4 a, b;
};

// Where the halves of unit `k` of a row begin, and its first angle (-1: not rotated).
struct Place {
  int a, b, angle;
};
__device__ __forceinline__ Place place_of(int k, int rope, bool interleaved) {
  if (!interleaved && 16 * k < rope) return {8 * k, 8 * k + rope / 2, 8 * k};
  return {16 * k, 16 * k + 8, 16 * k < rope ? 8 * k : -1};
}

struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(Angles &r, const float *row, int rope, int angle) {
  const float4 *c = reinterpret_cast<const float4 *>(row + angle), *s = reinterpret_cast<const float4 *>(row + rope / 2 + angle);
  const float4 x[4] = {__ldg(c), __ldg(c + 1), __ldg(s), __ldg(s + 1)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.c[4 * i] = x[i].x, r.c[4 * i + 1] = x[i].y, r.c[4 * i + 2] = x[i].z, r.c[4 * i + 3] = x[i].w;
    r.s[4 * i] = x[2 + i].x, r.s[4 * i + 1] = x[2 + i].y, r.s[4 * i + 2] = x[2 + i].z, r.s[4 * i + 3] = x[2 + i].w;
  }
}

template <typename T>
__device__ __forceinline__ void unpack_item(const Item &x, float (&f)[16]) {
  const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 y = unpack2(w[i], T{});
    f[2 * i] = y.x;
    f[2 * i + 1] = y.y;
  }
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}
__device__ __forceinline__ void rotate(float (&f)[16], const Angles &r, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(f[2 * i], f[2 * i + 1], r.c[i], r.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(f[i], f[8 + i], r.c[i], r.s[i]);
  }
}

template <typename T>
__device__ __forceinline__ Item pack_item(const float (&f)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = tc::pack2(f[2 * i], f[2 * i + 1], T{});
  return {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}
__device__ __forceinline__ uint4 code_item(const float (&f)[16]) {
  return make_uint4(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]), codes4(f[8], f[9], f[10], f[11]),
                    codes4(f[12], f[13], f[14], f[15]));
}

// Whether token t takes part, and its row of the table: a padding token does not, a position past the table is reported.
__device__ __forceinline__ bool token_row(const RopeParams &p, int64_t t, const float **row) {
  *row = p.table;
  if (!p.rope) return true;
  const int pos = __ldg(p.positions + t);
  if (pos >= p.num_positions) record_error(p.err, PA_ERR_DEVICE_CHECK);
  if (pos < 0 || pos >= p.num_positions) return false;
  *row += (int64_t)pos * p.rope;
  return true;
}

// One token's rows [0, rows): its q heads, then (unless a block-scaled launch's other warps do them) its k and v heads.
// Thread: unit `tid % units` of the rows tid / units, + threads / units, ..., kBatch of them in flight together.
template <typename T, bool kFp8, int kBatch>
__device__ __forceinline__ void token_rows(const RopeParams &p, int64_t t, int rows, int tid, int threads) {
  const int d = p.head_dim, units = d >> 4, k = tid & (units - 1), step = threads / units;
  const Place at = place_of(k, p.rope, p.interleaved);
  // 0: a query, 1: K, 2: V, and its head
  auto kind_of = [&](int h) { return h < p.num_q_heads ? 0 : h < p.num_q_heads + p.num_kv_heads ? 1 : 2; };
  auto head_of = [&](int h, int kind) { return kind == 0 ? h : kind == 1 ? h - p.num_q_heads : h - p.num_q_heads - p.num_kv_heads; };
  int64_t slot = rows > p.num_q_heads ? __ldg(p.slots + t) : -1;
  Item x[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * step, kind = kind_of(h);
      if (h >= rows) continue;
      const T *src = static_cast<const T *>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) + t * (kind ? p.stride : p.q_stride) + (int64_t)head_of(h, kind) * d;
      x[i] = {*reinterpret_cast<const uint4 *>(src + at.a), *reinterpret_cast<const uint4 *>(src + at.b)};
    }
  };
  load(tid / units);                       // (beside the position and the slot)
  const float *row;
  if (!token_row(p, t, &row)) return;
  Angles ang;
  if (at.angle >= 0) load_angles(ang, row, p.rope, at.angle);
  if (slot >= p.num_blocks * p.block_size) {
    record_error(p.err, PA_ERR_DEVICE_CHECK);
    slot = -1;
  }
  const int64_t blk = slot < 0 ? 0 : slot / p.block_size, off = slot < 0 ? 0 : slot - blk * p.block_size;
  for (int h0 = tid / units; h0 < rows; h0 += kBatch * step) {
    if (h0 >= kBatch * step) load(h0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * step, kind = kind_of(h), hh = head_of(h, kind);
      if (h >= rows || (kind && slot < 0)) continue;
      const bool turned = kind < 2 && at.angle >= 0;
      float f[16];
      if (turned || (kFp8 && kind)) unpack_item<T>(x[i], f);
      if (turned) rotate(f, ang, p.interleaved);
      if (kFp8 && kind) {
        const float *hs = kind == 1 ? p.k_hs : p.v_hs;
        const float s = hs ? __ldg(hs + hh) : kind == 1 ? p.k_scale : p.v_scale;
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = __fdiv_rn(f[e], s);
        const uint4 c = code_item(f);
        uint8_t *dst = static_cast<uint8_t *>(kind == 1 ? p.k_cache : p.v_cache) + ((blk * p.num_kv_heads + hh) * p.block_size + off) * d;
        *reinterpret_cast<uint2 *>(dst + at.a) = make_uint2(c.x, c.y);
        *reinterpret_cast<uint2 *>(dst + at.b) = make_uint2(c.z, c.w);
      } else {
        if (turned) x[i] = pack_item<T>(f);
        T *dst = kind == 0 ? static_cast<T *>(p.q_out) + (t * p.num_q_heads + hh) * d
                           : static_cast<T *>(kind == 1 ? p.k_cache : p.v_cache) + ((blk * p.num_kv_heads + hh) * p.block_size + off) * d;
        *reinterpret_cast<uint4 *>(dst + at.a) = x[i].a;
        *reinterpret_cast<uint4 *>(dst + at.b) = x[i].b;
      }
    }
  }
}

// q may be q_out: no __restrict__, and plain loads of the rows; a thread reads its 16 elements before it writes them
template <typename T, bool kFp8, int kBatch>
__global__ void __launch_bounds__(512) rope_kernel(const RopeParams p) {
  token_rows<T, kFp8, kBatch>(p, blockIdx.x, p.num_q_heads + 2 * p.num_kv_heads, threadIdx.x, blockDim.x);
}

// The smallest power of two 2^e, -64 <= e <= 32, with amax <= 448 * 2^e = 1.75 * 2^(8 + e), or 2^32.
__device__ __forceinline__ float power_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return __uint_as_float((uint32_t)(max(kMinScaleExp, min(kMaxScaleExp, e)) + 127) << 23);
}

// The new tokens t0 + 0..31 of one block (bit i of `mine`: token t0 + i is one), KV head h, K or V, by one warp.
template <typename T, int D, int kBs>
__device__ __forceinline__ void scaled_block(const RopeParams &p, int64_t t0, uint32_t mine, int64_t blk, int first, int h, bool is_v) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kIt = kBs / kRows;   // lanes per row, rows per step, steps
  const int lane = threadIdx.x & 31;
  const bool rope = !is_v && p.rope;
  const Place at = place_of(lane % kLanes, is_v ? 0 : p.rope, p.interleaved);
  const T *src = static_cast<const T *>(is_v ? p.v : p.k) + (int64_t)h * D;
  float *scales = (is_v ? p.v_scales : p.k_scales) + blk * p.num_kv_heads + h;
  const float was = first > 0 ? __ldg(scales) : 1.f;
  Item x[kIt];
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = i * kRows + lane / kLanes;
    x[i] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (mine >> r & 1) {
      const T *row = src + (t0 + r) * p.stride;
      x[i] = {__ldg(reinterpret_cast<const uint4 *>(row + at.a)), __ldg(reinterpret_cast<const uint4 *>(row + at.b))};
    }
  }
  auto values = [&](int i, float (&f)[16]) {   // of step i's row, rotated
    unpack_item<T>(x[i], f);
    const int r = i * kRows + lane / kLanes;
    if (rope && at.angle >= 0 && (mine >> r & 1)) {
      Angles ang;
      load_angles(ang, p.table + (int64_t)__ldg(p.positions + t0 + r) * p.rope, p.rope, at.angle);
      rotate(f, ang, p.interleaved);
    }
  };
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    if (!(mine >> (i * kRows) & ((1u << kRows) - 1))) continue;
    float f[16];
    values(i, f);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float y = fabsf(f[e]);
      if (y <= 3.4028235e38f) amax = fmaxf(amax, y);   // (an infinity saturates, a NaN stays one)
    }
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  float scale = power_for(amax);
  uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + (blk * p.num_kv_heads + h) * (kBs * D);
  if (first > 0) {
    if (!block_scale_ok(was)) {
      if (lane == 0) record_error(p.err, PA_ERR_DEVICE_CHECK);
      return;
    }
    if (amax <= kMaxCode * was) {
      scale = was;
    } else {
      // the tokens the block holds, by its new scale (code * was / scale is exact in fp32 if `was` is a power of two as scale is;
      // another one's 24 bits times a code's 4 are rounded to fp32 first)
      const float by = was / scale;
      for (int e = lane; e < first * (D / 16); e += 32) {
        const uint4 c = *reinterpret_cast<const uint4 *>(pool + e * 16);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        float f[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 lo = unpack2_e4m3(w[i]), hi = unpack2_e4m3(w[i] >> 16);
          f[4 * i] = lo.x * by, f[4 * i + 1] = lo.y * by, f[4 * i + 2] = hi.x * by, f[4 * i + 3] = hi.y * by;
        }
        *reinterpret_cast<uint4 *>(pool + e * 16) = code_item(f);
      }
    }
  }
  if (lane == 0) *scales = scale;
  const bool power = (__float_as_uint(scale) & 0x7fffffu) == 0;   // x / scale is x times an exact reciprocal
  const float inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = i * kRows + lane / kLanes;
    if (!(mine >> (i * kRows) & ((1u << kRows) - 1))) continue;
    float f[16];
    values(i, f);
    if (power) {
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] *= inv;
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = __fdiv_rn(f[e], scale);
    }
    if (mine >> r & 1) {
      const uint4 c = code_item(f);
      uint8_t *dst = pool + (__ldg(p.slots + t0 + r) - blk * kBs) * D;
      *reinterpret_cast<uint2 *>(dst + at.a) = make_uint2(c.x, c.y);
      *reinterpret_cast<uint2 *>(dst + at.b) = make_uint2(c.z, c.w);
    }
  }
}

// Rows in flight per thread of the queries: where the blocks' rows take 124 registers and more there are 16 warps per SM,
// which need 8 (4 x 2048 tokens, 64 heads: 63 us; with 4: 69); at 80 registers 4 (a ragged batch: 6.0 us; with 8: 6.9).
template <int D, int kBs>
constexpr int kQueryBatch = D * kBs >= 2048 ? 8 : 4;

// CTAs from unit_ctas on: the queries, q_threads threads a token.  The others, by warps: warp w takes the blocks whose first new
// token is one of tokens g * window .. + window - 1, KV head and side w % (2 Hkv), g = w / (2 Hkv).  A window of one
// token spreads a decode step over the GPU; a window of 32 leaves few warps without a block of a long prompt.
template <typename T, int D, int kBs>
__global__ void __launch_bounds__(kThreads) rope_scaled_kernel(const RopeParams p, int unit_ctas, int q_threads, int window) {
  if ((int)blockIdx.x >= unit_ctas) {
    const int group = threadIdx.x / q_threads;
    const int64_t t = (int64_t)(blockIdx.x - unit_ctas) * (kThreads / q_threads) + group;
    if (t < p.num_tokens) token_rows<T, false, kQueryBatch<D, kBs>>(p, t, p.num_q_heads, threadIdx.x - group * q_threads, q_threads);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int sides = 2 * p.num_kv_heads, hs = (int)(w % sides);
  const int64_t t0 = w / sides * window;
  if (t0 >= p.num_tokens) return;
  // blocks of the tokens t0 - 32 + lane, t0 + lane, t0 + 32 + lane (-1: none, or it does not take part), and slots in them
  const int64_t slots = p.num_blocks * kBs;
  int blk[3], off[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int64_t t = t0 + 32 * (i - 1) + lane;
    const bool here = t >= 0 && t < p.num_tokens;
    const int64_t s = here ? __ldg(p.slots + t) : -1;
    const int pos = here && p.rope ? __ldg(p.positions + t) : 0;
    // (each token is reported by the warps whose window holds it)
    if (i == 1 && lane < window && hs == 0 && pos >= 0 && (s >= slots || (p.rope && pos >= p.num_positions)))
      record_error(p.err, PA_ERR_DEVICE_CHECK);
    const bool ok = s >= 0 && s < slots && pos >= 0 && (!p.rope || pos < p.num_positions);
    blk[i] = ok ? (int)(s / kBs) : -1;
    off[i] = ok ? (int)(s % kBs) : kBs;
  }
  // candidates: tokens of the window whose neighbour in front is of another block
  int before = __shfl_up_sync(0xffffffffu, blk[1], 1);
  const int last = __shfl_sync(0xffffffffu, blk[0], 31);
  if (lane == 0) before = last;
  uint32_t todo = __ballot_sync(0xffffffffu, lane < window && blk[1] >= 0 && blk[1] != before);
  while (todo) {
    const int i = __ffs(todo) - 1;
    todo &= todo - 1;
    const int b = __shfl_sync(0xffffffffu, blk[1], i);
    // the kBs - 1 tokens in front of token i, and those from it on, that are of the block
    const uint64_t same = (uint64_t)__ballot_sync(0xffffffffu, blk[0] == b) | (uint64_t)__ballot_sync(0xffffffffu, blk[1] == b) << 32;
    const uint32_t next = __ballot_sync(0xffffffffu, blk[2] == b);
    if (same >> (33 + i - kBs) & ((1ull << (kBs - 1)) - 1)) continue;   // not its first new token
    const uint32_t from = (uint32_t)(same >> (32 + i)) | (i ? next << (32 - i) : 0u);
    const uint32_t mine = kBs == 32 ? from : from & 0xffffu;
    int first = min(blk[1] == b && lane >= i && lane < i + kBs ? off[1] : kBs, blk[2] == b && lane + 32 < i + kBs ? off[2] : kBs);
    first = __reduce_min_sync(0xffffffffu, first);
    scaled_block<T, D, kBs>(p, t0 + i, mine, b, first, hs >> 1, hs & 1);
  }
}

template <typename T, int D, int kBs>
cudaError_t launch_scaled(const RopeParams &p, cudaStream_t s) {
  // about 32 warps per SM while the tokens last
  int window = 1;
  while (window < 32 && (int64_t)p.num_tokens * 2 * p.num_kv_heads > (int64_t)window * 64 * kPlanSms) window *= 2;
  const int64_t warps = ((int64_t)p.num_tokens + window - 1) / window * 2 * p.num_kv_heads;
  const int64_t units = (warps + kThreads / 32 - 1) / (kThreads / 32);
  // 2 or 4 of a token's rows per thread while all threads are resident at once (64 tokens: 4.0 us; 4.7 with 8), kQueryBatch beyond that
  const int64_t q_units = (int64_t)p.num_q_heads * (D / 16);
  const int64_t resident = 512ll * kPlanSms;
  const int rows = p.num_tokens * q_units <= 2 * resident ? 2 : p.num_tokens * q_units <= 4 * resident ? 4 : kQueryBatch<D, kBs>;
  int q_threads = 32;
  while (q_threads < kThreads && q_threads * rows < q_units) q_threads *= 2;
  const int per_cta = kThreads / q_threads;
  const int64_t q_ctas = p.num_q_heads ? ((int64_t)p.num_tokens + per_cta - 1) / per_cta : 0;
  if (units + q_ctas > 2147483647ll) return cudaErrorInvalidValue;
  rope_scaled_kernel<T, D, kBs><<<(unsigned)(units + q_ctas), kThreads, 0, s>>>(p, (int)units, q_threads, window);
  return cudaGetLastError();
}

template <typename T, bool kFp8, int kBatch>
cudaError_t launch_rows(const RopeParams &p, int64_t units, int most, cudaStream_t s) {
  // kBatch units per thread, in as few turns of at most `most` threads as the token's need
  const int64_t want = (units + kBatch - 1) / kBatch, turns = (want + most - 1) / most;
  const int threads = (int)(((want + turns - 1) / turns + 31) / 32 * 32);
  rope_kernel<T, kFp8, kBatch><<<p.num_tokens, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_of(const RopeParams &p, cudaStream_t s) {
  if (p.k_scales) {
    if (p.head_dim == 64) return p.block_size == 16 ? launch_scaled<T, 64, 16>(p, s) : launch_scaled<T, 64, 32>(p, s);
    return p.block_size == 16 ? launch_scaled<T, 128, 16>(p, s) : launch_scaled<T, 128, 32>(p, s);
  }
  // 2 rows per thread while all threads are resident at once, 4 beyond that, in CTAs small enough for one to start as another
  // ends (4 x 2048 tokens, 64 + 2 x 8 heads, bf16 cache: turns of 128 threads 52.4 us, of 64 52.7, of 192 and more 59;
  // fp8 cache: 64.8, 60.6, 65.4)
  const int64_t units = ((int64_t)p.num_q_heads + 2 * p.num_kv_heads) * (p.head_dim / 16);
  const bool few = (units + 1) / 2 * p.num_tokens <= 2048ll * kPlanSms;
  if (p.fp8) return few ? launch_rows<T, true, 2>(p, units, 512, s) : launch_rows<T, true, 4>(p, units, 64, s);
  return few ? launch_rows<T, false, 2>(p, units, 512, s) : launch_rows<T, false, 4>(p, units, 128, s);
}

// grid.x = pair, grid.y = 0 (K) / 1 (V): a block's rows and its heads' scales.
__global__ void __launch_bounds__(kThreads) copy_blocks_scaled_kernel(char *k_cache, char *v_cache, float *k_scales, float *v_scales,
                                                                    const int32_t *pairs, int64_t num_blocks,
                                                                    int64_t block_bytes, int32_t heads, int32_t *err) {
  const int64_t src = __ldg(pairs + 2 * blockIdx.x), dst = __ldg(pairs + 2 * blockIdx.x + 1);
  if (src < 0 || dst < 0 || src >= num_blocks || dst >= num_blocks) {
    if (threadIdx.x == 0 && blockIdx.y == 0) record_error(err, PA_ERR_DEVICE_CHECK);
    return;
  }
  char *pool = blockIdx.y ? v_cache : k_cache;
  float *scales = blockIdx.y ? v_scales : k_scales;
  const uint4 *from = reinterpret_cast<const uint4 *>(pool + src * block_bytes);
  uint4 *to = reinterpret_cast<uint4 *>(pool + dst * block_bytes);
  for (int64_t i = threadIdx.x; i < block_bytes >> 4; i += kThreads) to[i] = from[i];
  for (int h = threadIdx.x; h < heads; h += kThreads) scales[dst * heads + h] = scales[src * heads + h];
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeParams &p, pa_dtype in_dtype, cudaStream_t s) {
  return in_dtype == PA_BF16 ? launch_of<__nv_bfloat16>(p, s) : launch_of<__half>(p, s);
}

cudaError_t launch_copy_blocks_scaled(void *k_cache, void *v_cache, const pa_kv_cache &c, float *k_scales, float *v_scales,
                                      const int32_t *pairs, int32_t num_pairs, int32_t *err, cudaStream_t s) {
  copy_blocks_scaled_kernel<<<dim3(num_pairs, 2), kThreads, 0, s>>>(
      static_cast<char *>(k_cache), static_cast<char *>(v_cache), k_scales, v_scales, pairs, c.num_blocks,
      (int64_t)c.num_kv_heads * c.block_size * c.head_dim, c.num_kv_heads, err);
  return cudaGetLastError();
}

}  // namespace pa
