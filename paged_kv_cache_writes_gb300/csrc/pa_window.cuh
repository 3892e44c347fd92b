// pa_window.cuh -- which cached tokens a sliding window with first tokens that
// stay visible lets a query see, and how the kernels walk over them.
//
// A query at position t sees p <= t with p < sinks or p > t - window.  With
// low = max(0, t + 1 - window) the visible tokens are [0, min(sinks, low)) and
// [low, t].  The kernels read whole cache blocks, so they walk a shortened
// ("packed") sequence: the blocks holding a visible first token, then the
// blocks from the one holding `low` on, with the blocks between them left out.
// What the two ends of that cut hold but the query does not see is one range
// of packed tokens, [gap_lo, gap_hi), shorter than two blocks; everything else
// about the sequence (tiles, partitions, causal limit) is unchanged, in packed
// coordinates.  Entries of the block table between the two parts are not read.
#pragma once

#include <stdint.h>

namespace pa {

struct WindowSpan {
  int32_t head_blocks;   // blocks of first tokens in front of the cut
  int32_t skip_blocks;   // blocks left out after them
  int32_t gap_lo, gap_hi;  // packed tokens that are not visible (gap_lo >= gap_hi: none)
};

// low: the first position inside the window (0 if it reaches back to the
// start); bs_log2: log2 of the block size.
__host__ __device__ __forceinline__ WindowSpan window_span(int32_t low, int32_t sinks, int32_t bs_log2) {
  WindowSpan w;
  const int32_t s = sinks < low ? sinks : low;
  const int32_t bs = 1 << bs_log2;
  w.head_blocks = (int32_t)(((uint32_t)s + bs - 1) >> bs_log2);
  const int32_t skip = (low >> bs_log2) - w.head_blocks;
  w.skip_blocks = skip > 0 ? skip : 0;
  w.gap_lo = s;
  w.gap_hi = low - (w.skip_blocks << bs_log2);
  return w;
}

// First position of the window of the last of `len` tokens.
__host__ __device__ __forceinline__ int32_t window_low(int32_t len, int32_t window) {
  return len > window ? len - window : 0;
}

// Most tokens the packed sequence can have.
__host__ __forceinline__ int64_t window_max_packed(int64_t max_len, int64_t window, int64_t sinks, int64_t bs) {
  const int64_t most = (sinks + bs - 1) / bs * bs + window + bs - 1;
  return max_len < most ? max_len : most;
}

}  // namespace pa
