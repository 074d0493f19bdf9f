// Which sequences of a packed batch count.  Sequence s has the rows cu[s] .. cu[s + 1] - 1; it counts
// when 0 <= cu[s] <= cu[s + 1] <= tokens and no earlier bound within [0, tokens] lies behind its
// start.  Sequences that count therefore share no rows: grids, workspaces and slot ranges are sized for
// `tokens` rows in all, whatever the bounds on the device are.
//
// While every sequence's own bounds are in order, no bound steps back and nothing more is to be
// looked at.  The kernels take that for granted, notice at a barrier that they have anyway when it does not
// hold, and only then find the largest earlier bounds (with a vote and a barrier of its own in each of its
// four launches, attention of single tokens in 32 sequences took 76.4 us; so 75.3, and 74.7 unchecked).
#pragma once

#include <cstdint>

namespace nvfp4 {

__device__ __forceinline__ bool bounds_ok(int64_t b, int64_t e, int64_t tokens) { return b >= 0 && e >= b && e <= tokens; }

// Largest usable bound of the sequences up to each thread's, THREADS of them at a time.  A thread whose
// sequence (if `have`) starts at b gets the largest bound in [0, tokens] of those before and its own;
// `high`, uniform over the block, is that of the batches before.  It may be 0 in front of the first call
// where all earlier sequences' own bounds were in order: then none exceeds the next one's start.
// All threads call; s_max: shared.
template <int THREADS>
__device__ __forceinline__ int bound_scan(bool have, int64_t b, int64_t tokens, int &high, int (&s_max)[THREADS / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = have && b >= 0 && b <= tokens ? static_cast<int>(b) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = max(v, x);
  }
  if (lane == 31) s_max[warp] = v;
  __syncthreads();
  v = max(v, high);
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) v = max(v, s_max[w]);
    high = max(high, s_max[w]);
  }
  __syncthreads();
  return v;
}

}  // namespace nvfp4
