// packed.hpp - sequences of different lengths packed one after the other: sequence s has the
// tokens cu[s] .. cu[s + 1] - 1.  Which sequence a workgroup's item belongs to is found on the
// device, by a wave, 64 sequences at a time.
#pragma once

#include "device.hpp"

namespace smcsd {

// The largest s in [0, S) with first(s, cu[s]) <= x, where first does not decrease (0 if there is none),
// with its bounds and context (ctx null: 0): every wave for itself, two rounds of loads for up to 4096
// sequences.  A lane that looks at a sequence loads all of it, and the wave takes what it finds from there.
struct Sequence {
  int s, begin, end, ctx;
};
template <class F>
__device__ __forceinline__ Sequence sequence_of(const int32_t *cu, const int32_t *ctx, int S, int64_t x, F first) {
  const int lane = threadIdx.x % kWave;
  int lo = 0, n = S;
  for (;;) {
    const int step = (n + kWave - 1) / kWave;
    const int at = lo + min(lane * step, n - 1);
    const int32_t begin = cu[at], end = cu[at + 1], have = ctx ? ctx[at] : 0;
    const bool below = lane * step < n && first(at, begin) <= x;
    const int count = max(1, (int)__popcll(__ballot(below)));
    if (step == 1) {
      const int w = count - 1;
      return Sequence{__builtin_amdgcn_readfirstlane(lo + w), __builtin_amdgcn_readlane(begin, w), __builtin_amdgcn_readlane(end, w),
                      __builtin_amdgcn_readlane(have, w)};
    }
    lo += (count - 1) * step;
    n = min(step, n - (count - 1) * step);
  }
}

// Whether the workgroup's share of the S pairs is in order; pairs are shared out over the grid.
__device__ __forceinline__ bool lengths_in_order(const int32_t *cu, int S, int T) {
  bool good = true;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < S; i += (int64_t)gridDim.x * blockDim.x) {
    const int32_t a = cu[i], b = cu[i + 1];
    good &= a >= 0 && b >= a && b <= T;
  }
  return good;
}

}  // namespace smcsd
