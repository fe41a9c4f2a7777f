// packed.cuh -- sequences laid end to end: cu[b] .. cu[b + 1] are the rows of sequence b.
#pragma once
#include <stdint.h>

namespace da {
namespace {

// The sequence of token t: the last b with cu[b] <= t (cu is non-decreasing; whatever it
// holds, the result is in [0, B)). Two rounds of 32-way counting: B <= 1024.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t, int lane) {
  const int step = (B + 31) / 32;
  const int i0 = min((lane + 1) * step, B);
  const int c0 = __popc(__ballot_sync(0xffffffffu, (lane + 1) * step < B && __ldg(cu + i0) <= t)) * step;
  const int i1 = c0 + 1 + lane;
  const int c1 = __popc(__ballot_sync(0xffffffffu, lane < step && i1 < B && __ldg(cu + min(i1, B)) <= t));
  return min(c0 + c1, B - 1);
}

}  // namespace
}  // namespace da
