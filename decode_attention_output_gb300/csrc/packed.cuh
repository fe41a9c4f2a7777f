// packed.cuh -- sequences laid end to end: cu[b] .. cu[b + 1] are the rows of sequence b. What the kernels over such
// rows share: a token's sequence, its place in a paged cache, e4m3 codes.
#pragma once
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

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

// The sequence of token t and its position there, or false for a row of no sequence and for one
// older than its sequence's first token.
template <bool WRITE>
__device__ __forceinline__ bool token_place(const CacheParams& p, int t, int lane, int* seq, long long* place) {
  const int b = find_sequence(p.cu, p.B, t, lane);
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  if (t < c0 || t >= c1) return false;  // a row of no sequence
  long long pos = t - c0;
  if (WRITE) pos += (long long)__ldg(p.seq_lens + b) - ((long long)c1 - c0);
  *seq = b;
  *place = pos;
  return pos >= 0;  // older than the sequence's first token
}

// Where position pos of sequence b lives; one past the table, or whose block is none of the pool's,
// is not written (false) and reads as zeros (block -1).
template <bool WRITE>
__device__ __forceinline__ bool place_block(const CacheParams& p, int b, long long pos, int lane, int* block, int* row) {
  const long long at = pos >> p.block_shift;
  int blk = -1;
  if (at < p.max_blocks && in_bounds(b >= 0 && b < p.B && b * p.bt_stride + at < p.table_span, p.err))
    blk = __ldg(p.table + b * p.bt_stride + at);
  *row = (int)(pos & ((1ll << p.block_shift) - 1));
  *block = blk;
  if ((unsigned)blk < (unsigned)p.num_blocks) return true;
  if (lane == 0) atomicOr(p.err, kErrBlockTable);  // past the table, or a block outside the pool
  *block = -1;
  return !WRITE;  // such a token is not written, and reads as zeros
}

// Where token t lives: flat row index parts (block, row in the block), or false where the
// token has no place. Whole warps call it; `lane` 0's error report counts once.
template <bool WRITE>
__device__ __forceinline__ bool locate(const CacheParams& p, int t, int lane, int* block, int* row) {
  int b;
  long long pos;
  return token_place<WRITE>(p, t, lane, &b, &pos) && place_block<WRITE>(p, b, pos, lane, block, row);
}

// Two floats to e4m3 codes (lo in the low byte), round to nearest even, saturating.
__device__ __forceinline__ unsigned e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace
}  // namespace da
