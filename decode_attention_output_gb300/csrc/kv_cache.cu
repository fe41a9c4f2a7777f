// kv_cache.cu -- the tokens of packed sequences into a paged KV cache and back.
//
// Write: token t of the packed k / v [T][Hkv][D] (sequence b holds rows cu[b] .. cu[b + 1],
// the last n_b of its seq_lens[b] tokens) goes to position seq_lens[b] - n_b + t - cu[b] of
// sequence b, i.e. to row pos % block_size of block table[b][pos / block_size]. A bf16 pool
// takes the rows as they are; an e4m3 pool takes, per (token, head) row x of K and of V,
//   e = the least integer with max |x| <= 448 * 2^e   (448: the largest e4m3 value)
//   code = e4m3(x * 2^-e)  (round to nearest even),   scale = 2^e.
// A power of two makes the scaling exact and the stored bits independent of how a quotient is
// rounded, and every code * scale is a bf16 value: reading back rounds nothing. It costs no
// precision against max / 448: e4m3 is a float format, the scale only picks its range.
// e stays in [-124, 120]: 2^-124 times the smallest code step 2^-9 is the smallest bf16
// subnormal, and 120 covers the largest bf16 value; under it codes end at 240, since 256 * 2^120
// is past that value. A row of zeros has scale 1; infinities do not count in the maximum and
// saturate to the largest code, NaN becomes the NaN code.
//
// Read: the first cu[b + 1] - cu[b] tokens of each sequence, code * scale, packed to bf16.
//
// Bound by bytes (T * Hkv * 2 * (256 + 132) at D = 128). A warp takes one token and a few of
// its heads: half a warp holds a 128-dim row (16 bytes of bf16 a lane), one half K and the
// other V, so the maximum is four shuffles, rows leave as whole 128-byte lines and the token's
// place (a search of cu, its block) is found once, while the rows are already on their way.
#include "kernels.h"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kCacheWarps = 4;

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

// Where token t lives: flat row index parts (block, row in the block), or false where the
// token has no place. Whole warps call it; `lane` 0's error report counts once.
template <bool WRITE>
__device__ __forceinline__ bool locate(const CacheParams& p, int t, int lane, int* block, int* row) {
  const int b = find_sequence(p.cu, p.B, t, lane);
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  if (t < c0 || t >= c1) return false;  // a row of no sequence
  long long pos = t - c0;
  if (WRITE) pos += (long long)__ldg(p.seq_lens + b) - ((long long)c1 - c0);
  if (pos < 0) return false;  // older than the sequence's first token
  const long long at = pos >> p.block_shift;
  int blk = -1;
  if (at < p.max_blocks) blk = __ldg(p.table + b * p.bt_stride + at);
  *row = (int)(pos & ((1ll << p.block_shift) - 1));
  *block = blk;
  if ((unsigned)blk < (unsigned)p.num_blocks) return true;
  if (lane == 0) atomicOr(p.err, kErrBlockTable);  // past the table, or a block outside the pool
  *block = -1;
  return !WRITE;  // such a token is not written, and reads as zeros
}

// Largest finite magnitude of eight bf16 values, as bf16 bits (order of the bits = order of
// the magnitudes; infinities and NaN, from 0x7f80 up, count as zero).
__device__ __forceinline__ unsigned amax_bits(const uint4& x) {
  unsigned m = 0;
  const unsigned w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned a = w[i] & 0x7fff7fffu;
    m = __vmaxu2(m, a & ~__vcmpgeu2(a, 0x7f807f80u));
  }
  return max(m & 0xffffu, m >> 16);
}

// Two floats to e4m3 codes (lo in the low byte), round to nearest even, saturating.
__device__ __forceinline__ unsigned e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DIM, bool KV8, bool WRITE, int HG>
__global__ void __launch_bounds__(kCacheWarps * 32) kv_cache_kernel(const CacheParams p) {
  constexpr int kLanes = DIM / 8;         // lanes of a row, 8 elements each
  constexpr int kRows = 32 / kLanes;      // rows a warp holds at once
  constexpr int kIt = 2 * HG / kRows;     // K and V rows of HG heads
  static_assert(!KV8 || DIM == kHeadDim, "e4m3 pools: head dim 128");
  const int lane = threadIdx.x & 31, col = (lane % kLanes) * 8;
  pdl_wait_primary();
  const long long unit = (long long)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  const int t = (int)(unit / p.head_groups), h0 = (int)(unit - (long long)t * p.head_groups) * HG;
  if (t >= p.T) return;
  auto tensor = [&](int it) { return (it * kRows + lane / kLanes) & 1; };
  auto head = [&](int it) { return h0 + ((it * kRows + lane / kLanes) >> 1); };
  auto token_row = [&](int it) {
    return (tensor(it) ? p.v + t * p.v_st + head(it) * p.v_sh : p.k + t * p.k_st + head(it) * p.k_sh) + col;
  };
  auto page_at = [&](int it, int block, int row) {  // element offset in the pool
    return (tensor(it) ? block * p.vp_sb + head(it) * p.vp_sh + row * p.vp_sr
                       : block * p.kp_sb + head(it) * p.kp_sh + row * p.kp_sr) + col;
  };
  auto scale_at = [&](int it, int block, int row) { return block * p.sc_sb + head(it) * p.sc_sh + tensor(it) * p.sc_st + row; };
  int block = 0, row = 0;
  if (WRITE) {
    uint4 x[kIt];
#pragma unroll
    for (int it = 0; it < kIt; ++it)
      x[it] = head(it) < p.Hkv ? ldg_stream_v4(token_row(it)) : make_uint4(0, 0, 0, 0);
    if (!locate<true>(p, t, lane, &block, &row)) return;
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      if constexpr (KV8) {
        unsigned m = amax_bits(x[it]);
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        // m = (1 + f / 128) 2^(E - 127); it fits 448 2^e = 1.75 2^(8 + e) with e = E - 135 when
        // f <= 96, else with one more: adding 31 carries into E exactly when f > 96
        const int e = m == 0 ? 0 : min(max((int)((m + 31u) >> 7) - 135, -124), 120);
        const float inv = __int_as_float((127 - e) << 23);
        const unsigned w[4] = {x[it].x, x[it].y, x[it].z, x[it].w};
        unsigned c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = e4m3x2(bf16lo_to_f32(w[i]) * inv, bf16hi_to_f32(w[i]) * inv);
        if (e == 120) {  // codes 0x78 .. 0x7e (256 .. 448) become 0x77 (240); 0x7f is NaN
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < 16; b += 8) {
              const unsigned mag = c[i] >> b & 0x7fu;
              if (mag > 0x77u && mag < 0x7fu) c[i] -= (mag - 0x77u) << b;
            }
        }
        if (head(it) < p.Hkv) {
          uint8_t* pool = static_cast<uint8_t*>(tensor(it) ? p.v_pages : p.k_pages);
          *reinterpret_cast<uint2*>(pool + page_at(it, block, row)) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
          if (col == 0) p.scales[scale_at(it, block, row)] = __int_as_float((127 + e) << 23);
        }
      } else if (head(it) < p.Hkv) {
        __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(tensor(it) ? p.v_pages : p.k_pages);
        *reinterpret_cast<uint4*>(pool + page_at(it, block, row)) = x[it];
      }
    }
  } else {
    if (!locate<false>(p, t, lane, &block, &row)) return;
    uint4 x[kIt];
    float s[kIt];
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      x[it] = make_uint4(0, 0, 0, 0);
      s[it] = 0.f;
      if (head(it) < p.Hkv && block >= 0) {
        if constexpr (KV8) {
          const uint8_t* pool = static_cast<const uint8_t*>(tensor(it) ? p.v_pages : p.k_pages);
          const uint2 c = *reinterpret_cast<const uint2*>(pool + page_at(it, block, row));
          x[it].x = c.x;
          x[it].y = c.y;
          s[it] = p.scales[scale_at(it, block, row)];
        } else {
          const __nv_bfloat16* pool = static_cast<const __nv_bfloat16*>(tensor(it) ? p.v_pages : p.k_pages);
          x[it] = *reinterpret_cast<const uint4*>(pool + page_at(it, block, row));
        }
      }
    }
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      if (KV8) {  // e4m3 -> f16 (exact) -> f32, times the scale, rounded once to bf16
        const unsigned c[2] = {x[it].x, x[it].y};
        unsigned o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned h = e4m3x2_to_f16x2(c[i >> 1] >> (16 * (i & 1)));
          o[i] = pack_bf16x2(f16lo_to_f32(h) * s[it], f16hi_to_f32(h) * s[it]);
        }
        x[it] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (head(it) < p.Hkv) *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(token_row(it))) = x[it];
    }
  }
}

template <int DIM, bool KV8, bool WRITE>
cudaError_t launch_heads(CacheParams& p, bool pdl, cudaStream_t stream) {
  // A warp takes four heads of a token; one head where that would leave SMs without a warp
  // (a decode step's few tokens).
  const int hg = (long long)p.T * ((p.Hkv + 3) / 4) >= 4096 ? 4 : 1;
  p.head_groups = (p.Hkv + hg - 1) / hg;
  const long long blocks = ((long long)p.T * p.head_groups + kCacheWarps - 1) / kCacheWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kCacheWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return hg == 4 ? cudaLaunchKernelEx(&cfg, kv_cache_kernel<DIM, KV8, WRITE, 4>, (const CacheParams)p)
                 : cudaLaunchKernelEx(&cfg, kv_cache_kernel<DIM, KV8, WRITE, 1>, (const CacheParams)p);
}

}  // namespace

cudaError_t launch_cache(CacheParams& p, int dim, bool kv8, bool write, bool pdl, cudaStream_t stream) {
  if (kv8) {
    if (dim != kHeadDim) return cudaErrorInvalidValue;
    return write ? launch_heads<kHeadDim, true, true>(p, pdl, stream) : launch_heads<kHeadDim, true, false>(p, pdl, stream);
  }
  if (dim == kHeadDimWide)
    return write ? launch_heads<kHeadDimWide, false, true>(p, pdl, stream)
                 : launch_heads<kHeadDimWide, false, false>(p, pdl, stream);
  if (dim != kHeadDim) return cudaErrorInvalidValue;
  return write ? launch_heads<kHeadDim, false, true>(p, pdl, stream) : launch_heads<kHeadDim, false, false>(p, pdl, stream);
}

}  // namespace da
