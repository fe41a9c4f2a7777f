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
// Bound by bytes (T * Hkv * 2 * (256 + 132) at D = 128) once the instructions are few: a warp
// takes one token and as many as eight of its heads (a divisor of Hkv, so that no row needs a
// test). Half a warp holds a 128-dim row (16 bytes of bf16 a lane), one half K and the other V:
// the maximum is four shuffles of packed 16-bit maxima, rows leave as whole 128-byte lines, a
// row's addresses are one addition from the last head's, and the token's place (a search of
// cu, its block) is found once, while the rows are already on their way. Measured at 8 heads:
// 46.6k tokens written into blocks of 16 in 47 us (6.1 TB/s; 75 us with four heads a warp and
// three times the instructions a row, which then set the pace), 200k read in 183 us (6.8 TB/s,
// the rate of a copy).
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kCacheWarps = 4;

// Largest magnitudes of a lane's eight bf16 values, as two packed bf16 bit patterns (their
// order is the magnitudes' order). Infinities and NaN, 0x7f80 and more, only with ALL.
template <bool ALL>
__device__ __forceinline__ unsigned amax_bits(const uint4& x) {
  unsigned a[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
  if (!ALL)
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] &= ~__vcmpgeu2(a[i], 0x7f807f80u);
  return __vmaxu2(__vmaxu2(a[0], a[1]), __vmaxu2(a[2], a[3]));
}
// ... over the lanes of a row
template <int LANES>
__device__ __forceinline__ unsigned row_max(unsigned m) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
  return max(m & 0xffffu, m >> 16);
}

template <int DIM, bool KV8, bool WRITE, int HG>
__global__ void __launch_bounds__(kCacheWarps * 32) kv_cache_kernel(const CacheParams p) {
  constexpr int kLanes = DIM / 8;      // lanes of a row, 8 elements each
  constexpr int kPer = kLanes / 16;    // tensors a lane takes part in: K or V, or (D = 256) both
  static_assert(!KV8 || DIM == kHeadDim, "e4m3 pools: head dim 128");
  const int lane = threadIdx.x & 31, col = (lane % kLanes) * 8;
  pdl_wait_primary();
  const long long unit = (long long)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  const int t = (int)(unit / p.head_groups), h0 = (int)(unit - (long long)t * p.head_groups) * HG;
  if (t >= p.T) return;
  int block = 0, row = 0;
  // Element offsets of this lane's share of the first head's row, and from head to head
  const bool is_v[2] = {kPer == 1 && lane >= kLanes, true};
  auto token_row = [&](int q) {
    return is_v[q] ? const_cast<__nv_bfloat16*>(p.v) + t * p.v_st + h0 * p.v_sh + col
                   : const_cast<__nv_bfloat16*>(p.k) + t * p.k_st + h0 * p.k_sh + col;
  };
  auto token_step = [&](int q) { return is_v[q] ? p.v_sh : p.k_sh; };
  auto page_row = [&](int q) {
    return is_v[q] ? block * p.vp_sb + h0 * p.vp_sh + row * p.vp_sr + col : block * p.kp_sb + h0 * p.kp_sh + row * p.kp_sr + col;
  };
  auto page_step = [&](int q) { return is_v[q] ? p.vp_sh : p.kp_sh; };
  auto pool = [&](int q) { return is_v[q] ? p.v_pages : p.k_pages; };
  // checked build: this lane's HG shares of rows lie inside the tokens, the pool and the scales
  auto tokens_ok = [&](int q) {
    const long long at = token_row(q) - (is_v[q] ? p.v : p.k);
    return in_bounds(h0 + HG <= p.Hkv && at >= 0 && at + (HG - 1) * token_step(q) + 8 <= (is_v[q] ? p.v_span : p.k_span), p.err);
  };
  auto page_ok = [&](int q) {
    const long long at = page_row(q);
    return in_bounds(row < 1 << p.block_shift && at >= 0 && at + (HG - 1) * page_step(q) + 8 <= (is_v[q] ? p.vp_span : p.kp_span), p.err);
  };
  auto scale_ok = [&] {
    const long long at = block * p.sc_sb + h0 * p.sc_sh + (is_v[0] ? p.sc_st : 0) + row;
    return in_bounds(at >= 0 && at + (HG - 1) * p.sc_sh < p.sc_span, p.err);
  };
  if (WRITE) {
    uint4 x[kPer][HG];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const __nv_bfloat16* from = token_row(q);
      const long long step = token_step(q);
#pragma unroll
      for (int h = 0; h < HG; ++h, from += step) x[q][h] = tokens_ok(q) ? ldg_stream_v4(from) : make_uint4(0, 0, 0, 0);
    }
    if (!locate<true>(p, t, lane, &block, &row)) return;
    if constexpr (KV8) {
      uint8_t* to = static_cast<uint8_t*>(pool(0)) + page_row(0);
      const long long step = page_step(0);
      const bool in = page_ok(0) && scale_ok();
      float* scale = p.scales + block * p.sc_sb + h0 * p.sc_sh + (is_v[0] ? p.sc_st : 0) + row;
#pragma unroll
      for (int h = 0; h < HG; ++h, to += step, scale += p.sc_sh) {
        const uint4 y = x[0][h];
        unsigned m = row_max<kLanes>(amax_bits<true>(y));
        if (__any_sync(0xffffffffu, m >= 0x7f80u)) m = row_max<kLanes>(amax_bits<false>(y));
        // m = (1 + f / 128) 2^(E - 127); it fits 448 2^e = 1.75 2^(8 + e) with e = E - 135 when
        // f <= 96, else with one more: adding 31 carries into E exactly when f > 96
        const int e = m == 0 ? 0 : min(max((int)((m + 31u) >> 7) - 135, -124), 120);
        const float inv = __int_as_float((127 - e) << 23);
        const unsigned w[4] = {y.x, y.y, y.z, y.w};
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
        if (in) *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
        if (col == 0 && in) *scale = __int_as_float((127 + e) << 23);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(pool(q)) + page_row(q);
        const long long step = page_step(q);
        if (!page_ok(q)) continue;
#pragma unroll
        for (int h = 0; h < HG; ++h, to += step) *reinterpret_cast<uint4*>(to) = x[q][h];
      }
    }
  } else {
    if (!locate<false>(p, t, lane, &block, &row)) return;
    if constexpr (KV8) {
      uint2 x[HG];
      float s[HG];
      const uint8_t* from = static_cast<const uint8_t*>(pool(0)) + page_row(0);
      const long long step = page_step(0);
      const float* scale = p.scales + block * p.sc_sb + h0 * p.sc_sh + (is_v[0] ? p.sc_st : 0) + row;
      if (block >= 0 && !(page_ok(0) && scale_ok())) block = -1;
      if (!tokens_ok(0)) return;
#pragma unroll
      for (int h = 0; h < HG; ++h, from += step, scale += p.sc_sh) {
        x[h] = block >= 0 ? __ldg(reinterpret_cast<const uint2*>(from)) : make_uint2(0, 0);
        s[h] = block >= 0 ? __ldg(scale) : 0.f;
      }
      __nv_bfloat16* to = token_row(0);
      const long long to_step = token_step(0);
#pragma unroll
      for (int h = 0; h < HG; ++h, to += to_step) {  // e4m3 -> f16 (exact) -> f32, times the scale, rounded once to bf16
        uint32_t f[4], o[4];
        e4m3x4_to_f16x4(x[h].x, f[0], f[1]);
        e4m3x4_to_f16x4(x[h].y, f[2], f[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(f16lo_to_f32(f[i]) * s[h], f16hi_to_f32(f[i]) * s[h]);
        *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        uint4 x[HG];
        const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(pool(q)) + page_row(q);
        const long long step = page_step(q);
        if (block >= 0 && !page_ok(q)) block = -1;
        if (!tokens_ok(q)) continue;
#pragma unroll
        for (int h = 0; h < HG; ++h, from += step)
          x[h] = block >= 0 ? __ldg(reinterpret_cast<const uint4*>(from)) : make_uint4(0, 0, 0, 0);
        __nv_bfloat16* to = token_row(q);
        const long long to_step = token_step(q);
#pragma unroll
        for (int h = 0; h < HG; ++h, to += to_step) *reinterpret_cast<uint4*>(to) = x[h];
      }
    }
  }
}

template <int DIM, bool KV8, bool WRITE>
cudaError_t launch_heads(CacheParams& p, bool pdl, cudaStream_t stream) {
  // A warp takes the most heads of a token that divide Hkv, up to eight; one where that would
  // leave SMs without a warp (a decode step's few tokens).
  int hg = 8;
  while (p.Hkv % hg || (hg > 1 && (long long)p.T * (p.Hkv / hg) < 4096)) hg /= 2;
  p.head_groups = p.Hkv / hg;
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
  const CacheParams& c = p;
  switch (hg) {
    case 8: return cudaLaunchKernelEx(&cfg, kv_cache_kernel<DIM, KV8, WRITE, 8>, c);
    case 4: return cudaLaunchKernelEx(&cfg, kv_cache_kernel<DIM, KV8, WRITE, 4>, c);
    case 2: return cudaLaunchKernelEx(&cfg, kv_cache_kernel<DIM, KV8, WRITE, 2>, c);
    default: return cudaLaunchKernelEx(&cfg, kv_cache_kernel<DIM, KV8, WRITE, 1>, c);
  }
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
