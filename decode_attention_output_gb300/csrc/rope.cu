// rope.cu -- norms per head and the position rotation of queries and keys, and the same on the way into a paged cache.
//
// Per (token, head) row x of D dims, in fp32 and rounded once at the end:
//   y = x * r * w,  r = (sum x^2 / D + eps)^-1/2                      (with a weight; y = x without)
//   z_a = y_a c - y_b s,  z_b = y_b c + y_a s    for the R / 2 pairs (a, b) of dims, the others as they are
// c, s = table[p][i], table[p][R / 2 + i]: pair i's angle at the token's position p on that pair's axis. Pairs are (i, i + R / 2), or
// neighbours (2 i, 2 i + 1). Without a norm products and their sum are rounded one by one (no fused multiply-add): the largest
// value of a row decides its scale in an e4m3 cache, and this way it is what the written formula gives. With one the weights
// go into the cosines and sines, a token's for all its heads, and r comes last.
//
// Into the cache: a key's z is rounded once, to bf16 or to e4m3 codes over 2^e with the least e that holds the row, as
// kv_cache.cu does for values; the values are its rows unchanged. Queries go to packed rows.
//
// A row is read and written once, 4 D bytes (a key into an e4m3 cache 3 D + 4), which bounds rows without a norm; with one, and with
// positions of several axes, instruction issue does (70% of the slots in a profile). A lane holds dims 4 l .. 4 l + 3 and
// their partners, so that neither pairing needs a shuffle and a call may work in place; the norm's sum is four shuffles a row, four
// rows side by side. A warp takes one token and eight rows of its heads (two where tokens are few), so that the token's place,
// its position and its cosines and sines are found once, while the rows are already on their way.
// Measured (32 / 8 heads), over rows that are not in L2: 8191 tokens without norms 29 us (5.9 TB/s), with them 36, and positions of
// three axes 38 (the same rows again and again: 27, 32, 35); 46.6k tokens with norms into a bf16 cache 181 (6.0 TB/s), into an e4m3
// one 219; four chunks of 509 to 512 tokens into an e4m3 one 11.1 (again and again 10.4); one token of each of 64 sequences 3.8.
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kRopeWarps = 4;

// Two products, two x * y + c: of what stands in the same place of each.
__device__ __forceinline__ unsigned long long bits2(float2 x) { return *reinterpret_cast<unsigned long long*>(&x); }
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(x)), "l"(bits2(y)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(x)), "l"(bits2(y)), "l"(bits2(c)));
  return *reinterpret_cast<float2*>(&r);
}

// Four weights of dims `at` .. `at` + 3.
__device__ __forceinline__ float4 four_weights(const void* w, bool f32, int at) {
  if (f32) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + at));
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + at));
  return make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
}

__device__ __forceinline__ uint2 ldg_stream_v2(const void* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

// The least e with max <= 448 * 2^e for a row's largest magnitude (its fp32 bits), in [-124, 120]; 0 for a row of zeros.
__device__ __forceinline__ int e4m3_exponent(unsigned m) {
  // m = (1 + f / 2^23) 2^(E - 127); it fits 448 2^e = 1.75 2^(8 + e) with e = E - 135 when f <= 0.75 * 2^23, else with
  // one more: adding 0x1fffff carries into E exactly when f is past that
  return m == 0 ? 0 : min(max((int)((m + 0x1fffffu) >> 23) - 135, -124), 120);
}

enum Dest { kPacked, kPages16, kPages8 };  // where keys go

// ROWS: rows of a warp, per lane group that holds one. NORM: there is a weight, of q or of k.
template <int DIM, bool HALVES, int DEST, int ROWS, bool NORM>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const RopeParams p) {
  constexpr int kLanes = DIM / 8, kAt = 32 / kLanes;  // lanes of a row; rows at a time
  constexpr int kRows = ROWS * kAt;
  const CacheParams& cp = p.cache;
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  pdl_wait_primary();
  const long long unit = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int t = (int)(unit / p.groups), g = (int)(unit - (long long)t * p.groups);
  if (t >= p.T) return;
  const bool is_q = g < p.q_groups, is_k = !is_q && g < p.q_groups + p.k_groups;
  const int heads = is_q ? p.Hq : cp.Hkv;
  const int h0 = (is_q ? g : is_k ? g - p.q_groups : g - p.q_groups - p.k_groups) * kRows + sub;

  // This lane's two runs of four dims. Pairs of halves: dims 4 l and the same of the other half, and
  // behind the R rotated ones two runs that stay. Neighbours: any two runs.
  const int eighth = p.R / 8;
  int d0 = 4 * l, d1 = 4 * l + DIM / 2;
  bool turn0 = d0 < p.R, turn1 = d1 < p.R;
  if (HALVES) {
    turn0 = turn1 = l < eighth;
    d0 = turn0 ? 4 * l : 4 * (l + eighth);
    d1 = turn0 ? 4 * (l + eighth) : 4 * l + DIM / 2;
  }

  const __nv_bfloat16* from = is_q ? p.q + t * p.q_st : is_k ? cp.k + t * cp.k_st : cp.v + t * cp.v_st;
  const long long from_sh = is_q ? p.q_sh : is_k ? cp.k_sh : cp.v_sh;
  const __nv_bfloat16* from_end = is_q ? p.q + p.q_span : is_k ? cp.k + cp.k_span : cp.v + cp.v_span;
  uint2 x[ROWS][2];
  const __nv_bfloat16* at_row = from + h0 * from_sh;
#pragma unroll
  for (int i = 0; i < ROWS; ++i, at_row += kAt * from_sh) {
    const __nv_bfloat16* at = at_row;
    const bool ok = h0 + i * kAt < heads && in_bounds(at + DIM <= from_end, p.err);
    x[i][0] = ok ? ldg_stream_v2(at + d0) : make_uint2(0, 0);
    x[i][1] = ok ? ldg_stream_v2(at + d1) : make_uint2(0, 0);
  }

  // The token's place, and with it its position unless the caller gives one
  int seq = 0, block = 0, row = 0;
  long long place = 0;
  if (DEST != kPacked) {
    if (!token_place<true>(cp, t, lane, &seq, &place)) return;
    if (!is_q && !place_block<true>(cp, seq, place, lane, &block, &row)) return;
  }

  float c[4], s[4];  // halves: of this lane's four pairs; neighbours: two of each run
  if (DEST == kPacked || is_q || is_k) {
    bool far = false;  // a position that the table does not hold: an angle of 0
    if (p.axes == nullptr) {
      const long long pos = p.pos ? (long long)__ldg(p.pos + t) : place;
      far = pos < 0 || pos >= p.P;
      const float* tr = p.table + (far ? 0 : pos) * p.table_st;
      const float *c0 = tr + (HALVES ? 4 * l : 2 * l), *c1 = tr + (HALVES ? 4 * l + 2 : 2 * l + DIM / 4);
      const bool t0 = turn0 && !far && in_bounds((HALVES ? 4 * l + 4 : 2 * l + 2) <= p.R / 2, p.err);
      const bool t1 = turn1 && !far && in_bounds((HALVES ? 4 * l + 4 : 2 * l + DIM / 4 + 2) <= p.R / 2, p.err);
      const float2 one = make_float2(1.f, 1.f), zero = make_float2(0.f, 0.f);
      const float2 ca = t0 ? __ldg(reinterpret_cast<const float2*>(c0)) : one, cb = t1 ? __ldg(reinterpret_cast<const float2*>(c1)) : one;
      const float2 sa = t0 ? __ldg(reinterpret_cast<const float2*>(c0 + p.R / 2)) : zero,
                   sb = t1 ? __ldg(reinterpret_cast<const float2*>(c1 + p.R / 2)) : zero;
      c[0] = ca.x, c[1] = ca.y, c[2] = cb.x, c[3] = cb.y;
      s[0] = sa.x, s[1] = sa.y, s[2] = sb.x, s[3] = sb.y;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pair = HALVES ? 4 * l + i : i < 2 ? 2 * l + i : 2 * l + DIM / 4 + i - 2;
        const bool turn = i < 2 ? turn0 : turn1;
        const int axis = turn ? __ldg(p.axes + pair) : 0;
        const bool known = (unsigned)axis < (unsigned)p.A;
        const int pos = turn && known ? __ldg(p.pos + axis * p.pos_sa + t) : 0;
        const bool off = !known || (unsigned)pos >= (unsigned)p.P;
        const float* at = p.table + (long long)pos * p.table_st + pair;
        far |= turn && off;
        c[i] = turn && !off ? __ldg(at) : 1.f;
        s[i] = turn && !off ? __ldg(at + p.R / 2) : 0.f;
      }
    }
    if (__any_sync(0xffffffffu, far) && lane == 0) atomicOr(p.err, kErrPosition);
  } else {
    turn0 = turn1 = false;
  }
  // A lane's dims as firsts and seconds of its four pairs, two by two: (first, first), (second, second)
  auto firsts_of = [&](float2 (&first)[2], float2 (&second)[2], const float4& run0, const float4& run1) {
    if (HALVES) {
      first[0] = make_float2(run0.x, run0.y), first[1] = make_float2(run0.z, run0.w);
      second[0] = make_float2(run1.x, run1.y), second[1] = make_float2(run1.z, run1.w);
    } else {
      first[0] = make_float2(run0.x, run0.z), second[0] = make_float2(run0.y, run0.w);
      first[1] = make_float2(run1.x, run1.z), second[1] = make_float2(run1.y, run1.w);
    }
  };
  // z_a = (a aa + b ba) r, z_b = (b bb + a ab) r, with the weights in the factors (r = 1 without)
  const void* weight = !NORM ? nullptr : is_q ? p.q_weight : is_k ? p.k_weight : nullptr;
  const bool w32 = is_q ? p.q_weight_f32 : p.k_weight_f32;
  float2 aa[2], ab[2], ba[2], bb[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    aa[k] = bb[k] = make_float2(c[2 * k], c[2 * k + 1]);
    ab[k] = make_float2(s[2 * k], s[2 * k + 1]);
    ba[k] = make_float2(-s[2 * k], -s[2 * k + 1]);
  }
  if (NORM && weight) {
    float2 w_first[2], w_second[2];
    firsts_of(w_first, w_second, four_weights(weight, w32, d0), four_weights(weight, w32, d1));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      aa[k] = mul2(aa[k], w_first[k]);
      ab[k] = mul2(ab[k], w_first[k]);
      ba[k] = mul2(ba[k], w_second[k]);
      bb[k] = mul2(bb[k], w_second[k]);
    }
  }

  // Where the rows go
  const bool packed = is_q || DEST == kPacked;
  __nv_bfloat16* to = is_q ? p.q_out + t * p.qo_st : p.k_out + t * p.ko_st;
  long long to_sh = is_q ? p.qo_sh : p.ko_sh;
  const __nv_bfloat16* to_end = is_q ? p.q_out + p.qo_span : p.k_out + p.ko_span;
  if (!packed) {
    const long long at = is_k ? block * cp.kp_sb + row * cp.kp_sr : block * cp.vp_sb + row * cp.vp_sr;
    to_sh = is_k ? cp.kp_sh : cp.vp_sh;
    void* pool = is_k ? cp.k_pages : cp.v_pages;
    if (DEST == kPages8) {
      to = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(pool) + at);
      to_end = reinterpret_cast<const __nv_bfloat16*>(static_cast<uint8_t*>(pool) + (is_k ? cp.kp_span : cp.vp_span));
    } else {
      to = static_cast<__nv_bfloat16*>(pool) + at;
      to_end = static_cast<const __nv_bfloat16*>(pool) + (is_k ? cp.kp_span : cp.vp_span);
    }
  }

  // The rows' reciprocal roots, whose shuffles wait for one another only within a row
  float root[ROWS];
  if (NORM && weight) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      float2 q = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 u = make_float2(bf16lo_to_f32(x[i][k].x), bf16hi_to_f32(x[i][k].x)), v = make_float2(bf16lo_to_f32(x[i][k].y), bf16hi_to_f32(x[i][k].y));
        q = fma2(v, v, fma2(u, u, q));
      }
      root[i] = q.x + q.y;
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < ROWS; ++i) root[i] += __shfl_xor_sync(0xffffffffu, root[i], off);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) root[i] = rsqrtf(root[i] * (1.f / DIM) + p.eps);
  }

#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i * kAt;
    float2 first[2], second[2];
    firsts_of(first, second, make_float4(bf16lo_to_f32(x[i][0].x), bf16hi_to_f32(x[i][0].x), bf16lo_to_f32(x[i][0].y), bf16hi_to_f32(x[i][0].y)),
              make_float4(bf16lo_to_f32(x[i][1].x), bf16hi_to_f32(x[i][1].x), bf16lo_to_f32(x[i][1].y), bf16hi_to_f32(x[i][1].y)));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 a = first[k], b = second[k];
      const bool turn = HALVES || k == 0 ? turn0 : turn1;
      if (NORM && weight) {
        first[k] = mul2(a, aa[k]);
        second[k] = mul2(b, bb[k]);
        if (turn) {
          first[k] = fma2(b, ba[k], first[k]);
          second[k] = fma2(a, ab[k], second[k]);
        }
        first[k] = mul2(first[k], make_float2(root[i], root[i]));
        second[k] = mul2(second[k], make_float2(root[i], root[i]));
      } else if (turn) {  // each product and their sum rounded once
        first[k] = make_float2(__fadd_rn(__fmul_rn(a.x, aa[k].x), __fmul_rn(b.x, ba[k].x)), __fadd_rn(__fmul_rn(a.y, aa[k].y), __fmul_rn(b.y, ba[k].y)));
        second[k] = make_float2(__fadd_rn(__fmul_rn(b.x, bb[k].x), __fmul_rn(a.x, ab[k].x)), __fadd_rn(__fmul_rn(b.y, bb[k].y), __fmul_rn(a.y, ab[k].y)));
      }
    }
    // in the order of the dims again: this lane's first run, then its second
    float y[8];
    if (HALVES) {
      y[0] = first[0].x, y[1] = first[0].y, y[2] = first[1].x, y[3] = first[1].y;
      y[4] = second[0].x, y[5] = second[0].y, y[6] = second[1].x, y[7] = second[1].y;
    } else {
      y[0] = first[0].x, y[1] = second[0].x, y[2] = first[0].y, y[3] = second[0].y;
      y[4] = first[1].x, y[5] = second[1].x, y[6] = first[1].y, y[7] = second[1].y;
    }
    if (DEST == kPages8 && !is_q) {
      unsigned m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(y[k]) & 0x7fffffffu);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (__any_sync(0xffffffffu, m >= 0x7f800000u)) {  // infinities and NaN do not count
        m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const unsigned b = __float_as_uint(y[k]) & 0x7fffffffu;
          m = max(m, b < 0x7f800000u ? b : 0u);
        }
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
      }
      const int e = e4m3_exponent(m);
      const float inv = __int_as_float((127 - e) << 23);
      unsigned code[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) code[k] = e4m3x2(y[2 * k] * inv, y[2 * k + 1] * inv);
      if (e == 120) {  // codes 0x78 .. 0x7e (256 .. 448) become 0x77 (240), as 256 * 2^120 is no bf16 value; 0x7f is NaN
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int b = 0; b < 16; b += 8) {
            const unsigned mag = code[k] >> b & 0x7fu;
            if (mag > 0x77u && mag < 0x7fu) code[k] -= (mag - 0x77u) << b;
          }
      }
      uint8_t* at = reinterpret_cast<uint8_t*>(to) + h * to_sh;
      const long long sc = block * cp.sc_sb + h * cp.sc_sh + (is_k ? 0 : cp.sc_st) + row;
      if (h < heads && in_bounds(at + DIM <= reinterpret_cast<const uint8_t*>(to_end) && sc < cp.sc_span, p.err)) {
        *reinterpret_cast<unsigned*>(at + d0) = __byte_perm(code[0], code[1], 0x5410);
        *reinterpret_cast<unsigned*>(at + d1) = __byte_perm(code[2], code[3], 0x5410);
        if (l == 0) cp.scales[sc] = __int_as_float((127 + e) << 23);
      }
    } else {
      __nv_bfloat16* at = to + h * to_sh;
      if (h < heads && in_bounds(at + DIM <= to_end, p.err)) {
        const bool as_is = DEST == kPages16 && !is_q && !is_k;  // values: their bits, of NaN too
        *reinterpret_cast<uint2*>(at + d0) = as_is ? x[i][0] : make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
        *reinterpret_cast<uint2*>(at + d1) = as_is ? x[i][1] : make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      }
    }
  }
}

template <int DIM, bool HALVES, int DEST, bool NORM>
cudaError_t launch_rows(RopeParams& p, bool pdl, cudaStream_t stream) {
  constexpr int kAt = 32 / (DIM / 8);
  auto plan = [&](int rows) {
    const int each = rows * kAt;
    p.q_groups = (p.Hq + each - 1) / each;
    p.k_groups = (p.cache.Hkv + each - 1) / each;
    p.groups = p.q_groups + p.k_groups * (DEST == kPacked ? 1 : 2);
    return (long long)p.T * p.groups;
  };
  // Four rows of each lane group, or one where that would leave SMs without a warp (a decode step's few tokens). Eight took
  // registers from other warps: 46.6k tokens into an e4m3 cache 264 us, against 230.
  const bool many = plan(4) >= 4096;
  const long long warps = many ? plan(4) : plan(1), blocks = (warps + kRopeWarps - 1) / kRopeWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kRopeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const RopeParams& c = p;
  return many ? cudaLaunchKernelEx(&cfg, rope_kernel<DIM, HALVES, DEST, 4, NORM>, c) : cudaLaunchKernelEx(&cfg, rope_kernel<DIM, HALVES, DEST, 1, NORM>, c);
}

template <int DIM, int DEST>
cudaError_t launch_pairs(RopeParams& p, bool halves, bool pdl, cudaStream_t stream) {
  if (p.q_weight || p.k_weight)
    return halves ? launch_rows<DIM, true, DEST, true>(p, pdl, stream) : launch_rows<DIM, false, DEST, true>(p, pdl, stream);
  return halves ? launch_rows<DIM, true, DEST, false>(p, pdl, stream) : launch_rows<DIM, false, DEST, false>(p, pdl, stream);
}

}  // namespace

cudaError_t launch_rope(RopeParams& p, int dim, bool halves, bool pages, bool kv8, bool pdl, cudaStream_t stream) {
  if (dim == kHeadDim) {
    if (!pages) return launch_pairs<kHeadDim, kPacked>(p, halves, pdl, stream);
    return kv8 ? launch_pairs<kHeadDim, kPages8>(p, halves, pdl, stream) : launch_pairs<kHeadDim, kPages16>(p, halves, pdl, stream);
  }
  if (dim != kHeadDimWide || (pages && kv8)) return cudaErrorInvalidValue;
  return pages ? launch_pairs<kHeadDimWide, kPages16>(p, halves, pdl, stream) : launch_pairs<kHeadDimWide, kPacked>(p, halves, pdl, stream);
}

}  // namespace da
