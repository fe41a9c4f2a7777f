// chunk_few.cu -- attention of a few new tokens of each sequence over a paged cache: decode_attn_chunk where sequences have
// one token, or a few drafted ones.
//
// An item is 16 rows of one (sequence, KV head): npos = floor(16 / G) query positions x the G heads that share the KV head.
// Its keys go by in units of 16 (e4m3: 32), those of the first `sinks` and from the window's beginning on. The
// units of all items, laid end to end, are cut into equal parts, one for each CTA (one per SM, fewer where little is
// left to each), whatever the sequences' lengths: an item that lies in several CTAs leaves a state in the
// workspace from each, and the last of them to end joins them in order.
//
//  * Bound by the bytes of K and V. The 128-row tiles of prefill.cuh would be idle but for 16 rows and take 1.3 us
//    a tile of 128 keys, the time of one softmax, whatever its bytes; here a warp works on a unit of its own
//    (mma.sync, 16 rows being one tile's height) and the eight of a CTA meet at the item's end only.
//  * K and V go from memory to the registers that the matrix instructions take them from. Which of a row's dims meet which
//    lane and step is free as long as Q's follow: lane t of the four that hold a key takes its 16-byte pieces t, t + 4,
//    ..., and for V, where an instruction wants two keys' values of one dim in a register, a lane takes one piece of two keys
//    and exchanges halves of its own registers. A unit's 16 loads are issued as soon as the last one's
//    registers have been used: 8 KB a warp, 64 KB an SM on their way.
//  * Softmax as in prefill.cuh: the running maximum lags by up to 2^8, the weights enter P V as bf16, sums are fp32. e4m3:
//    code * scale, rounded once to bf16 (exact for power-of-two scales).
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kWarpsF = 8, kThreadsF = kWarpsF * 32;
constexpr int kRowF = 132;       // floats of a row of the merge buffer (128 and padding)
constexpr int kMostParts = 48;   // of an item
constexpr float kSlackF = 8.f;   // log2 units the maximum may lag
constexpr float kNegInfF = -__builtin_huge_valf();

// Shared memory: the sequences' units (prefix sums), then the warps' states.
constexpr size_t kOffState = ((kMaxBatch + 1) * 8 + 15) & ~(size_t)15;
constexpr size_t kOffMl = kOffState + (size_t)kWarpsF * 16 * kRowF * 4;
constexpr size_t kOffLast = kOffMl + kWarpsF * 16 * 2 * 4;
constexpr size_t kSmemF = kOffLast + 16;

// Units that a sequence's queries see: those of the first keys, and from the window's beginning on.
struct Units {
  int ns, skip, n;
  __device__ __forceinline__ int at(int u) const { return u < ns ? u : u + skip; }
};
template <int KEYS>
__device__ __forceinline__ Units units_of(int lo, int lk, int sinks) {
  Units u;
  const int first = lo / KEYS, ns = (sinks + KEYS - 1) / KEYS;
  u.ns = first > ns ? ns : 0;
  u.skip = first > ns ? first - ns : 0;
  u.n = max((lk + KEYS - 1) / KEYS - u.skip, 1);  // (a sequence without a key gets its rows of zeros)
  return u;
}

__device__ __forceinline__ uint4 ldg_piece(const uint8_t* p, bool ok) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (ok) v = ldg_stream_v4(p);
  return v;
}
// (x.x a.x, x.y a.y) as bf16, of an f16 pair
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t f16x2, float2 a) {
  return pack_bf16x2(f16lo_to_f32(f16x2) * a.x, f16hi_to_f32(f16x2) * a.y);
}

template <bool KV8>
__global__ void __launch_bounds__(kThreadsF, 1) chunk_few_kernel(const __grid_constant__ FewParams p) {
  constexpr int kKeys = KV8 ? 32 : 16, kNT = kKeys / 8;  // keys of a unit, in tiles of 8
  extern __shared__ __align__(16) uint8_t smem[];
  long long* prefix = reinterpret_cast<long long*>(smem);
  float* state = reinterpret_cast<float*>(smem + kOffState);
  float* ml = reinterpret_cast<float*>(smem + kOffMl);
  int* last = reinterpret_cast<int*>(smem + kOffLast);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int G = p.G, npos = p.npos;
  pdl_wait_primary();

  // A sequence: its rows of q, its tokens, the first key of its first query's window.
  struct Seq {
    int q0, lq, lk, lo;
  };
  auto sequence = [&](int b) {
    Seq s;
    s.q0 = min(max(__ldg(p.cu + b), 0), p.Tq);
    s.lq = min(max(__ldg(p.cu + b + 1), s.q0), p.Tq) - s.q0;
    s.lk = min(max(__ldg(p.lens + b), 0), p.cap);
    s.lo = max(0, s.lk - s.lq - p.window + 1);
    return s;
  };
  if (tid == 0) *last = 0;
  __syncthreads();
  for (int b = tid; b < p.B; b += kThreadsF) {
    const Seq s = sequence(b);
    const int n = units_of<kKeys>(s.lo, s.lk, p.sinks).n;
    prefix[b + 1] = (long long)((s.lq + npos - 1) / npos) * p.Hkv * n;
    if (s.lq > 0) atomicMax(last, n);
  }
  __syncthreads();
  if (warp == 0) {
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      long long v = b0 + lane < p.B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
      }
      if (b0 + lane < p.B) prefix[b0 + lane + 1] = base + v;
      base += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) prefix[0] = 0;
  }
  __syncthreads();
  const long long total = prefix[p.B];
  // As many CTAs take part as leave each 256 keys, and the longest item in 48 parts at most: one CTA joins them
  const int ctas = (int)min((long long)gridDim.x, max(total / max(p.least, *last / kMostParts), 1ll));
  if ((int)blockIdx.x >= ctas) return;
  auto begin_of = [&](int c) { return total * c / ctas; };
  auto owner = [&](long long f) { return (int)(((f + 1) * ctas - 1) / total); };
  const long long f1 = begin_of(blockIdx.x + 1);

  for (long long f = begin_of(blockIdx.x); f < f1;) {
    // ------------------------------------------------------------ the segment
    int b = 0;
    for (int step = 512; step > 0; step >>= 1)  // the last b with prefix[b] <= f: B <= 1024
      if (b + step < p.B && prefix[b + step] <= f) b += step;
    const Seq sq = sequence(b);
    const Units un = units_of<kKeys>(sq.lo, sq.lk, p.sinks);
    const long long within = f - prefix[b], item = within / un.n;
    const int rg = (int)(item / p.Hkv), kvh = (int)(item - (long long)rg * p.Hkv);
    const int u0 = (int)(within - item * un.n), u1 = (int)min((long long)un.n, u0 + (f1 - f));
    const long long item0 = f - u0;  // the item's first unit
    const int pos0 = rg * npos, most = min(npos, sq.lq - pos0);  // its first query and how many
    const int shift = sq.lk - sq.lq;                             // position of the sequence's first query
    const int end = min(sq.lk, pos0 + most + shift);             // keys that its last query sees
    const int low = max(0, pos0 + shift - p.window + 1);         // the first of its first query's window
    f += u1 - u0;

    // Q, in the order of dims that K's pieces give: step s holds dims 4 e of piece (16 bytes of a key) ...
    uint32_t aq[8][4];
    int lim[2], from[2];  // of rows g and g + 8: keys seen before lim, and from `from` on (or before sinks)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i, pos = pos0 + r / G;
      const bool ok = r < most * G;
      lim[i] = ok ? min(sq.lk, pos + shift + 1) : 0;
      from[i] = pos + shift - p.window + 1;
      const __nv_bfloat16* row = p.q + (long long)(sq.q0 + pos) * p.q_st + (long long)(kvh * G + r % G) * p.q_sh;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int dim = KV8 ? (t + 4 * (s >> 2)) * 16 + (s & 3) * 4 : (t + 4 * (s >> 1)) * 8 + (s & 1) * 4;
        uint2 v = make_uint2(0, 0);
        if (ok && in_bounds(row + 128 <= p.q + p.q_span, p.err)) v = __ldg(reinterpret_cast<const uint2*>(row + dim));
        aq[s][i] = v.x;
        aq[s][2 + i] = v.y;
      }
    }

    // The blocks of both halves of this warp's next 32 units, a unit a lane.
    int ids[2], ids_at = u0 + warp;
    auto seen = [&](int key) { return key < end && (key >= low || key < p.sinks); };
    auto load_ids = [&] {
      const int key = un.at(ids_at + lane * kWarpsF) * kKeys;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k0 = key + i * (kKeys / 2), k1 = k0 + kKeys / 2 - 1;
        // some key of the half is seen: its first or last, or the sinks or the end fall inside
        const bool need = ids_at + lane * kWarpsF < u1 && k0 < end && (k0 < p.sinks || k1 >= low);
        const long long at = b * p.bt_stride + (k0 >> p.block_shift);
        ids[i] = need && in_bounds(at < p.table_span, p.err) ? __ldg(p.table + at) : -1;
        if (need && (unsigned)ids[i] >= (unsigned)p.num_blocks) {
          atomicOr(p.err, kErrBlockTable);
          ids[i] = -1;
        }
      }
    };
    // The rows' addresses in unit u: pool + block * sb + head * sh + row * sr, as bytes
    uint4 kx[8], vx[8];
    float ks[KV8 ? kNT : 1];
    float2 vs[KV8 ? kNT : 1];
    auto load_k = [&](int u) {
      const int key0 = un.at(u) * kKeys, src = (u - ids_at) / kWarpsF;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int id = __shfl_sync(0xffffffffu, ids[i], src);
        const uint8_t* pool = p.k_pages + id * p.kp_sb + kvh * p.kp_sh;
#pragma unroll
        for (int n = 0; n < kNT / 2; ++n) {
          const int nt = i * (kNT / 2) + n, key = key0 + nt * 8 + g;
          const int row = key & ((1 << p.block_shift) - 1);
          const uint8_t* at = pool + row * p.kp_sr + t * 16;
          const bool ok = id >= 0 && u < u1 && seen(key) && in_bounds(at + (KV8 ? 80 : 208) - p.k_pages <= p.kp_span, p.err);
#pragma unroll
          for (int j = 0; j < 8 / kNT; ++j) kx[nt * (8 / kNT) + j] = ldg_piece(at + j * 64, ok);
          if constexpr (KV8) {
            const float* sc = p.scales + id * p.sc_sb + kvh * p.sc_sh + row;
            ks[nt] = ok && in_bounds(sc - p.scales < p.sc_span, p.err) ? __ldg(sc) : 0.f;
          }
        }
      }
    };
    auto load_v = [&](int u) {
      const int key0 = un.at(u) * kKeys, src = (u - ids_at) / kWarpsF;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int id = __shfl_sync(0xffffffffu, ids[i], src);
        const uint8_t* pool = p.v_pages + id * p.vp_sb + kvh * p.vp_sh;
#pragma unroll
        for (int n = 0; n < kNT / 2; ++n) {
          const int nt = i * (kNT / 2) + n, key = key0 + nt * 8 + 2 * t;
          const int row = key & ((1 << p.block_shift) - 1);
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // two keys of every eight
            const uint8_t* at = pool + (row + k) * p.vp_sr + g * 16;
            const bool ok = id >= 0 && u < u1 && seen(key + k) && in_bounds(at + (KV8 ? 16 : 144) - p.v_pages <= p.vp_span, p.err);
#pragma unroll
            for (int j = 0; j < 4 / kNT; ++j) vx[(nt * 2 + k) * (4 / kNT) + j] = ldg_piece(at + j * 128, ok);
          }
          if constexpr (KV8) {
            const float* sc = p.scales + id * p.sc_sb + kvh * p.sc_sh + p.sc_st + row;
            const bool any = id >= 0 && u < u1 && in_bounds(sc + 1 - p.scales < p.sc_span, p.err);
            const float2 s2 = any && (seen(key) || seen(key + 1)) ? __ldg(reinterpret_cast<const float2*>(sc)) : make_float2(0.f, 0.f);
            vs[nt] = make_float2(seen(key) ? s2.x : 0.f, seen(key + 1) ? s2.y : 0.f);
          }
        }
      }
    };

    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m[2] = {kNegInfF, kNegInfF}, l[2] = {0.f, 0.f};
    // ------------------------------------------------------------ units
    load_ids();
    load_k(u0 + warp);
    load_v(u0 + warp);
    for (int u = u0 + warp; u < u1; u += kWarpsF) {
      const bool refill = (u + kWarpsF - ids_at) / kWarpsF == 32;
      float x[kNT][4];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          if constexpr (KV8) {
            const uint4 k = kx[nt * 2 + (s >> 2)];
            const uint32_t codes = (s & 3) == 0 ? k.x : (s & 3) == 1 ? k.y : (s & 3) == 2 ? k.z : k.w;
            uint32_t lo, hi;
            e4m3x4_to_f16x4(codes, lo, hi);
            const float2 sc = make_float2(ks[nt], ks[nt]);
            mma_bf16_16816(x[nt], aq[s], scaled_bf16x2(lo, sc), scaled_bf16x2(hi, sc));
          } else {
            const uint4 k = kx[nt * 4 + (s >> 1)];
            mma_bf16_16816(x[nt], aq[s], s & 1 ? k.z : k.x, s & 1 ? k.w : k.y);
          }
        }
      }
      const int key0 = un.at(u) * kKeys;
      if (refill) {  // (V's loads of the next unit want its blocks too, this one's are under way)
        ids_at = u + kWarpsF;
        load_ids();
      }
      load_k(u + kWarpsF);
      // Every key of the unit seen by every row?
      const bool whole = key0 + kKeys <= min(sq.lk, pos0 + shift + 1) && (key0 >= pos0 + most - 1 + shift - p.window + 1 || key0 + kKeys <= p.sinks);
      float top[2] = {kNegInfF, kNegInfF};
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[nt][i] *= p.scale_log2;
          const int key = key0 + nt * 8 + 2 * t + (i & 1);
          if (!whole && !(key < lim[i >> 1] && (key >= from[i >> 1] || key < p.sinks))) x[nt][i] = kNegInfF;
          top[i >> 1] = fmaxf(top[i >> 1], x[nt][i]);
        }
      if (__any_sync(0xffffffffu, top[0] > m[0] + kSlackF || top[1] > m[1] + kSlackF)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float r = top[i];
          r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 1));
          r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 2));
          const float mn = fmaxf(m[i], r), a = m[i] == kNegInfF ? 0.f : fast_exp2(m[i] - mn);
          m[i] = mn;
          l[i] *= a;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j][2 * i] *= a;
            o[j][2 * i + 1] *= a;
          }
        }
      }
      uint32_t w[kNT][2];  // weights of rows g and g + 8
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ref = m[i] == kNegInfF ? 0.f : m[i];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const float a = fast_exp2(x[nt][2 * i] - ref), c = fast_exp2(x[nt][2 * i + 1] - ref);
          l[i] += a + c;
          w[nt][i] = pack_bf16x2(a, c);
        }
      }
#pragma unroll
      for (int kk = 0; kk < kNT / 2; ++kk) {
        const uint32_t a[4] = {w[2 * kk][0], w[2 * kk][1], w[2 * kk + 1][0], w[2 * kk + 1][1]};
        if constexpr (KV8) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // dims 16 g + 4 q ..
            uint32_t bb[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 r0 = vx[(2 * kk + h) * 2], r1 = vx[(2 * kk + h) * 2 + 1];
              const uint32_t c0 = q == 0 ? r0.x : q == 1 ? r0.y : q == 2 ? r0.z : r0.w, c1 = q == 0 ? r1.x : q == 1 ? r1.y : q == 2 ? r1.z : r1.w;
              uint32_t d0, d1, d2, d3;  // (first key, second key) of a dim
              e4m3x4_to_f16x4(__byte_perm(c0, c1, 0x5140), d0, d1);
              e4m3x4_to_f16x4(__byte_perm(c0, c1, 0x7362), d2, d3);
              bb[h][0] = scaled_bf16x2(d0, vs[2 * kk + h]);
              bb[h][1] = scaled_bf16x2(d1, vs[2 * kk + h]);
              bb[h][2] = scaled_bf16x2(d2, vs[2 * kk + h]);
              bb[h][3] = scaled_bf16x2(d3, vs[2 * kk + h]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) mma_bf16_16816(o[q * 4 + e], a, bb[0][e], bb[1][e]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // pieces g and g + 8
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              auto word = [&](int i) {
                const uint4 v = vx[i * 2 + h];
                return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
              };
#pragma unroll
              for (int e = 0; e < 2; ++e)
                mma_bf16_16816(o[h * 8 + q * 2 + e], a, __byte_perm(word(0), word(1), e ? 0x7632 : 0x5410),
                               __byte_perm(word(2), word(3), e ? 0x7632 : 0x5410));
            }
          }
        }
      }
      load_v(u + kWarpsF);
    }

    // ------------------------------------------------------------ the warps' states meet
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    __syncthreads();  // the last segment's have been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* row = state + (warp * 16 + g + 8 * i) * kRowF;
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)  // column 2 t + e of tile j: the dim that lane g = 2 t + e loaded as its j-th
          row[KV8 ? (2 * t + e) * 16 + j : (2 * t + e + 8 * (j >> 3)) * 8 + (j & 7)] = o[j][2 * i + e];
      if (t == 0) {
        ml[(warp * 16 + g + 8 * i) * 2] = m[i];
        ml[(warp * 16 + g + 8 * i) * 2 + 1] = l[i];
      }
    }
    __syncthreads();
    const int r = tid >> 4, d0 = (tid & 15) * 8;  // this thread's row and dims from here on
    float top = kNegInfF, sum = 0.f, y[8] = {};
    auto add = [&](const float* from_o, float fm, float fl, float ref) {  // ref: the largest maximum
      const float c = fm == kNegInfF ? (fl == 0.f ? 0.f : 1.f) : fast_exp2(fm - ref);  // (no maximum: no key, or NaN scores)
      sum += fl * c;
      const float4 a = *reinterpret_cast<const float4*>(from_o), e = *reinterpret_cast<const float4*>(from_o + 4);
      if (c != 0.f) {
        y[0] += a.x * c, y[1] += a.y * c, y[2] += a.z * c, y[3] += a.w * c;
        y[4] += e.x * c, y[5] += e.y * c, y[6] += e.z * c, y[7] += e.w * c;
      }
    };
#pragma unroll
    for (int w = 0; w < kWarpsF; ++w) top = fmaxf(top, ml[(w * 16 + r) * 2]);
#pragma unroll
    for (int w = 0; w < kWarpsF; ++w) add(state + (w * 16 + r) * kRowF + d0, ml[(w * 16 + r) * 2], ml[(w * 16 + r) * 2 + 1], top);
    bool write = true;
    if (u1 - u0 < un.n) {
      // Part of an item: its state to the workspace (a CTA starts at most one item that it does not end, and ends or
      // passes through at most one that it did not start).
      const int slot = 2 * blockIdx.x + (u0 == 0 ? 1 : 0);
      const int c0 = owner(item0), c1 = owner(item0 + un.n - 1);
      if (in_bounds(slot < p.slots && c1 < p.slots / 2, p.err)) {
        float* to = p.part_o + ((long long)slot * 16 + r) * 128 + d0;
        *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(y[4], y[5], y[6], y[7]);
        if ((tid & 15) == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * 16 + r) * 2) = make_float2(top, sum);
      }
      __syncthreads();
      if (tid == 0) {
        const int done = atomic_add_acq_rel_gpu(p.counters + c0, 1) == c1 - c0;
        if (done) p.counters[c0] = 0;  // as the next call finds it
        *last = done;
      }
      __syncthreads();
      write = *last != 0;
      if (write) {  // the last of its CTAs: all states, in order
        top = kNegInfF;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.f;
        auto slot_of = [&](int c) { return (long long)(2 * c + (c == c0 ? 1 : 0)) * 16 + r; };
        for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(p.part_ml + slot_of(c) * 2));
#pragma unroll 4
        for (int c = c0; c <= c1; ++c) {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(p.part_ml + slot_of(c) * 2));
          const float* from_o = p.part_o + slot_of(c) * 128 + d0;
          const float4 a = __ldcg(reinterpret_cast<const float4*>(from_o)), e = __ldcg(reinterpret_cast<const float4*>(from_o + 4));
          const float both[8] = {a.x, a.y, a.z, a.w, e.x, e.y, e.z, e.w};
          const float k = v.x == kNegInfF ? (v.y == 0.f ? 0.f : 1.f) : fast_exp2(v.x - top);
          sum += v.y * k;
          if (k != 0.f)
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += both[i] * k;
        }
      }
    }
    if (write && r < most * G) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      __nv_bfloat16* to = p.out + (long long)(sq.q0 + pos0 + r / G) * p.o_st + (long long)(kvh * G + r % G) * p.o_sh + d0;
      uint4 v = make_uint4(pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv), pack_bf16x2(y[4] * inv, y[5] * inv),
                           pack_bf16x2(y[6] * inv, y[7] * inv));
      if (sum == 0.f) v = make_uint4(0, 0, 0, 0);
      if (in_bounds(to >= p.out && to + 8 <= p.out + p.out_span, p.err)) *reinterpret_cast<uint4*>(to) = v;
    }
  }
}

template <bool KV8>
cudaError_t launch_few(const FewParams& p, int grid, bool pdl, cudaStream_t stream) {
  static int configured[64] = {0};  // the shared-memory opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(chunk_few_kernel<KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemF);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreadsF);
  cfg.dynamicSmemBytes = kSmemF;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, chunk_few_kernel<KV8>, p);
}

}  // namespace

cudaError_t launch_chunk_few(const FewParams& p, int grid, bool kv8, bool pdl, cudaStream_t stream) {
  return kv8 ? launch_few<true>(p, grid, pdl, stream) : launch_few<false>(p, grid, pdl, stream);
}

}  // namespace da
