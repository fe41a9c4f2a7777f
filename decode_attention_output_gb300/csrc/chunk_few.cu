// chunk_few.cu -- attention of a few new tokens of each sequence over a paged cache: decode_attn_chunk where sequences have
// one token, or a few drafted ones.
//
// An item is 8 or 16 rows of one (sequence, KV head): npos = floor(rows / G) query positions x the G heads that share the KV
// head.
// Its keys go by in units of 16 (e4m3: 32), those of the first `sinks` and from the window's beginning on. The units of all
// items, laid end to end, are cut into equal parts, one for each CTA (one an SM, or two half as large where items of e4m3 codes
// are many: one's products then hide the other's beginnings and ends; fewer where little is left to each), whatever the
// sequences' lengths: an item that lies in several CTAs leaves a state in the workspace from each, and the last of them
// to end joins them in order.
//
//  * Bound by the bytes of K and V. The 128-row tiles of prefill.cuh would be idle but for 16 rows and take 1.3 us
//    a tile of 128 keys, the time of one softmax, whatever its bytes; here a warp works on a unit of its own
//    (mma.sync) and those of a CTA meet at the item's end only. S^T = K Q^T and O^T = V^T P^T: keys and dims are the
//    instruction's 16 rows, queries its 8 columns, so that eight of them cost half of sixteen.
//  * A warp copies its units of K and V by TMA (4 KB each, a copy each where a block holds a unit), two units ahead and on
//    into the next item's: 16 KB a warp, 128 KB an SM on their way. Which of a row's dims meet which lane and step of the
//    matrix instructions is free as long as Q's follow: of a key, lane t of four takes the 16-byte pieces t, t + 4, ...; for V,
//    where an instruction wants two keys' values of one dim in a register, a lane takes one piece of two keys and exchanges halves
//    of its own registers. The copies' 128-byte swizzle lets eight lanes reach all banks in both.
//  * bf16: softmax as in prefill.cuh: the running maximum lags by up to 2^8, the weights enter P V as bf16, sums are fp32.
//  * e4m3: codes are widened to f16 (exact, half an instruction each; to bf16 with their scale 2.5, which set the pace: 270 us
//    for the 32 sequences). K's scale multiplies the score; q's rows become f16 over a power of two that puts the
//    largest under 2^15 (exact down to 2^-32 of it). V's scale joins the weight, w v f as f16: f, a power of two a row, keeps the
//    largest w v (of rows of V that are not all zero: those have a scale of 1 whatever the others have) between 1 and 2^8,
//    so that smaller ones are off by 2^-25 of it at most. The products are taken as (w v) f: v f can be infinite where w is 0.
// Measured (32 / 8 heads): four drafted tokens of each of 32 sequences over 8k, bf16 168 us (6.5 TB/s), e4m3 122, eight of each 170
// and 246 (two items of 16 rows, each of which widens all codes); one token each of 64 sequences over 16k, 64 / 8 heads, 615 us
// (7.0 TB/s) and 335; of 64 over 1k 56 and 43; of 256 sequences of 100 tokens 33 and 34; of one over 2k 10 and 11.
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kRowF = 132;       // floats of a row of the merge buffer (128 and padding)
constexpr int kMostParts = 48;   // of an item
constexpr int kAlignedMore = 16;  // units
constexpr float kSlackF = 8.f;   // log2 units the maximum may lag
constexpr float kVScaleUnit = 0x1p-8f;  // V's scales are held times this: a weight (up to 2^8) times one stays finite
constexpr float kNegInfF = -__builtin_huge_valf();

constexpr int kStagesF = 2;
constexpr uint32_t kHalfUnit = 4096;                // K or V of a unit
constexpr uint32_t kScalesF = 256, kUnitBytes = 2 * kHalfUnit;
// Shared memory of a CTA of WARPS: two units of each warp (K, V, scales of 32 keys), their barriers, the warps' states, the
// sequences' units (prefix sums)
template <int WARPS>
struct FewSmem {
  static constexpr size_t kScales = (size_t)WARPS * kStagesF * kUnitBytes;
  static constexpr size_t kBars = kScales + (size_t)WARPS * kStagesF * kScalesF;
  static constexpr size_t kMl = kBars + WARPS * kStagesF * 8;
  static constexpr size_t kState = (kMl + WARPS * 16 * 2 * 4 + 15) & ~(size_t)15;
  static constexpr size_t kLast = kState + (size_t)WARPS * 16 * kRowF * 4;
  static constexpr size_t kPrefix = kLast + 16;
  static constexpr size_t kAll = 1024 + kPrefix + (kMaxBatch + 1) * 8;
};
static_assert(FewSmem<8>::kAll <= kMaxDynSmem && 2 * (FewSmem<4>::kAll + 1024) <= kMaxDynSmem + 1024, "the kernel exceeds an SM's shared memory");

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

__device__ __forceinline__ uint4 lds_piece(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// The maximum over the eight lanes that hold other keys of the same rows.
__device__ __forceinline__ float max_of_keys(float r) {
  r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 4));
  r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 8));
  return fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 16));
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// 2^e, e clamped to what a float holds
__device__ __forceinline__ float power_of_2(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
// floor(log2 x) of a positive float (subnormal ones: -127)
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23 & 0xffu) - 127; }

// A sequence: its rows of q, its tokens, the first key of its first query's window.
struct Seq {
  int q0, lq, lk, lo;
};
__device__ __forceinline__ Seq sequence(const FewParams& p, int b) {
  Seq s;
  s.q0 = min(max(__ldg(p.cu + b), 0), p.Tq);
  s.lq = min(max(__ldg(p.cu + b + 1), s.q0), p.Tq) - s.q0;
  if (s.lq > p.most_lq) s.lq = 0;
  s.lk = min(max(__ldg(p.lens + b), 0), p.cap);
  s.lo = max(0, s.lk - s.lq - p.window + 1);
  return s;
}

// A segment: an item's units of one worker, from the flat unit f on and before f1 (ALONE: to the item's end).
struct Segment {
  int b, q0, lk, kvh, u0, u1, pos0, most, shift, end, low;
  long long item0;  // the item's first unit
  Units un;
};
template <int KEYS, bool ALONE>
__device__ __forceinline__ Segment segment_of(const FewParams& p, const long long* prefix, long long f, long long f1) {
  Segment s;
  s.b = 0;
  for (int step = p.B > 1 ? 1 << (31 - __clz(p.B - 1)) : 0; step > 0; step >>= 1)  // the last b with prefix[b] <= f
    if (s.b + step < p.B && prefix[s.b + step] <= f) s.b += step;
  const Seq sq = sequence(p, s.b);
  s.un = units_of<KEYS>(sq.lo, sq.lk, p.sinks);
  const long long within = f - prefix[s.b], item = within / s.un.n;
  const int rgs = (sq.lq + p.npos - 1) / p.npos;  // of a KV head one behind the other: their keys are in L2
  s.kvh = (int)(item / rgs);
  const int rg = (int)(item - (long long)s.kvh * rgs);
  s.u0 = (int)(within - item * s.un.n);
  s.u1 = ALONE ? s.un.n : (int)min((long long)s.un.n, s.u0 + (f1 - f));
  s.item0 = f - s.u0;
  s.q0 = sq.q0;
  s.lk = sq.lk;
  s.pos0 = rg * p.npos;  // its first query, and how many
  s.most = min(p.npos, sq.lq - s.pos0);
  s.shift = sq.lk - sq.lq;  // position of the sequence's first query
  s.end = min(sq.lk, s.pos0 + s.most + s.shift);       // keys that its last query sees
  s.low = max(0, s.pos0 + s.shift - p.window + 1);  // the first of its first query's window
  return s;
}

// Where segments are long the kernel's code stays in the instruction cache by being called, not inlined twice (one
// token each of eight sequences over 8k, e4m3: 39.7 us inlined, 38.3 called). Where each unit or two is a segment the call costs more than that
// (one token each of 256 sequences of 100: 39 us inlined, 41 called).
template <int KEYS>
__device__ __noinline__ Segment segment_called(const FewParams& p, const long long* prefix, long long f, long long f1) {
  return segment_of<KEYS, false>(p, prefix, f, f1);
}

// The items, or parts of them, of worker `me` of `workers`. ALONE: a worker is a warp and takes items as a whole; else it is a
// CTA, whose warps take an item's units in turn.
// NB: blocks of eight rows of an item
template <bool KV8, int NB, int WARPS, bool ALONE>
__device__ __forceinline__ void run_items(const FewParams& p, uint8_t* smem, const uint8_t* smem_raw, int workers, int me) {
  constexpr int kKeys = KV8 ? kFewKeys8 : kFewKeys16, kKT = kKeys / 16;  // keys of a unit, in tiles of 16
  constexpr float kUnitBack = KV8 ? 1.f / kVScaleUnit : 1.f;  // of an item's O
  constexpr int kRows = 8 * NB, kDims = kRows * 4 / WARPS;  // rows of an item; dims of a thread where states are joined
  const long long* prefix = reinterpret_cast<const long long*>(smem + FewSmem<WARPS>::kPrefix);
  float* state = reinterpret_cast<float*>(smem + FewSmem<WARPS>::kState);
  float* ml = reinterpret_cast<float*>(smem + FewSmem<WARPS>::kMl);
  int* last = reinterpret_cast<int*>(smem + FewSmem<WARPS>::kLast);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int G = p.G;
  const long long total = prefix[p.B];
  const int first = ALONE ? 0 : warp;             // this warp's units of a segment
  constexpr int step = ALONE ? 1 : WARPS;
  const long long each = total / workers;
  const int rest = (int)(total - each * workers);
  auto begin_of = [&](int c) { return each * c + (int)((unsigned)rest * (unsigned)c / (unsigned)workers); };  // total * c / workers
  auto owner = [&](long long f) { return (int)(((f + 1) * workers - 1) / total); };

  long long f1 = begin_of(me + 1);
  auto segment = [&](long long f) {
    if constexpr (ALONE) return segment_of<kKeys, true>(p, prefix, f, f1);
    else return segment_called<kKeys>(p, prefix, f, f1);
  };
  const uint32_t units = smem_u32(smem) + warp * kStagesF * kUnitBytes;
  const uint32_t scales = smem_u32(smem + FewSmem<WARPS>::kScales) + warp * kStagesF * kScalesF;
  const uint32_t bars = smem_u32(smem + FewSmem<WARPS>::kBars) + warp * kStagesF * 8;
  auto sm_ok = [&](uint32_t addr, uint32_t bytes) { return smem_in_bounds(smem_u32(smem_raw), addr, bytes, p.err); };

  // The loads, which run ahead of the products and on into the next segments: the segment, this warp's next unit of it, and the
  // blocks of both halves of 32 units from ids_at on, a unit a lane.
  struct {
    long long next;  // the first unit behind the segment
    Units un;
    int b, kvh, u, u1, end, low;
  } ld;
  int ids[2] = {-1, -1}, ids_at = 0, loaded = 0;
  auto begin_loads = [&](const Segment& s, long long f) {
    ld.next = f + s.u1 - s.u0;
    ld.un = s.un;
    ld.b = s.b;
    ld.kvh = s.kvh;
    ld.u = s.u0 + first;
    ld.u1 = s.u1;
    ld.end = s.end;
    ld.low = s.low;
    ids_at = -1;
  };
  auto load_unit = [&] {
    while (ld.u >= ld.u1 && ld.next < f1) begin_loads(segment(ld.next), ld.next);
    if (ld.u >= ld.u1) return;  // nothing is left
    if (ids_at < 0 || (ld.u - ids_at) / step == 32) {
      ids_at = ld.u;
      const int u = ids_at + lane * step, key = ld.un.at(u) * kKeys;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k0 = key + i * (kKeys / 2), k1 = k0 + kKeys / 2 - 1;
        const bool need = u < ld.u1 && k0 < ld.end && (k0 < p.sinks || k1 >= ld.low);  // some key of the half is seen
        const long long at = ld.b * p.bt_stride + (k0 >> p.block_shift);
        ids[i] = need && in_bounds(at < p.table_span, p.err) ? __ldg(p.table + at) : -1;
        if (need && (unsigned)ids[i] >= (unsigned)p.num_blocks) atomicOr(p.err, kErrBlockTable);
        // halves that no row of the item sees, and blocks that are none of the pool's, are past its end: zeros
        if ((unsigned)ids[i] >= (unsigned)p.num_blocks) ids[i] = p.num_blocks;
      }
    }
    const int src = (ld.u - ids_at) / step, key0 = ld.un.at(ld.u) * kKeys, row = key0 & ((1 << p.block_shift) - 1);
    const int id0 = __shfl_sync(0xffffffffu, ids[0], src), id1 = __shfl_sync(0xffffffffu, ids[1], src);
    // A copy of the unit, or one of each half where a block holds no more. (Where one half only is seen, the copy of both
    // brings the block's other rows too; they are masked.)
    const bool split = (1 << p.block_shift) < kKeys;
    const int st = loaded & 1;
    const uint32_t to = units + st * kUnitBytes, bar = bars + st * 8, sc = scales + st * kScalesF;
    __syncwarp();  // the stage has been read
    if (lane == 0 && sm_ok(to, kUnitBytes) && sm_ok(sc, kScalesF) && in_bounds(ld.kvh < p.Hkv, p.err)) {
      mbar_arrive_expect_tx(bar, kUnitBytes + (KV8 ? kScalesF : 0));
      const int blk = split ? id0 : min(id0, id1);
      tma_load_5d(to, &p.tm_k, bar, 0, row, 0, ld.kvh, blk);
      tma_load_5d(to + kHalfUnit, &p.tm_v, bar, 0, row, 0, ld.kvh, blk);
      if (KV8) tma_load_4d(sc, &p.tm_scales, bar, row, 0, ld.kvh, blk);
      if (split) {
        const int row1 = (key0 + kKeys / 2) & ((1 << p.block_shift) - 1);
        tma_load_5d(to + kHalfUnit / 2, &p.tm_k, bar, 0, row1, 0, ld.kvh, id1);
        tma_load_5d(to + kHalfUnit + kHalfUnit / 2, &p.tm_v, bar, 0, row1, 0, ld.kvh, id1);
        if (KV8) tma_load_4d(sc + kScalesF / 2, &p.tm_scales, bar, row1, 0, ld.kvh, id1);
      }
    }
    __syncwarp();
    ++loaded;
    ld.u += step;
  };

  long long f = begin_of(me);
  if (ALONE) {  // items as a whole: those that begin in this warp's share
    auto next_item = [&](long long x) {
      if (x >= total) return total;
      const Segment s = segment(x);
      return s.u0 == 0 ? x : s.item0 + s.un.n;
    };
    f = next_item(f);
    f1 = next_item(f1);
  }
  if (f >= f1) return;
  // Addresses in a stage. K: key g of every eight, pieces t and t + 4 of 128 bytes, in the order that gives two keys' lanes
  // different banks. V: keys 2 t and 2 t + 1, piece g. Scales: a copy's K scales, then its V scales.
  const bool split = (1 << p.block_shift) < kKeys, odd = g & 1;
  const uint32_t eight = !KV8 && split ? 2048 : 1024;   // from eight keys to the next
  const uint32_t second = split ? 1024 : 2048;          // bf16: from a row's first 64 dims to the others
  const uint32_t k_at = g * 128 + (((t + 4 * (g & 1)) ^ g) << 4);
  const uint32_t v_at = 2 * t * 128 + ((g ^ (2 * t)) << 4), v_at1 = (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) << 4);
  // K's scale of key g of the nt-th eight; V's lies `scale_v` behind
  const uint32_t scale_v = split ? 64 : 128;
  auto scale_at = [&](int nt) { return (uint32_t)(split ? (nt >> 1) * 128 + (nt & 1) * 32 : nt * 32) + g * 4; };

  Segment sg = segment(f);
  begin_loads(sg, f);
#pragma unroll 1
  for (int i = 0; i < kStagesF; ++i) load_unit();
  int used = 0;       // units taken
  bool alive = true;  // no wait has run out
  while (true) {
    // Q, in the order of dims that K's pieces give: row g of each block of eight. e4m3: f16 over a power of two.
    uint32_t bq[NB][8][2];
    int e_row[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + g, pos = sg.pos0 + r / G;
      const bool ok = r < sg.most * G;
      const __nv_bfloat16* row = p.q + (long long)(sg.q0 + pos) * p.q_st + (long long)(sg.kvh * G + r % G) * p.q_sh;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int dim = KV8 ? (t + 4 * (s >> 2)) * 16 + (s & 3) * 4 : (t + 4 * (s >> 1)) * 8 + (s & 1) * 4;
        uint2 v = make_uint2(0, 0);
        if (ok && in_bounds(row + 128 <= p.q + p.q_span, p.err)) v = __ldg(reinterpret_cast<const uint2*>(row + dim));
        bq[nb][s][0] = v.x;
        bq[nb][s][1] = v.y;
      }
      e_row[nb] = 0;
      if constexpr (KV8) {
        unsigned top = 0;  // the row's largest magnitude, a bf16 pattern
#pragma unroll
        for (int s = 0; s < 8; ++s) top = __vmaxu2(top, __vmaxu2(bq[nb][s][0] & 0x7fff7fffu, bq[nb][s][1] & 0x7fff7fffu));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top & 0xffffu, top >> 16);
        // (a row of zeros, or one with an infinity or NaN: as it is; in two halves, as 2^-112 and less are no floats)
        const int e = top == 0 || top >= 0x7f80u ? 0 : 14 - ((int)(top >> 7) - 127);
        const float a = power_of_2(e / 2), c = power_of_2(e - e / 2);
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) bq[nb][s][k] = pack_f16x2(bf16lo_to_f32(bq[nb][s][k]) * a * c, bf16hi_to_f32(bq[nb][s][k]) * a * c);
        e_row[nb] = e;
      }
    }
    // This lane's scores: keys g and g + 8 of every sixteen, rows 2 t and 2 t + 1 of every eight. The rows see keys before lim
    // and from `from` on (or before sinks); factor turns products into log2 units.
    int lim[NB][2], from[NB][2];
    float factor[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nb * 8 + 2 * t + e, pos = sg.pos0 + r / G;
        lim[nb][e] = r < sg.most * G ? min(sg.lk, pos + sg.shift + 1) : 0;
        from[nb][e] = pos + sg.shift - p.window + 1;
        factor[nb][e] = p.scale_log2;
        if constexpr (KV8) {
          const int x = __shfl_sync(0xffffffffu, e_row[nb], (2 * t + e) * 4);
          factor[nb][e] = fminf(fmaxf(p.scale_log2 * power_of_2(-(x / 2)) * power_of_2(-(x - x / 2)), -3.4e38f), 3.4e38f);
        }
      }
    float o[NB][8][4], m[NB][2], l[NB][2];
    float fv[NB][2], largest[NB][2];  // e4m3: V's factor, and the largest weight times V scale (times kVScaleUnit) so far
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[nb][j][0] = o[nb][j][1] = o[nb][j][2] = o[nb][j][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nb][e] = kNegInfF;
        l[nb][e] = 0.f;
        fv[nb][e] = 1.f / kVScaleUnit;
        largest[nb][e] = 0.f;
      }
    }
    const int all_before = min(sg.lk, sg.pos0 + sg.shift + 1), all_from = sg.pos0 + sg.most - 1 + sg.shift - p.window + 1;
    for (int u = sg.u0 + first; u < sg.u1 && alive; u += step) {
      const int st = used & 1;
      alive = mbar_wait_bounded(bars + st * 8, used >> 1 & 1, p.err, kErrWaitFull, nullptr);
      alive = __all_sync(0xffffffffu, alive);
      ++used;
      const uint32_t kv = units + st * kUnitBytes, sc = scales + st * kScalesF;
      float x[kKT][NB][4];
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) x[kt][nb][0] = x[kt][nb][1] = x[kt][nb][2] = x[kt][nb][3] = 0.f;
      // S^T = K Q^T: sixteen keys by eight rows
#pragma unroll
      for (int h = 0; h < (KV8 ? 1 : 2); ++h) {
        uint4 k[kKT][2][2];  // pieces t and t + 4 of keys g and g + 8
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = kv + (2 * kt + i) * eight + h * second + k_at;
            const uint4 a = lds_piece(at), c = lds_piece(at ^ 64);
            k[kt][i][0] = odd ? c : a;
            k[kt][i][1] = odd ? a : c;
          }
#pragma unroll
        for (int s = 0; s < (KV8 ? 8 : 4); ++s)
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt) {
            uint32_t a[4];
            if constexpr (KV8) {
              e4m3x4_to_f16x4(word_of(k[kt][0][s >> 2], s & 3), a[0], a[2]);
              e4m3x4_to_f16x4(word_of(k[kt][1][s >> 2], s & 3), a[1], a[3]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_f16_16816(x[kt][nb], a, bq[nb][s][0], bq[nb][s][1]);
            } else {
              a[0] = word_of(k[kt][0][s >> 1], 2 * (s & 1));
              a[1] = word_of(k[kt][1][s >> 1], 2 * (s & 1));
              a[2] = word_of(k[kt][0][s >> 1], 2 * (s & 1) + 1);
              a[3] = word_of(k[kt][1][s >> 1], 2 * (s & 1) + 1);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_bf16_16816(x[kt][nb], a, bq[nb][h * 4 + s][0], bq[nb][h * 4 + s][1]);
            }
          }
      }
      const int key0 = sg.un.at(u) * kKeys;
      auto seen = [&](int key) { return key < sg.end && (key >= sg.low || key < p.sinks); };  // by some row of the item
      const bool whole = key0 + kKeys <= all_before && (key0 >= all_from || key0 + kKeys <= p.sinks);  // every key seen by every row
      float top[NB][2];
      bool over = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        top[nb][0] = top[nb][1] = kNegInfF;
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& v = x[kt][nb][i];
            v *= factor[nb][i & 1];
            if (KV8) v *= lds_f32(sc + scale_at(2 * kt + (i >> 1)));
            const int key = key0 + kt * 16 + 8 * (i >> 1) + g;
            if (!whole && !(key < lim[nb][i & 1] && (key >= from[nb][i & 1] || key < p.sinks))) v = kNegInfF;
            top[nb][i & 1] = fmaxf(top[nb][i & 1], v);
          }
        over = over || top[nb][0] > m[nb][0] + kSlackF || top[nb][1] > m[nb][1] + kSlackF;
      }
      const bool grow = __any_sync(0xffffffffu, over);
      float a[NB][2];  // what the sums and O so far are worth against the new maximum
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          a[nb][e] = 1.f;
          if (grow) {
            const float mn = fmaxf(m[nb][e], max_of_keys(top[nb][e]));
            a[nb][e] = m[nb][e] == kNegInfF ? 0.f : fast_exp2(m[nb][e] - mn);
            m[nb][e] = mn;
            l[nb][e] *= a[nb][e];
            largest[nb][e] *= a[nb][e];
          }
          const float ref = m[nb][e] == kNegInfF ? 0.f : m[nb][e];
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int i = e; i < 4; i += 2) {
              x[kt][nb][i] = fast_exp2(x[kt][nb][i] - ref);
              l[nb][e] += x[kt][nb][i];
            }
        }
      if constexpr (KV8) {
        float vs[kKT][2];
        bool redo = grow;
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            vs[kt][i] = lds_f32(sc + scale_at(2 * kt + i) + scale_v) * kVScaleUnit;
            if (!whole && !seen(key0 + kt * 16 + 8 * i + g)) vs[kt][i] = 0.f;  // (0 times a scale that belongs to no key is not 0)
          }
        // The weight first: of a key that a row does not see it is 0, and the scale times the row's factor may be infinite.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[kt][nb][i] *= vs[kt][i >> 1];
        auto big = [&](int nb, int e) {  // the largest weight times V scale of this lane's
          float r = 0.f;
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt) r = fmaxf(r, fmaxf(fabsf(x[kt][nb][e]), fabsf(x[kt][nb][2 + e])));
          return r;
        };
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float r = big(nb, e);
            redo = redo || (largest[nb][e] == 0.f && r > 0.f) || r * fv[nb][e] > 256.f;
          }
        if (__any_sync(0xffffffffu, redo)) {
          unsigned some = 0;  // keys 2 t and 2 t + 1 of every eight: does V's row hold a code that is not 0?
#pragma unroll
          for (int k = 0; k < 4 * kKT; ++k) {
            const uint4 v = lds_piece(kv + kHalfUnit + (k >> 1) * eight + (k & 1 ? v_at1 : v_at));
            some |= ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) ? 1u << k : 0u;
          }
          some |= __shfl_xor_sync(0xffffffffu, some, 4);
          some |= __shfl_xor_sync(0xffffffffu, some, 8);
          some |= __shfl_xor_sync(0xffffffffu, some, 16);
          some = __shfl_sync(0xffffffffu, some, g >> 1) >> (g & 1);  // key g's of every eight
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(some >> (2 * (2 * kt + (i >> 1))) & 1u))
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) x[kt][nb][i] = 0.f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              largest[nb][e] = fmaxf(largest[nb][e], max_of_keys(big(nb, e)));
              float to = fv[nb][e];  // the largest times it stays between 1 and 2^8
              if (largest[nb][e] > 0.f && !(largest[nb][e] * to >= 1.f && largest[nb][e] * to <= 256.f)) to = power_of_2(-exponent_of(largest[nb][e]));
              a[nb][e] *= fminf(to / fv[nb][e], 0x1p127f);
              fv[nb][e] = to;
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[kt][nb][i] *= fv[nb][i & 1];
      }
      // V: key 2 t + k of the nt-th eight, piece g. What no row sees may hold anything: zeros.
      auto load_v = [&](int nt, int k, uint32_t off) {
        uint4 v = lds_piece(kv + kHalfUnit + nt * eight + off + (k ? v_at1 : v_at));
        if (!whole && !seen(key0 + nt * 8 + 2 * t + k)) v = make_uint4(0, 0, 0, 0);
        return v;
      };
      bool scaled = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) scaled = scaled || a[nb][0] != 1.f || a[nb][1] != 1.f;
      if (__any_sync(0xffffffffu, scaled)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nb][j][i] *= a[nb][i & 1];
      }
      // O^T += V^T P^T: sixteen dims by eight rows. A lane's dims of a tile are neighbours of its piece.
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt) {
        uint32_t w[NB][2];  // weights of keys 2 t, 2 t + 1 of both eights, row g
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            w[nb][i] = movmatrix_trans(KV8 ? pack_f16x2(x[kt][nb][2 * i], x[kt][nb][2 * i + 1]) : pack_bf16x2(x[kt][nb][2 * i], x[kt][nb][2 * i + 1]));
#pragma unroll
        for (int h = 0; h < (KV8 ? 1 : 2); ++h) {  // bf16: pieces g and g + 8
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = load_v(2 * kt + (i >> 1), i & 1, h * second);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (KV8) {
              uint32_t b[2][4];  // (first key, second key) of dims 16 g + 4 q ..
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t c0 = word_of(v[2 * i], q), c1 = word_of(v[2 * i + 1], q);
                e4m3x4_to_f16x4(__byte_perm(c0, c1, 0x5140), b[i][0], b[i][1]);
                e4m3x4_to_f16x4(__byte_perm(c0, c1, 0x7362), b[i][2], b[i][3]);
              }
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const uint32_t d[4] = {b[0][e], b[0][e + 1], b[1][e], b[1][e + 1]};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_f16_16816(o[nb][q * 2 + (e >> 1)], d, w[nb][0], w[nb][1]);
              }
            } else {
              uint32_t d[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                d[i] = __byte_perm(word_of(v[i & 2], q), word_of(v[(i & 2) + 1], q), i & 1 ? 0x7632 : 0x5410);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_bf16_16816(o[nb][h * 4 + q], d, w[nb][0], w[nb][1]);
            }
          }
        }
      }
      if (alive) load_unit();
    }

    // ------------------------------------------------------------ the warps' states meet
    f += sg.u1 - sg.u0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 4);
        l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 8);
        l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 16);
      }
    if (ALONE) {  // (the pairs of dims of a piece are neighbours)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nb * 8 + 2 * t + e;
          const float inv = l[nb][e] == 0.f ? 0.f : kUnitBack / l[nb][e], back = KV8 ? 1.f / fv[nb][e] : 1.f;
          __nv_bfloat16* to = p.out + (long long)(sg.q0 + sg.pos0 + r / G) * p.o_st + (long long)(sg.kvh * G + r % G) * p.o_sh;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = l[nb][e] == 0.f ? 0u : pack_bf16x2(o[nb][h * 4 + q][e] * back * inv, o[nb][h * 4 + q][2 + e] * back * inv);
            __nv_bfloat16* at = to + (KV8 ? 16 * g + 8 * h : (g + 8 * h) * 8);
            if (r < sg.most * G && in_bounds(at >= p.out && at + 8 <= p.out + p.out_span, p.err))
              *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      if (f >= f1) break;
      sg = segment(f);
      continue;
    }
    __syncthreads();  // the last segment's have been read
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = warp * kRows + nb * 8 + 2 * t + e;
        const float back = KV8 ? 1.f / fv[nb][e] : 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)  // (the pair of dims whose words made tile j)
          *reinterpret_cast<float2*>(state + r * kRowF + (KV8 ? 16 * g + 2 * j : (g + 8 * (j >> 2)) * 8 + 2 * (j & 3))) =
              make_float2(o[nb][j][e] * back, o[nb][j][2 + e] * back);
        if (g == 0) *reinterpret_cast<float2*>(ml + r * 2) = make_float2(m[nb][e], l[nb][e]);
      }
    __syncthreads();
    const int r = tid / (128 / kDims), d0 = tid % (128 / kDims) * kDims;  // this thread's row and dims from here on
    float top = kNegInfF, sum = 0.f, y[kDims] = {};
    auto add = [&](const float4* c, float pm, float pl) {  // a state's O, maximum and sum; top: the largest maximum
      const float k = pm == kNegInfF ? (pl == 0.f ? 0.f : 1.f) : fast_exp2(pm - top);  // (no maximum: no key, or NaN scores)
      sum += pl * k;
      if (k != 0.f)
#pragma unroll
        for (int i = 0; i < kDims; i += 4) {
          y[i] += c[i / 4].x * k, y[i + 1] += c[i / 4].y * k;
          y[i + 2] += c[i / 4].z * k, y[i + 3] += c[i / 4].w * k;
        }
    };
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[(w * kRows + r) * 2]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 s = *reinterpret_cast<const float2*>(ml + (w * kRows + r) * 2);
      add(reinterpret_cast<const float4*>(state + (w * kRows + r) * kRowF + d0), s.x, s.y);
    }
    bool write = true;
    if (sg.u1 - sg.u0 < sg.un.n) {
      // Part of an item: its state to the workspace (a CTA starts at most one item that it does not end, and ends or
      // passes through at most one that it did not start).
      const int slot = 2 * blockIdx.x + (sg.u0 == 0 ? 1 : 0);
      const int c0 = owner(sg.item0), c1 = owner(sg.item0 + sg.un.n - 1);
      if (in_bounds(slot < p.slots && c1 < p.slots / 2, p.err)) {
        float* to = p.part_o + ((long long)slot * kRows + r) * 128 + d0;
#pragma unroll
        for (int i = 0; i < kDims; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        if (d0 == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * kRows + r) * 2) = make_float2(top, sum);
      }
      __syncthreads();
      if (tid == 0) {
        const int ended = atomic_add_acq_rel_gpu(p.counters + c0, 1) == c1 - c0;
        if (ended) p.counters[c0] = 0;  // as the next call finds it
        *last = ended;
      }
      __syncthreads();
      write = *last != 0;
      if (write && r < sg.most * G) {  // the last of its CTAs: all states, in order
        auto slot_of = [&](int c) { return (long long)(2 * c + (c == c0 ? 1 : 0)) * kRows + r; };
        top = kNegInfF;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kDims; ++i) y[i] = 0.f;
#pragma unroll 8
        for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(p.part_ml + slot_of(c) * 2));
#pragma unroll 8
        for (int c = c0; c <= c1; ++c) {
          const float2 s = __ldcg(reinterpret_cast<const float2*>(p.part_ml + slot_of(c) * 2));
          float4 part[kDims / 4];
#pragma unroll
          for (int i = 0; i < kDims / 4; ++i) part[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + slot_of(c) * 128 + d0) + i);
          add(part, s.x, s.y);
        }
      }
    }
    if (write && r < sg.most * G) {
      const float inv = sum == 0.f ? 0.f : kUnitBack / sum;
      __nv_bfloat16* to = p.out + (long long)(sg.q0 + sg.pos0 + r / G) * p.o_st + (long long)(sg.kvh * G + r % G) * p.o_sh + d0;
      if (in_bounds(to >= p.out && to + kDims <= p.out + p.out_span, p.err))
#pragma unroll
        for (int i = 0; i < kDims; i += 4)
          *reinterpret_cast<uint2*>(to + i) =
              sum == 0.f ? make_uint2(0, 0) : make_uint2(pack_bf16x2(y[i] * inv, y[i + 1] * inv), pack_bf16x2(y[i + 2] * inv, y[i + 3] * inv));
    }
    if (f >= f1) break;
    sg = segment(f);
  }
  for (; used < loaded; ++used)  // (a wait has run out: what is still on its way must not land behind the CTA's end)
    mbar_wait_bounded(bars + (used & 1) * 8, used >> 1 & 1, p.err, kErrWaitDrain, nullptr, kWaitLimitNs / 10);
}

template <bool KV8, int NB, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 8 / WARPS) chunk_few_kernel(const __grid_constant__ FewParams p) {
  constexpr int kKeys = KV8 ? kFewKeys8 : kFewKeys16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  long long* prefix = reinterpret_cast<long long*>(smem + FewSmem<WARPS>::kPrefix);
  int* last = reinterpret_cast<int*>(smem + FewSmem<WARPS>::kLast);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, npos = p.npos;
  if (lane == 0) {
    for (int i = 0; i < kStagesF; ++i) mbar_init(smem_u32(smem + FewSmem<WARPS>::kBars) + (warp * kStagesF + i) * 8, 1);
    fence_barrier_init();
    if (warp == 0) {
      prefetch_tensormap(&p.tm_k);
      prefetch_tensormap(&p.tm_v);
      if (KV8) prefetch_tensormap(&p.tm_scales);
    }
  }
  pdl_wait_primary();

  if (tid == 0) last[0] = last[1] = 0;
  __syncthreads();
  for (int b = tid; b < p.B; b += WARPS * 32) {
    const Seq s = sequence(p, b);
    const int n = units_of<kKeys>(s.lo, s.lk, p.sinks).n;
    prefix[b + 1] = (long long)((s.lq + npos - 1) / npos) * p.Hkv * n;
    if (s.lq > 0) {
      atomicMax(last, n);
      atomicAdd(last + 1, (s.lq + npos - 1) / npos * p.Hkv);
    }
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
  if (total == 0) return;
  const int longest = last[0];
  // As many CTAs take part as leave each 256 keys, and the longest item in 48 parts at most: one CTA joins them
  int workers = (int)min((long long)gridDim.x, max(total / max(p.least, longest / kMostParts), 1ll));
  // Items all alike to the unit (one sequence's, or sequences of one length) and few: so many CTAs that none has parts of two, of which each costs it 5 us, if that leaves
  // none many units more (one token over 2k, e4m3, 65 units of each of 8 heads: 16.1 -> 10.7 us)
  const int items = last[1], whole = items > 0 ? workers / items * items : 0;
  if (whole > 0 && total == (long long)longest * items && total / whole - total / workers <= kAlignedMore) workers = whole;
  // Many short items: a warp each, from its first unit to its last, and nothing to join. In units a warp, that takes the
  // longer of its share and an item, and one more in part; items shared by a CTA's warps cost the time of two units
  // each on top. (256 sequences of 100 tokens, 8 KV heads: 86 us by CTAs.)
  const long long share = total / (workers * WARPS);
  const bool alone = max(share, (long long)longest) + longest / 2 < share + 2ll * (last[1] / workers + 1);
  if (alone) run_items<KV8, NB, WARPS, true>(p, smem, smem_raw, gridDim.x * WARPS, warp * gridDim.x + blockIdx.x);
  else if ((int)blockIdx.x < workers) run_items<KV8, NB, WARPS, false>(p, smem, smem_raw, workers, blockIdx.x);
}

template <bool KV8, int NB, int WARPS>
cudaError_t launch_few(const FewParams& p, int grid, bool pdl, cudaStream_t stream) {
  static int configured[64] = {0};  // the shared-memory opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(chunk_few_kernel<KV8, NB, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FewSmem<WARPS>::kAll);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = FewSmem<WARPS>::kAll;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, chunk_few_kernel<KV8, NB, WARPS>, p);
}

}  // namespace

cudaError_t launch_chunk_few(const FewParams& p, int grid, bool kv8, int rows, int warps, bool pdl, cudaStream_t stream) {
  if (!kv8) return rows == 8 ? launch_few<false, 1, 8>(p, grid, pdl, stream) : launch_few<false, 2, 8>(p, grid, pdl, stream);
  if (warps == 4) return rows == 8 ? launch_few<true, 1, 4>(p, grid, pdl, stream) : launch_few<true, 2, 4>(p, grid, pdl, stream);
  return rows == 8 ? launch_few<true, 1, 8>(p, grid, pdl, stream) : launch_few<true, 2, 8>(p, grid, pdl, stream);
}

}  // namespace da
