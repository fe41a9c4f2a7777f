// prefill.cuh -- causal attention of packed queries on the 5th-generation tensor cores: over packed prompts
// (prefill.cu) or over a paged cache (prefill_paged.cu), with a window and a few first tokens if asked for.
//
// For query i of a sequence (Lq queries, the last of its Lk tokens) and query head h:
//   S_ij = q_i . k_j (KV head h / G),  j < i + Lk - Lq + 1
//   O_i  = sum_j 2^(s S_ij - m_i) v_j / sum_j 2^(s S_ij - m_i),   s = scale * log2 e.
//
// Work item: 256 rows of one (sequence, KV head), as two tiles of 128: a tile's rows are
// npos = floor(128 / G) query positions x the G heads that share the KV head, so both tiles
// use every K and V tile that is brought in, whatever G is, and short prompts fill tiles.
// Items are taken heaviest (last positions) first within each sequence: the grid has a CTA per
// item, and a CTA that runs takes over the next one that has not started (cluster launch
// control), so that items of very different length even out and set-up and pipeline carry on
// across them (taking items blockIdx, blockIdx + gridDim, ... left 16 ragged prompts at 75 steps
// on the longest CTA of 62 on average, 8192 tokens at 476 of 445).
//
//  * tcgen05.mma M = N = 128: S = Q K^T from shared memory into TMEM, then O += P V with P
//    (bf16) in TMEM and V as the N-major B operand. TMEM, all 512 columns: one S (128), a P
//    for each tile (64 each), an O for each tile (128 each).
//  * The work is a stream of steps (item, K/V tile) that runs on across items, through four
//    parties that only wait for data: one warp issues S = Q K^T for the two tiles in turn, a
//    warpgroup per tile does the softmax, another warp issues O += P V, a producer loads. A
//    softmax thread holds one row (no shuffles; the row's maximum, sum and O correction are
//    one thread's), takes its S into registers and frees it at once. An item's O is stored
//    when its tile's next step has its weights.
//  * A step's MMAs compute for 2048 cycles and keep the tensor pipe busy for 86% of it (2400
//    cycles). One issuing warp, with P over its S (PV(r), then S(r + 1)), took 2860: each side
//    waited for the other in turn, and every wait costs an issuing warp some 200 cycles in which
//    nothing else is issued. Issued by one lane in a branch, an MMA took 100 cycles.
//  * The running maximum lags as in the decode kernel: O in TMEM is only rescaled when a row's
//    maximum grows by more than 2^8, by the thread that owns the row.
//  * With few rows over many keys (a few new tokens of long sequences) there are fewer items
//    than SMs: each is then cut into parts of its K/V tiles, which leave fp32 (O, m, l) in the
//    workspace, and a second kernel joins them in order.
//  * One producer warp streams K and V tiles (32 KB) by TMA through a ring of five stages, in
//    the order of their use; it also finds the items (a scan of the offsets) and passes them on.
//    A stage takes K and V tiles in turn and has a "full" barrier for each: a wait for the parity of
//    one that both shared could pass on the tile before the one that it waits for.
//  * With a window an item takes tiles from its first row's first key on, not from a multiple of 128 (16
//    ragged prompts, window 777: 175 -> 166 us; pages are taken by whole boxes, from a multiple); the first
//    keys, where they are few, lie in its first tile before that key, for which there would else be a tile
//    more (a window of 1024, 4 first keys: 457 -> 441 us).
// Measured: 8192 tokens, 64 / 8 heads 667 us (1.65 PFLOP/s; a short run, before the power limit
// lowers the clock, 581 us); four chunks of 512 over 7.7k 180 us (1.48); 16 ragged prompts of up
// to 2048 112 us (1.09): a step costs 1.2 us, an item 2.8 us more (its output, the diagonal's
// masks, the hand-over), of which 16 ragged prompts have 11 on each SM. In a window: 16384 tokens, 64 / 8 heads, window 1024,
// 4 first keys 446 to 454 us under the power limit, 16 ragged prompts of up to 2048, 32 / 8 heads,
// window 777 167 to 169: nine and seven steps an item, and the softmax warps, which also store the last item's
// output, are busy for nine tenths of them.
#pragma once
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace da {
namespace {

enum KeySource {
  kPackedKeys,  // rows of k and v, laid end to end
  kPages16,     // a paged bf16 cache
  kGathered     // a paged cache's tokens as a kernel before this one has laid them out (chunk_gather.cu)
};

constexpr int kN = 128;                         // keys per tile
constexpr uint32_t kHalf = 128 * 128;           // 128 rows x 64 dims bf16
constexpr uint32_t kTileP = 2 * kHalf;          // 128 rows x 128 dims
constexpr int kSoftWarps = 8;                   // four per tile
constexpr float kSlackP = 8.f;                  // log2 units the maximum may lag
constexpr float kNegInfP = -__builtin_huge_valf();

struct Item {  // in shared memory, as ints
  int lq, lk, q0, k0, p0, kvh;  // lq < 0: no more items
  int j0, end0, end1;           // K/V tiles from j0 on, to the end of each tile of rows
  int clear;                    // the V tile whose end is another sequence's (-1: none)
  int part;                     // of the item (-1: the item is whole)
  // With a window, j0, end0 and end1 count the tiles that some row of the item sees: tile j is the one of
  // keys 128 j .. of the sequence while j < ns, and the one of 128 j + skip .. from there on. lo: the
  // least key in the first row's window. merged: so many rows of the first tile, which lie before lo, hold the sequence's first keys.
  int ns, skip, lo, merged;
};
constexpr int kItems = 4;  // items on their way from the producer
constexpr int kStagesP = 5;  // K / V ring
enum Bar {
  kQFull,                          // per tile: queries landed / free
  kQEmpty = kQFull + 2,
  kSFull = kQEmpty + 2,            // per tile: its S is in TMEM
  kPFull = kSFull + 2,             // per tile: its P is in TMEM, O is corrected
  kPvDone = kPFull + 2,            // per tile: its PV has completed
  kSFree = kPvDone + 2,            // the S columns have been read
  kSIssued,                        // per tile: the MMAs of its S are on their way
  kNext = kSIssued + 2,                           // the next item's index has been answered
  kItemFull, kItemEmpty = kItemFull + kItems,
  // A stage holds a K tile and a V tile in turn, for an issuer each, who tests only its own tiles: with one barrier for both
  // the test would also pass while the other's tile before it is still on its way.
  kKFull = kItemEmpty + kItems, kVFull = kKFull + kStagesP, kKvEmpty = kVFull + kStagesP,
  kBars = kKvEmpty + kStagesP
};
constexpr uint32_t kTmemP = 128, kTmemO = 256;  // columns: S, P0, P1, O0, O1

// two softmax warpgroups and a third: the producer, the issuers of S and of PV, and a spare warp
constexpr int kThreadsP = (kSoftWarps + 4) * 32;
// registers a thread: 168 at launch; the third warpgroup gives 80 of its own to the softmax,
// whose threads hold a row of 128 scores (2 * 208 + 88 = 3 * 168)
constexpr int kRegsSoft = 208, kRegsRest = 88;
constexpr size_t kOffRing = 2 * kTileP;
constexpr size_t kOffBars = kOffRing + (size_t)kStagesP * kTileP;
constexpr size_t kOffItems = kOffBars + kBars * 8;
constexpr size_t kOffNext = (kOffItems + kItems * sizeof(Item) + 15) & ~(size_t)15;  // answer to the request for the next item
constexpr size_t kOffFlags = kOffNext + 16;
constexpr size_t kSmemP = 1024 + kOffFlags + 16;
static_assert(kSmemP <= kMaxDynSmem, "prefill kernel exceeds 227 KB of shared memory");

// K/V tiles that npos query positions from `first` on need, of Lq and Lk tokens: those up to
// the last position's last key.
__device__ __forceinline__ int kv_tiles(int first, int npos, int lq, int lk) {
  const int last = min(first + npos, lq) - 1;
  return first < lq ? max(0, last + lk - lq + kN) / kN : 0;
}
// Parts that an item of `top` tiles is cut into, and the first tile of one. Four tiles or more
// each, and none below twelve, where leaving and joining the parts costs more than they save
// (Hq 32, Hkv 8, 64 new tokens over 1200: 17.4 us whole, 18.3 cut; over 1500: 20.5 and 17.7; over
// 8000: 77.7 and 26.0. With many rows the crossing lies higher, as more is left and joined:
// 1773 tokens, Hq 8, Hkv 1: 22.1 whole, 23.6 cut).
__device__ __forceinline__ int item_parts(int top, int parts) {
  return top < kPrefillCutTiles ? 1 : max(1, min(top / kPrefillPartTiles, parts));
}
__device__ __forceinline__ int part_begin(int part, int top, int n) { return (int)((long long)part * top / n); }

// Keys that npos query positions from `first` on see without a window.
__device__ __forceinline__ int kv_keys(int first, int npos, int lq, int lk) {
  return first < lq ? max(0, min(first + npos, lq) + lk - lq) : 0;
}

// The tiles that a window and the first `sinks` keys leave of an item whose first position is p0 (see Item). ANY: they may begin at
// any key, the window's first or, where the first keys fit a tile, those (eight at a time, as a copy's swizzle has it) in rows
// before it; else at multiples of a tile.
struct Seen {
  int ns, skip, lo, merged;
  // of the tiles that hold keys before `keys`
  __device__ __forceinline__ int count(int keys) const {
    return keys <= ns * kN ? (keys + kN - 1) / kN : max(ns, (keys - skip + kN - 1) / kN);
  }
};
template <bool ANY>
__device__ __forceinline__ Seen seen_tiles(int p0, int lq, int lk, int window, int sinks) {
  Seen w;
  w.lo = max(0, p0 + lk - lq - window + 1);
  const int rows = (sinks + 7) & ~7, ns = (sinks + kN - 1) / kN, from = ANY ? w.lo : w.lo / kN * kN;
  w.ns = w.skip = w.merged = 0;
  if (ANY && sinks > 0 && rows <= kN && w.lo > rows) {
    w.skip = w.lo - rows;
    w.merged = rows;
  } else if (from > ns * kN) {
    w.ns = ns;
    w.skip = from - ns * kN;
  }
  return w;
}
// Bits below n of a 32-bit word, 0 <= n <= 32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : (1u << n) - 1u; }

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(u[0]),
      "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
      "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]),
      "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]),
      "r"(u[29]), "r"(u[30]), "r"(u[31]), "r"(taddr)
      : "memory");
}
// Waits for the thread's TMEM loads; their 32 registers are read behind the wait only.
__device__ __forceinline__ void tmem_ld_wait_x32(float* r) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(r[i]));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One thread's work of a converged warp. The whole warp runs the issuing code and each
// instruction elects its thread, so that descriptors stay in uniform registers: issued from a
// branch that one lane takes, an MMA cost about 100 cycles against the 64 it computes for.
#define DA_ELECT "elect.sync _|e, 0xffffffff;\n\t"

// D[tmem] (+)= A[smem] x B[smem]
__device__ __forceinline__ void warp_umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t" DA_ELECT
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] x B[smem]
__device__ __forceinline__ void warp_umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t" DA_ELECT
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_umma_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t" DA_ELECT
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// mbar_wait_bounded in few instructions, for a whole warp: the issuing warp's code competes with
// the softmax loop for the instruction cache. Lanes may leave the loop apart, and what follows
// (TMEM loads and stores, elections, shuffles) needs them together.
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, int* err, int code, int* abort_flag) {
  if (!mbar_try_wait(bar, parity)) {
    const unsigned long long t0 = globaltimer_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
      if (*(volatile int*)abort_flag) break;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        atomicOr(err, code);
        *(volatile int*)abort_flag = 1;
        break;
      }
    }
  }
  __syncwarp();
}
// Has a warp given up? One answer for the whole warp, so that its lanes leave their loops together.
__device__ __forceinline__ bool given_up(const int* abort_flag) {
  return __any_sync(0xffffffffu, *(const volatile int*)abort_flag != 0);
}
// Asks for a CTA of the grid that has not started, to run it here; the 16-byte answer lands at
// `dst` and completes on `bar`.
__device__ __forceinline__ void request_next_cta(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
               "r"(bar)
               : "memory");
}
// The answer: that CTA's blockIdx.x, or -1: none is left (the request must not be repeated).
__device__ __forceinline__ int next_cta(uint32_t src) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "mov.b32 %0, -1;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=&r"(x)
      : "r"(src)
      : "memory");
  return x;
}
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// (x, y) * (a, a) + (c, c)
__device__ __forceinline__ float2 fma2(float2 x, float a, float c) {
  unsigned long long r, xx = *reinterpret_cast<unsigned long long*>(&x), aa, cc;
  asm("mov.b64 %0, {%1, %1};" : "=l"(aa) : "f"(a));
  asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(xx), "l"(aa), "l"(cc));
  return *reinterpret_cast<float2*>(&r);
}
// Lanes with bit D of t give `lo` and lanes without it `hi`; each takes the other's.
template <int D>
__device__ __forceinline__ void exchange(uint32_t (&lo)[4], uint32_t (&hi)[4], int t) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, t & D ? lo[k] : hi[k], D);
    lo[k] = t & D ? got : lo[k];
    hi[k] = t & D ? hi[k] : got;
  }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&x)), "l"(*reinterpret_cast<unsigned long long*>(&y)));
  return *reinterpret_cast<float2*>(&r);
}

// Rows one behind the other can be loaded eight at a time.
__host__ __device__ constexpr bool merges(int src, bool window) { return window && src != kPages16; }

template <int SRC, bool WINDOW>
__global__ void __launch_bounds__(kThreadsP, 1) prefill_kernel(const __grid_constant__ PrefillParams p) {
  static_assert(SRC == kPackedKeys || WINDOW, "over a cache the window is always looked at");
  constexpr bool kCached = SRC != kPackedKeys, kMerge = merges(SRC, WINDOW);
  constexpr uint32_t kIdescS = umma_idesc_bf16(128, kN, /*A MN-major*/ false, /*B MN-major*/ false);
  constexpr uint32_t kIdescO = umma_idesc_bf16(128, 128, /*A MN-major*/ false, /*B MN-major*/ true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
  Item* items = reinterpret_cast<Item*>(smem + kOffItems);
  int* flags = reinterpret_cast<int*>(smem + kOffFlags);  // [0] abort, [1] TMEM address
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  // Guards of the bounds-checked build (constant true otherwise): shared memory that copies and
  // plain stores write, rows of the output and of the workspace.
  auto sm_ok = [&](uint32_t addr, uint32_t bytes) { return smem_in_bounds(smem_u32(smem_raw), addr, bytes, p.err); };
  auto out_ok = [&](const __nv_bfloat16* at, int n) { return in_bounds(at >= p.out && at + n <= p.out + p.out_span, p.err); };
  auto part_ok = [&](long long slot) { return in_bounds(slot >= 0 && slot < p.part_rows, p.err); };
  const uint32_t q_smem = smem_u32(smem), ring = q_smem + kOffRing;
  const int G = p.G, npos = p.npos;

  if (warp == kSoftWarps + 1) {
    tmem_alloc(smem_u32(flags + 1), 512);
    tmem_relinquish();
  } else if (tid == kSoftWarps * 32) {
    prefetch_tensormap(&p.tm_q);
    if (kCached || p.Tk > 0) {
      prefetch_tensormap(&p.tm_k);
      prefetch_tensormap(&p.tm_v);
    }
    for (int i = 0; i < kBars; ++i) {
      const bool soft = i == kPFull || i == kPFull + 1 || i == kSFree;  // an arrival per warp of a tile
      mbar_init(bar(i), soft ? 4 : (i >= kItemEmpty && i < kItemEmpty + kItems ? kSoftWarps + 2 : 1));
    }
    flags[0] = 0;
    fence_barrier_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = (uint32_t)flags[1];
  pdl_wait_primary();

  if (warp == kSoftWarps) {
    // ------------------------------------------------------------ producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    int base = 0, b0 = 0;  // row blocks of the sequences before b0 (a multiple of 32) and b0
    int total = 0x7fffffff;  // row blocks in all, once known
    int kv = 0, qn[2] = {0, 0};
    // Paged: the blocks of 32 boxes (a block's tokens, at most a tile's) at a time, a box a lane, and
    // of the 32 behind them, so that a block's number is at hand when its box is asked for.
    int ids = 0, ids_next = 0, ids_at = -2;
    auto box_seen = [&](const Item& it, int box) {  // does some row of the item see a token of it?
      const int key = box << p.box_shift;
      return key < it.lk && (key < p.sinks || key + (1 << p.box_shift) > it.lo);
    };
    auto box_ids = [&](const Item& it, int group) {
      const int box = group * 32 + lane;
      const long long at = (long long)it.k0 * p.bt_stride + (box >> (p.block_shift - p.box_shift));  // (k0: the sequence)
      return box_seen(it, box) && in_bounds(at < p.table_span, p.err) ? __ldg(p.table + at) : -1;
    };
    // Tile t of the item's keys or values: a box a lane (a half of its dims a lane where it is shorter than a
    // tile). Boxes that no row sees, and blocks outside the pool, are past the pool's end: zeros.
    auto load_pages = [&](const CUtensorMap* map, const Item& it, int t) {
      const int nb = kN >> p.box_shift, group = t * nb >> 5;
      if (group != ids_at) {
        ids = group == ids_at + 1 ? ids_next : box_ids(it, group);
        ids_next = box_ids(it, group + 1);
        ids_at = group;
      }
      const int i = nb > 1 ? lane >> 1 : lane, box = t * nb + i;
      int blk = __shfl_sync(0xffffffffu, ids, box & 31);
      const bool mine = i < nb;
      if ((unsigned)blk >= (unsigned)p.num_blocks) {
        if (mine && box_seen(it, box)) atomicOr(p.err, kErrBlockTable);
        blk = p.num_blocks;
      }
      const int row = (box << p.box_shift) & ((1 << p.block_shift) - 1), half = nb > 1 ? lane & 1 : 0;
      if (!in_bounds((unsigned)blk <= (unsigned)p.num_blocks && (unsigned)it.kvh < (unsigned)p.Hkv && t >= 0, p.err)) blk = p.num_blocks;
      int s = kv % kStagesP;
      if (!sm_ok(ring + s * kTileP, kTileP)) s = 0;
      mbar_wait_warp(bar(kKvEmpty + s), ((kv / kStagesP) & 1) ^ 1, p.err, kErrWaitEmpty, flags);
      const uint32_t full = bar((kv & 1 ? kVFull : kKFull) + s);
      ++kv;
      if (lane == 0) mbar_arrive_expect_tx(full, kTileP);
      __syncwarp();
      if (mine) tma_load_5d(ring + s * kTileP + half * kHalf + ((uint32_t)i << p.box_shift) * 128, map, full, 0, row, half, it.kvh, blk);
    };
    auto load_kv = [&](const CUtensorMap* map, int row, int kvh) {
      int s = kv % kStagesP;
      if (!sm_ok(ring + s * kTileP, kTileP)) s = 0;
      mbar_wait_warp(bar(kKvEmpty + s), ((kv / kStagesP) & 1) ^ 1, p.err, kErrWaitEmpty, flags);
      const uint32_t full = bar((kv & 1 ? kVFull : kKFull) + s);
      ++kv;
      if (lane == 0) {
        mbar_arrive_expect_tx(full, kTileP);
        tma_load_4d(ring + s * kTileP, map, full, 0, row, 0, kvh);
      }
    };
    // A tile from `row` on, but its first `merged` rows from `row0` on: eight rows of half the dims a lane.
    auto load_merged = [&](const CUtensorMap* map, int row0, int merged, int row, int kvh) {
      int s = kv % kStagesP;
      if (!sm_ok(ring + s * kTileP, kTileP)) s = 0;
      mbar_wait_warp(bar(kKvEmpty + s), ((kv / kStagesP) & 1) ^ 1, p.err, kErrWaitEmpty, flags);
      const uint32_t full = bar((kv & 1 ? kVFull : kKFull) + s);
      ++kv;
      if (lane == 0) mbar_arrive_expect_tx(full, kTileP);
      __syncwarp();
      const int at = (lane >> 1) * 8;
      tma_load_4d(ring + s * kTileP + (lane & 1) * kHalf + at * 128, map, full, 0, (at < merged ? row0 : row) + at, lane & 1, kvh);
    };
    const uint32_t next_smem = smem_u32(smem + kOffNext);
    int x = blockIdx.x, n = 0, asked = 0;
    auto ask = [&] {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kNext), 16);
        request_next_cta(next_smem, bar(kNext));
      }
    };
    auto answer = [&] {
      mbar_wait_warp(bar(kNext), asked & 1, p.err, kErrWaitFull, flags);
      ++asked;
      x = next_cta(next_smem);
      fence_proxy_async_smem();  // the answer has been read before the next one is written
      __syncwarp();
    };
    // Item x: the sequence that holds row block x / Hkv, looked for 32 sequences at a time.
    // lq < 0: none (x < 0, or past the last: the grid has CTAs for the most there can be).
    auto find = [&] {
      Item it;
      const int xi = x < 0 ? 0 : x / p.parts, part = x - xi * p.parts;
      const int mb = x < 0 ? total : xi / p.Hkv;
      it.kvh = x < 0 ? 0 : xi - mb * p.Hkv;
      it.lq = -1;
      it.lk = it.q0 = it.k0 = it.p0 = it.j0 = it.end0 = it.end1 = 0;
      it.ns = it.skip = it.lo = it.merged = 0;
      it.clear = it.part = -1;
      if (mb >= total) return it;
      if (mb < base) base = b0 = 0;
      while (b0 < p.B) {
        const int b = b0 + lane;
        int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
        if (b < p.B) {
          q0 = min(max(__ldg(p.cu_q + b), 0), p.Tq);
          q1 = min(max(__ldg(p.cu_q + b + 1), q0), p.Tq);
          if constexpr (kCached) {
            k1 = min(max(__ldg(p.cu_k + b), 0), p.Tk);  // (the sequences' lengths, and the table's capacity)
            if (SRC == kGathered && q1 - q0 <= p.few_lq) q1 = q0;
          } else {
            k0 = min(max(__ldg(p.cu_k + b), 0), p.Tk);
            k1 = min(max(__ldg(p.cu_k + b + 1), k0), p.Tk);
          }
        }
        const int nb = (q1 - q0 + 2 * npos - 1) / (2 * npos);
        int end = nb;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, end, off);
          if (lane >= off) end += o;
        }
        const unsigned after = __ballot_sync(0xffffffffu, base + end > mb);
        if (after) {
          const int src = __ffs(after) - 1;
          it.lq = __shfl_sync(0xffffffffu, q1 - q0, src);
          it.lk = __shfl_sync(0xffffffffu, k1 - k0, src);
          it.q0 = __shfl_sync(0xffffffffu, q0, src);
          it.k0 = kCached ? b0 + src : __shfl_sync(0xffffffffu, k0, src);
          it.p0 = (__shfl_sync(0xffffffffu, base + end, src) - 1 - mb) * 2 * npos;  // last block first
          break;
        }
        base += __shfl_sync(0xffffffffu, end, 31);
        b0 += 32;
      }
      if (it.lq < 0) {
        total = base;
        return it;
      }
      if constexpr (WINDOW) {
        const Seen w = seen_tiles<kMerge>(it.p0, it.lq, it.lk, p.window, p.sinks);
        it.ns = w.ns;
        it.skip = w.skip;
        it.lo = w.lo;
        it.merged = w.merged;
        it.end0 = w.count(kv_keys(it.p0, npos, it.lq, it.lk));
        it.end1 = w.count(kv_keys(it.p0 + npos, npos, it.lq, it.lk));
      } else {
        it.end0 = kv_tiles(it.p0, npos, it.lq, it.lk);
        it.end1 = kv_tiles(it.p0 + npos, npos, it.lq, it.lk);
        it.clear = it.lk % kN != 0 && it.k0 + it.lk < p.Tk ? it.lk / kN : -1;
      }
      ids_at = -2;
      if (p.parts > 1) {
        const int top = max(it.end0, it.end1), n = item_parts(top, p.parts);
        if (part >= n) it.lq = -1;  // fewer tiles than parts: not this one
        if (n > 1) {
          it.part = part;
          it.j0 = part_begin(part, top, n);
          it.end0 = min(it.end0, part_begin(part + 1, top, n));
          it.end1 = min(it.end1, part_begin(part + 1, top, n));
        }
      }
      return it;
    };
    Item it = find();
    while (true) {
      while (x >= 0 && it.lq < 0 && !given_up(flags)) {
        ask();
        answer();
        it = find();
      }
      const int slot = n % kItems;
      mbar_wait_warp(bar(kItemEmpty + slot), ((n / kItems) & 1) ^ 1, p.err, kErrWaitEmpty, flags);
      if (lane == 0 && sm_ok(smem_u32(items + slot), sizeof(Item))) {
        items[slot] = it;
        mbar_arrive(bar(kItemFull + slot));
      }
      if (it.lq < 0 || given_up(flags)) break;
      ++n;
      // The queries of both tiles, which come into shared memory when the item before has had
      // its last S computed, are on their way into L2 until then.
      if (lane < 4) tma_prefetch_4d(&p.tm_q, 0, it.kvh * G, it.q0 + it.p0 + (lane >> 1) * npos, lane & 1);
      const int top = max(it.end0, it.end1);
      if (top <= it.j0) ask();
      const Seen laid = seen_tiles<false>(0, it.lq, it.lk, p.window, p.sinks);  // kGathered: the keys that lie there
      for (int j = it.j0; j < top && !given_up(flags); ++j) {
        if (j == max(it.j0, top - 3)) ask();  // late, so that no item waits behind a long one
        const int key = j * kN + (WINDOW && j >= it.ns ? it.skip : 0);
        if constexpr (SRC == kPages16) {
          load_pages(&p.tm_k, it, key / kN);
          load_pages(&p.tm_v, it, key / kN);
        } else {
          const int row0 = SRC == kGathered ? (it.k0 * p.Hkv + it.kvh) * p.gather_rows : it.k0, head = SRC == kGathered ? 0 : it.kvh;
          const int merged = kMerge && j == 0 ? it.merged : 0;
          const int row = row0 + key - (SRC == kGathered && key + merged >= laid.ns * kN + laid.skip ? laid.skip : 0);
          if (merged > 0) {
            load_merged(&p.tm_k8, row0, merged, row, head);
            load_merged(&p.tm_v8, row0, merged, row, head);
          } else {
            load_kv(&p.tm_k, row, head);
            load_kv(&p.tm_v, row, head);
          }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (j > it.j0 || (w ? it.end1 : it.end0) <= it.j0) continue;
          mbar_wait_warp(bar(kQEmpty + w), (qn[w] & 1) ^ 1, p.err, kErrWaitEmpty, flags);
          ++qn[w];
          if (lane == 0 && sm_ok(q_smem + w * kTileP, kHalf + (uint32_t)(npos * G) * 128) && in_bounds(npos * G <= 128, p.err)) {
            mbar_arrive_expect_tx(bar(kQFull + w), (uint32_t)(npos * G) * 256);
            for (int c = 0; c < 2; ++c)
              tma_load_4d(q_smem + w * kTileP + c * kHalf, &p.tm_q, bar(kQFull + w), 0, it.kvh * G,
                          it.q0 + it.p0 + w * npos, c);
          }
        }
      }
      if (given_up(flags)) break;
      answer();
      it = find();
    }
    if (given_up(flags))  // with an answer on its way
      mbar_wait_bounded(bar(kNext), asked & 1, p.err, kErrWaitDrain, nullptr, kWaitLimitNs / 10);
    // every stage released (all MMAs that read them done, and so every copy) before the CTA may end
    for (int i = kv > kStagesP ? kv - kStagesP : 0; i < kv; ++i)
      mbar_wait_bounded(bar(kKvEmpty + i % kStagesP), (i / kStagesP) & 1, p.err, kErrWaitDrain, nullptr, kWaitLimitNs / 10);
    for (int w = 0; w < 2; ++w)
      if (qn[w]) mbar_wait_bounded(bar(kQEmpty + w), (qn[w] - 1) & 1, p.err, kErrWaitDrain, nullptr, kWaitLimitNs / 10);
  } else if (warp == kSoftWarps + 1 || warp == kSoftWarps + 2) {
    // ------------------------------------------- MMA issuers: S = Q K^T; O += P V
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    const bool pv = warp == kSoftWarps + 2;
    auto wait = [&](int b, int parity, int code) { wait_bar(bar(b), parity, p.err, code, flags); };
    const uint64_t q_desc = umma_smem_desc(q_smem, 16, 1024);
    const uint64_t kv_desc = pv ? umma_smem_desc(ring, kHalf, 1024) : umma_smem_desc(ring, 16, 1024);
    int ks = pv ? 1 : 0, kph = 0;  // ring position of the next V or K tile (they alternate)
    int tn = 0;                    // bit w: the parity that tile w's P (or Q) completes next
    int sn = 0, pn0 = 0, pn1 = 0;
    for (int n = 0;; ++n) {
      const int slot = n % kItems;
      wait(kItemFull + slot, (n / kItems) & 1, kErrWaitFull);
      const int j0 = uniform(items[slot].j0), end0 = uniform(items[slot].end0), end1 = uniform(items[slot].end1);
      const int lk = items[slot].lk, clear_at = pv ? items[slot].clear : -1;
      const int ns = WINDOW ? items[slot].ns : 0, skip = WINDOW ? items[slot].skip : 0, lo = WINDOW ? items[slot].lo : 0;
      const int merged = WINDOW ? items[slot].merged : 0;
      const bool none = items[slot].lq < 0 || given_up(flags);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kItemEmpty + slot));
      __syncwarp();
      if (none) break;
      for (int j = j0; j < max(end0, end1); ++j) {
        const int stage = ks;
        wait((pv ? kVFull : kKFull) + stage, kph, kErrWaitFull);
        ks += 2;
        if (ks >= kStagesP) ks -= kStagesP;
        if (ks == (pv ? 1 : 0)) kph ^= 1;  // every stage has held one of its tiles
        const uint64_t b = kv_desc + (uint64_t)(stage * (kTileP >> 4));
        // A V tile that ends inside another sequence's rows: their weights are 0, but 0 times a
        // NaN or infinity there is not, so those rows are cleared before the MMAs see them. With a window
        // also those before it (their blocks may be another sequence's by now).
        if constexpr (WINDOW) {
          const int base = j * kN + (j < ns ? 0 : skip);
          const int a = merged > 0 && j == 0 ? p.sinks : min(max(p.sinks - base, 0), kN), c = min(max(lo - base, 0), kN), e = min(max(lk - base, 0), kN);
          if (pv && (c > a || e < kN)) {
            uint4* tile = reinterpret_cast<uint4*>(smem + kOffRing + stage * kTileP);
            for (int i = lane; i < kN * 8; i += 32) {
              const int r = i >> 3;
              if (!((r >= a && r < c) || r >= e) || !sm_ok(smem_u32(tile + i), kHalf + 16)) continue;
              tile[i] = make_uint4(0, 0, 0, 0);
              tile[i + kHalf / 16] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (!WINDOW && j == clear_at) {
          uint4* tile = reinterpret_cast<uint4*>(smem + kOffRing + stage * kTileP);
          for (int i = lk % kN * 8 + lane; i < kN * 8 && sm_ok(smem_u32(tile + i), kHalf + 16); i += 32) {
            tile[i] = make_uint4(0, 0, 0, 0);
            tile[i + kHalf / 16] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          const int end = w ? end1 : end0;
          if (j >= end) continue;
          if (pv) {  // O_w += P_w V
            wait(kPFull + w, tn >> w & 1, kErrWaitMma);
            tn ^= 1 << w;
            // Behind the tile's next S, which the softmax waits for, rather than mixed with it
            // (8192 tokens x 64 heads in a short run: 575 us, 640 without this); after some polls
            // regardless, as that S may itself be waiting, for its K tile or for the softmax.
            ++(w ? pn1 : pn0);
            if (j + 1 < end) {
#pragma unroll 1
              for (int i = 0; i < 16 && !mbar_try_wait(bar(kSIssued + w), (w ? pn1 : pn0) & 1); ++i) {
              }
            }
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              warp_umma_ts(tmem + kTmemO + w * 128, tmem + kTmemP + w * 64 + kk * 8, b + ((kk * 16 * 128) >> 4), kIdescO,
                           kk > 0 || j > j0);
            warp_umma_commit(bar(kPvDone + w));
          } else {  // S = Q_w K^T
            if (j == j0) {
              wait(kQFull + w, tn >> w & 1, kErrWaitFull);
              tn ^= 1 << w;
            }
            wait(kSFree, (sn & 1) ^ 1, kErrWaitMma);
            ++sn;
            tc_fence_after_sync();
            const uint64_t a = q_desc + (uint64_t)(w * (kTileP >> 4));
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
              warp_umma_ss(tmem, a + off, b + off, kIdescS, kk != 0);
            }
            warp_umma_commit(bar(kSFull + w));
            if (lane == 0) mbar_arrive(bar(kSIssued + w));
            __syncwarp();
            if (j == end - 1) warp_umma_commit(bar(kQEmpty + w));
          }
        }
        warp_umma_commit(bar(kKvEmpty + stage));
      }
    }
  } else if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;  // tile, row of it (= TMEM lane)
    const uint32_t s_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t p_tmem = s_tmem + kTmemP + w * 64, o_tmem = s_tmem + kTmemO + w * 128;
    const int off = r / G, g = r - off * G;               // position in the tile, head of the group
    const int off0 = (warp & 3) * 32 / G;                 // of the warp's first row
    const float sl2 = p.scale_log2;
    const bool neg = sl2 < 0.f;
    int step = 0;
    float m = kNegInfP, l = 0.f;
    bool big = false;  // a row of the warp has a maximum past 2^24
    __nv_bfloat16* out = nullptr;  // this row of the item in work (null: no such row)
    long long slot_out = -1;       // its row in the workspace (-1: a whole item; -2: a part, no such row)
    // The O of the tile's last item, complete with PV of its last step (waited for here)
    auto pv_done = [&] {
      if (step > 0) wait_bar(bar(kPvDone + w), (step - 1) & 1, p.err, kErrWaitMma, flags);
      tc_fence_after_sync();
    };
    auto store = [&](__nv_bfloat16* to, float sum) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const bool none = sum == 0.f;  // a row without a key: zeros, whatever its O columns hold
      // Four lanes exchange their rows' 16-byte pieces, so that they write 64 bytes of one row
      // at a time: a store of 16 bytes to each of 32 rows takes the load-store unit 32 cycles.
      const int t = lane & 3;
      __nv_bfloat16* rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rows[i] = reinterpret_cast<__nv_bfloat16*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), (lane & ~3) + i));
#pragma unroll 1  // (run once an item: the time goes into fetching the instructions)
      for (int c = 0; c < 4; ++c) {
        float o[32];
        tmem_ld_x32(o_tmem + c * 32, o);
        tmem_ld_wait_x32(o);
        uint32_t y[4][4];  // 16-byte pieces of this row, then piece t of the four rows
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[i][k] = none ? 0u : pack_bf16x2(o[i * 8 + 2 * k] * inv, o[i * 8 + 2 * k + 1] * inv);
        exchange<1>(y[0], y[1], t);
        exchange<1>(y[2], y[3], t);
        exchange<2>(y[0], y[2], t);
        exchange<2>(y[1], y[3], t);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (rows[i] && out_ok(rows[i] + c * 32 + t * 8, 8))
            *reinterpret_cast<uint4*>(rows[i] + c * 32 + t * 8) = make_uint4(y[i][0], y[i][1], y[i][2], y[i][3]);
      }
    };
    // A part's row: O as it is, the sum and the reference maximum.
    auto store_part = [&](float sum, float ref) {
      if (slot_out >= 0 && part_ok(slot_out)) {
        p.part_ml[slot_out * 2] = ref;
        p.part_ml[slot_out * 2 + 1] = sum;
      }
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld_32x32b_x16(o_tmem + c * 16, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(o[i]));
        if (slot_out >= 0 && part_ok(slot_out))
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(p.part_o + slot_out * 128 + c * 16 + i * 4) =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    };
    auto finish = [&](float sum, float ref) {
      if (slot_out == -1) store(out, sum);
      else store_part(sum, ref);
    };
    for (int n = 0;; ++n) {
      const int slot = n % kItems;
      wait_bar(bar(kItemFull + slot), (n / kItems) & 1, p.err, kErrWaitFull, flags);
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kItemEmpty + slot));
      if (it.lq < 0 || given_up(flags)) break;
      const int first = it.p0 + w * npos, pos = first + off;
      const bool row_ok = off < npos && pos < it.lq;
      const int lim = min(it.lk, pos + it.lk - it.lq + 1);            // keys of this row
      const int lim0 = min(it.lk, first + off0 + it.lk - it.lq + 1);  // the least of the warp's rows
      const int low = pos + it.lk - it.lq - p.window + 1;             // this row's window begins there
      const int low1 = first + ((warp & 3) * 32 + 31) / G + it.lk - it.lq - p.window + 1;  // the last of the warp's rows
      const int end = w ? it.end1 : it.end0;
      __nv_bfloat16* to = row_ok ? p.out + (long long)(it.q0 + pos) * p.o_st + (long long)(it.kvh * G + g) * p.o_sh : nullptr;
      if (it.part < 0 && end == 0 && to && out_ok(to, 128)) {  // no key at all
#pragma unroll
        for (int i = 0; i < 16; ++i) *reinterpret_cast<uint4*>(to + i * 8) = make_uint4(0, 0, 0, 0);
      }
      for (int j = it.j0; j < end; ++j, ++step) {
        wait_bar(bar(kSFull + w), step & 1, p.err, kErrWaitMma, flags);
        tc_fence_after_sync();
        float s[kN];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_x32(s_tmem + c * 32, s + c * 32);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait_x32(s + c * 32);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree));
        const int base = j * kN + (WINDOW && j >= it.ns ? it.skip : 0);
        // some row of the warp ends inside this tile, or its window begins behind a key of it that is none of the first
        if (base + kN > lim0 || (WINDOW && base < low1 && base + kN > p.sinks)) {
          const float none = neg ? -kNegInfP : kNegInfP;
          const int left = lim - base, kept = it.merged > 0 && j == 0 ? p.sinks : p.sinks - base;  // columns that are first keys
#pragma unroll
          for (int h = 0; h < 4; ++h) {  // a bit per key (tests of single bits share an instruction)
            uint32_t keep = low_bits(min(max(left - 32 * h, 0), 32));
            if constexpr (WINDOW)
              keep &= ~low_bits(min(max(low - base - 32 * h, 0), 32)) | low_bits(min(max(kept - 32 * h, 0), 32));
#pragma unroll
            for (int c = 0; c < 32; ++c) s[32 * h + c] = keep >> c & 1u ? s[32 * h + c] : none;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = s[c];
        if (!neg) {
#pragma unroll
          for (int c = 4; c < kN; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], s[c], s[c + 1]);
          mx[0] = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        } else {
#pragma unroll
          for (int c = 4; c < kN; ++c) mx[c & 3] = fminf(mx[c & 3], s[c]);
          mx[0] = fminf(fminf(mx[0], mx[1]), fminf(mx[2], mx[3]));
        }
        const float xm = mx[0] * sl2;
        const float l_old = l, m_old = m;
        if (j == it.j0) {
          m = kNegInfP;
          l = 0.f;
        }
        const bool grow = row_ok && xm > m + kSlackP;
        const bool any = __any_sync(0xffffffffu, grow);
        const float al = grow ? fast_exp2(m - xm) : 1.f;
        m = grow ? xm : m;
        l *= al;
        // The weights' exponent is one fused s * sl2 - m, and m a rounded product: past 2^24 they part
        // by whole powers of two, past 2^32 by more than fp32 holds. There the products are rounded
        // first, as the maximum's is.
        if (any) big = __any_sync(0xffffffffu, (__float_as_uint(m) & 0x7fffffffu) - 0x4b800000u < 0x34000000u);
        if (big) {
#pragma unroll
          for (int c = 0; c < kN; ++c) s[c] *= sl2;
        }
        const float mul = big ? 1.f : sl2;
        const float mr = m == kNegInfP ? 0.f : -m;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float2 x = fma2(make_float2(s[2 * i], s[2 * i + 1]), mul, mr);
          x.x = fast_exp2(x.x);
          x.y = fast_exp2(x.y);
          sum[i & 1] = add2(sum[i & 1], x);
          pk[i] = pack_bf16x2(x.x, x.y);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        pv_done();
        if (j == it.j0) {
          if (step > 0) finish(l_old, m_old);
          out = to;
          slot_out = it.part < 0 ? -1
                                 : row_ok ? ((long long)it.part * p.Tq + it.q0 + pos) * (p.G * p.Hkv) + it.kvh * G + g : -2;
        } else if (any) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld_x32(o_tmem + c * 32, o);
            tmem_ld_wait_x32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= al;
            tmem_st_x32(o_tmem + c * 32, reinterpret_cast<uint32_t*>(o));
          }
        }
        tmem_st_x32(p_tmem, pk);
        tmem_st_x32(p_tmem + 32, pk + 32);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + w));
      }
    }
    pv_done();
    if (step > 0) finish(l, m);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kSoftWarps + 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that were cut: a warp per (token, head), four dims a lane.
template <int SRC, bool WINDOW>
__global__ void __launch_bounds__(128) prefill_join_kernel(const __grid_constant__ PrefillParams p) {
  const int lane = threadIdx.x & 31, Hq = p.G * p.Hkv;
  pdl_wait_primary();
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(unit / Hq), h = (int)(unit - (long long)t * Hq);
  if (t >= p.Tq) return;
  const int b = find_sequence(p.cu_q, p.B, t, lane);
  const int q0 = min(max(__ldg(p.cu_q + b), 0), p.Tq), q1 = min(max(__ldg(p.cu_q + b + 1), q0), p.Tq);
  const int first = min(max(__ldg(p.cu_k + b), 0), p.Tk);
  const int k0 = SRC == kPackedKeys ? first : 0, k1 = SRC == kPackedKeys ? min(max(__ldg(p.cu_k + b + 1), k0), p.Tk) : first;
  if (t < q0 || t >= q1) return;  // a row of no sequence
  if (SRC == kGathered && q1 - q0 <= p.few_lq) return;
  const int lq = q1 - q0, lk = k1 - k0, p0 = (t - q0) / (2 * p.npos) * 2 * p.npos;
  int end0, end1;
  if (WINDOW) {
    const Seen w = seen_tiles<merges(SRC, WINDOW)>(p0, lq, lk, p.window, p.sinks);
    end0 = w.count(kv_keys(p0, p.npos, lq, lk));
    end1 = w.count(kv_keys(p0 + p.npos, p.npos, lq, lk));
  } else {
    end0 = kv_tiles(p0, p.npos, lq, lk);
    end1 = kv_tiles(p0 + p.npos, p.npos, lq, lk);
  }
  const int top = max(end0, end1), n = item_parts(top, p.parts), end = t - q0 - p0 < p.npos ? end0 : end1;
  if (n == 1) return;  // whole: it has been written
  float m = kNegInfP, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < n && part_begin(i, top, n) < end; ++i) {  // (parts past the row's last key hold nothing)
    const long long slot = ((long long)i * p.Tq + t) * Hq + h;
    if (!in_bounds(slot < p.part_rows, p.err)) continue;
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot * 2);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot * 128 + lane * 4);
    if (ml.x == kNegInfP && ml.y == 0.f) continue;  // the part's keys all lie past the row
    const float mn = fmaxf(m, ml.x), a = m == kNegInfP ? 0.f : fast_exp2(m - mn);
    const float c = ml.x == kNegInfP ? 1.f : fast_exp2(ml.x - mn);  // (no maximum: NaN scores)
    l = l * a + ml.y * c;
    o.x = o.x * a + v.x * c;
    o.y = o.y * a + v.y * c;
    o.z = o.z * a + v.z * c;
    o.w = o.w * a + v.w * c;
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 y = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (l == 0.f) y = make_uint2(0u, 0u);
  __nv_bfloat16* to = p.out + (long long)t * p.o_st + (long long)h * p.o_sh + lane * 4;
  if (in_bounds(to + 4 <= p.out + p.out_span, p.err)) *reinterpret_cast<uint2*>(to) = y;
}

template <int SRC, bool WINDOW>
cudaError_t launch_prefill_as(const PrefillParams& p, int grid, bool pdl, cudaStream_t stream) {
  static int configured[64] = {0};  // the shared-memory opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(prefill_kernel<SRC, WINDOW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemP);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = kSmemP;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, prefill_kernel<SRC, WINDOW>, p);
  if (e != cudaSuccess || p.parts == 1) return e;
  cfg.gridDim = dim3((unsigned)(((long long)p.Tq * p.G * p.Hkv + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefill_join_kernel<SRC, WINDOW>, p);
}

}  // namespace
}  // namespace da
