// kernels.h -- parameter blocks and launchers shared by the C-ABI layer (api.cu)
// and the kernels. Host and device code both include it; it holds no method
// arithmetic beyond the tiling constants.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace da {

// ----------------------------------------------------------- split-KV attention
// Head dims the kernel implements: 128, and 256 (the two-halves contraction of a
// D = 256 GQA decode). A stage always holds 32 KB: a K tile and a V tile of
// tile_tokens(D) tokens x D dims in 64-dim boxes of 128-byte swizzled rows.
constexpr int kHeadDim = 128;
constexpr int kHeadDimWide = 256;
__host__ __device__ constexpr int tile_tokens(int dim) { return dim == kHeadDimWide ? 32 : 64; }
constexpr int kTile = 64;                      // tokens per pipeline stage at D = 128
constexpr int kGroupWarps = 4;                 // consumer warps per group; each owns 16 tokens of a stage
constexpr int kGroups = 2;                     // consumer groups take alternate stages
constexpr int kConsumerThreads = kGroups * kGroupWarps * 32;
// Producer warps of the attention kernel: one per consumer group (each issues the tiles of
// its group's stages) for a paged cache, where small blocks mean several copies per tile and
// one lane's issue rate set the pace; for a contiguous cache when kContigTwoProducers.
constexpr bool kContigTwoProducers = true;
// A paged fp8 cache has more and smaller copies (a third one per box for the scales, 2 KB of K
// in a block of 16): four.
__host__ __device__ constexpr int attn_producers(bool paged, bool fused, bool scores, bool kv8 = false) {
  return paged && kv8 ? 4 : paged || (kContigTwoProducers && !fused && !scores) ? 2 : 1;
}
__host__ __device__ constexpr int attn_threads(int producers) { return kConsumerThreads + 32 * producers; }
constexpr int kMaxStages = 6;                  // even stage counts: stage s always belongs to group s % 2
constexpr int kKTileBytes = 16384;             // K tile: tile_tokens(D) x D x bf16 (both head dims)
constexpr int kStageBytes = 2 * kKTileBytes;   // K tile + V tile
__host__ __device__ constexpr int box_bytes(int dim) { return tile_tokens(dim) * 128; }  // 64 dims of a tile
__host__ __device__ constexpr int q_row_bytes(int dim) { return dim * 2 + 16; }  // + 16 B pad: conflict-free
                                                                                 // fragment loads
constexpr int kMaxGroup = 16;
constexpr int kMaxBatch = 1024;
constexpr int kMergeRow = 132;                 // floats per head row of the merge scratch (128 + pad); at
                                               // D = 256 a warp holds one 128-dim half of the output
constexpr int kMaxAttnCtas = 512;              // persistent CTAs of the attention kernel (and so parts
                                               // per sequence) at most
static_assert(tile_tokens(kHeadDim) * kHeadDim * 2 == kKTileBytes, "K tile bytes at D = 128");
static_assert(tile_tokens(kHeadDimWide) * kHeadDimWide * 2 == kKTileBytes, "K tile bytes at D = 256");
// Shared-memory carve-up of the attention kernel; nb = 8-head blocks (1 or 2),
// stages = pipeline depth (even, so that a stage always belongs to one consumer group),
// dim = head dim (128 or 256).
struct AttnSmem {
  int nb, batch, stages, dim, stage_bytes;
  __host__ __device__ constexpr AttnSmem(int nb_, int batch_, int stages_, int dim_ = kHeadDim,
                                         int stage_bytes_ = kStageBytes)
      : nb(nb_), batch(batch_), stages(stages_), dim(dim_), stage_bytes(stage_bytes_) {}
  __host__ __device__ constexpr int heads() const { return 8 * nb; }
  __host__ __device__ constexpr size_t q_slot() const { return (size_t)heads() * q_row_bytes(dim); }
  __host__ __device__ constexpr size_t off_q() const { return (size_t)stages * stage_bytes; }
  __host__ __device__ constexpr size_t off_merge_o() const { return off_q() + stages * q_slot(); }
  __host__ __device__ constexpr size_t off_merge_ml() const {
    return off_merge_o() + (size_t)kGroupWarps * heads() * kMergeRow * 4;
  }
  __host__ __device__ constexpr size_t off_bars() const { return off_merge_ml() + (size_t)kGroupWarps * heads() * 2 * 4; }
  // barriers: full[S], empty[S] (attention); full[8], empty[8], accum[2] (fused projection)
  __host__ __device__ constexpr size_t off_flags() const { return off_bars() + (2 * stages + 18) * 8; }
  // flags: int [16]: [0] abort, [1] last CTA of a sequence, [2] last CTA of a column tile (fused
  // step), [3] TMEM address, [8..15] this CTA's range of tiles and the cursor at its first tile
  __host__ __device__ constexpr size_t off_prefix() const { return off_flags() + 64; }
  __host__ __device__ constexpr size_t off_lens() const { return off_prefix() + (size_t)(batch + 1) * 4; }
  // paged caches: kIdTiles rows of 16 block ids (one 64-byte TMA box per tile), rows
  // 128 bytes apart (a tensor copy's shared-memory destination is 128-byte aligned)
  __host__ __device__ constexpr size_t off_ids() const { return (off_lens() + (size_t)batch * 4 + 127) & ~(size_t)127; }
  // cluster mode: this CTA's merged states of the sequences it shares with other CTAs of its
  // cluster (slot 0: its first segment, slot 1: its last), read by those CTAs:
  // O [2][heads][dim], then (m, l) [2][heads][2], then the merge duties int [2][4] (and 16
  // bytes of padding)
  __host__ __device__ constexpr size_t off_cpart() const { return off_ids() + kIdTiles * kIdStride * 4; }
  __host__ __device__ constexpr size_t cpart_bytes() const { return 2 * (size_t)heads() * (dim + 2) * 4 + 48; }
  // the cluster-mode states only in clusters (at most half as many sequences as SMs)
  __host__ __device__ constexpr size_t total(bool cluster = false) const {
    return 1024 + off_cpart() + (cluster ? cpart_bytes() : 0);
  }
  // paged fp8 caches: the scales of each stage's 128 tokens, after everything else (one
  // box's K scales then its V scales, 128-byte aligned for the tensor copies)
  __host__ __device__ constexpr size_t off_scales(bool cluster) const {
    return (off_cpart() + (cluster ? cpart_bytes() : 0) + 127) & ~(size_t)127;
  }
  __host__ __device__ constexpr size_t total_scaled(bool cluster = false) const {
    return 1024 + off_scales(cluster) + (size_t)stages * kScaleStageBytes;
  }
  static constexpr int kScaleStageBytes = 2 * 128 * 4;
  static constexpr int kIdTiles = 8;
  static constexpr int kIdRow = 16;     // entries a row receives
  static constexpr int kIdStride = 32;  // entries between rows (128 bytes)
};

constexpr size_t kMaxDynSmem = 232448;  // 227 KB per CTA on sm_100-class GPUs
constexpr size_t attn_smem_bytes(int batch, int nb, int stages, int dim = kHeadDim, int stage_bytes = kStageBytes,
                                 bool cluster = false) {
  return AttnSmem(nb, batch, stages, dim, stage_bytes).total(cluster);
}
// fp8 (e4m3) caches: a tile is 128 tokens (128 x 128 dims x 1 byte of K and of V), so a
// stage holds the same 32 KB and the ring the same 4 stages as for bf16.
constexpr int kTileFp8 = 128;
static_assert(AttnSmem(2, kMaxBatch, 4).total_scaled() <= kMaxDynSmem && AttnSmem(2, 128, 4).total_scaled(true) <= kMaxDynSmem,
              "attention kernel (paged fp8) exceeds 227 KB of shared memory");
static_assert(AttnSmem(2, kMaxBatch, 4).total() <= kMaxDynSmem, "attention kernel exceeds 227 KB of shared memory");
// Cluster mode needs room for two parked states: every group width at D = 128, up to
// eight heads per group at D = 256 (the host checks each launch; wider groups at D = 256
// merge through L2).
static_assert(AttnSmem(2, 128, 4).total(true) <= kMaxDynSmem, "cluster mode (D = 128) exceeds 227 KB");
static_assert(AttnSmem(1, 128, 4, kHeadDimWide).total(true) <= kMaxDynSmem, "cluster mode (D = 256) exceeds 227 KB");
static_assert(AttnSmem(2, kMaxBatch, 4, kHeadDimWide).total() <= kMaxDynSmem,
              "attention kernel (D = 256) exceeds 227 KB of shared memory");
// 4 stages by default (measured faster than 6 on the GB300: deeper rings slowed the
// stream); 6 on request when it fits this batch and group width (D = 128 only).
constexpr int attn_stages_for(int batch, int nb, int requested, bool cluster = false) {
  return requested == kMaxStages && attn_smem_bytes(batch, nb, kMaxStages, kHeadDim, kStageBytes, cluster) <= kMaxDynSmem
             ? kMaxStages
             : 4;
}

struct AttnParams {
  CUtensorMap tm_k;  // [B][Hkv][Lcap][D] bf16, box 64 dims x tile_tokens(D) tokens, 128B swizzle
  CUtensorMap tm_v;
  const __nv_bfloat16* q;
  long long q_sb, q_sh;  // element strides of q [B][Hq][D]
  const int* seq_lens;
  __nv_bfloat16* attn;   // [B][Hq][D] bf16 result
  long long a_sb, a_sh;
  float* scores;         // [B][Hq][Lcap] fp32 (scores-only mode)
  long long s_sb, s_sh;
  float* part_o;         // [slots][gpad][D] unnormalised partial outputs
  float* part_ml;        // [slots][gpad][2]   (running max in log2 units, sum)
  long long part_slots;  // slots of part_o / part_ml (checked in the bounds-checked build)
  int* counters;         // [B*Hkv] completion counters (zero between calls)
  int* err;              // device error word
  int B, Hkv, G, Lcap;
  int gpad;              // 8 or 16 (heads per group rounded up to the MMA width)
  float scale_log2;      // scale * log2(e)
  // Optional region the next kernel reads (the projection weights): pulled into L2
  // in pieces while the K/V stream runs. prefetch_bytes = 0 disables it.
  const char* prefetch;
  long long prefetch_bytes;
  int stages;            // requested pipeline depth (4 or 6)
  // Fused step only (decode_attn_fwd in one launch): the projection of this kernel's
  // own attention output (attn, contiguous [B][K]) by W_o, on tcgen05 after a grid barrier.
  CUtensorMap tm_w;      // W_o [K][N] bf16: box 64 columns x 64 rows, 128B swizzle
  CUtensorMap tm_x;      // attention output [B][K] bf16: box 64 k x npad rows, 128B swizzle
  __nv_bfloat16* y;      // [B][N]
  long long y_sb;
  float* proj_part;      // [slots][B][128] fp32 split-K partials
  long long proj_part_floats;  // floats of proj_part (checked in the bounds-checked build)
  int* proj_counters;    // [column tiles], zero between calls
  int* grid_sync;        // [2]: arrivals, departures of the grid barrier, zero between calls
  unsigned long long sync_limit_ns;  // the grid barrier's wait limit (0: two seconds)
  int sync_extra;        // arrivals the grid barrier waits for beyond the grid (0; a test sets 1
                         // to make the wait run out)
  int N, K, kb_per_tile, units;  // units = column tiles x k-blocks of 64
  int attn_workers;      // CTAs that take attention tiles (<= grid); the fused step may leave
                         // some CTAs free to start on W_o at once
  // Paged cache only: tm_k / tm_v map [num_blocks][Hkv][block_size][D]; token t of sequence b
  // is row t % block_size of block block_table[b * bt_stride + t / block_size].
  const int* block_table;
  long long bt_stride;
  long long bt_entries;  // flat extent of the table, (B - 1) * bt_stride + max_blocks
  int block_size, num_blocks;
  int block_shift;       // log2(block_size)
  CUtensorMap tm_table;  // the table as one flat int32 array (one row), box 16 entries
  // fp8 (e4m3) caches only: K = k_cache * k_scale, V = v_cache * v_scale
  float k_scale, v_scale;
  // paged fp8 caches: a scale per token and KV head instead, [num_blocks][Hkv][2][block_size]
  // fp32 (K's, then V's), box min(block size, 128) tokens x 2
  CUtensorMap tm_scales;
  // paged fp8 caches: 1, 2: tm_k maps both pools, the third coordinate choosing K (1) or V (2)
  // first, and one copy brings a box of both; 0: a copy from each of tm_k and tm_v
  int kv_pair;
  // Cluster mode (> 1): the grid is launched in clusters of `cluster` consecutive CTAs; the
  // tiles are split over the CTAs as always, and a sequence whose parts all lie in one
  // cluster merges them in distributed shared memory (the others through L2).
  int cluster;
  // Paged fp8 caches. Sequences of equal length: cluster mode while a batch row has at most
  // chip_row_tiles tiles (of all its KV heads). Otherwise seq_parts(tiles, seq_ctas, seq_least)
  // CTAs each (seq_ctas = workers / sequences; 0: the tiles split over all workers), unless the
  // longest one's would be all seq_ctas and it has more than own_slope * T + own_slack tiles.
  int chip_row_tiles, seq_ctas, seq_least;
  float own_slope, own_slack[2];  // (slack: of equal lengths, of ragged ones)
  int pdl;  // 1: launched with programmatic dependent launch (waits before any global access)
  // > 0: each CTA lets the next kernel launch when it reaches the tile this many before the
  // end of its range; 0: right after set-up
  int trigger_at;
  // floor(n / d) = (n * split_mul) >> split_shift, exact for 0 <= n < 2^31, for the two worker
  // counts d that split the tiles over the CTAs: [0] min(grid, attn_workers), [1] (cluster
  // mode) min(that, B * Hkv * cluster). A worker count that differs is divided the plain way.
  unsigned long long split_mul[2];
  int split_div[2], split_shift[2];
};
constexpr int kMaxAttnCluster = 8;  // portable cluster size

// CTAs for each of several sequences of `tiles` 128-token tiles, `most` at hand for each: one up
// to four tiles (a tile per group of warps); then parts of two tiles, of four from eight parts on,
// and more than 64 parts only once they hold 16 tiles, as the one CTA that joins a sequence's
// parts pays for each (one sequence of 8192 tokens: 10.7 us in 16 parts, 11.1 in 32, 14.3 in 64;
// of 131072: 24.8 in 64, 29.2 in 152). At least `least` where there are tiles for them.
__host__ __device__ inline int seq_parts(int tiles, int most, int least) {
  const int small = tiles / 2 < 8 ? tiles / 2 : 8, mid = tiles / 4 < 64 ? tiles / 4 : 64, large = tiles / 16;
  int k = tiles <= 4 ? 1 : (small > mid ? small : mid);
  k = k > large ? k : large;
  const int low = least < tiles ? least : tiles;
  k = k > low ? k : low;
  return k < most ? k : most;
}

// Paged caches: a power of two from 8 tokens (tiles are cut into blocks, or blocks hold
// whole tiles; the producer's index arithmetic is shifts and masks).
// A paged fp8 cache: from 16 (a tile of 128 tokens then has at most eight boxes, whose ids
// fit a row of the id ring, and a box's scales are a multiple of 128 bytes).
constexpr int kMinBlock = 8, kMinBlockFp8 = 16;
__host__ __device__ constexpr bool paged_block_ok(int block_size, int dim, bool kv8 = false) {
  return block_size >= (kv8 ? kMinBlockFp8 : kMinBlock) && block_size <= (1 << 20) && (block_size & (block_size - 1)) == 0 && dim > 0;
}

constexpr int kProjWBytes = 2 * 64 * 128;  // one stage of W_o: 128 columns x 64 k-rows
// Phase-B stages re-cut the attention ring (kStages x kStageBytes) into W_o + X tiles.
__host__ __device__ constexpr int proj_stage_bytes(int npad) { return kProjWBytes + ((npad * 128 + 1023) / 1024) * 1024; }
__host__ __device__ constexpr int proj_stages(int npad) {
  return (4 * kStageBytes) / proj_stage_bytes(npad) < 8 ? (4 * kStageBytes) / proj_stage_bytes(npad) : 8;
}

// grid = number of persistent CTAs; nb = 1 for G <= 8, 2 for G <= 16; dim = head dim
// (128 or 256); npad = 0 for the attention alone, else the batch padding (16/32/64/128)
// of the fused projection (a cooperative launch: every CTA must be resident for the
// grid barrier; D = 128 only).
cudaError_t launch_attention(const AttnParams& p, int grid, int nb, int dim, bool scores_only, cudaStream_t stream,
                             int npad = 0);
// The D = 256 instantiations (their own translation unit).
cudaError_t launch_attention_d256(const AttnParams& p, int grid, int nb, bool scores_only, cudaStream_t stream);
// Attention over a paged cache (p.block_table set), D = 128 or 256.
cudaError_t launch_attention_paged(const AttnParams& p, int grid, int nb, int dim, cudaStream_t stream);
// Attention over an fp8 (e4m3) cache, D = 128 (p.k_scale, p.v_scale set).
cudaError_t launch_attention_fp8(const AttnParams& p, int grid, int nb, cudaStream_t stream);
// Attention over a paged fp8 cache with a scale per token and KV head, D = 128 (p.block_table,
// p.tm_scales set).
cudaError_t launch_attention_paged_fp8(const AttnParams& p, int grid, int nb, cudaStream_t stream);
// Clusters of `cluster` attention CTAs (one per SM) that can be resident at once on the
// current device (the GPCs' SM counts leave some SMs out); 0 if the query fails.
int attn_max_active_clusters(int cluster);

// ------------------------------------------------------------ prompt attention
constexpr int kMaxPrefillParts = 32, kPrefillPartTiles = 4, kPrefillCutTiles = 12;
struct PrefillParams {
  CUtensorMap tm_q;  // q [Tq][Hq][128] bf16: box 64 dims x G heads x npos tokens, 128B swizzle
  CUtensorMap tm_k;  // k, v [Tk][Hkv][128]: box 64 dims x 128 tokens x both halves of the dims
  CUtensorMap tm_v;
  __nv_bfloat16* out;  // [Tq][Hq][128]
  long long o_st, o_sh;
  const int *cu_q, *cu_k;  // [B + 1]; over pages cu_k is [B], the sequences' lengths, and Tk their capacity
  int* err;
  int B, Hkv, G, Tq, Tk;
  int npos;            // query positions per tile, floor(128 / G)
  float scale_log2;    // scale * log2(e), never 0
  long long out_span;      // elements of out from its first to one past its last (bounds-checked build)
  int parts;           // an item's K/V tiles are cut into at most so many parts (1: none is cut)
  float* part_o;       // [parts][Tq][Hq][128] unnormalised outputs of the parts
  float* part_ml;      // [parts][Tq][Hq][2] their maxima (log2 units) and sums
  long long part_rows;  // rows of both (0: no item is cut)
  // A query at position i sees keys i - window + 1 .. i and those below `sinks` (no window: 2^30)
  int window, sinks;
  CUtensorMap tm_k8, tm_v8;  // with first keys: k and v by boxes of 64 dims x 8 tokens (not over pages)
  // Pages: tm_k and tm_v map [num_blocks][Hkv][block_size][128], a box of 2^box_shift = min(block size, 128) tokens
  const int* table;
  long long bt_stride, table_span;
  int num_blocks, block_shift, box_shift;
  // ... or rows of bf16 that launch_gather has laid out, tm_k and tm_v as of [B * Hkv * gather_rows][1][128] packed tokens
  int gather_rows;
  int few_lq;  // sequences of so many queries and fewer are another kernel's: their rows are left as they are
};
// grid = as many CTAs as there can be work items; those that run take over the others.
cudaError_t launch_prefill(const PrefillParams& p, int grid, bool pdl, cudaStream_t stream);
// ... with a window
cudaError_t launch_prefill_window(const PrefillParams& p, int grid, bool pdl, cudaStream_t stream);
// ... over a paged bf16 cache, or over its gathered tokens
cudaError_t launch_prefill_paged(const PrefillParams& p, int grid, bool gathered, bool pdl, cudaStream_t stream);

// The tokens of a paged cache that a chunk's queries see, as rows of bf16 [batch][heads][rows][128].
struct GatherParams {
  const uint8_t *k_pages, *v_pages;  // [num_blocks][Hkv][block_size][128] bf16 or e4m3; strides and spans in bytes
  long long kp_sb, kp_sh, kp_sr, vp_sb, vp_sh, vp_sr, kp_span, vp_span;
  const float* scales;               // [num_blocks][Hkv][2][block_size] (e4m3); strides in floats
  long long sc_sb, sc_sh, sc_st, sc_span;
  const int *cu, *lens, *table;      // [batch + 1], [batch], [batch][max_blocks]
  long long bt_stride, table_span;
  __nv_bfloat16 *k_out, *v_out;
  long long span;                    // elements of each
  int* err;
  int heads, rows, Tq, cap, num_blocks, block_shift, window, sinks;
  int few_lq;                        // sequences of so many new tokens and fewer are another kernel's: left out
};
// CTAs of a (sequence, head) at most, each with every so many-th of its tiles: a table's capacity may be far past the lengths (and in
// a mixed batch most sequences have none: 32 for those)
constexpr int kGatherCtas = 64;
cudaError_t launch_gather(const GatherParams& p, int batch, bool kv8, bool pdl, cudaStream_t stream);

// ---------------------------------- attention of a few new tokens over a paged cache
struct FewParams {
  const __nv_bfloat16* q;  // [Tq][Hq][128]
  __nv_bfloat16* out;
  long long q_st, q_sh, o_st, o_sh;
  // [num_blocks][Hkv][block_size][128] bf16 or e4m3, a box of a unit's 16 (e4m3: 32) tokens or of a block's where it has
  // fewer; e4m3: the scales [num_blocks][Hkv][2][block_size]
  CUtensorMap tm_k, tm_v, tm_scales;
  const int *cu, *lens, *table;      // [B + 1], [B], [B][max_blocks]
  long long bt_stride;
  int* err;
  int* counters;                     // a CTA each, zero between calls
  float *part_o, *part_ml;           // [2 * CTAs][rows][128], [2 * CTAs][rows][2]: states of items that lie in several CTAs
  int slots;                         // 2 * CTAs
  int B, Hkv, G, Tq, cap;
  int npos;                          // query positions of an item, floor(rows / G)
  int most_lq;                       // sequences with more rows are another kernel's: theirs are left as they are
  int num_blocks, block_shift, window, sinks;
  float scale_log2;
  int least;                         // units that a CTA takes at least
  // elements from the first to one past the last (bounds-checked build)
  long long q_span, out_span, table_span;
};
constexpr int kFewRows = 16, kFewKeys16 = 16, kFewKeys8 = 32;
// rows: of an item, 8 or 16; warps: of a CTA, 8, or (e4m3) 4 with two CTAs an SM
cudaError_t launch_chunk_few(const FewParams& p, int grid, bool kv8, int rows, int warps, bool pdl, cudaStream_t stream);

// ------------------------------------------------ paged cache: writing and reading
struct CacheParams {
  const __nv_bfloat16 *k, *v;  // [T][Hkv][D] packed tokens (read: the destinations)
  long long k_st, k_sh, v_st, v_sh;
  const int* cu;               // [B + 1] offsets of the sequences in the packed tokens
  const int* table;            // [B][max_blocks]
  long long bt_stride;
  const int* seq_lens;         // [B] tokens of each sequence, the new ones among them (write only)
  void *k_pages, *v_pages;     // [num_blocks][Hkv][block_size][D] bf16 or e4m3
  long long kp_sb, kp_sh, kp_sr, vp_sb, vp_sh, vp_sr;
  float* scales;               // [num_blocks][Hkv][2][block_size] (e4m3 pools)
  long long sc_sb, sc_sh, sc_st;
  int* err;
  int B, Hkv, T, max_blocks, block_shift, num_blocks;
  int head_groups;             // set by the launcher
  // elements from the first to one past the last (bounds-checked build)
  long long k_span, v_span, kp_span, vp_span, sc_span, table_span;
};
cudaError_t launch_cache(CacheParams& p, int dim, bool kv8, bool write, bool pdl, cudaStream_t stream);

// --------------------- norms per head and the position rotation, apart or into a paged cache
struct RopeParams {
  CacheParams cache;          // keys (and for pages values and the pools); keys to packed rows: k, k_st, k_sh, Hkv, k_span alone
  const __nv_bfloat16* q;     // [T][Hq][D]
  __nv_bfloat16 *q_out, *k_out;
  long long q_st, q_sh, qo_st, qo_sh, ko_st, ko_sh;
  const void *q_weight, *k_weight;  // [D] bf16 or fp32, null: no norm
  int q_weight_f32, k_weight_f32;
  float eps;
  const float* table;         // [P][R] fp32: cosines, then sines
  long long table_st;
  int P, R;
  const int* pos;             // [A][T] positions (null: the tokens' places in their sequences)
  long long pos_sa;
  int A;
  const int* axes;            // [R / 2] the axis of each pair (null: one axis)
  int* err;
  int T, Hq;                  // heads of q: 0 where there is none
  int groups, q_groups, k_groups;  // set by the launcher: warps of a token, of its queries, of its keys
  long long q_span, qo_span, ko_span;  // elements from the first to one past the last (bounds-checked build)
};
cudaError_t launch_rope(RopeParams& p, int dim, bool halves, bool pages, bool kv8, bool pdl, cudaStream_t stream);

// ------------------------------------------------------- projection: GEMV path
constexpr int kGemvThreads = 256;
constexpr int kGemvCols = 256;  // 32 lanes x 8 columns
constexpr int kGemvMaxKc = 1024;

struct GemvParams {
  const __nv_bfloat16* x;  // [B][K]
  long long x_sb;
  const __nv_bfloat16* w;  // [K][N] row-major
  long long w_sk;
  __nv_bfloat16* y;        // [B][N]
  long long y_sb;
  float* part;             // [ksplit][B][N] fp32 split-K partials
  int* counters;           // [batch chunks][column blocks]
  int* err;                // device error word (bounds-checked build)
  int B, K, N, kc, ksplit;
};

// bt = batch rows per CTA (1, 2, 4 or 8); grid = (col blocks, ksplit, batch chunks).
cudaError_t launch_gemv(const GemvParams& p, int bt, bool pdl, cudaStream_t stream);
size_t gemv_smem_bytes(int bt, int kc);


// ------------------------------------------- projection: tcgen05 tensor-core path
constexpr int kUmmaThreads = 128;  // warp 0: TMA producer, warp 1: MMA issuer, all four: epilogue
constexpr int kUmmaBM = 128;       // hidden columns per tile (the MMA's M, swap-AB)
constexpr int kUmmaBK = 64;        // k rows per pipeline stage

struct UmmaParams {
  CUtensorMap tm_w;  // W [K][N] bf16 row-major: box 64 columns x 64 rows, 128B swizzle
  CUtensorMap tm_x;  // X [B][K] bf16: box 64 k x npad batch rows, 128B swizzle
  __nv_bfloat16* y;  // [B][N]
  long long y_sb;
  float* part;       // [ksplit][B][N] fp32 split-K partials (null: the cluster reduction)
  int* counters;     // [batch chunks][column tiles]
  int* err;
  int B, K, N, ksplit;
  int prefetch;      // 1: pull the k-blocks past the first ring fill into L2 before the PDL wait
  int cluster;       // 1: the ksplit slices of a column tile are one cluster (ksplit <= 8)
};
constexpr int kMaxClusterSplit = 8;  // portable cluster size

// ---------------------------- projection of a single-row batch with W staged on chip
constexpr int kOnchipThreads = 512;   // thread t: 8 columns (piece t % 8 of column tile t / 64), rows (t / 8) % 8 + 8 i
constexpr int kOnchipCols = 512;      // columns of a CTA's group (1 KB of every row of W)
constexpr int kOnchipRegKblocks = 3;  // k-blocks (64 rows) a CTA holds in registers (8 x 16 bytes each per thread)

struct OnchipParams {
  CUtensorMap tm_w;          // W [K][N] bf16 row-major: box 64 columns x 64 rows, 128B swizzle
  const __nv_bfloat16* x;    // [K] the attention output of the one batch row (16-byte aligned)
  const __nv_bfloat16* w;    // W, for the register-held k-blocks
  long long w_sk;            // row stride of W in elements
  __nv_bfloat16* y;          // [N]
  float* part;               // [N / 512 groups][k-ranges][512] fp32 parts
  int* counters;             // [N / 512] completion counters, zero between calls
  int* err;
  int K, N;                  // K a multiple of 64, N of 512
  int kb;                    // K / 64
  int smem_kblocks;          // k-blocks a CTA stages in shared memory (the rest of its range in registers)
};
size_t onchip_smem_bytes(int smem_kblocks, int K);
int onchip_max_smem_kblocks(int K);
// grid = (N / 512 column groups, kgroups k-ranges): one CTA per SM that the attention leaves
// free; each CTA's k-range is at most smem_kblocks + kOnchipRegKblocks k-blocks.
cudaError_t launch_onchip(const OnchipParams& p, int kgroups, bool pdl, cudaStream_t stream);

size_t umma_smem_bytes(int npad);
// grid = (ceil(N / 128), ksplit, ceil(B / npad)); npad in {16, 32, 64, 128}.
cudaError_t launch_umma(const UmmaParams& p, int npad, bool pdl, cudaStream_t stream);

}  // namespace da
