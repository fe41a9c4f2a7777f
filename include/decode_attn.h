/*
 * decode_attn.h -- C ABI of libdecode_attn.so: one decode step of grouped-query
 * attention over a bf16 KV cache, followed by the output projection, on one
 * NVIDIA GB300 (sm_103a).
 *
 * The computation is the one of the page "PyPTO 开箱性能调优实战 Decode
 * Attention 多 Matmul 独立 TileShape 配置 F-16" (eliteato.com/news/26629),
 * section "代码对比": three contractions with their own result types
 *
 *   scores_fp32 = q_grouped . k_cache^T                 (fp32 scores)
 *   weights     = softmax(scale * scores_fp32)          (the "vector ops")
 *   attn_output = weights . v_cache                     (bf16)
 *   result      = attn_output_flat . o_weight           (bf16)
 *
 * and the shapes of its table "三个 Matmul 的 Shape 特征分析" (QK^T: M = query
 * heads per KV head, K = head_dim = 128, N = kv_len; attn.V: M = heads per KV
 * head, K = kv_len, N = 128; output_proj: M = batch, K = heads * 128,
 * N = hidden). Head dim 256 is the page's other GQA decode (section "仓库源码
 * 佐证": QK^T contracts D = 256 in two halves of 128, attn.V has N = D = 256);
 * every entry point takes D = 128 or D = 256, read from q's last extent (those over an
 * fp8 cache, decode_attn_prefill, decode_attn_prefill_window and decode_attn_chunk: D = 128).
 *
 * Conventions shared by every entry point
 *  - Every tensor argument is a da_tensor_t descriptor. Its data pointer is a
 *    DEVICE pointer owned by the caller; the library never frees or keeps it.
 *  - Strides are in elements. The innermost dimension must be contiguous
 *    (stride 1); every other stride of an input must be a multiple of 16 bytes
 *    (8 bf16 elements, 16 e4m3 elements) and every base pointer 16-byte aligned
 *    (TMA and 16-byte vector loads need it).
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream). Every call only enqueues work on it and returns; nothing is
 *    synchronised, nothing is copied back to the host.
 *  - All arguments are validated on the host before anything is launched; on
 *    a failure the call returns a negative da_status_t and launches nothing.
 *    A failed launch returns DA_ERR_CUDA.
 *  - The library owns one workspace per device (partial results of the split
 *    KV pass and of the split-K projection, completion counters, the bf16
 *    attention intermediate). When a call needs more, it is grown in stream
 *    order on that call's stream (cudaMallocAsync of a new block of the power of two
 *    that holds it, from 32 MiB on, or of what is needed where there is no room for that;
 *    cudaMemsetAsync of its header; no device-wide synchronisation). The
 *    old blocks are kept until decode_attn_release, so a graph captured before can be
 *    replayed; together they are smaller than the new one (but where room was short).
 *    A call that would have to grow it while its stream is being captured
 *    returns DA_ERR_NOMEM: the first call with the largest shapes must precede the
 *    capture. Calls on different streams of the same device share it, graph replays
 *    among them: the caller must order them (their work must not overlap on the GPU).
 *    Host threads may call at the same time; each call's launches are enqueued in one go.
 *  - seq_lens lives on the device. Each length is clamped to [0, Lcap] on the
 *    device; a length of 0 gives an all-zero attention row.
 *  - Bounded device waits: every wait inside a kernel gives up after about
 *    two seconds, records a code that decode_attn_last_device_error() returns,
 *    and the kernel then finishes without waiting further (its output is not
 *    valid).
 */
#ifndef DECODE_ATTN_H
#define DECODE_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of da_tensor_t.dtype. */
enum { DA_DTYPE_BF16 = 1, DA_DTYPE_F32 = 2, DA_DTYPE_I32 = 3, DA_DTYPE_E4M3 = 4 /* fp8 e4m3 (OCP "fn") */ };

/* A strided view of caller-owned device memory (DLPack-like). */
typedef struct da_tensor {
  void* data;        /* device pointer */
  int32_t dtype;     /* DA_DTYPE_* */
  int32_t ndim;      /* number of valid entries in shape/stride, 1..4 */
  int64_t shape[4];
  int64_t stride[4]; /* in elements */
} da_tensor_t;

typedef enum {
  DA_OK = 0,
  DA_ERR_NULL = -1,        /* a required pointer or descriptor is NULL */
  DA_ERR_DTYPE = -2,       /* wrong element type */
  DA_ERR_SHAPE = -3,       /* inconsistent or unsupported shape */
  DA_ERR_STRIDE = -4,      /* innermost dim not contiguous, or a stride not a multiple of 8 */
  DA_ERR_ALIGN = -5,       /* base pointer not 16-byte aligned */
  DA_ERR_UNSUPPORTED = -6, /* valid request outside what the kernels implement */
  DA_ERR_NOMEM = -7,       /* the workspace could not be grown */
  DA_ERR_CUDA = -8,        /* a CUDA runtime call or launch failed */
  DA_ERR_OPTION = -9,      /* unknown option key or value out of range */
  DA_ERR_DEVICE = -10,     /* a kernel recorded a device-side error (bounded wait ran out) */
  DA_ERR_SCRATCH = -11     /* decode_attn_only_noalloc: the call needs more than its fixed scratch */
} da_status_t;

/* Limits checked on the host. */
#define DA_HEAD_DIM 128      /* D: the default head dim */
#define DA_HEAD_DIM_WIDE 256 /* D: the other head dim the kernels implement */
#define DA_MAX_GROUP 16  /* G = Hq / Hkv */
#define DA_MAX_BATCH 1024

/*
 * decode_attn_fwd -- the whole step: attention, then the output projection.
 * Page: "PyPTO 开箱性能调优实战 Decode Attention 多 Matmul 独立 TileShape 配置
 * F-16", section "代码对比" (the three matmuls) and the shape table.
 *
 *   q        [B, Hq, D]          bf16  the new token's queries, D = 128 or 256
 *   k_cache  [B, Hkv, Lcap, D]   bf16  keys; token t of sequence b is row t
 *   v_cache  [B, Hkv, Lcap, D]   bf16  values, same shape as k_cache
 *   seq_lens [B]                 int32 valid tokens per sequence (device)
 *   o_weight [Hq*D, N]           bf16  row-major; row k = h*D + d
 *   out      [B, N]              bf16  written
 *   scale    softmax scale applied to the fp32 scores (usually 1/sqrt(D))
 *
 * Query head h attends with KV head h / (Hq / Hkv) over tokens t < seq_lens[b].
 * Requires Hq % Hkv == 0, Hq / Hkv <= 16, B <= 1024, N % 8 == 0; any other D
 * returns DA_ERR_SHAPE.
 * Returns DA_OK or a negative da_status_t.
 */
int decode_attn_fwd(const da_tensor_t* q, const da_tensor_t* k_cache, const da_tensor_t* v_cache,
                    const da_tensor_t* seq_lens, const da_tensor_t* o_weight, const da_tensor_t* out,
                    float scale, void* stream);

/*
 * decode_attn_only -- the attention half: attn_out[b, h, :] =
 * softmax(scale * q[b,h] . K[b, h/G]^T) . V[b, h/G] over t < seq_lens[b],
 * written as bf16 (the page's `attn_output`, DT_BF16).
 *   attn_out [B, Hq, D] bf16, caller-allocated, any strides obeying the
 *   conventions. Other arguments as decode_attn_fwd.
 */
int decode_attn_only(const da_tensor_t* q, const da_tensor_t* k_cache, const da_tensor_t* v_cache,
                     const da_tensor_t* seq_lens, const da_tensor_t* attn_out, float scale,
                     void* stream);

/*
 * decode_attn_only_noalloc -- decode_attn_only for callers that must not allocate
 * device memory at run time: for example a serving process whose GPU memory is
 * reserved up front by its own allocator or memory pool (an allocation outside
 * it can fail, or take memory the pool was sized to own), or a request path with
 * a latency bound, where growing the library workspace (a stream-ordered pool
 * allocation that may have to map new device memory) is not allowed. The pages
 * have no counterpart; this is a deployment convenience, with the same arguments
 * and the same result as decode_attn_only.
 *
 * Scratch: a fixed 8 MiB device array inside the library, held by every GPU that
 * loads it until the process exits. It is never allocated or freed and no
 * allocating routine is called. The split-KV partials need one slot per
 * (sequence, KV head) pair plus one per persistent CTA: on a 152-SM GB300 with
 * the default grid that allows B*Hkv up to 1738 when Hq/Hkv <= 8 and up to 793
 * when Hq/Hkv <= 16 at D = 128; at D = 256 up to 800 and 324. A larger call
 * returns DA_ERR_SCRATCH and launches nothing.
 *
 * - The first call on a device looks up the array's device address (no
 *   allocation); make that first call before any stream capture.
 * - Every call clears the error word and its completion counters with
 *   cudaMemsetAsync on `stream` before the kernel, because the array keeps the
 *   previous call's contents.
 * - All calls share the one array: calls whose work overlaps on the GPU (other
 *   streams, other host threads) race on it and must be serialised by the caller.
 * - Device-side wait timeouts are recorded in the array's own error word, which
 *   decode_attn_last_device_error() reads and clears together with the
 *   workspace's (until the next call of this entry point clears it).
 */
int decode_attn_only_noalloc(const da_tensor_t* q, const da_tensor_t* k_cache, const da_tensor_t* v_cache,
                             const da_tensor_t* seq_lens, const da_tensor_t* attn_out, float scale,
                             void* stream);

/*
 * decode_attn_fwd_paged / decode_attn_only_paged -- decode_attn_fwd / decode_attn_only
 * over a paged KV cache: the keys and values live in a pool of fixed-size blocks and
 * a per-sequence block table lists the blocks of each sequence in token order. The
 * pages have no paged cache; the computation is exactly that of the contiguous entry
 * points on the cache the table describes,
 *
 *   K[b, j, t, :] = k_pages[block_table[b, t / block_size], j, t % block_size, :]
 *
 * for t < seq_lens[b] (and the same for V).
 *   k_pages     [num_blocks, Hkv, block_size, D] bf16  the key pool (device). Any strides
 *               obeying the conventions, so a pool stored as [num_blocks, block_size,
 *               Hkv, D] is passed as the view with dims 1 and 2 swapped.
 *   v_pages     same shape as k_pages (its own strides)
 *   block_table [B, max_blocks] int32 (device), rows contiguous, base 16-byte aligned
 *               (it is read by TMA): entry i of row b is the pool block holding tokens
 *               [i * block_size, (i + 1) * block_size) of sequence b. Only the first
 *               ceil(seq_lens[b] / block_size) entries of a row are used (a few entries
 *               past them may be fetched, never past the table's last entry).
 *   seq_lens    [B] int32 (device), clamped to [0, max_blocks * block_size]
 *   q, o_weight, out, attn_out, scale: as decode_attn_fwd / decode_attn_only.
 * block_size: a power of two from 8 to 2^20; anything else returns DA_ERR_UNSUPPORTED.
 * (Blocks of 32 tokens and more stream at 90-95% of the contiguous rate on GB300; 16
 * at about 75%, 8 at about 55%.) A table entry outside [0, num_blocks) that
 * is read sets bit 64 of the device error word (decode_attn_last_device_error) and that
 * block reads as zeros. The fused option does not apply: two launches.
 */
int decode_attn_fwd_paged(const da_tensor_t* q, const da_tensor_t* k_pages, const da_tensor_t* v_pages,
                          const da_tensor_t* block_table, const da_tensor_t* seq_lens, const da_tensor_t* o_weight,
                          const da_tensor_t* out, float scale, void* stream);
int decode_attn_only_paged(const da_tensor_t* q, const da_tensor_t* k_pages, const da_tensor_t* v_pages,
                           const da_tensor_t* block_table, const da_tensor_t* seq_lens, const da_tensor_t* attn_out,
                           float scale, void* stream);

/*
 * decode_attn_fwd_fp8 / decode_attn_only_fp8 -- decode_attn_fwd / decode_attn_only over
 * an fp8 KV cache: k_cache and v_cache hold e4m3 codes (DA_DTYPE_E4M3, the OCP "fn"
 * format: 4 exponent bits with bias 7, 3 mantissa bits, no infinities), and the keys and
 * values are
 *
 *   K = k_cache * k_scale,   V = v_cache * v_scale       (one float scale per cache)
 *
 * The pages have no fp8 cache; the computation is exactly that of the bf16 entry points
 * on these K and V. The cache bytes halve; q, o_weight and the outputs stay bf16.
 *   k_cache, v_cache [B, Hkv, Lcap, 128] e4m3; strides multiples of 16 elements (bytes)
 *   k_scale, v_scale finite floats (DA_ERR_UNSUPPORTED otherwise)
 *   other arguments as decode_attn_fwd / decode_attn_only
 * Head dim 128 only (D = 256 returns DA_ERR_UNSUPPORTED); the fused option does not apply.
 * The kernels widen the codes to f16 (exact) and multiply them with q rounded to f16,
 * which is exact for 2^-17 <= |q| <= 65504 (and 0); smaller |q| goes to the nearest
 * multiple of 2^-24, larger |q| is clamped to 65504. The softmax weights enter P.V as
 * f16 (bf16 on the bf16 path).
 */
int decode_attn_fwd_fp8(const da_tensor_t* q, const da_tensor_t* k_cache, const da_tensor_t* v_cache,
                        const da_tensor_t* seq_lens, const da_tensor_t* o_weight, const da_tensor_t* out, float scale,
                        float k_scale, float v_scale, void* stream);
int decode_attn_only_fp8(const da_tensor_t* q, const da_tensor_t* k_cache, const da_tensor_t* v_cache,
                         const da_tensor_t* seq_lens, const da_tensor_t* attn_out, float scale, float k_scale,
                         float v_scale, void* stream);

/*
 * decode_attn_fwd_paged_fp8 / decode_attn_only_paged_fp8 -- decode_attn_fwd_paged /
 * decode_attn_only_paged over a paged fp8 cache with a scale for every token and KV head, the
 * cache that decode_attn_cache_write fills:
 *
 *   K[b, j, t, :] = k_pages[i, j, r, :] * kv_scales[i, j, 0, r]
 *   V[b, j, t, :] = v_pages[i, j, r, :] * kv_scales[i, j, 1, r]
 *   i = block_table[b, t / block_size],  r = t % block_size
 *
 *   k_pages, v_pages [num_blocks, Hkv, block_size, 128] e4m3; strides multiples of 16 elements
 *   kv_scales [num_blocks, Hkv, 2, block_size] fp32 (K's scales, then V's); strides multiples
 *             of 4 elements. Any finite values, in any mixture; V's of 2^-100 and more in
 *             magnitude keep the accuracy of the other entry points (smaller ones lose it
 *             gradually), 0 makes the row zero. A token whose softmax weight is below 2^-126 of
 *             the largest counts as none.
 *   other arguments as decode_attn_fwd_paged / decode_attn_only_paged
 * block_size: a power of two from 16 to 2^20. Head dim 128 only (D = 256 returns
 * DA_ERR_UNSUPPORTED). q and the softmax weights as in decode_attn_fwd_fp8. A table entry
 * outside the pool sets bit 64 of the error word and its block reads as zeros.
 */
int decode_attn_fwd_paged_fp8(const da_tensor_t* q, const da_tensor_t* k_pages, const da_tensor_t* v_pages,
                              const da_tensor_t* kv_scales, const da_tensor_t* block_table,
                              const da_tensor_t* seq_lens, const da_tensor_t* o_weight, const da_tensor_t* out,
                              float scale, void* stream);
int decode_attn_only_paged_fp8(const da_tensor_t* q, const da_tensor_t* k_pages, const da_tensor_t* v_pages,
                               const da_tensor_t* kv_scales, const da_tensor_t* block_table,
                               const da_tensor_t* seq_lens, const da_tensor_t* attn_out, float scale, void* stream);

/*
 * decode_attn_prefill -- causal attention over whole prompts: the queries of B packed sequences
 * of different lengths (tokens laid end to end, no padding) over their keys and values.
 *
 *   q [Tq, Hq, 128] bf16, k and v [Tk, Hkv, 128] bf16; out [Tq, Hq, 128] bf16, written
 *   cu_seqlens_q, cu_seqlens_k [B + 1] int32 (device): sequence b holds rows
 *     cu_seqlens_q[b] .. cu_seqlens_q[b + 1] of q and out, and rows cu_seqlens_k[b] ..
 *     cu_seqlens_k[b + 1] of k and v: Lq queries, which are the LAST Lq of its Lk tokens
 *     (Lq < Lk: a prompt whose beginning is cached already, see decode_attn_cache_read)
 *   scale  softmax scale, any float (its product with log2 e finite)
 *
 * Query i of a sequence (0 <= i < Lq) attends keys j <= i + Lk - Lq; query head h attends with
 * KV head h / (Hq / Hkv). A query without a key (Lk < Lq: the first Lq - Lk ones) gives a row
 * of zeros. Rows of q that belong to no sequence are left as they were in out. Offsets must
 * not decrease; they are clamped to [0, Tq] and [0, Tk], and whatever they hold nothing but
 * rows of out is written (where they do decrease, which rows is unspecified).
 * Other sequences' rows never reach a sequence's output, whatever they hold; a NaN or infinity
 * in a sequence's own k or v can make any output row of that sequence and KV head non-finite.
 * Requires Hq % Hkv == 0, Hq / Hkv <= 16, B <= 1024, D = 128 (256 returns DA_ERR_UNSUPPORTED);
 * out 16-byte aligned with strides multiples of 8 elements, like the inputs.
 * The softmax weights enter P.V as bf16, unnormalised; sums and the accumulation are fp32.
 * With few queries over many keys the keys are cut into parts that meet in the workspace
 * (by Tq, Tk, B, the head counts and the sequence's own lengths); results do not depend on timing.
 */
int decode_attn_prefill(const da_tensor_t* q, const da_tensor_t* k, const da_tensor_t* v,
                        const da_tensor_t* cu_seqlens_q, const da_tensor_t* cu_seqlens_k, const da_tensor_t* out,
                        float scale, void* stream);

/*
 * decode_attn_prefill_window -- decode_attn_prefill in which the query at position i of its sequence
 * sees keys i - window + 1 .. i and those below `sinks` (the first tokens, which stay visible):
 *   window  0: no window (sinks is not looked at), else >= 1;  sinks >= 0
 * Tiles that no row of a work item sees are not read. Everything else as decode_attn_prefill
 * (position i of a sequence's query r is r + Lk - Lq). Negative numbers return DA_ERR_UNSUPPORTED.
 */
int decode_attn_prefill_window(const da_tensor_t* q, const da_tensor_t* k, const da_tensor_t* v,
                               const da_tensor_t* cu_seqlens_q, const da_tensor_t* cu_seqlens_k, const da_tensor_t* out,
                               float scale, int32_t window, int32_t sinks, void* stream);

/*
 * decode_attn_chunk -- attention of new tokens over a paged cache that holds their keys and values
 * already: the next chunk of prompts, drafted tokens, or one token a sequence, in any mixture. What
 * decode_attn_cache_read and decode_attn_prefill give together, without the copy.
 *
 *   q, out      [Tq, Hq, 128] bf16; 16-byte aligned, strides multiples of 8 elements
 *   k_pages, v_pages [num_blocks, Hkv, block_size, 128] bf16 or e4m3, any strides obeying the conventions
 *   kv_scales   [num_blocks, Hkv, 2, block_size] fp32 for e4m3 pools; NULL for bf16
 *   block_table [B, max_blocks] int32 (device), rows contiguous
 *   cu_seqlens  [B + 1] int32 (device): rows cu_seqlens[b] .. cu_seqlens[b + 1] of q are the last tokens
 *   seq_lens    [B] int32 (device) of the seq_lens[b] tokens of sequence b, clamped to
 *               [0, max_blocks * block_size]
 *   scale, window, sinks: as decode_attn_prefill_window
 *
 * The query at position i sees keys 0 .. i, or with a window i - window + 1 .. i and those below
 * `sinks`. A query without a key gives a row of zeros; rows of q that belong to no sequence
 * are left as they were in out. An e4m3 key or value is code * scale, rounded to bf16 where a call has many
 * rows (exact for the powers of two that decode_attn_cache_write gives; scales: any finite values, V's from 2^-100 on in
 * magnitude, or 0).
 * Table entries and tokens that no query of the call sees are not read: blocks that a window has
 * left behind may belong to others by now, and what rows past seq_lens hold does not matter. An entry outside
 * the pool that is read sets bit 64 of the device error word and its block reads as zeros. A NaN or infinity in a
 * key or value that some query of a sequence sees can make any output row of that sequence and KV head non-finite.
 * block_size: a power of two from 8 (e4m3: 16) to 2^20. Other limits as decode_attn_prefill. The softmax weights enter
 * P.V unnormalised as bf16, or (e4m3, few rows) with V's scale as f16, off by 2^-25 of the row's largest product
 * of weight and scale at most; weights below 2^-126 of the row's largest count as 0. A score has to stay in fp32's range, and so
 * have its product with codes before their scale and a row's sum of values times weights (up to 2^8 each before the division; values
 * up to 2^90 always do).
 *
 * By Tq * G / B (rows of a sequence and KV head on average) and the pool: few rows are taken 8 or 16 at a time over
 * K and V as they lie, and items that several CTAs share meet in the workspace; many rows 256 at a time, over
 * bf16 blocks of 64 tokens and more as they lie, and else over a bf16 copy of the tokens that the call sees in
 * the workspace: so much of the tables' capacity at a time as a block of 4 GiB holds (or one head of one sequence, if that has more), the
 * rest after it. Where the device or the option "workspace_mib" has no such block, half as much at a time, and so on; a size that the device
 * did not have is not asked for again until decode_attn_release or a larger block. DA_ERR_NOMEM where one head of one sequence does not fit.
 * Of a batch over such a copy, of more than 24 rows on average and of more (sequence, KV head) pairs than SMs, each sequence goes
 * the way of its own rows. Else the average decides for all: a long chunk among very many single tokens is then taken 16 rows at a
 * time (1280 new tokens and 255 single ones over 8k, e4m3, 32 / 8 heads: 1977 us; in two calls 184 + 658), and single tokens among few
 * long chunks 256 at a time. Where the host knows the lengths, such a batch is better called in two.
 */
int decode_attn_chunk(const da_tensor_t* q, const da_tensor_t* k_pages, const da_tensor_t* v_pages, const da_tensor_t* kv_scales,
                      const da_tensor_t* block_table, const da_tensor_t* cu_seqlens, const da_tensor_t* seq_lens,
                      const da_tensor_t* out, float scale, int32_t window, int32_t sinks, void* stream);

/*
 * decode_attn_cache_write -- the keys and values of new tokens into a paged cache, as
 * decode_attn_*_paged (bf16 pools: copied) or decode_attn_*_paged_fp8 (e4m3 pools: quantised)
 * read them.
 *
 *   k, v        [T, Hkv, D] bf16: the new tokens of B packed sequences
 *   cu_seqlens  [B + 1] int32 (device): sequence b holds rows cu_seqlens[b] .. cu_seqlens[b + 1]
 *   block_table [B, max_blocks] int32 (device), rows contiguous
 *   seq_lens    [B] int32 (device): tokens of each sequence, the new ones among them: its n
 *               rows are tokens seq_lens[b] - n .. seq_lens[b] - 1 (a decode step after its
 *               token: n = 1 and the same seq_lens that its attention takes)
 *   k_pages, v_pages [num_blocks, Hkv, block_size, D] bf16 (D = 128 or 256) or e4m3 (D = 128),
 *               any strides obeying the conventions; written
 *   kv_scales   [num_blocks, Hkv, 2, block_size] fp32, written, for e4m3 pools; NULL for bf16
 *
 * e4m3: per token and head, of K and of V alike, scale = 2^e with the least e for which the
 * row's largest finite magnitude is at most 448 * 2^e (e in [-124, 120]; 1 for a row of
 * zeros), code = e4m3(x / scale), rounded to nearest even; infinities become the largest code,
 * +-448, NaN the NaN code. Every code * scale is a bf16 value (under 2^120, for rows that pass
 * 2.98e38, codes end at +-240 for that).
 * Nothing else in the pools is touched. Rows that belong to no sequence, and tokens before a
 * sequence's first (a negative position), are not written; a token past max_blocks *
 * block_size, or whose table entry lies outside the pool, is not written and sets bit 64 of the
 * device error word. Two tokens of one call must not share a place (a block that two
 * sequences share is for reading only): what such a row holds afterwards is unspecified.
 * block_size: a power of two from 8 (e4m3: 16) to 2^20. B <= 1024.
 */
int decode_attn_cache_write(const da_tensor_t* k, const da_tensor_t* v, const da_tensor_t* cu_seqlens,
                            const da_tensor_t* block_table, const da_tensor_t* seq_lens, const da_tensor_t* k_pages,
                            const da_tensor_t* v_pages, const da_tensor_t* kv_scales, void* stream);

/*
 * decode_attn_cache_read -- the first tokens of B sequences out of a paged cache (bf16 or
 * e4m3), packed: row cu_seqlens[b] + t of k_out and v_out [T, Hkv, D] bf16 is token t of
 * sequence b, 0 <= t < cu_seqlens[b + 1] - cu_seqlens[b] (e4m3: code * scale, rounded once to
 * bf16; exact for what decode_attn_cache_write wrote). The k and v of decode_attn_prefill for
 * prompts whose beginning is cached. Other arguments and limits as decode_attn_cache_write;
 * rows that belong to no sequence are left as they were; a token past max_blocks * block_size,
 * or whose table entry lies outside the pool, reads as zeros and sets bit 64.
 * k_out, v_out 16-byte aligned with strides multiples of 8 elements.
 */
int decode_attn_cache_read(const da_tensor_t* k_pages, const da_tensor_t* v_pages, const da_tensor_t* kv_scales,
                           const da_tensor_t* block_table, const da_tensor_t* cu_seqlens, const da_tensor_t* k_out,
                           const da_tensor_t* v_out, void* stream);

/*
 * decode_attn_rope -- the norms per head and the position rotation of packed tokens' queries and
 * keys, in one pass: what stands between their projection and an attention.
 *
 *   q [T, Hq, D], k [T, Hkv, D] bf16, D = 128 or 256; q_out and k_out like them, written, apart
 *              or the same memory as their inputs (in place; no other overlap). q with q_out, or k
 *              with k_out, may be NULL.
 *   cos_sin    [P, R] fp32: of the R / 2 pairs of dims that are rotated, the cosines and then the
 *              sines at each position; R a multiple of 8, at most D
 *   positions  [T] int32 (device), or [A, T] for positions of A axes (A <= 4: time, height,
 *              width); the last dimension contiguous
 *   q_weight, k_weight [D] bf16 or fp32, contiguous and 16-byte aligned: the norm's weights; NULL:
 *              no norm
 *   axes       [R / 2] int32 (device), contiguous: the position axis that each pair follows; NULL: axis 0
 *              (A > 1 needs it)
 *   eps        finite, >= 0
 *   interleaved  0: pair i is dims (i, i + R / 2); 1: dims (2 i, 2 i + 1)
 *
 * Per row: y = x / sqrt(mean(x^2) + eps) * weight where there is one; then (a, b) becomes
 * (a c - b s, b c + a s) for each pair; dims from R on keep y. All in fp32 (the mean's sum too),
 * rounded once to bf16 (with a weight, a row whose squares' sum leaves fp32's range gives zeros, infinities or NaN).
 * A position outside [0, P), or an axis outside [0, A), counts as an angle of
 * 0 and sets bit 128 of the device error word.
 */
int decode_attn_rope(const da_tensor_t* q, const da_tensor_t* k, const da_tensor_t* cos_sin, const da_tensor_t* positions,
                     const da_tensor_t* q_out, const da_tensor_t* k_out, const da_tensor_t* q_weight, const da_tensor_t* k_weight,
                     const da_tensor_t* axes, float eps, int32_t interleaved, void* stream);

/*
 * decode_attn_rope_cache_write -- decode_attn_rope of the new tokens' q and k, with k and v going
 * straight into a paged cache: decode_attn_rope and decode_attn_cache_write in one launch.
 *
 *   q, q_out [T, Hq, D] bf16, or both NULL; k, v [T, Hkv, D] bf16
 *   cos_sin, q_weight, k_weight, axes, eps, interleaved: as decode_attn_rope
 *   positions  as decode_attn_rope, or NULL: each token's place in its sequence (one axis)
 *   cu_seqlens, block_table, seq_lens, k_pages, v_pages, kv_scales: as decode_attn_cache_write
 *
 * A bf16 pool holds what decode_attn_rope gives for k, and v unchanged. An e4m3 pool's codes and
 * scales of k come from the rotated fp32 values directly (one rounding: they can differ by one from
 * those of the bf16 values), by the rule of decode_attn_cache_write; v's are that function's own.
 * Tokens that decode_attn_cache_write would not write are not written; q_out is left as it was in
 * rows that belong to no sequence and in those before a sequence's first token. Bits 64 and 128
 * of the device error word as in those two functions.
 */
int decode_attn_rope_cache_write(const da_tensor_t* q, const da_tensor_t* k, const da_tensor_t* v, const da_tensor_t* cos_sin,
                                 const da_tensor_t* cu_seqlens, const da_tensor_t* block_table, const da_tensor_t* seq_lens,
                                 const da_tensor_t* q_out, const da_tensor_t* k_pages, const da_tensor_t* v_pages,
                                 const da_tensor_t* kv_scales, const da_tensor_t* positions, const da_tensor_t* q_weight,
                                 const da_tensor_t* k_weight, const da_tensor_t* axes, float eps, int32_t interleaved, void* stream);

/*
 * decode_attn_scores -- the first contraction alone: the page's `scores_fp32`
 * (q_grouped . k_cache^T, b_trans=True), unscaled, in fp32.
 *   scores [B, Hq, Lcap] fp32: scores[b, h, t] is written for t < seq_lens[b]
 *   only; entries at t >= seq_lens[b] are left as they were.
 * A checking and tuning hook; it runs the attention kernel's QK^T code.
 */
int decode_attn_scores(const da_tensor_t* q, const da_tensor_t* k_cache,
                       const da_tensor_t* seq_lens, const da_tensor_t* scores, void* stream);

/*
 * decode_attn_oproj -- the last contraction alone: out = attn_flat . o_weight
 * (the page's output_proj: M = batch, K = Hq*128, N = hidden), bf16 operands,
 * fp32 accumulation, bf16 result.
 *   attn_flat [B, K] bf16;  o_weight [K, N] bf16 row-major;  out [B, N] bf16.
 * Requires N % 8 == 0 and K % 8 == 0.
 */
int decode_attn_oproj(const da_tensor_t* attn_flat, const da_tensor_t* o_weight,
                      const da_tensor_t* out, void* stream);

/*
 * Tuning options (process-wide; 0 = automatic). Keys:
 *   "attn_ctas"     CTAs of the persistent attention kernel (0: one per SM, fewer for
 *                   small problems: about four tiles each by the cache capacity;
 *                   at most 512; paged fp8 caches: a tile each up to 16 tiles of
 *                   capacity a sequence, and where the longest sequence allows it
 *                   each one gets CTAs of its own; a set count is kept, its tiles
 *                   split evenly)
 *   "oproj_path"    0 auto, 1 CUDA-core GEMV, 2 tcgen05 tensor-core GEMM, 3 (decode_attn_fwd
 *                   at batch 1) o_weight staged in the shared memory and registers of the
 *                   SMs the attention leaves free while the attention runs, then a CUDA-core
 *                   product (correct, measured slower on GB300; auto where it does not fit)
 *   "oproj_splitk"  split-K factor of the projection (0: auto, two CTAs per SM, at
 *                   most 8, at most 6 when K > 4096)
 *   "attn_cluster"  1 (default): where there is room for two or more CTAs per
 *                   (batch, KV head) sequence, the attention kernel is launched in
 *                   thread-block clusters of up to 8 CTAs (decode_attn_fwd: only
 *                   above about four tiles per SM). When every sequence has the same
 *                   length, each gets the CTAs of one cluster and their partial
 *                   states merge in distributed shared memory; otherwise the tiles
 *                   are split evenly over the whole grid as in the flat mode, and
 *                   only the sequences whose parts fall in one cluster merge on
 *                   chip (the rest through L2). 2: as 1, and decode_attn_fwd
 *                   takes clusters at every size too. 0: always the flat grid.
 *                   Paged fp8 caches: clusters of 4 where few sequences have a
 *                   long capacity, and on chip only while they are short, as 8
 *                   CTAs a sequence would leave the other SMs idle.
 *                   Results agree within the rounding of the merge order.
 *   "oproj_cluster" 1 (default): the split-K slices of a tcgen05 column tile form a
 *                   thread-block cluster and reduce in distributed shared memory
 *                   (split-K <= 8); 0: through global partials and an atomic counter
 *   "gemm_min_batch" smallest batch that takes the tensor-core GEMM in auto mode
 *                   (default 1: every batch; the GEMV measured slower on GB300)
 *   "pdl"           1 (default): launch the projection with programmatic
 *                   dependent launch so it overlaps the attention kernel's tail
 *   "attn_pdl"      1 (default): launch the attention kernel with programmatic
 *                   dependent launch too; it waits for the previous kernel in the
 *                   stream to complete before its first global-memory access (every
 *                   input is read after that), so only its start-up overlaps
 *   "attn_trigger"  3 (default): in decode_attn_fwd each attention CTA lets the
 *                   projection kernel launch when it reaches the tile this many
 *                   before the end of its range, so that the projection's early
 *                   o_weight loads overlap the attention's last tiles and merges
 *                   rather than queue in front of its K/V stream; 0: right after
 *                   the attention's set-up. Timing only: results are identical.
 *   "l2_prefetch"   0 (default) or 1: in decode_attn_fwd the attention kernel
 *                   pulls o_weight into L2 while it streams K/V, so that the
 *                   projection reads o_weight from L2 (measured slower on GB300:
 *                   the prefetch competes with the K/V stream)
 *   "attn_stages"   4 (default) or 6: depth of the attention kernel's K/V ring
 *                   (6 only at D = 128, bf16 or fp8 cache, and when it fits in shared
 *                   memory for the batch)
 *   "fused"         0 (default): decode_attn_fwd runs two launches (attention,
 *                   projection); 1: one persistent cooperative launch (attention,
 *                   a bounded grid barrier, tcgen05 projection) when batch <= 128
 *                   (correct, but measured slower on GB300 so far); head dim 128
 *                   only: at D = 256 decode_attn_fwd always takes two launches
 *   "fused_attn_ctas" attention workers of the fused step (0: about four 64-token
 *                   tiles each, at most one per SM; the other CTAs start on o_weight)
 *   "oproj_prefetch" 0 (default) or 1: in decode_attn_fwd each tcgen05 projection CTA
 *                   pulls the part of its o_weight slice that its ring does not hold
 *                   into L2 before it waits for the attention kernel (measured no
 *                   faster on GB300)
 *   "workspace_mib" 0 (default): a block of the workspace is as large as calls need; else at most
 *                   so many MiB (up to 1048576). A call that needs more returns DA_ERR_NOMEM, but
 *                   decode_attn_chunk takes its tokens in smaller shares. Blocks that are there stay.
 *   "grid_wait_us"  test hook: the fused step's grid-barrier wait limit in microseconds
 *                   (0, the default: two seconds; at most 2000000)
 *   "grid_wait_extra" test hook, 0 (default) or 1: the fused step's grid barrier waits
 *                   for this many arrivals beyond the grid, so that with 1 the wait runs
 *                   out, records error bit 32 and the kernel completes with an invalid
 *                   result (a failure that touches no bad address and hangs nothing)
 * Returns DA_OK or DA_ERR_OPTION.
 */
int decode_attn_set_option(const char* key, int64_t value);
int decode_attn_get_option(const char* key, int64_t* value);

/*
 * decode_attn_last_device_error -- synchronises `stream`, then reports in
 * *host_code the device error word of the current device (the bitwise OR of the
 * workspace's word and the no-allocation scratch's word): 0 when no kernel
 * recorded an error. Codes (bits): 1 a consumer gave up waiting for a K/V stage,
 * 2 a producer gave up waiting for a free stage, 4 copies still in flight at
 * exit, 8 a tensor-core completion never arrived, 32 the fused step's grid
 * barrier did not complete, 64 a paged cache's block table named a block outside
 * the pool, 128 a position outside the table of cosines and sines. A non-zero word is cleared, and with it the completion counters and
 * grid-barrier words beside it (a CTA that gave up left them short of the count
 * that resets them), so that the next call starts clean. Returns DA_OK, or
 * DA_ERR_CUDA when the synchronisation or a copy failed.
 */
int decode_attn_last_device_error(void* stream, int32_t* host_code);
/* The same call under its earlier name. */
int decode_attn_device_error(void* stream, int32_t* host_code);

/* Frees the workspace of every device (synchronises those devices). Graphs captured before
 * must not be replayed afterwards. */
void decode_attn_release(void);

/* A static, human-readable name for a da_status_t. */
const char* decode_attn_status_str(int code);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_ATTN_H */
