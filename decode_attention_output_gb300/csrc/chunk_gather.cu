// chunk_gather.cu -- the tokens that a call of decode_attn_chunk sees, out of a paged cache's e4m3 or small blocks, as bf16 rows
// one behind the other: what the 128-row tiles of prefill.cuh take by one copy each.
//
// Tile j of a (sequence, KV head) is the j-th tile of 128 keys that some query of the sequence sees (all up to the end, or
// with a window those of the first `sinks` keys and from its beginning on). e4m3: code * scale, rounded once to bf16, as
// decode_attn_cache_read gives it. Rows that no query sees are left as they are.
//
// Bound by bytes; read once and written once whatever the number of queries, where widening in the attention is done for every
// 256 rows of queries (four chunks of 512 tokens over 7.7k, 32 / 8 heads: 328 us widened there, 181 over a bf16 cache). A CTA
// takes a tile of one head at a time, all its loads before its stores. (CTAs that walk all tiles in equal shares, however many:
// 100 new tokens each of 32 sequences over 4k, e4m3: 336 -> 346 us in all.)
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace da {
namespace {

constexpr int kGatherThreads = 256;

// A sequence's tokens (none: nothing of it is laid out) and its first that a window sees; of its tiles the first ns are
// those of `sinks`, then `skip` are left out.
struct Kept {
  int lk, lo, ns, skip;
};
__device__ __forceinline__ Kept kept(const GatherParams& p, int b) {
  Kept s;
  const int q0 = min(max(__ldg(p.cu + b), 0), p.Tq), lq = min(max(__ldg(p.cu + b + 1), q0), p.Tq) - q0;
  s.lk = lq <= p.few_lq ? 0 : min(max(__ldg(p.lens + b), 0), p.cap);
  s.lo = max(0, s.lk - lq - p.window + 1);
  const int first = s.lo / 128;
  s.ns = (p.sinks + 127) / 128;
  s.skip = max(0, first - s.ns);
  return s;
}

template <bool KV8>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int kPieces = KV8 ? 8 : 16, kAt = kGatherThreads / kPieces, kPasses = 128 / kAt;  // 16-byte pieces of a row; rows at a time
  const int c = threadIdx.x % kPieces, row0 = threadIdx.x / kPieces;
  pdl_wait_primary();
  const int b = blockIdx.y, h = blockIdx.z;
  const Kept s = kept(p, b);
  const int lk = s.lk, lo = s.lo, tiles = lk > 0 ? (lk + 127) / 128 - s.skip : 0;
  for (int j = blockIdx.x; j < tiles; j += gridDim.x) {
    const int t = s.skip > 0 && j >= s.ns ? j + s.skip : j;
    uint4 x[2][kPasses];
    float f[2][KV8 ? kPasses : 1];
    bool seen[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int key = t * 128 + i * kAt + row0, row = key & ((1 << p.block_shift) - 1);
      seen[i] = key < lk && (key >= lo || key < p.sinks);
      const long long entry = b * p.bt_stride + (key >> p.block_shift);
      const int id = seen[i] && in_bounds(entry < p.table_span, p.err) ? __ldg(p.table + entry) : -1;
      bool ok = (unsigned)id < (unsigned)p.num_blocks;
      if (seen[i] && !ok) atomicOr(p.err, kErrBlockTable);  // reads as zeros
      const long long k_at = id * p.kp_sb + h * p.kp_sh + row * p.kp_sr + c * 16, v_at = id * p.vp_sb + h * p.vp_sh + row * p.vp_sr + c * 16;
      ok = ok && in_bounds(k_at + 16 <= p.kp_span && v_at + 16 <= p.vp_span, p.err);
      x[0][i] = ok ? ldg_stream_v4(p.k_pages + k_at) : make_uint4(0, 0, 0, 0);
      x[1][i] = ok ? ldg_stream_v4(p.v_pages + v_at) : make_uint4(0, 0, 0, 0);
      if constexpr (KV8) {
        const long long sc = id * p.sc_sb + h * p.sc_sh + row;
        ok = ok && in_bounds(sc + p.sc_st < p.sc_span, p.err);
        f[0][i] = ok ? __ldg(p.scales + sc) : 0.f;
        f[1][i] = ok ? __ldg(p.scales + sc + p.sc_st) : 0.f;
      }
    }
    const long long to = (((long long)b * p.heads + h) * p.rows + j * 128 + row0) * 128 + c * (KV8 ? 16 : 8);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const long long first = to + (long long)i * kAt * 128;  // of this store
      if (!seen[i] || !in_bounds(j * 128 + 128 <= p.rows && first >= 0 && first + (KV8 ? 16 : 8) <= p.span, p.err)) continue;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        __nv_bfloat16* at = (v ? p.v_out : p.k_out) + first;
        if constexpr (KV8) {
          const uint32_t w[4] = {x[v][i].x, x[v][i].y, x[v][i].z, x[v][i].w};
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t lo2, hi2;
            e4m3x4_to_f16x4(w[k], lo2, hi2);
            o[2 * k] = pack_bf16x2(f16lo_to_f32(lo2) * f[v][i], f16hi_to_f32(lo2) * f[v][i]);
            o[2 * k + 1] = pack_bf16x2(f16lo_to_f32(hi2) * f[v][i], f16hi_to_f32(hi2) * f[v][i]);
          }
          *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(at + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
          *reinterpret_cast<uint4*>(at) = x[v][i];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_gather(const GatherParams& p, int batch, bool kv8, bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(p.rows / 128, p.few_lq ? kGatherCtas / 2 : kGatherCtas), (unsigned)batch, (unsigned)p.heads);
  cfg.blockDim = dim3(kGatherThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return kv8 ? cudaLaunchKernelEx(&cfg, gather_kernel<true>, p) : cudaLaunchKernelEx(&cfg, gather_kernel<false>, p);
}

}  // namespace da
