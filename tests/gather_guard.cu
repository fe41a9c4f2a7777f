// Calls the kernel that lays tokens out with one sequence of one KV head and 128 tokens in blocks of 16 (tests/test_gather_guard.py).
#include <string.h>

#include "kernels.h"

extern "C" int gather_one_tile(const void* k_pages, const void* v_pages, const float* scales, const int* cu, const int* lens, const int* table,
                               void* k_out, void* v_out, int* err, int kv8, long long span, void* stream) {
  da::GatherParams p;
  memset(&p, 0, sizeof(p));
  const int es = kv8 ? 1 : 2;
  p.k_pages = static_cast<const uint8_t*>(k_pages);
  p.v_pages = static_cast<const uint8_t*>(v_pages);
  p.kp_sb = p.kp_sh = p.vp_sb = p.vp_sh = 16 * 128 * es;
  p.kp_sr = p.vp_sr = 128 * es;
  p.kp_span = p.vp_span = 8 * 16 * 128 * es;
  p.scales = scales;
  p.sc_sb = p.sc_sh = 2 * 16;
  p.sc_st = 16;
  p.sc_span = 8 * 2 * 16;
  p.cu = cu;
  p.lens = lens;
  p.table = table;
  p.bt_stride = p.table_span = 8;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.span = span;
  p.err = err;
  p.heads = 1;
  p.rows = p.cap = 128;
  p.Tq = 1;
  p.num_blocks = 8;
  p.block_shift = 4;
  p.window = 1 << 30;
  return (int)da::launch_gather(p, 1, kv8 != 0, false, static_cast<cudaStream_t>(stream));
}
