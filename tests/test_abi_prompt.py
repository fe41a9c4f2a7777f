"""Host-side refusals of the prompt attention, the cache's writing and reading and the paged e4m3 step: the documented
status codes, before anything touches the device (fake device addresses, without a GPU only)."""
import ctypes

import pytest

from decode_attention_output_gb300 import binding
from test_abi import ALIGN, DTYPE, FAKE, NULL, OK, SHAPE, STRIDE, UNSUP, cpu_only, desc, lib  # noqa: F401

I32, F32, E4M3 = binding.DA_DTYPE_I32, binding.DA_DTYPE_F32, binding.DA_DTYPE_E4M3


def refs(a, *names):
    return [ctypes.byref(a[n]) if a[n] is not None else None for n in names]


# ------------------------------------------------------------------ prompt attention
def prefill_args(Tq=70, Tk=90, Hq=8, Hkv=2, B=3, **over):
    a = dict(q=desc([Tq, Hq, 128]), k=desc([Tk, Hkv, 128]), v=desc([Tk, Hkv, 128]), cq=desc([B + 1], I32),
             ck=desc([B + 1], I32), out=desc([Tq, Hq, 128]))
    a.update(over)
    return a


def call_prefill(lib, a, scale=0.1):  # noqa: F811
    return lib.decode_attn_prefill(*refs(a, "q", "k", "v", "cq", "ck", "out"), ctypes.c_float(scale), None)


BAD_PREFILL = [
    ("q_dtype", dict(q=desc([70, 8, 128], F32)), DTYPE),
    ("k_dtype", dict(k=desc([90, 2, 128], E4M3)), DTYPE),
    ("cu_dtype", dict(cq=desc([4], F32)), DTYPE),
    ("q_2d", dict(q=desc([70, 1024])), SHAPE),
    ("head_dim_64", dict(q=desc([70, 8, 64]), k=desc([90, 2, 64]), v=desc([90, 2, 64]), out=desc([70, 8, 64])), SHAPE),
    ("head_dim_256", dict(q=desc([70, 8, 256]), k=desc([90, 2, 256]), v=desc([90, 2, 256]), out=desc([70, 8, 256])), UNSUP),
    ("heads_not_multiple", dict(q=desc([70, 7, 128]), out=desc([70, 7, 128])), SHAPE),
    ("group_17", dict(q=desc([70, 34, 128]), out=desc([70, 34, 128])), UNSUP),
    ("v_tokens", dict(v=desc([91, 2, 128])), SHAPE),
    ("out_heads", dict(out=desc([70, 4, 128])), SHAPE),
    ("offsets_differ", dict(ck=desc([5], I32)), SHAPE),
    ("no_offsets", dict(cq=desc([0], I32), ck=desc([0], I32)), SHAPE),
    ("batch_too_large", dict(cq=desc([1026], I32), ck=desc([1026], I32)), UNSUP),
    ("offsets_strided", dict(cq=desc([4], I32, strides=[2])), STRIDE),
    ("offsets_misaligned", dict(ck=desc([4], I32, addr=FAKE + 2)), ALIGN),
    ("q_misaligned", dict(q=desc([70, 8, 128], addr=FAKE + 8)), ALIGN),
    ("out_misaligned", dict(out=desc([70, 8, 128], addr=FAKE + 2)), ALIGN),
    ("out_stride_odd", dict(out=desc([70, 8, 128], strides=[8 * 132, 132, 1])), STRIDE),
    ("k_broadcast", dict(k=desc([90, 2, 128], strides=[128, 0, 1])), STRIDE),
    ("v_inner_stride", dict(v=desc([90, 2, 128], strides=[512, 256, 2])), STRIDE),
    ("null_v", dict(v=None), NULL),
    ("null_offsets", dict(cq=None), NULL),
    ("null_out_data", dict(out=desc([70, 8, 128], addr=None)), NULL),
]


@cpu_only
@pytest.mark.parametrize("name,over,code", BAD_PREFILL, ids=[c[0] for c in BAD_PREFILL])
def test_prefill_rejects(lib, name, over, code):  # noqa: F811
    assert call_prefill(lib, prefill_args(**over)) == code


@cpu_only
def test_prefill_scale_and_empty(lib):  # noqa: F811
    assert call_prefill(lib, prefill_args(), scale=float("inf")) == UNSUP
    assert call_prefill(lib, prefill_args(), scale=float("nan")) == UNSUP
    assert call_prefill(lib, prefill_args(), scale=3e38) == UNSUP  # times log2 e: no float
    a = prefill_args(Tq=0, Tk=0)
    for n in ("q", "k", "v", "out"):
        a[n].data = None
    assert call_prefill(lib, a) == OK
    assert call_prefill(lib, prefill_args(B=0)) == OK


# ------------------------------------------------------------ writing and reading the cache
def cache_args(T=9, H=2, D=128, B=3, nblk=10, bs=16, mb=4, dtype=E4M3, **over):
    a = dict(k=desc([T, H, D]), v=desc([T, H, D]), cu=desc([B + 1], I32), table=desc([B, mb], I32), lens=desc([B], I32),
             kp=desc([nblk, H, bs, D], dtype), vp=desc([nblk, H, bs, D], dtype),
             sc=desc([nblk, H, 2, bs], F32) if dtype == E4M3 else None)
    a.update(over)
    return a


def call_cache(lib, a):  # noqa: F811
    return (lib.decode_attn_cache_write(*refs(a, "k", "v", "cu", "table", "lens", "kp", "vp", "sc"), None),
            lib.decode_attn_cache_read(*refs(a, "kp", "vp", "sc", "table", "cu", "k", "v"), None))


BAD_CACHE = [
    ("k_dtype", dict(k=desc([9, 2, 128], F32)), DTYPE),
    ("pool_f32", dict(kp=desc([10, 2, 16, 128], F32)), DTYPE),
    ("pools_differ", dict(vp=desc([10, 2, 16, 128])), DTYPE),
    ("scales_bf16", dict(sc=desc([10, 2, 2, 16])), DTYPE),
    ("scales_missing", dict(sc=None), NULL),
    ("scales_for_bf16", dict(kp=desc([10, 2, 16, 128]), vp=desc([10, 2, 16, 128])), DTYPE),
    ("scales_one_tensor", dict(sc=desc([10, 2, 1, 16], F32)), SHAPE),
    ("scales_rows", dict(sc=desc([10, 2, 2, 32], F32)), SHAPE),
    ("scales_stride", dict(sc=desc([10, 2, 2, 16], F32, strides=[2 * 34, 34, 17, 1])), STRIDE),
    ("heads_differ", dict(kp=desc([10, 3, 16, 128], E4M3), vp=desc([10, 3, 16, 128], E4M3), sc=desc([10, 3, 2, 16], F32)), SHAPE),
    ("v_tokens", dict(v=desc([8, 2, 128])), SHAPE),
    ("cu_length", dict(cu=desc([3], I32)), SHAPE),
    ("cu_dtype", dict(cu=desc([4], F32)), DTYPE),
    ("table_1d", dict(table=desc([12], I32)), SHAPE),
    ("table_inner_stride", dict(table=desc([3, 4], I32, strides=[8, 2])), STRIDE),
    ("table_rows_overlap", dict(table=desc([3, 4], I32, strides=[3, 1])), STRIDE),
    ("block_size_8", dict(kp=desc([10, 2, 8, 128], E4M3), vp=desc([10, 2, 8, 128], E4M3), sc=desc([10, 2, 2, 8], F32)), UNSUP),
    ("block_size_48", dict(kp=desc([10, 2, 48, 128], E4M3), vp=desc([10, 2, 48, 128], E4M3), sc=desc([10, 2, 2, 48], F32)), UNSUP),
    ("e4m3_d256", dict(k=desc([9, 2, 256]), v=desc([9, 2, 256]), kp=desc([10, 2, 16, 256], E4M3), vp=desc([10, 2, 16, 256], E4M3)),
     UNSUP),
    ("head_dim_64", dict(k=desc([9, 2, 64]), v=desc([9, 2, 64]), kp=desc([10, 2, 16, 64], E4M3), vp=desc([10, 2, 16, 64], E4M3)),
     SHAPE),
    ("empty_pool", dict(kp=desc([0, 2, 16, 128], E4M3), vp=desc([0, 2, 16, 128], E4M3), sc=desc([0, 2, 2, 16], F32)), SHAPE),
    ("batch_too_large", dict(table=desc([1025, 4], I32), cu=desc([1026], I32), lens=desc([1025], I32)), UNSUP),
    ("k_misaligned", dict(k=desc([9, 2, 128], addr=FAKE + 8)), ALIGN),
    ("pool_misaligned", dict(kp=desc([10, 2, 16, 128], E4M3, addr=FAKE + 8)), ALIGN),
    ("pool_row_stride", dict(vp=desc([10, 2, 16, 128], E4M3, strides=[2 * 16 * 136, 16 * 136, 136, 1])), STRIDE),
    ("null_k", dict(k=None), NULL),
    ("null_table", dict(table=None), NULL),
    ("null_cu", dict(cu=None), NULL),
]


@cpu_only
@pytest.mark.parametrize("name,over,code", BAD_CACHE, ids=[c[0] for c in BAD_CACHE])
def test_cache_rejects(lib, name, over, code):  # noqa: F811
    assert call_cache(lib, cache_args(**over)) == (code, code)


@cpu_only
def test_cache_write_needs_lengths(lib):  # noqa: F811
    for lens, code in ((None, NULL), (desc([2], I32), SHAPE), (desc([3], F32), DTYPE), (desc([3], I32, strides=[2]), STRIDE)):
        assert call_cache(lib, cache_args(lens=lens))[0] == code


@cpu_only
def test_cache_accepts_on_the_host(lib):  # noqa: F811
    """Valid calls without a token or a sequence launch nothing."""
    for kw in (dict(), dict(dtype=binding.DA_DTYPE_BF16, bs=8), dict(dtype=binding.DA_DTYPE_BF16, D=256), dict(bs=1 << 20)):
        a = cache_args(T=0, **kw)
        a["k"].data = a["v"].data = None
        assert call_cache(lib, a) == (OK, OK)
        a = cache_args(B=0, **kw)
        a["table"].data = a["lens"].data = None
        assert call_cache(lib, a) == (OK, OK)


# ------------------------------------------------------------- a token over the e4m3 pages
def step_args(B=2, Hq=8, Hkv=2, nblk=10, bs=16, mb=4, N=256, **over):
    a = dict(q=desc([B, Hq, 128]), kp=desc([nblk, Hkv, bs, 128], E4M3), vp=desc([nblk, Hkv, bs, 128], E4M3),
             sc=desc([nblk, Hkv, 2, bs], F32), table=desc([B, mb], I32), lens=desc([B], I32), w=desc([Hq * 128, N]),
             out=desc([B, N]), attn=desc([B, Hq, 128]))
    a.update(over)
    return a


def call_step(lib, a, scale=0.1):  # noqa: F811
    names = ("q", "kp", "vp", "sc", "table", "lens")
    return (lib.decode_attn_fwd_paged_fp8(*refs(a, *names, "w", "out"), ctypes.c_float(scale), None),
            lib.decode_attn_only_paged_fp8(*refs(a, *names, "attn"), ctypes.c_float(scale), None))


BAD_STEP = [
    ("pool_bf16", dict(kp=desc([10, 2, 16, 128]), vp=desc([10, 2, 16, 128])), DTYPE),
    ("v_bf16", dict(vp=desc([10, 2, 16, 128])), DTYPE),
    ("scales_missing", dict(sc=None), NULL),
    ("scales_dtype", dict(sc=desc([10, 2, 2, 16])), DTYPE),
    ("scales_3d", dict(sc=desc([10, 2, 32], F32)), SHAPE),
    ("scales_blocks", dict(sc=desc([9, 2, 2, 16], F32)), SHAPE),
    ("scales_misaligned", dict(sc=desc([10, 2, 2, 16], F32, addr=FAKE + 4)), ALIGN),
    ("block_size_8", dict(kp=desc([10, 2, 8, 128], E4M3), vp=desc([10, 2, 8, 128], E4M3), sc=desc([10, 2, 2, 8], F32)), UNSUP),
    ("block_size_24", dict(kp=desc([10, 2, 24, 128], E4M3), vp=desc([10, 2, 24, 128], E4M3), sc=desc([10, 2, 2, 24], F32)), UNSUP),
    ("d256", dict(q=desc([2, 8, 256]), kp=desc([10, 2, 16, 256], E4M3), vp=desc([10, 2, 16, 256], E4M3), w=desc([2048, 256]),
                  attn=desc([2, 8, 256])), UNSUP),
    ("group_32", dict(q=desc([2, 64, 128]), w=desc([64 * 128, 256]), attn=desc([2, 64, 128])), UNSUP),
    ("table_misaligned", dict(table=desc([2, 4], I32, addr=FAKE + 4)), ALIGN),
    ("null_pool", dict(kp=None), NULL),
]


@cpu_only
@pytest.mark.parametrize("name,over,code", BAD_STEP, ids=[c[0] for c in BAD_STEP])
def test_step_rejects(lib, name, over, code):  # noqa: F811
    assert call_step(lib, step_args(**over)) == (code, code)


@cpu_only
def test_step_scale_and_empty(lib):  # noqa: F811
    assert call_step(lib, step_args(), scale=float("nan")) == (UNSUP, UNSUP)
    for bs in (16, 64, 4096):
        a = step_args(B=0, bs=bs)
        for n in ("q", "table", "lens", "out", "attn"):
            a[n].data = None
        assert call_step(lib, a) == (OK, OK)
