"""Host-side refusals of decode_attn_chunk and decode_attn_prefill_window: the documented status codes, before anything touches
the device (fake device addresses, without a GPU only), and tensors that are not on the current device."""
import ctypes

import pytest
import torch

import decode_attention_output_gb300 as da
from decode_attention_output_gb300 import binding
from test_abi import ALIGN, DTYPE, FAKE, NULL, OK, SHAPE, STRIDE, UNSUP, cpu_only, desc, lib  # noqa: F401
from test_abi_prompt import BAD_PREFILL, E4M3, F32, I32, prefill_args, refs

NAMES = ("q", "kp", "vp", "sc", "table", "cu", "lens", "out")


def chunk_args(T=9, Hq=8, H=2, D=128, B=3, nblk=10, bs=16, mb=4, dtype=E4M3, **over):
    a = dict(q=desc([T, Hq, D]), kp=desc([nblk, H, bs, D], dtype), vp=desc([nblk, H, bs, D], dtype),
             sc=desc([nblk, H, 2, bs], F32) if dtype == E4M3 else None, table=desc([B, mb], I32), cu=desc([B + 1], I32),
             lens=desc([B], I32), out=desc([T, Hq, D]))
    a.update(over)
    return a


def call_chunk(lib, a, scale=0.1, window=0, sinks=0):  # noqa: F811
    return lib.decode_attn_chunk(*refs(a, *NAMES), ctypes.c_float(scale), window, sinks, None)


BF16 = binding.DA_DTYPE_BF16
BAD = [
    ("q_dtype", dict(q=desc([9, 8, 128], F32)), DTYPE),
    ("out_heads", dict(out=desc([9, 4, 128])), SHAPE),
    ("out_stride", dict(out=desc([9, 8, 128], strides=[8 * 132, 132, 1])), STRIDE),
    ("q_misaligned", dict(q=desc([9, 8, 128], addr=FAKE + 8)), ALIGN),
    ("pool_f32", dict(kp=desc([10, 2, 16, 128], F32)), DTYPE),
    ("pools_differ", dict(vp=desc([10, 2, 16, 128])), DTYPE),
    ("pool_shapes", dict(vp=desc([9, 2, 16, 128], E4M3)), SHAPE),
    ("pool_3d", dict(kp=desc([10, 16, 128], E4M3)), SHAPE),
    ("pool_misaligned", dict(kp=desc([10, 2, 16, 128], E4M3, addr=FAKE + 8)), ALIGN),
    ("scales_missing", dict(sc=None), NULL),
    ("scales_rows", dict(sc=desc([10, 2, 2, 32], F32)), SHAPE),
    ("scales_for_bf16", dict(kp=desc([10, 2, 16, 128]), vp=desc([10, 2, 16, 128])), DTYPE),
    ("block_size_8", dict(kp=desc([10, 2, 8, 128], E4M3), vp=desc([10, 2, 8, 128], E4M3), sc=desc([10, 2, 2, 8], F32)), UNSUP),
    ("block_size_48", dict(kp=desc([10, 2, 48, 128], E4M3), vp=desc([10, 2, 48, 128], E4M3), sc=desc([10, 2, 2, 48], F32)), UNSUP),
    ("heads_not_multiple", dict(q=desc([9, 7, 128]), out=desc([9, 7, 128])), SHAPE),
    ("group_17", dict(q=desc([9, 34, 128]), out=desc([9, 34, 128])), UNSUP),
    ("head_dim_256", dict(q=desc([9, 8, 256]), out=desc([9, 8, 256]), kp=desc([10, 2, 16, 256], E4M3), vp=desc([10, 2, 16, 256], E4M3),
                          sc=desc([10, 2, 2, 16], F32)), UNSUP),
    ("head_dim_64", dict(q=desc([9, 8, 64]), out=desc([9, 8, 64]), kp=desc([10, 2, 16, 64], E4M3), vp=desc([10, 2, 16, 64], E4M3)), SHAPE),
    ("pool_dim", dict(kp=desc([10, 2, 16, 256], E4M3), vp=desc([10, 2, 16, 256], E4M3)), SHAPE),
    ("empty_pool", dict(kp=desc([0, 2, 16, 128], E4M3), vp=desc([0, 2, 16, 128], E4M3), sc=desc([0, 2, 2, 16], F32)), SHAPE),
    ("table_1d", dict(table=desc([12], I32)), SHAPE),
    ("table_dtype", dict(table=desc([3, 4], F32)), DTYPE),
    ("table_inner_stride", dict(table=desc([3, 4], I32, strides=[8, 2])), STRIDE),
    ("table_rows_overlap", dict(table=desc([3, 4], I32, strides=[3, 1])), STRIDE),
    ("table_misaligned", dict(table=desc([3, 4], I32, addr=FAKE + 2)), ALIGN),
    ("cu_length", dict(cu=desc([3], I32)), SHAPE),
    ("cu_strided", dict(cu=desc([4], I32, strides=[2])), STRIDE),
    ("lens_length", dict(lens=desc([4], I32)), SHAPE),
    ("lens_dtype", dict(lens=desc([3], F32)), DTYPE),
    ("lens_strided", dict(lens=desc([3], I32, strides=[2])), STRIDE),
    ("batch_too_large", dict(table=desc([1025, 4], I32), cu=desc([1026], I32), lens=desc([1025], I32)), UNSUP),
    ("capacity", dict(table=desc([3, 1 << 27], I32)), UNSUP),
    ("null_q", dict(q=None), NULL),
    ("null_table", dict(table=None), NULL),
    ("null_lens_data", dict(lens=desc([3], I32, addr=None)), NULL),
    ("null_out_data", dict(out=desc([9, 8, 128], addr=None)), NULL),
]


@cpu_only
@pytest.mark.parametrize("name,over,code", BAD, ids=[c[0] for c in BAD])
def test_chunk_rejects(lib, name, over, code):  # noqa: F811
    assert call_chunk(lib, chunk_args(**over)) == code


def call_window(lib, a, scale=0.1, window=5, sinks=1):  # noqa: F811
    return lib.decode_attn_prefill_window(*refs(a, "q", "k", "v", "cq", "ck", "out"), ctypes.c_float(scale), window, sinks, None)


@cpu_only
@pytest.mark.parametrize("name,over,code", BAD_PREFILL, ids=[c[0] for c in BAD_PREFILL])
def test_window_rejects(lib, name, over, code):  # noqa: F811
    assert call_window(lib, prefill_args(**over)) == code


@cpu_only
def test_numbers_and_empty_calls(lib):  # noqa: F811
    for window, sinks in ((-1, 0), (4, -1), (0, -5)):
        assert call_chunk(lib, chunk_args(), window=window, sinks=sinks) == UNSUP
        assert call_window(lib, prefill_args(), window=window, sinks=sinks) == UNSUP
    for scale in (float("inf"), float("nan"), 3e38):
        assert call_chunk(lib, chunk_args(), scale=scale) == UNSUP and call_window(lib, prefill_args(), scale=scale) == UNSUP
    for kw in (dict(), dict(dtype=BF16, bs=8), dict(bs=1 << 20)):
        a = chunk_args(T=0, **kw)
        a["q"].data = a["out"].data = None
        assert call_chunk(lib, a) == OK
        a = chunk_args(B=0, **kw)
        a["table"].data = a["lens"].data = None
        assert call_chunk(lib, a) == OK
    a = prefill_args(Tq=0, Tk=0)
    for n in ("q", "k", "v", "out"):
        a[n].data = None
    assert call_window(lib, a) == OK


def test_windows_that_do_not_fit_are_refused(lib):  # noqa: F811
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16)
    k, c = torch.empty((0, 2, 128), dtype=torch.bfloat16), torch.zeros(0, dtype=torch.int32)
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        da.decode_attn_prefill_window(q, k, k, c, c, q, 0.1, 1 << 31, stream=0)
    with pytest.raises(TypeError):
        da.decode_attn_prefill_window(q, k, k, c, c, q, 0.1, 1.5, stream=0)


def chunk_calls(device):
    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=device)

    i32 = torch.int32
    chunk = dict(q=new(2, 4, 128), kp=new(4, 2, 16, 128, dtype=torch.float8_e4m3fn), vp=new(4, 2, 16, 128, dtype=torch.float8_e4m3fn),
                 sc=torch.ones((4, 2, 2, 16), device=device), table=new(2, 2, dtype=i32), cu=new(3, dtype=i32), lens=new(2, dtype=i32), out=new(2, 4, 128))
    prompt = dict(q=new(2, 4, 128), k=new(2, 2, 128), v=new(2, 2, 128), cu_q=new(3, dtype=i32), cu_k=new(3, dtype=i32), out=new(2, 4, 128))
    return [("decode_attn_chunk", chunk, (0.1,)), ("decode_attn_prefill_window", prompt, (0.1, 5))]


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors' addresses: without a GPU only")
@pytest.mark.parametrize("at", [0, 1])
def test_host_tensors_are_refused(at, lib):  # noqa: F811
    name, tensors, rest = chunk_calls("cpu")[at]
    with pytest.raises(ValueError, match="expected a CUDA tensor, got one on cpu"):
        getattr(da, name)(*tensors.values(), *rest, stream=0)
    for n in tensors:
        descs = []
        for m, t in tensors.items():
            d = binding.describe(t)
            d.data = None if m == n else FAKE
            descs.append(d)
        assert getattr(lib, name)(*(ctypes.byref(d) for d in descs), ctypes.c_float(0.1), 5, 0, None) == NULL, n


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 1])
def test_one_host_tensor_among_cuda_tensors_is_refused(at):
    torch.cuda.set_device(0)
    name, tensors, rest = chunk_calls("cuda:0")[at]
    for n, t in tensors.items():
        with pytest.raises(ValueError, match="expected a CUDA tensor, got one on cpu"):
            getattr(da, name)(*{**tensors, n: t.cpu()}.values(), *rest)
    getattr(da, name)(*tensors.values(), *rest)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
