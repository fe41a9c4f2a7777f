"""Host-side refusals of the rotating entry points: the documented status codes, before anything touches the device (fake
device addresses, without a GPU only), and tensors that are not on the current device."""
import ctypes

import pytest
import torch

import decode_attention_output_gb300 as da
from decode_attention_output_gb300 import binding
from test_abi import ALIGN, DTYPE, FAKE, NULL, OK, SHAPE, STRIDE, UNSUP, cpu_only, desc, lib  # noqa: F401
from test_abi_prompt import E4M3, F32, I32, refs

ROPE = ("q", "k", "tab", "pos", "qo", "ko", "qw", "kw", "axes")
APPEND = ("q", "k", "v", "tab", "cu", "table", "lens", "qo", "kp", "vp", "sc", "pos", "qw", "kw", "axes")


def rope_args(T=9, Hq=8, H=2, D=128, R=128, P=50, A=0, B=3, nblk=10, bs=16, mb=4, dtype=E4M3, **over):
    a = dict(q=desc([T, Hq, D]), k=desc([T, H, D]), v=desc([T, H, D]), tab=desc([P, R], F32),
             pos=desc([A, T] if A else [T], I32), qo=desc([T, Hq, D]), ko=desc([T, H, D]), qw=desc([D]), kw=desc([D], F32),
             axes=desc([R // 2], I32) if A else None, cu=desc([B + 1], I32), table=desc([B, mb], I32), lens=desc([B], I32),
             kp=desc([nblk, H, bs, D], dtype), vp=desc([nblk, H, bs, D], dtype), sc=desc([nblk, H, 2, bs], F32) if dtype == E4M3 else None)
    a.update(over)
    return a


def call_rope(lib, a, eps=1e-6, inter=0):  # noqa: F811
    return lib.decode_attn_rope(*refs(a, *ROPE), ctypes.c_float(eps), inter, None)


def call_append(lib, a, eps=1e-6, inter=0):  # noqa: F811
    return lib.decode_attn_rope_cache_write(*refs(a, *APPEND), ctypes.c_float(eps), inter, None)


BAD = [
    ("q_dtype", dict(q=desc([9, 8, 128], F32)), DTYPE),
    ("q_out_dtype", dict(qo=desc([9, 8, 128], F32)), DTYPE),
    ("q_tokens", dict(q=desc([8, 8, 128]), qo=desc([8, 8, 128])), SHAPE),
    ("q_out_heads", dict(qo=desc([9, 4, 128])), SHAPE),
    ("q_dim", dict(q=desc([9, 8, 256]), qo=desc([9, 8, 256])), SHAPE),
    ("head_dim_64", dict(q=desc([9, 8, 64]), qo=desc([9, 8, 64]), k=desc([9, 2, 64]), v=desc([9, 2, 64]), ko=desc([9, 2, 64]),
                         kp=desc([10, 2, 16, 64], E4M3), vp=desc([10, 2, 16, 64], E4M3)), SHAPE),
    ("q_misaligned", dict(q=desc([9, 8, 128], addr=FAKE + 8)), ALIGN),
    ("q_out_stride", dict(qo=desc([9, 8, 128], strides=[8 * 132, 132, 1])), STRIDE),
    ("q_without_out", dict(qo=None), NULL),
    ("out_without_q", dict(q=None), NULL),
    ("table_dtype", dict(tab=desc([50, 128])), DTYPE),
    ("table_1d", dict(tab=desc([50], F32)), SHAPE),
    ("table_wide", dict(tab=desc([50, 136], F32)), SHAPE),
    ("table_empty", dict(tab=desc([0, 128], F32)), SHAPE),
    ("table_r_100", dict(tab=desc([50, 100], F32)), UNSUP),
    ("table_rows_overlap", dict(tab=desc([50, 128], F32, strides=[64, 1])), STRIDE),
    ("table_misaligned", dict(tab=desc([50, 128], F32, addr=FAKE + 8)), ALIGN),
    ("table_null", dict(tab=None), NULL),
    ("weight_dtype", dict(qw=desc([128], I32)), DTYPE),
    ("weight_length", dict(kw=desc([64], F32)), SHAPE),
    ("weight_2d", dict(kw=desc([1, 128])), SHAPE),
    ("weight_stride", dict(qw=desc([128], strides=[2])), STRIDE),
    ("weight_misaligned", dict(qw=desc([128], addr=FAKE + 2)), ALIGN),
    ("positions_dtype", dict(pos=desc([9], F32)), DTYPE),
    ("positions_tokens", dict(pos=desc([8], I32)), SHAPE),
    ("positions_3d", dict(pos=desc([1, 1, 9], I32)), SHAPE),
    ("positions_stride", dict(pos=desc([9], I32, strides=[2])), STRIDE),
    ("positions_misaligned", dict(pos=desc([9], I32, addr=FAKE + 2)), ALIGN),
    ("axes_missing", dict(pos=desc([3, 9], I32)), NULL),
    ("five_axes", dict(pos=desc([5, 9], I32), axes=desc([64], I32)), UNSUP),
    ("axes_length", dict(axes=desc([32], I32)), SHAPE),
    ("axes_dtype", dict(axes=desc([64], F32)), DTYPE),
    ("axes_stride", dict(axes=desc([64], I32, strides=[2])), STRIDE),
    ("axes_null_data", dict(axes=desc([64], I32, addr=None)), NULL),
    ("k_tokens", dict(k=desc([8, 2, 128])), SHAPE),
    ("k_misaligned", dict(k=desc([9, 2, 128], addr=FAKE + 8)), ALIGN),
]


@cpu_only
@pytest.mark.parametrize("name,over,code", BAD, ids=[c[0] for c in BAD])
def test_both_reject(lib, name, over, code):  # noqa: F811
    assert call_rope(lib, rope_args(**over)) == code
    assert call_append(lib, rope_args(**over)) == code


@cpu_only
def test_rope_rejects(lib):  # noqa: F811
    assert call_rope(lib, rope_args(q=None, qo=None, k=None, ko=None)) == NULL
    assert call_rope(lib, rope_args(ko=None)) == NULL
    assert call_rope(lib, rope_args(ko=desc([9, 3, 128]))) == SHAPE
    assert call_rope(lib, rope_args(pos=None)) == NULL
    for call in (call_rope, call_append):
        for eps in (-1e-6, float("nan"), float("inf")):
            assert call(lib, rope_args(), eps=eps) == UNSUP
        assert call(lib, rope_args(), inter=2) == UNSUP


APPEND_BAD = [
    ("axes_without_positions", dict(pos=None, axes=desc([64], I32)), SHAPE),
    ("v_tokens", dict(v=desc([8, 2, 128])), SHAPE),
    ("null_v", dict(v=None), NULL),
    ("null_lens", dict(lens=None), NULL),
    ("scales_missing", dict(sc=None), NULL),
    ("scales_for_bf16", dict(kp=desc([10, 2, 16, 128]), vp=desc([10, 2, 16, 128])), DTYPE),
    ("block_size_48", dict(kp=desc([10, 2, 48, 128], E4M3), vp=desc([10, 2, 48, 128], E4M3), sc=desc([10, 2, 2, 48], F32)), UNSUP),
    ("cu_length", dict(cu=desc([3], I32)), SHAPE),
    ("batch_too_large", dict(table=desc([1025, 4], I32), cu=desc([1026], I32), lens=desc([1025], I32)), UNSUP),
]


@cpu_only
@pytest.mark.parametrize("name,over,code", APPEND_BAD, ids=[c[0] for c in APPEND_BAD])
def test_append_rejects(lib, name, over, code):  # noqa: F811
    assert call_append(lib, rope_args(**over)) == code


@cpu_only
def test_nothing_to_do(lib):  # noqa: F811
    a = rope_args(T=0)
    for n in ("q", "k", "v", "qo", "ko", "pos"):
        a[n].data = None
    assert call_rope(lib, a) == OK and call_append(lib, a) == OK
    assert call_append(lib, rope_args(B=0)) == OK


def rope_calls(device):
    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=device)

    i32 = torch.int32
    a = dict(q=new(2, 4, 128), k=new(2, 2, 128), v=new(2, 2, 128), tab=new(8, 128, dtype=torch.float32), cu=new(3, dtype=i32),
             table=new(2, 2, dtype=i32), lens=new(2, dtype=i32), qo=new(2, 4, 128), ko=new(2, 2, 128), kp=new(4, 2, 16, 128, dtype=torch.float8_e4m3fn),
             vp=new(4, 2, 16, 128, dtype=torch.float8_e4m3fn), sc=torch.ones((4, 2, 2, 16), device=device), pos=new(2, 2, dtype=i32),
             qw=new(128), kw=new(128), axes=new(64, dtype=i32))
    return [("rope", da.decode_attn_rope, {n: a[n] for n in ROPE}), ("rope_cache_write", da.decode_attn_rope_cache_write, {n: a[n] for n in APPEND})]


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors' addresses: without a GPU only")
@pytest.mark.parametrize("at", [0, 1])
def test_host_tensors_are_refused(at, lib):  # noqa: F811
    name, fn, tensors = rope_calls("cpu")[at]
    with pytest.raises(ValueError, match="expected a CUDA tensor, got one on cpu"):
        fn(*tensors.values(), stream=0)
    c_fn = getattr(lib, "decode_attn_" + name)
    for n in tensors:
        descs = []
        for m, t in tensors.items():
            d = binding.describe(t)
            d.data = None if m == n else FAKE
            descs.append(d)
        assert c_fn(*(ctypes.byref(d) for d in descs), ctypes.c_float(1e-6), 0, None) == NULL, n


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 1])
def test_one_host_tensor_among_cuda_tensors_is_refused(at):
    torch.cuda.set_device(0)
    _, fn, tensors = rope_calls("cuda:0")[at]
    for n, t in tensors.items():
        with pytest.raises(ValueError, match="expected a CUDA tensor, got one on cpu"):
            fn(*{**tensors, n: t.cpu()}.values())
    fn(*tensors.values())
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
