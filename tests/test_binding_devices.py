"""The entry points refuse tensors that are not on the current CUDA device before the library sees their addresses:
lengths, offsets and block tables are easily left on the host."""
import ctypes

import pytest
import torch

import decode_attention_output_gb300 as da
from decode_attention_output_gb300 import binding
from decode_attention_output_gb300 import build as lib_build

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _library():
    lib_build.build()
    binding.load()


def calls(dev, bs=16, N=64):
    """(name, function, its tensors by name, its other arguments) of every entry point that takes tensors."""
    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=dev)

    i32 = torch.int32
    q, k, lens, w, out = new(2, 4, 128), new(2, 2, 32, 128), new(2, dtype=i32), new(512, N), new(2, N)
    k8, pages, pages8 = new(2, 2, 32, 128, dtype=E4M3), new(4, 2, bs, 128), new(4, 2, bs, 128, dtype=E4M3)
    scales, table, cu = torch.ones((4, 2, 2, bs), device=dev), new(2, 2, dtype=i32), new(3, dtype=i32)
    attn, new_k = torch.zeros_like(q), new(2, 2, 128)
    cont, cont8 = dict(q=q, k=k, v=k.clone(), lens=lens), dict(q=q, k=k8, v=k8.clone(), lens=lens)
    paged = dict(q=q, k=pages, v=pages.clone(), table=table, lens=lens)
    paged8 = dict(q=q, k=pages8, v=pages8.clone(), scales=scales, table=table, lens=lens)
    write = dict(k=new_k, v=new_k.clone(), cu=cu, table=table, lens=lens, kp=pages8, vp=pages8.clone(), scales=scales)
    read = dict(kp=pages8, vp=pages8.clone(), scales=scales, table=table, cu=cu, k=new_k, v=new_k.clone())
    prompt = dict(q=q, k=new_k, v=new_k.clone(), cu_q=cu, cu_k=cu.clone(), out=attn)
    return [
        ("fwd", da.decode_attn_fwd, dict(cont, w=w, out=out), (0.1,)),
        ("only", da.decode_attn_only, dict(cont, attn=attn), (0.1,)),
        ("only_noalloc", da.decode_attn_only_noalloc, dict(cont, attn=attn), (0.1,)),
        ("fwd_paged", da.decode_attn_fwd_paged, dict(paged, w=w, out=out), (0.1,)),
        ("only_paged", da.decode_attn_only_paged, dict(paged, attn=attn), (0.1,)),
        ("fwd_fp8", da.decode_attn_fwd_fp8, dict(cont8, w=w, out=out), (0.1, 1.0, 1.0)),
        ("only_fp8", da.decode_attn_only_fp8, dict(cont8, attn=attn), (0.1, 1.0, 1.0)),
        ("fwd_paged_fp8", da.decode_attn_fwd_paged_fp8, dict(paged8, w=w, out=out), (0.1,)),
        ("only_paged_fp8", da.decode_attn_only_paged_fp8, dict(paged8, attn=attn), (0.1,)),
        ("prefill", da.decode_attn_prefill, prompt, (0.1,)),
        ("cache_write", da.decode_attn_cache_write, write, ()),
        ("cache_read", da.decode_attn_cache_read, read, ()),
        ("scores", da.decode_attn_scores, dict(q=q, k=k, lens=lens, scores=torch.zeros((2, 4, 32), device=dev)), ()),
        ("oproj", da.decode_attn_oproj, dict(x=new(2, 512), w=w, out=out), ()),
    ]


NAMES = [c[0] for c in calls("meta")]


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors' addresses: without a GPU only")
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dev", ["cpu", "meta"])
def test_host_tensors_are_refused(name, dev):
    _, fn, tensors, rest = calls(dev)[NAMES.index(name)]
    with pytest.raises(ValueError, match=f"expected a CUDA tensor, got one on {dev}"):
        fn(*tensors.values(), *rest, stream=0)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_one_host_tensor_among_cuda_tensors_is_refused(name):
    torch.cuda.set_device(0)
    _, fn, tensors, rest = calls("cuda:0")[NAMES.index(name)]
    for at, t in tensors.items():
        args = dict(tensors)
        args[at] = t.cpu()
        with pytest.raises(ValueError, match="expected a CUDA tensor, got one on cpu"):
            fn(*args.values(), *rest)
    fn(*tensors.values(), *rest)  # as they are: accepted
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0


@pytest.mark.gpu
def test_tensors_without_elements_may_lie_anywhere():
    """Nothing is read from them (an empty batch)."""
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16)
    k = torch.empty((0, 2, 32, 128), dtype=torch.bfloat16)
    da.decode_attn_only(q, k, k, torch.empty((0,), dtype=torch.int32), q.clone(), 0.1)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: without a GPU only")
@pytest.mark.parametrize("name", NAMES)
def test_the_library_refuses_a_null_address_of_every_tensor(name):
    """What the binding relies on: each tensor with elements but no address is DA_ERR_NULL, whatever the others are."""
    full = {"fwd": "decode_attn_fwd", "only": "decode_attn_only", "only_noalloc": "decode_attn_only_noalloc"}
    lib = binding.load()
    fn = getattr(lib, full.get(name, "decode_attn_" + name))
    _, _, tensors, rest = calls("cpu")[NAMES.index(name)]
    for at in tensors:
        descs = []
        for n, t in tensors.items():
            d = binding.describe(t)
            d.data = None if n == at else 0x10000000
            descs.append(d)
        assert fn(*(ctypes.byref(d) for d in descs), *rest, None) == -1, at


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors' addresses: without a GPU only")
def test_a_wrong_type_is_told_first():
    """The library looks at a tensor's type before its address."""
    _, fn, tensors, rest = calls("cpu")[NAMES.index("prefill")]
    tensors["q"] = tensors["q"].float()
    with pytest.raises(da.DecodeAttnError) as e:
        fn(*tensors.values(), *rest, stream=0)
    assert e.value.code == -2
