"""The workspace and CUDA graphs: a call that would have to grow it during a capture is refused, and a graph captured
before a growth can be replayed after it."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import assert_within, prefill_ref, token_ref
from test_parity_paged_fp8 import DEV, SCALE, _library, case, on  # noqa: F401

pytestmark = pytest.mark.gpu
DA_ERR_NOMEM = -7


def larger_call():
    """A decode call whose partial results take 68 MB, more than a first workspace."""
    q = torch.zeros((1024, 16, 128), dtype=torch.bfloat16, device=DEV)
    k = torch.ones((1024, 16, 8, 128), dtype=torch.bfloat16, device=DEV)
    lens = torch.full((1024,), 8, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    da.decode_attn_only(q, k, k, lens, out, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out, torch.ones_like(out))


def entry_points():
    x = case(2, 8, 2, [300, 90], 16, seed=31)
    a = on(x)
    attn, out = torch.zeros_like(a[0]), torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((8 * 128, 64), dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    return {"step": lambda: da.decode_attn_fwd_paged_fp8(*a, w, out, SCALE),
            "token": lambda: da.decode_attn_only_paged_fp8(*a, attn, SCALE),
            "prompt": lambda: da.decode_attn_prefill(a[0], kv, kv, cu, cu, attn, SCALE),
            "write": lambda: da.decode_attn_cache_write(kv, kv, cu, a[4], a[5], a[1], a[2], a[3]),
            "read": lambda: da.decode_attn_cache_read(a[1], a[2], a[3], a[4], cu, kv.clone(), kv.clone()),
            "bf16": lambda: da.decode_attn_only(a[0], kv[:, :, None], kv[:, :, None], a[5], attn, SCALE)}


@pytest.mark.parametrize("name", ["step", "token", "prompt", "write", "read", "bf16"])
def test_a_first_call_during_a_capture_is_refused(name):
    call = entry_points()[name]
    torch.cuda.synchronize()
    da.decode_attn_release()
    graph = torch.cuda.CUDAGraph()
    status = None
    with torch.cuda.graph(graph):
        torch.zeros((8,), device=DEV)  # (something in the graph)
        try:
            call()
        except da.DecodeAttnError as e:
            status = e.code
    assert status == DA_ERR_NOMEM
    call()  # not captured: the workspace is there from now on
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        call()
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0


def test_a_graph_captured_before_a_growth_replays_after_it():
    torch.cuda.synchronize()
    da.decode_attn_release()
    x = case(3, 8, 2, [9000, 5, 1300], 64, seed=32)
    a = on(x)
    g = torch.Generator().manual_seed(33)
    q, k, v = (torch.randn((n, h, 128), generator=g).to(torch.bfloat16) for n, h in ((40, 8), (4000, 2), (4000, 2)))
    cu_q, cu_k = [0, 40], [0, 4000]
    p = [t.to(DEV) for t in (q, k, v)] + [torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cu_q, cu_k)]
    token, prompt = torch.empty_like(a[0]), torch.empty_like(p[0])

    def both():  # parts of a sequence, and of a prompt, meet in the workspace
        da.decode_attn_only_paged_fp8(*a, token, SCALE)
        da.decode_attn_prefill(*p, prompt, SCALE)

    both()
    torch.cuda.synchronize()
    first = token.clone(), prompt.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    larger_call()
    for _ in range(3):
        token.fill_(math.nan)
        prompt.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, first[0]) and torch.equal(prompt, first[1])
        larger_call()
    ref, tol = token_ref(*x, SCALE)
    assert_within(token.cpu(), ref, tol, "token")
    ref, tol, _ = prefill_ref(q, k, v, cu_q, cu_k, SCALE)
    assert_within(prompt.cpu(), ref, tol, "prompt")
    x[4][1, 0] = x[1].shape[0] + 3  # an error that the replay records where the graph was captured
    a[4].copy_(x[4])
    graph.replay()
    assert da.decode_attn_last_device_error() == 64
    assert da.decode_attn_last_device_error() == 0
