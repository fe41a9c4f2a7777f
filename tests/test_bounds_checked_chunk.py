"""The bounds-checked build on decode_attn_chunk and decode_attn_prefill_window: guarded are the rows of q and the outputs, block
tables, pools and scales, the workspace's states and laid-out tokens, and the shared memory that copies and stores reach. Outputs lie
in larger buffers whose other bytes must not change."""
import pytest
import torch

import decode_attention_output_gb300 as da
from chunk_helpers import attend_ref
from prompt_helpers import assert_within
from test_bounds_checked import DEV, Padded, _checked_library  # noqa: F401
from test_bounds_checked_prompt import clean, i32
from test_chunk import CHUNKS, SCALE, WINDOWS, Cache
from test_cache import cu

pytestmark = pytest.mark.gpu


def padded(T, H):
    out = Padded((T, H, 128), torch.bfloat16)
    return out, out.big.view(torch.int16).clone()


def check(out, before, ref, tol, have):
    clean(out)
    assert_within(out.view.cpu()[have], ref[have], tol[have], "rows")
    rest = 1 + torch.nonzero(~have).flatten().to(DEV)
    assert torch.equal(out.big.view(torch.int16)[rest], before[rest])


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,lq,lk,bs,window,sinks", CHUNKS + [(4, 1, [1] * 300, [i % 90 for i in range(300)], 16, 0, 0)], ids=str)
def test_chunk_in_bounds(Hq, Hkv, lq, lk, bs, window, sinks, kv8):
    if kv8 and bs < 16:
        pytest.skip("e4m3 pools: blocks of 16 and more")
    g = torch.Generator().manual_seed(91)
    cache = Cache(g, lk, Hkv, bs, kv8, spare=0)
    c = cu(lq, first=1)
    q = torch.randn((c[-1] + 2, Hq, 128), generator=g).to(torch.bfloat16)
    out, before = padded(c[-1] + 2, Hq)
    kp, vp, sc = cache.on()
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, cache.table.to(torch.int32).to(DEV), i32(c), i32(lk), out.view, SCALE, window, sinks)
    check(out, before, *attend_ref(q, *cache.tokens, c, SCALE, window, sinks))


@pytest.mark.parametrize("Hq,Hkv,lq,lk,window,sinks", WINDOWS, ids=str)
def test_window_in_bounds(Hq, Hkv, lq, lk, window, sinks):
    g = torch.Generator().manual_seed(92)
    cq, ck = cu(lq, first=1), cu(lk, first=2)
    q, k, v = (torch.randn((n + 2, h, 128), generator=g).to(torch.bfloat16) for n, h in ((cq[-1], Hq), (ck[-1], Hkv), (ck[-1], Hkv)))
    out, before = padded(cq[-1] + 2, Hq)
    da.decode_attn_prefill_window(q.to(DEV), k.to(DEV), v.to(DEV), i32(cq), i32(ck), out.view, SCALE, window, sinks)
    check(out, before, *attend_ref(q, *([x[a:b] for a, b in zip(ck, ck[1:])] for x in (k, v)), cq, SCALE, window, sinks))
