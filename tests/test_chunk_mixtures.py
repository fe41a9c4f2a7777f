"""decode_attn_chunk on batches of prompts' chunks and single tokens over pools whose tokens are laid out first: each sequence
goes the way of its own rows, whatever the others have."""
import pytest
import torch

import decode_attention_output_gb300 as da
from chunk_helpers import attend_ref
from test_cache import DEV, _library, bits, cu, i32  # noqa: F401
from test_chunk import SCALE, Cache, canvas, check

pytestmark = pytest.mark.gpu

KINDS = [(True, 16), (True, 64), (False, 16), (False, 32)]
MIXTURES = [  # Hq, Hkv, queries, keys, window, sinks; more than an SM's items of few rows for each of 152
    (16, 8, [300] + [1] * 20, [700, 0, 5] + [37 * i for i in range(18)], 0, 0),
    (8, 8, [1] * 10 + [800] + [1] * 10, [90 + i for i in range(10)] + [800] + [2, 1000] + [64] * 8, 0, 0),
    (32, 8, [7, 12, 13, 100, 11, 1, 0] * 3, [7, 900, 300, 99, 11, 0, 50] * 3, 0, 0),  # 48 rows, 52, more queries than keys
    (32, 8, [3, 4, 5, 260, 12, 13, 0] * 3, [400, 4, 1000, 1000, 12, 300, 9] * 3, 100, 4),
    (32, 2, [2] * 70 + [500] * 8, [60 + i for i in range(70)] + [500, 900] * 4, 130, 129),
    (160, 160, [40, 1], [300, 500], 0, 0), (12, 4, [0] * 40 + [700] + [0] * 5, [10] * 46, 0, 0),
]


@pytest.mark.parametrize("kv8,bs", KINDS, ids=str)
@pytest.mark.parametrize("Hq,Hkv,lq,lk,window,sinks", MIXTURES, ids=lambda x: str(x)[:24])
def test_mixture(Hq, Hkv, lq, lk, window, sinks, kv8, bs):
    g = torch.Generator().manual_seed(101)
    cache = Cache(g, lk, Hkv, bs, kv8)
    c = cu(lq, first=2)
    q = torch.randn((c[-1] + 3, Hq, 128), generator=g).to(torch.bfloat16)
    kp, vp, sc = cache.on()
    out = canvas(q)
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, cache.table.to(torch.int32).to(DEV), i32(c), i32(lk), out, SCALE, window, sinks)
    check(out, *attend_ref(q, *cache.tokens, c, SCALE, window, sinks), "mixture")


def test_mixture_a_few_heads_at_a_time():
    """A table whose capacity's tokens fit the workspace's part for a few heads only; their items are cut along the keys."""
    g = torch.Generator().manual_seed(102)
    lq, lk = [40, 1], [9000, 700]
    cache = Cache(g, lk, 80, 16, True)
    wide = torch.full((2, 500_000 // 16), -1, dtype=torch.int32)
    wide[:, :cache.table.shape[1]] = cache.table
    c = cu(lq, first=1)
    q = torch.randn((c[-1] + 2, 160, 128), generator=g).to(torch.bfloat16)
    kp, vp, sc = cache.on()
    out = canvas(q)
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, wide.to(DEV), i32(c), i32(lk), out, SCALE)
    check(out, *attend_ref(q, *cache.tokens, c, SCALE), "heads")


@pytest.mark.parametrize("kv8,bs", KINDS, ids=str)
@pytest.mark.parametrize("window,sinks", [(0, 0), (15000, 300)], ids=str)
def test_long_tokens_laid_out(window, sinks, kv8, bs):
    """More tiles of a sequence than CTAs that lay them out, by itself and in a mixture; the shorter one's rows end inside a tile."""
    g = torch.Generator().manual_seed(104)
    for Hq, lq, lk in ((8, [70, 61], [20011, 9001]), (160, [30] + [1], [9001, 300])):
        Hkv = Hq // 2 if Hq > 8 else 1
        cache = Cache(g, lk, Hkv, bs, kv8)
        c = cu(lq, first=1)
        q = torch.randn((c[-1] + 2, Hq, 128), generator=g).to(torch.bfloat16)
        kp, vp, sc = cache.on()
        out = canvas(q)
        da.decode_attn_chunk(q.to(DEV), kp, vp, sc, cache.table.to(torch.int32).to(DEV), i32(c), i32(lk), out, SCALE, window, sinks)
        check(out, *attend_ref(q, *cache.tokens, c, SCALE, window, sinks), f"{Hq} heads")


@pytest.mark.parametrize("kv8", [False, True])
def test_equal_items_on_whole_ctas(kv8):
    """One sequence, or a few of the same length, over so many CTAs that none has parts of two items; and one unit more or fewer."""
    g = torch.Generator().manual_seed(105)
    for B, Hkv, n in ((1, 8, 2049), (1, 8, 2048), (1, 8, 2047), (1, 3, 5000), (2, 5, 777), (4, 8, 1600), (1, 1, 17), (19, 8, 300)):
        lk = [n] * B
        cache = Cache(g, lk, Hkv, 64, kv8)
        c = cu([1] * B)
        q = torch.randn((B, 4 * Hkv, 128), generator=g).to(torch.bfloat16)
        kp, vp, sc = cache.on()
        out = canvas(q)
        da.decode_attn_chunk(q.to(DEV), kp, vp, sc, cache.table.to(torch.int32).to(DEV), i32(c), i32(lk), out, SCALE)
        check(out, *attend_ref(q, *cache.tokens, c, SCALE), f"{B} {Hkv} {n}")


def test_mixture_captured_with_other_lengths():
    """One graph, replayed with other shares of the tokens: what was a chunk becomes a token, and the other way round."""
    g = torch.Generator().manual_seed(103)
    B = 24
    lk = [500 + 13 * i for i in range(B)]
    cache = Cache(g, lk, 8, 32, True)
    kp, vp, sc = cache.on()
    t, lens = cache.table.to(torch.int32).to(DEV), i32(lk)
    q = torch.randn((330, 16, 128), generator=g).to(torch.bfloat16)
    qd, out, c = q.to(DEV), canvas(q), i32([0] * (B + 1))
    run = lambda o: da.decode_attn_chunk(qd, kp, vp, sc, t, c, lens, o, SCALE)  # noqa: E731
    run(out)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        run(out)
    for lq in ([300] + [1] * 23, [1] * 23 + [300], [13] * 24, [100, 0, 25] + [1] * 20 + [24]):
        at = cu(lq)
        c.copy_(torch.tensor(at, dtype=torch.int32))
        out.fill_(7.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(out, *attend_ref(q, *cache.tokens, at, SCALE), str(lq[:3]))
        other = canvas(q)
        run(other)
        assert torch.equal(bits(other), bits(out))
