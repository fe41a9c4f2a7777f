"""A layer's attention as a server runs it with every operator between the projection and the output projection: prompts in chunks
(queries and keys normed and rotated, keys and values into the paged cache on the way, the chunk's attention over that cache),
drafted tokens, then single ones, with and without a window whose old blocks are given away; against 64 bits at every stage. And
whole prompts in a window, rotated apart, whose keys and values are written afterwards."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from chunk_helpers import attend_ref
from prompt_helpers import F64, assert_within, gather, token_ref
from rope_helpers import angles, rope_ref, table
from test_cache import DEV, _library, cu, i32  # noqa: F401

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)
EPS = 1e-5


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
@pytest.mark.parametrize("kv8", [False, True])
def test_chunks_drafts_and_tokens(kv8, window, sinks):
    g = torch.Generator().manual_seed(101)
    Hq, Hkv, bs, B = 8, 2, 16, 3
    steps = [[150, 1, 70], [90, 200, 1], [4, 3, 1], [4, 1, 4], [1, 1, 1], [1, 1, 1], [0, 1, 1]]
    most = -(-max(sum(s[b] for s in steps) for b in range(B)) // bs)
    nb = B * most + 3
    tab = torch.randperm(nb, generator=g)[: B * most].view(B, most)
    dt = tab.to(torch.int32).to(DEV)
    kind = torch.float8_e4m3fn if kv8 else torch.bfloat16
    pool = [torch.zeros((nb, Hkv, bs, 128), device=DEV).to(kind) for _ in range(2)] + [torch.ones((nb, Hkv, 2, bs), device=DEV) if kv8 else None]
    cs = table(512, 128)
    qw, kw = (torch.exp(0.3 * torch.randn(128, generator=g)).to(torch.bfloat16) for _ in range(2))
    lens = [0] * B
    for n in steps:
        c = cu(n)
        T = c[-1]
        qkv = torch.randn((T, Hq + 2 * Hkv, 128), generator=g).to(torch.bfloat16)  # as a projection leaves them
        d = qkv.to(DEV)
        before = list(lens)
        lens = [a + b for a, b in zip(lens, n)]
        q = torch.empty((T, Hq, 128), dtype=torch.bfloat16, device=DEV)
        place = torch.cat([torch.arange(a, b) for a, b in zip(before, lens)]).to(torch.int32)
        da.decode_attn_rope_cache_write(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], cs.to(DEV), i32(c), dt, i32(lens), q, *pool,
                                        q_weight=qw.to(DEV), k_weight=kw.to(DEV), eps=EPS)
        cos, sin, _ = angles(cs, place, None)
        ref, tol = rope_ref(qkv[:, :Hq], qw, EPS, cos, sin, False)
        assert_within(q.cpu(), ref, tol, "queries")
        cached = [None if x is None else x.cpu() for x in pool]
        tokens = []
        for at in range(2):
            rows = []
            for b in range(B):
                x = gather(cached[at].float(), tab, b, lens[b]).to(F64)
                if kv8:
                    x = x * gather(cached[2][:, :, at][..., None], tab, b, lens[b]).to(F64)
                rows.append(x.transpose(0, 1))
            tokens.append(rows)
        ref, tol = rope_ref(qkv[:, Hq:Hq + Hkv], kw, EPS, cos, sin, False)
        for at, (want, off) in enumerate(((ref, tol), (qkv[:, Hq + Hkv:].to(F64), torch.zeros_like(ref)))):
            for b in range(B):
                w, o = want[c[b]:c[b + 1]], off[c[b]:c[b + 1]]
                # e4m3: half a step of the code, whose scale holds the row's largest value in 448 steps at most
                extra = 2.0 ** -4 * w.abs() + 2.0 ** -10 * w.abs().amax(-1, keepdim=True) / 224 if kv8 else 1e-30
                assert_within(tokens[at][b][before[b]:], w, o + extra, "cached")
        out = torch.full((T, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        da.decode_attn_chunk(q, *pool, dt, i32(c), i32(lens), out, SCALE, window, sinks)
        ref, tol, _ = attend_ref(q.cpu(), *tokens, c, SCALE, window, sinks)
        assert_within(out.cpu(), ref, tol, f"chunk of {n}")
        if kv8 and not window and n == [1, 1, 1]:  # the decode step over the same cache
            attn = torch.empty((B, Hq, 128), dtype=torch.bfloat16, device=DEV)
            da.decode_attn_only_paged_fp8(q, *pool, dt, i32(lens), attn, SCALE)
            ref, tol = token_ref(q.cpu(), *cached, tab, lens, SCALE)
            assert_within(attn.cpu(), ref, tol, "decode")
        if window:  # blocks that no query will see again belong to others from here on
            for b in range(B):
                for i in range(-(-sinks // bs), max(0, (lens[b] - window + 1) // bs)):
                    dt[b, i] = -1
                    tab[b, i] = -1  # (reads as zeros: outside every window)
    assert da.decode_attn_last_device_error() == 0


def test_whole_prompts_in_a_window():
    g = torch.Generator().manual_seed(102)
    Hq, Hkv, bs, window, sinks = 6, 3, 32, 64, 2
    n = [200, 1, 90]
    c = cu(n)
    q, k, v = (torch.randn((c[-1], h, 128), generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    pos = torch.stack([torch.cat([torch.arange(x) for x in n]), *(torch.randint(0, 30, (c[-1],), generator=g) for _ in range(2))]).to(torch.int32)
    axes = torch.tensor([0] * 16 + [1] * 24 + [2] * 24, dtype=torch.int32)
    cs = table(256, 128)
    da.decode_attn_rope(q, k, cs.to(DEV), pos.to(DEV), q, k, axes=axes.to(DEV))  # in place
    out = torch.empty_like(q)
    da.decode_attn_prefill_window(q, k, v, i32(c), i32(c), out, SCALE, window, sinks)
    held = [[x.cpu()[a:b] for a, b in zip(c, c[1:])] for x in (k, v)]
    ref, tol, _ = attend_ref(q.cpu(), *held, c, SCALE, window, sinks)
    assert_within(out.cpu(), ref, tol, "prompts")
    # the cache that they leave, and one more token of each over it
    most = -(-(max(n) + 1) // bs)
    tab = torch.randperm(3 * most, generator=g).view(3, most)
    dt = tab.to(torch.int32).to(DEV)
    pool = [torch.zeros((3 * most, Hkv, bs, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    da.decode_attn_cache_write(k, v, i32(c), dt, i32(n), *pool)
    q1, k1, v1 = (torch.randn((3, h, 128), generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    lens = [x + 1 for x in n]
    pos1 = torch.tensor([n] * 3, dtype=torch.int32)  # text: all axes the same
    da.decode_attn_rope_cache_write(q1, k1, v1, cs.to(DEV), i32([0, 1, 2, 3]), dt, i32(lens), q1, *pool, positions=pos1.to(DEV), axes=axes.to(DEV))
    out = torch.empty_like(q1)
    da.decode_attn_chunk(q1, *pool, None, dt, i32([0, 1, 2, 3]), i32(lens), out, SCALE, window, sinks)
    tokens = [[gather(x.cpu().to(F64), tab, b, lens[b]).transpose(0, 1) for b in range(3)] for x in pool]
    for at, x in enumerate((k, v)):
        for b in range(3):
            assert torch.equal(tokens[at][b][:-1], x.cpu()[c[b]:c[b + 1]].to(F64))
    ref, tol, _ = attend_ref(q1.cpu(), *tokens, [0, 1, 2, 3], SCALE, window, sinks)
    assert_within(out.cpu(), ref, tol, "tokens")
    assert da.decode_attn_last_device_error() == 0
