"""A request as a server runs it, through every operator: a prompt in two chunks (attention, its keys and values
quantised into the paged cache, the cached beginning read back for the second chunk), then decode steps over that
cache, each token's keys and values written before its attention; against 64 bits at every stage."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import F64, assert_within, gather, prefill_ref, quantise_ref, token_ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SCALE = 1 / math.sqrt(128)


@pytest.mark.parametrize("Hq,Hkv,bs,chunks", [(8, 2, 16, ([130, 1, 60], [70, 200, 33])), (12, 4, 64, ([64], [300]))])
def test_prompt_in_chunks_then_tokens(Hq, Hkv, bs, chunks):
    from decode_attention_output_gb300 import build

    build.build()
    torch.cuda.set_device(0)
    g = torch.Generator().manual_seed(bs)
    B, steps = len(chunks[0]), 3
    most = -(-(max(a + b for a, b in zip(*chunks)) + steps) // bs)
    table = torch.randperm(B * most + 2, generator=g)[: B * most].view(B, most)
    dt = table.to(torch.int32).to(DEV)
    pool = [torch.zeros((B * most + 2, Hkv, bs, 128), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    pool.append(torch.ones((B * most + 2, Hkv, 2, bs), device=DEV))
    kept = [[torch.zeros((0, Hkv, 128), dtype=F64) for _ in range(B)] for _ in range(2)]  # what the cache stands for
    lens = [0] * B

    def rand(T, H):
        return torch.randn((T, H, 128), generator=g).to(torch.bfloat16)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def cu(n):
        return torch.tensor([0] + n).cumsum(0).tolist()

    def write(k, v, n):
        for b in range(B):
            lens[b] += n[b]
        c = cu(n)
        da.decode_attn_cache_write(k.to(DEV), v.to(DEV), i32(c), dt, i32(lens), *pool)
        for x, old in ((k, kept[0]), (v, kept[1])):
            codes, s = quantise_ref(x)
            y = codes.view(torch.float8_e4m3fn).float().to(F64) * s.to(F64)[..., None]
            for b in range(B):
                old[b] = torch.cat([old[b], y[c[b]:c[b + 1]]])

    for n in chunks:
        c = cu(n)
        q, k, v = rand(c[-1], Hq), rand(c[-1], Hkv), rand(c[-1], Hkv)
        write(k, v, n)
        # the whole sequences' tokens as they are cached, the chunk's among them
        ck = cu(lens)
        kk, vv = (torch.zeros((ck[-1], Hkv, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        da.decode_attn_cache_read(*pool, dt, i32(ck), kk, vv)
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        da.decode_attn_prefill(q.to(DEV), kk, vv, i32(c), i32(ck), out, SCALE)
        torch.cuda.synchronize()
        assert torch.equal(kk.cpu().to(F64), torch.cat(kept[0])) and torch.equal(vv.cpu().to(F64), torch.cat(kept[1]))
        ref, tol, _ = prefill_ref(q, torch.cat(kept[0]), torch.cat(kept[1]), c, ck, SCALE)
        assert_within(out.cpu(), ref, tol, f"chunk of {n}")

    N = 256
    w = (torch.randn((Hq * 128, N), generator=g) / math.sqrt(Hq * 128)).to(torch.bfloat16)
    dw = w.to(DEV)
    for _ in range(steps):
        q, k, v = rand(B, Hq), rand(B, Hkv), rand(B, Hkv)
        write(k, v, [1] * B)
        attn = torch.empty((B, Hq, 128), dtype=torch.bfloat16, device=DEV)
        out = torch.empty((B, N), dtype=torch.bfloat16, device=DEV)
        args = q.to(DEV), *pool, dt, i32(lens)
        da.decode_attn_only_paged_fp8(*args, attn, SCALE)
        da.decode_attn_fwd_paged_fp8(*args, dw, out, SCALE)
        torch.cuda.synchronize()
        cached = [p.cpu() for p in pool]
        for b in range(B):
            got = gather(cached[0].float(), table, b, lens[b]).to(F64) * gather(cached[2][:, :, 0][..., None], table, b, lens[b]).to(F64)
            assert torch.equal(got.transpose(0, 1), kept[0][b])
        ref, tol = token_ref(q, *cached, table, lens, SCALE)
        assert_within(attn.cpu(), ref, tol, "token")
        ref, tol = ref.reshape(B, -1), tol.reshape(B, -1)
        want = ref @ w.to(F64)
        bound = tol @ w.to(F64).abs() + Hq * 128 * 2.0 ** -23 * (ref.abs() @ w.to(F64).abs()) + 2.0 ** -8 * want.abs()
        assert_within(out.cpu(), want, bound * 1.01, "step")
    assert da.decode_attn_last_device_error() == 0
