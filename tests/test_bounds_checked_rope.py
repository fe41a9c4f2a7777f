"""The bounds-checked build on the rotating entry points: guarded are the rows that they read and write, the pools, scales and
block table, and the rows of the table of angles. Outputs and pools lie in larger buffers whose other bytes must not change."""
import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import assert_within, places
from rope_helpers import angles, rope_f32, rope_ref, table
from prompt_helpers import quantise_ref
from test_bounds_checked import DEV, Padded, _checked_library  # noqa: F401
from test_bounds_checked_prompt import Pool, clean, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,R,Hq,Hkv,inter,A", [(128, 128, 8, 2, False, 0), (128, 64, 5, 1, True, 0), (128, 24, 4, 4, False, 3),
                                                (256, 256, 3, 1, True, 2), (256, 128, 16, 8, False, 0)], ids=str)
@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_in_bounds(D, R, Hq, Hkv, inter, A, T, norm):
    g = torch.Generator().manual_seed(61)
    q, k = (torch.randn((T, h, D), generator=g).to(torch.bfloat16) for h in (Hq, Hkv))
    tab = table(90, R)
    pos = torch.randint(0, 90, (A, T) if A else (T,), generator=g).to(torch.int32)
    axes = torch.randint(0, A, (R // 2,), generator=g).to(torch.int32) if A else None
    w = torch.rand(D, generator=g).to(torch.bfloat16) if norm else None
    out = [Padded((T, h, D), torch.bfloat16) for h in (Hq, Hkv)]
    dw = w.to(DEV) if norm else None
    da.decode_attn_rope(q.to(DEV), k.to(DEV), tab.to(DEV), pos.to(DEV), out[0].view, out[1].view, dw, dw, axes.to(DEV) if A else None, 1e-6, inter)
    clean(*out)
    cos, sin, _ = angles(tab, pos, axes)
    for x, o in zip((q, k), out):
        assert_within(o.view.cpu(), *rope_ref(x, w, 1e-6, cos, sin, inter), "rows")


@pytest.mark.parametrize("dtype,D,Hkv,bs", [(torch.float8_e4m3fn, 128, 1, 16), (torch.float8_e4m3fn, 128, 6, 64),
                                            (torch.bfloat16, 128, 3, 8), (torch.bfloat16, 256, 4, 32)], ids=str)
@pytest.mark.parametrize("many", [False, True])
def test_append_in_bounds(dtype, D, Hkv, bs, many):
    g = torch.Generator().manual_seed(62)
    new = [700, 0, 1, 333] if many else [5, 0, 1]
    lens = [n + e for n, e in zip(new, (3, 9, 40, 0))]
    B, mb = len(new), -(-max(lens) // bs) + 1
    nb = B * mb + 2
    blocks = torch.randperm(nb, generator=g)[: B * mb].view(B, mb)
    wide = torch.full((B, mb + 5), 1 << 30, dtype=torch.int32)  # a padded table
    wide[:, :mb] = blocks
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    T = cu[-1] + 2  # rows behind the last sequence
    q, k, v = (torch.randn((T, h, D), generator=g).to(torch.bfloat16) for h in (2 * Hkv, Hkv, Hkv))
    tab, at = table(max(lens), D), torch.zeros(T, dtype=torch.int32)
    for b in range(B):
        at[cu[b]:cu[b + 1]] = torch.arange(lens[b] - new[b], lens[b])
    cos, sin, _ = angles(tab, at, None)
    kv8 = dtype == torch.float8_e4m3fn
    kp, vp = Pool((nb, Hkv, bs, D), dtype, g), Pool((nb, Hkv, bs, D), dtype, g)
    sc = Pool((nb, Hkv, 2, bs), torch.float32, g) if kv8 else None
    want = [p.bytes() for p in (kp, vp, sc) if p]
    views = [w.view(p.view.dtype)[1:-1] for w, p in zip(want, (kp, vp, sc))]
    pad = 8 if not kv8 else 16
    turned = rope_f32(k, cos, sin, False)
    for x, view, which in ((turned, views[0], 0), (v, views[1], 1)):
        codes, scale = quantise_ref(x) if kv8 else (None, None)
        for t, blk, row in places(blocks, cu, lens, bs):
            view[blk, :, row, pad:-pad] = (codes[t].view(dtype) if kv8 else x[t].to(torch.bfloat16)).to(DEV)
            if kv8:
                views[2][blk, :, which, 4 + row] = scale[t].to(DEV)
    qo = Padded((T, 2 * Hkv, D), torch.bfloat16)
    rest = qo.big[-3:].clone()
    da.decode_attn_rope_cache_write(q.to(DEV), k.to(DEV), v.to(DEV), tab.to(DEV), i32(cu), wide.to(DEV)[:, :mb], i32(lens), qo.view, kp.view,
                                    vp.view, sc.view if kv8 else None)
    clean(qo)
    for p, w in zip((kp, vp, sc), want):
        assert torch.equal(p.big, w)
    ref, tol = rope_ref(q, None, 1e-6, cos, sin, False)
    assert_within(qo.view.cpu()[:cu[-1]], ref[:cu[-1]], tol[:cu[-1]], "q")
    assert torch.equal(qo.big[-3:].view(torch.int16), rest.view(torch.int16))
