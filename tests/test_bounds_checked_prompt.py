"""The bounds-checked build on the prompt attention, the paged cache's writing and reading and the attention over a
paged e4m3 cache: guarded are the rows of the outputs, the tokens, pools, scales and block tables that the cache kernels
read and write (against the tensors' extents), the workspace rows of cut prompts, and the shared memory that copies and
stores reach. Every output lies in a larger buffer whose other bytes must not change; the error word is 0 and the
results are within the bounds of prompt_helpers."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import F64, assert_within, gather, places, prefill_ref, quantise_ref, token_ref
from test_bounds_checked import DEV, Padded, _checked_library, _Opt  # noqa: F401
from test_parity_paged_fp8 import SCALE, case, on

pytestmark = pytest.mark.gpu


def clean(*outs):
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0, "device error word set"
    for o in outs:
        assert o.canaries_intact(), "written outside its view"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


PROMPTS = [  # Hq, Hkv, new tokens, tokens in all
    (8, 2, [70, 0, 1, 300], [70, 5, 1, 300]), (4, 4, [129, 64], [400, 64]), (6, 2, [43, 100, 7], [43, 260, 3]),
    (32, 2, [20, 33], [20, 150]), (8, 1, [10], [5000]), (4, 1, [64, 3], [2600, 1700]), (8, 8, [5], [0]), (12, 1, [1000], [1900]),
]


@pytest.mark.parametrize("Hq,Hkv,lq,lk", PROMPTS, ids=str)
def test_prompt_in_bounds(Hq, Hkv, lq, lk):
    g = torch.Generator().manual_seed(41)
    cu_q, cu_k = ([0] + torch.tensor(n).cumsum(0).tolist() for n in (lq, lk))
    Tq, Tk = cu_q[-1] + 3, cu_k[-1] + 2  # rows behind the last sequence
    q, k, v = (torch.randn((n, h, 128), generator=g).to(torch.bfloat16) for n, h in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv)))
    ref, tol, have = prefill_ref(q, k, v, cu_q, cu_k, SCALE)
    out = Padded((Tq, Hq, 128), torch.bfloat16)
    before = out.big.view(torch.int16).clone()
    da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), i32(cu_q), i32(cu_k), out.view, SCALE)
    clean(out)
    assert_within(out.view.cpu()[have], ref[have], tol[have], "prompt")
    rest = 1 + torch.nonzero(~have).flatten().to(DEV)
    assert torch.equal(out.big.view(torch.int16)[rest], before[rest])


class Pool:
    """A pool [blocks, Hkv, bs, D] inside a larger buffer of random bytes, rows 16 bytes apart from one another."""

    def __init__(self, shape, dtype, g):
        size = torch.tensor([], dtype=dtype).element_size()
        pad = 16 // size
        self.big = torch.randint(0, 256, (shape[0] + 2, *shape[1:-1], (shape[-1] + 2 * pad) * size), generator=g, dtype=torch.uint8).to(DEV)
        self.view = self.big.view(dtype)[1:-1, ..., pad:-pad]
        assert self.view.shape == shape

    def bytes(self, of=None):
        return (self.big if of is None else of).clone()


@pytest.mark.parametrize("dtype,D,Hkv,bs", [(torch.float8_e4m3fn, 128, 1, 16), (torch.float8_e4m3fn, 128, 6, 32),
                                            (torch.float8_e4m3fn, 128, 8, 128), (torch.bfloat16, 128, 3, 8),
                                            (torch.bfloat16, 256, 4, 64)], ids=str)
@pytest.mark.parametrize("many", [False, True])
def test_cache_in_bounds(dtype, D, Hkv, bs, many):
    """Written rows get their codes and scales, every other byte of the three pools keeps its value; then they are read."""
    g = torch.Generator().manual_seed(42)
    new = [700, 0, 1, 333] if many else [5, 0, 1]
    lens = [n + e for n, e in zip(new, (3, 9, 40, 0))]
    B = len(new)
    mb = -(-max(lens) // bs) + 1
    nb = B * mb + 2
    table = torch.randperm(nb, generator=g)[: B * mb].view(B, mb)
    wide = torch.full((B, mb + 5), 1 << 30, dtype=torch.int32)  # a padded table
    wide[:, :mb] = table
    dt = wide.to(DEV)[:, :mb]
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    T = cu[-1] + 2  # rows behind the last sequence
    k, v = (torch.randn((T, Hkv, D), generator=g).to(torch.bfloat16) for _ in range(2))
    kv8 = dtype == torch.float8_e4m3fn
    kp, vp = Pool((nb, Hkv, bs, D), dtype, g), Pool((nb, Hkv, bs, D), dtype, g)
    sc = Pool((nb, Hkv, 2, bs), torch.float32, g) if kv8 else None
    want = [p.bytes() for p in (kp, vp, sc) if p]
    views = [w.view(p.view.dtype)[tuple(slice(1, -1) if i == 0 else slice(None) for i in range(3))] for w, p in zip(want, (kp, vp, sc))]
    pad = 16 // k.element_size() if not kv8 else 16
    for x, view, which in ((k, views[0], 0), (v, views[1], 1)):
        codes, scale = quantise_ref(x) if kv8 else (None, None)
        for t, blk, row in places(table, cu, lens, bs):
            view[blk, :, row, pad:-pad] = (codes[t].view(dtype) if kv8 else x[t]).to(DEV)
            if kv8:
                views[2][blk, :, which, 4 + row] = scale[t].to(DEV)
    da.decode_attn_cache_write(k.to(DEV), v.to(DEV), i32(cu), dt, i32(lens), kp.view, vp.view, sc.view if kv8 else None)
    clean()
    for p, w in zip((kp, vp, sc), want):
        assert torch.equal(p.big, w)
    first = [n // 2 for n in lens]
    ck = [0] + torch.tensor(first).cumsum(0).tolist()
    outs = [Padded((ck[-1] + 1, Hkv, D), torch.bfloat16) for _ in range(2)]
    last = [o.big.view(torch.int16)[-2].clone() for o in outs]
    for p in (kp, vp):  # the bytes that nothing wrote are random: no NaN codes
        p.view.copy_(torch.nan_to_num(p.view.float()).clamp(-400, 400).to(dtype))
    if kv8:
        sc.view.copy_(torch.exp2(torch.randint(-9, 4, sc.view.shape, generator=g).float()))
    da.decode_attn_cache_read(kp.view, vp.view, sc.view if kv8 else None, dt, i32(ck), outs[0].view, outs[1].view)
    clean(*outs)
    for which, (o, p) in enumerate(zip(outs, (kp, vp))):
        x = p.view.cpu().float()
        if kv8:
            x = x * sc.view.cpu()[:, :, which][..., None]
        ref = torch.cat([gather(x, table, b, n).transpose(0, 1) for b, n in enumerate(first)])
        assert torch.equal(o.view.cpu()[:-1].float(), ref.to(torch.bfloat16).float())
        assert torch.equal(o.big.view(torch.int16)[-2], last[which])


TOKENS = [  # B, Hq, Hkv, lengths, block size, options
    (3, 8, 2, [300, 0, 129], 16, {}), (2, 32, 2, [700, 64], 64, {}), (2, 4, 4, [100, 1], 256, {}), (4, 16, 4, [1024] * 4, 16, {}),
    (8, 8, 2, [1024, 0, 1, 700, 64, 1000, 333, 129], 32, {"attn_ctas": 5}), (3, 24, 2, [5000, 3, 900], 64, {"attn_ctas": 40}),
    (1, 8, 1, [9000], 128, {}), (24, 4, 1, [800 + 15 * b for b in range(24)], 16, {}),
]


@pytest.mark.parametrize("B,Hq,Hkv,lens,bs,opts", TOKENS, ids=[str(i) for i in range(len(TOKENS))])
def test_token_in_bounds(B, Hq, Hkv, lens, bs, opts):
    x = case(B, Hq, Hkv, lens, bs, seed=43)
    ref, tol = token_ref(*x, SCALE)
    g = torch.Generator().manual_seed(44)
    w = (torch.randn((Hq * 128, 264), generator=g) / math.sqrt(Hq * 128)).to(torch.bfloat16)
    attn, out = Padded((B, Hq, 128), torch.bfloat16), Padded((B, 264), torch.bfloat16)
    with _Opt(**opts):
        da.decode_attn_only_paged_fp8(*on(x), attn.view, SCALE)
        da.decode_attn_fwd_paged_fp8(*on(x), w.to(DEV), out.view, SCALE)
    clean(attn, out)
    assert_within(attn.view.cpu(), ref, tol, "attention")
    ref, tol, w = ref.reshape(B, -1), tol.reshape(B, -1), w.to(F64)
    want = ref @ w
    bound = tol @ w.abs() + Hq * 128 * 2.0 ** -23 * (ref.abs() @ w.abs()) + 2.0 ** -8 * want.abs()
    assert_within(out.view.cpu(), want, bound * 1.01 + 1e-30, "step")


def test_two_key_pools_and_one_pool_as_both():
    """Copies of one tensor each and of both at once, in either order of the pools."""
    x = case(2, 8, 2, [200, 33], 16, seed=45)
    q, k, v, scales, table, lens = on(x)
    ref, tol = token_ref(*x, SCALE)
    both = torch.empty((2, *k.shape), dtype=torch.uint8, device=DEV)
    for first in (0, 1):
        k2, v2 = both[first].view(k.dtype), both[1 - first].view(k.dtype)
        k2.view(torch.uint8).copy_(k.view(torch.uint8))
        v2.view(torch.uint8).copy_(v.view(torch.uint8))
        out = Padded((2, 8, 128), torch.bfloat16)
        da.decode_attn_only_paged_fp8(q, k2, v2, scales, table, lens, out.view, SCALE)
        clean(out)
        assert_within(out.view.cpu(), ref, tol, "token")
    ref, tol = token_ref(x[0], x[1], x[1], *x[3:], SCALE)
    da.decode_attn_only_paged_fp8(q, k, k, scales, table, lens, out.view, SCALE)
    clean(out)
    assert_within(out.view.cpu(), ref, tol, "one pool")
