"""decode_attn_cache_write and decode_attn_cache_read: codes, scales and copies bit for bit against the definition in
64 bits, every byte that is not a new token's left as it was, and what was written read back."""
import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import gather, places, quantise_ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _library():
    from decode_attention_output_gb300 import build

    build.build()
    da.load()
    torch.cuda.set_device(0)
    yield
    assert da.decode_attn_last_device_error() == 0


def cu(lengths, first=0):
    c = [first]
    for n in lengths:
        c.append(c[-1] + n)
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def tables(lens, bs, g, spare=3):
    most = max(1, max(-(-n // bs) for n in lens))
    blocks = len(lens) * most + spare
    return torch.randperm(blocks, generator=g)[: len(lens) * most].view(len(lens), most), blocks


def tokens(T, H, D, g):
    size = torch.exp(2 * torch.randn((T, H, 1), generator=g))
    return (torch.randn((T, H, D), generator=g) * size).to(torch.bfloat16)


def pools(blocks, H, bs, D, fp8):
    """Pools (and scales) of a bit pattern that nothing here writes."""
    if not fp8:
        return [torch.full((blocks, H, bs, D), 0x7FA5, dtype=torch.int16, device=DEV).view(torch.bfloat16) for _ in range(2)] + [None]
    k, v = (torch.full((blocks, H, bs, D), 0xFF, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    return [k, v, torch.full((blocks, H, 2, bs), float("nan"), dtype=torch.float32, device=DEV)]


def bits(t):
    return t.view(torch.uint8 if t.dtype == torch.float8_e4m3fn else (torch.int16 if t.dtype == torch.bfloat16 else torch.int32)).cpu()


def expected(before, k, v, table, c, seq_lens, bs, fp8):
    want = [None if t is None else t.cpu().clone() for t in before]
    for row, block, r in places(table, c, seq_lens, bs):
        for i, x in enumerate((k, v)):
            if fp8:
                codes, scale = quantise_ref(x[row])
                want[i].view(torch.uint8)[block, :, r] = codes
                want[2][block, :, i, r] = scale
            else:
                want[i][block, :, r] = x[row]
    return want


CASES = [  # new tokens, tokens before them, KV heads, block size
    ([1], [0], 1, 16),
    ([1, 1, 1, 1, 1], [0, 15, 16, 17, 300], 8, 16),
    ([70, 0, 33, 1], [0, 5, 31, 64], 3, 32),
    ([129], [1000], 5, 64),
    ([3] * 40, list(range(40)), 2, 16),           # more than 32 sequences
    ([700, 600], [3, 0], 8, 128),                 # four heads to a warp
    ([500, 900], [3, 0], 7, 256),
]


@pytest.mark.parametrize("fp8,D", [(True, 128), (False, 128), (False, 256)])
@pytest.mark.parametrize("new,old,H,bs", CASES, ids=[str(i) for i in range(len(CASES))])
def test_write_then_read(new, old, H, bs, fp8, D):
    g = torch.Generator().manual_seed(len(new) + bs)
    lens = [a + b for a, b in zip(new, old)]
    table, blocks = tables(lens, bs, g)
    first, spare = 2, 3  # rows before the first and behind the last sequence
    c = cu(new, first)
    k, v = tokens(c[-1] + spare, H, D, g), tokens(c[-1] + spare, H, D, g)
    pool = pools(blocks, H, bs, D, fp8)
    want = expected(pool, k, v, table, c, lens, bs, fp8)
    dt = table.to(torch.int32).to(DEV)
    da.decode_attn_cache_write(k.to(DEV), v.to(DEV), i32(c), dt, i32(lens), *pool)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    for name, p, w in zip(("k_pages", "v_pages", "kv_scales"), pool, want):
        if p is not None:
            assert torch.equal(bits(p), bits(w)), f"{name}: not the written tokens, or more than them"

    # the sequences that are all this call's, read back
    n = [a if b == 0 else 0 for a, b in zip(new, old)]
    cr = cu(n, first)
    outs = [torch.full((cr[-1] + spare, H, D), 0x7FA5, dtype=torch.int16, device=DEV).view(torch.bfloat16) for _ in range(2)]
    da.decode_attn_cache_read(*pool, dt, i32(cr), *outs)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    for i, out in enumerate(outs):
        got = out.cpu()
        for b in range(len(n)):
            x = gather(want[i].float(), table, b, n[b])
            if fp8:
                x = x * gather(want[2][:, :, i].float()[..., None], table, b, n[b])
            assert torch.equal(got[cr[b]:cr[b + 1]], x.transpose(0, 1).to(torch.bfloat16))
        assert (bits(got[:first]) == 0x7FA5).all() and (bits(got[cr[-1]:]) == 0x7FA5).all()


@pytest.mark.parametrize("fp8,D,bs", [(True, 128, 16), (True, 128, 64), (False, 128, 8), (False, 256, 32)])
def test_read(fp8, D, bs):
    """Any codes and scales, lengths from none to more than one block, a table with padded rows."""
    g = torch.Generator().manual_seed(bs)
    n, H = [0, 1, bs, bs + 1, 5 * bs - 1, 0, 77], 3
    table, blocks = tables(n, bs, g)
    pad = torch.full((len(n), table.shape[1] + 4), -1, dtype=torch.int32)
    pad[:, : table.shape[1]] = table
    k, v = (torch.randn((blocks, H, bs, D), generator=g) * 3 for _ in range(2))
    k, v = (x.to(torch.float8_e4m3fn if fp8 else torch.bfloat16) for x in (k, v))
    scales = torch.exp(torch.randn((blocks, H, 2, bs), generator=g)) if fp8 else None  # not powers of two
    c = cu(n)
    outs = [torch.zeros((c[-1], H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    da.decode_attn_cache_read(k.to(DEV), v.to(DEV), None if scales is None else scales.to(DEV), pad.to(DEV)[:, : table.shape[1]],
                              i32(c), *outs)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    for i, (pages, out) in enumerate(((k, outs[0]), (v, outs[1]))):
        for b in range(len(n)):
            x = gather(pages.float(), table, b, n[b])
            if fp8:
                x = x * gather(scales[:, :, i][..., None], table, b, n[b])  # one product in fp32, then bf16
            assert torch.equal(out.cpu()[c[b]:c[b + 1]], x.transpose(0, 1).to(torch.bfloat16))


def test_special_rows():
    """Zeros, infinities, NaN, subnormals, the largest values, every power of two and both sides of every border."""
    rows = [torch.zeros(128), torch.full((128,), -0.0)]
    base = torch.linspace(-1, 1, 128)
    for e in list(range(-133, 128)):
        rows.append(base * 2.0 ** e)
    for f in (447.0, 448.0, 450.0, 464.0, 480.0, 224.0, 226.0):
        rows.append(base * f)
    for x in (float("inf"), -float("inf"), float("nan")):
        r = base.clone()
        r[5] = x
        rows.append(r)
        rows.append(torch.full((128,), x))
    rows.append(torch.full((128,), 3.3895e38))
    r = torch.zeros(128)
    r[127] = 2.0 ** -133
    rows.append(r)
    x = torch.stack(rows).to(torch.bfloat16)[:, None]
    T, bs = len(rows), 16
    table = torch.arange(-(-T // bs)).view(1, -1)
    pool = pools(table.numel(), 1, bs, 128, True)
    da.decode_attn_cache_write(x.to(DEV), x.flip(0).contiguous().to(DEV), i32([0, T]), table.to(torch.int32).to(DEV), i32([T]), *pool)
    outs = [torch.zeros(x.shape, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    da.decode_attn_cache_read(*pool, table.to(torch.int32).to(DEV), i32([0, T]), *outs)
    torch.cuda.synchronize()
    want = expected(pools(table.numel(), 1, bs, 128, True), x, x.flip(0), table, [0, T], [T], bs, True)
    for p, w in zip(pool, want):
        if p.dtype == torch.float8_e4m3fn:  # NaN codes: either sign
            a, b = bits(p), bits(w)
            assert torch.equal(torch.where((a & 0x7F) == 0x7F, 0x7F, a), torch.where((b & 0x7F) == 0x7F, 0x7F, b))
        else:
            assert torch.equal(bits(p), bits(w))
    got, xf = outs[0].cpu().double(), x.double()
    fine = torch.isfinite(xf)
    size = torch.where(fine, xf.abs(), torch.zeros_like(xf)).amax(-1, keepdim=True)
    # a normal code is within 2^-4 of the value, a subnormal one (below 2^-6 of the scale, 448 of which the row's
    # largest fills more than half of) within half of its step 2^-9
    tol = torch.maximum(xf.abs() * 2.0 ** -4, torch.maximum(size / 224 * 2.0 ** -10, torch.tensor(2.0 ** -134, dtype=torch.float64)))
    assert ((got - xf).abs()[fine] <= tol[fine]).all()
    assert torch.isnan(got[torch.isnan(xf)]).all()
    assert torch.equal(torch.sign(got[torch.isinf(xf)]), torch.sign(xf[torch.isinf(xf)])) and torch.isfinite(got[torch.isinf(xf)]).all()


@pytest.mark.parametrize("fp8", [True, False])
def test_strided(fp8):
    """k and v as slices of one projection's output, pools stored token-major."""
    g = torch.Generator().manual_seed(2)
    H, bs, lens, new = 4, 32, [40, 100], [40, 60]
    table, blocks = tables(lens, bs, g)
    c = cu(new)
    kv = tokens(c[-1], 2 * H + 3, 128, g)
    k, v = kv[:, :H], kv[:, H:2 * H]
    plain, swapped = pools(blocks, H, bs, 128, fp8), pools(blocks, bs, H, 128, fp8)
    scales = plain[2]
    for p in plain[:2], [t.transpose(1, 2) for t in swapped[:2]]:
        d = kv.to(DEV)
        da.decode_attn_cache_write(d[:, :H], d[:, H:2 * H], i32(c), table.to(torch.int32).to(DEV), i32(lens), *p, scales)
        outs = [torch.zeros((c[-1], H, 256), dtype=torch.bfloat16, device=DEV)[:, :, 64:192] for _ in range(2)]
        da.decode_attn_cache_read(*p, scales, table.to(torch.int32).to(DEV), i32([0, 40, 40]), *outs)
        torch.cuda.synchronize()
        want = expected(pools(blocks, H, bs, 128, fp8), k, v, table, c, lens, bs, fp8)
        for i in range(2):
            assert torch.equal(bits(p[i].contiguous()), bits(want[i]))
            x = gather(want[i].float(), table, 0, 40)
            x = x * gather(want[2][:, :, i][..., None], table, 0, 40) if fp8 else x
            assert torch.equal(outs[i].cpu()[:40], x.transpose(0, 1).to(torch.bfloat16))


def test_places_outside():
    """Tokens before the first and past the table, and blocks outside the pool: the rest is written, bit 64 says so."""
    g = torch.Generator().manual_seed(4)
    bs, H = 16, 2
    table = torch.tensor([[0, 1], [2, 99], [-7, 3]])
    new, lens = [6, 20, 20], [4, 34, 20]  # 2 negative positions; position 32, 33 past the table, 16.. block 99; block -7
    c = cu(new)
    k, v = tokens(c[-1], H, 128, g), tokens(c[-1], H, 128, g)
    pool, want = pools(5, H, bs, 128, True), pools(5, H, bs, 128, True)
    da.decode_attn_cache_write(k.to(DEV), v.to(DEV), i32(c), table.to(torch.int32).to(DEV), i32(lens), *pool)
    assert da.decode_attn_last_device_error() == 64 and da.decode_attn_last_device_error() == 0
    want = [t.cpu() for t in want]
    for row, block, r in places(table, c, lens, bs):
        if 0 <= block < 5:
            for i, x in enumerate((k, v)):
                codes, s = quantise_ref(x[row])
                want[i].view(torch.uint8)[block, :, r] = codes
                want[2][block, :, i, r] = s
    for p, w in zip(pool, want):
        assert torch.equal(bits(p), bits(w))
    outs = [torch.ones((70, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pool[2].nan_to_num_(1.0)  # (rows that were never written)
    da.decode_attn_cache_read(*pool, table.to(torch.int32).to(DEV), i32([0, 4, 24, 64]), *outs)
    assert da.decode_attn_last_device_error() == 64
    got = outs[0].cpu()
    assert (got[20:24] == 0).all() and (got[24:40] == 0).all() and (got[56:64] == 0).all() and (got[64:] == 1).all()
    assert torch.equal(got[2:4].float(), (want[0].float()[0, :, 2:4] * want[2][0, :, 0, 2:4][..., None]).transpose(0, 1))


def test_offsets_of_any_kind_stay_inside():
    """Offsets that fall, start late or run past the tokens leave tokens without a sequence; nothing else happens."""
    g = torch.Generator().manual_seed(5)
    k = tokens(50, 2, 128, g)
    table = torch.arange(8).view(4, 2)
    for c in ([10, 5, 40, 40, 1 << 30], [-3, 10, 20, 30, 40], [60, 61, 62, 63, 64], [2 ** 31 - 1, -2 ** 31, 7, 9, 3]):
        pool = pools(8, 2, 16, 128, True)
        da.decode_attn_cache_write(k.to(DEV), k.to(DEV), i32(c), table.to(torch.int32).to(DEV), i32([32, 32, -2 ** 31, 2 ** 31 - 1]), *pool)
        assert da.decode_attn_last_device_error() in (0, 64)


def test_captured_other_stream_and_empty():
    g = torch.Generator().manual_seed(6)
    bs, H, B = 64, 8, 9
    table, blocks = tables([200] * B, bs, g)
    dt, c = table.to(torch.int32).to(DEV), i32(cu([1] * B))
    lens = i32([100] * B)
    k, v = tokens(B, H, 128, g).to(DEV), tokens(B, H, 128, g).to(DEV)
    pool = pools(blocks, H, bs, 128, True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        da.decode_attn_cache_write(k, v, c, dt, lens, *pool)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.decode_attn_cache_write(k, v, c, dt, lens, *pool)
        lens.add_(1)
    want = expected(pools(blocks, H, bs, 128, True), k.cpu(), v.cpu(), table, cu([1] * B), [100] * B, bs, True)
    for step in range(3):
        k.copy_(tokens(B, H, 128, g))
        v.copy_(tokens(B, H, 128, g))
        want = expected(want, k.cpu(), v.cpu(), table, cu([1] * B), [100 + step] * B, bs, True)
        graph.replay()
    torch.cuda.synchronize()
    for p, w in zip(pool, want):
        assert torch.equal(bits(p), bits(w))
    before = [bits(p) for p in pool]
    none = torch.empty((0, H, 128), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_cache_write(none, none, i32([0] * (B + 1)), dt, lens, *pool)
    da.decode_attn_cache_write(k, v, i32([0]), dt[:0], lens[:0], *pool)
    da.decode_attn_cache_read(*pool, dt, i32([0] * (B + 1)), none, none.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(bits(p), b) for p, b in zip(pool, before))
