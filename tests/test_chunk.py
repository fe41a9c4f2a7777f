"""decode_attn_chunk and decode_attn_prefill_window against 64 bits: windows and first tokens of every kind, pools of every
block size and stride, lengths from none to thousands, what no query sees filled with NaN, and rows that are not theirs left
as they were."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from chunk_helpers import attend_ref
from prompt_helpers import F64, assert_within, quantise_ref
from test_cache import DEV, _library, bits, cu, i32  # noqa: F401

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)
NAN = float("nan")


def packed(g, lq, lk, Hq, Hkv, tail=3):
    cq, ck = cu(lq), cu(lk)
    q, k, v = (torch.randn((n + tail, h, 128), generator=g).to(torch.bfloat16) for n, h in ((cq[-1], Hq), (ck[-1], Hkv), (ck[-1], Hkv)))
    return q, k, v, cq, ck


def canvas(q):
    return torch.full(q.shape, 7.5, dtype=torch.bfloat16, device=DEV)


def check(out, ref, tol, have, what):
    out = out.cpu()
    assert_within(out[have], ref[have], tol[have], what)
    assert (out[~have] == 7.5).all(), "a row of no sequence was written"
    assert da.decode_attn_last_device_error() == 0


WINDOWS = [  # Hq, Hkv, queries, keys, window, sinks
    (8, 2, [70, 0, 1, 300], [70, 5, 1, 300], 50, 0), (4, 4, [400], [400], 1, 0), (4, 4, [400], [400], 1, 1), (6, 2, [300], [300], 130, 4),
    (32, 2, [200, 33], [200, 150], 64, 129), (8, 1, [10], [5000], 777, 4), (8, 1, [10], [5000], 4900, 300), (16, 1, [1, 1, 1], [900, 1, 130], 128, 1),
    (8, 8, [5], [0], 3, 3), (7, 7, [43, 100], [30, 260], 20, 2), (12, 1, [1000], [1900], 256, 0), (4, 1, [64, 3], [2600, 1700], 2000, 500),
    (8, 2, [1], [20000], 8192, 4), (8, 2, [600], [600], 100000, 4), (8, 2, [900, 700], [900, 2000], 200, 120), (4, 1, [700], [800], 130, 8),
    (16, 2, [300], [1000], 257, 1), (1, 1, [400, 300], [400, 9000], 129, 121), (2, 2, [513], [513], 127, 1000), (1, 1, [1], [1], 1, 0), (10, 2, [777], [777], 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("Hq,Hkv,lq,lk,window,sinks", WINDOWS, ids=str)
def test_prefill_window(Hq, Hkv, lq, lk, window, sinks):
    g = torch.Generator().manual_seed(71)
    q, k, v, cq, ck = packed(g, lq, lk, Hq, Hkv)
    k[ck[-1]:], v[ck[-1]:] = NAN, NAN
    ref, tol, have = attend_ref(q, [k[a:b] for a, b in zip(ck, ck[1:])], [v[a:b] for a, b in zip(ck, ck[1:])], cq, SCALE, window, sinks)
    out = canvas(q)
    assert da.decode_attn_prefill_window(q.to(DEV), k.to(DEV), v.to(DEV), i32(cq), i32(ck), out, SCALE, window, sinks) is out
    check(out, ref, tol, have, "window")
    # keys outside every query's window are not looked at
    for b in range(len(lq)):
        lo, n = max(0, lk[b] - lq[b] - window + 1), min(sinks, lk[b])
        k[ck[b] + n:ck[b] + lo], v[ck[b] + n:ck[b] + lo] = NAN, NAN
    again = canvas(q)
    da.decode_attn_prefill_window(q.to(DEV), k.to(DEV), v.to(DEV), i32(cq), i32(ck), again, SCALE, window, sinks)
    assert torch.equal(bits(again), bits(out))


@pytest.mark.parametrize("lq,lk", [([300, 1, 0, 64], [300, 900, 4, 64]), ([3], [7000])], ids=str)
def test_no_window_is_the_plain_call(lq, lk):
    g = torch.Generator().manual_seed(72)
    q, k, v, cq, ck = packed(g, lq, lk, 8, 2)
    args = q.to(DEV), k.to(DEV), v.to(DEV), i32(cq), i32(ck)
    plain, zero, wide = canvas(q), canvas(q), canvas(q)
    da.decode_attn_prefill(*args, plain, SCALE)
    da.decode_attn_prefill_window(*args, zero, SCALE, 0, 5)
    da.decode_attn_prefill_window(*args, wide, SCALE, max(lk), 5)
    assert torch.equal(bits(zero), bits(plain)) and torch.equal(bits(wide), bits(plain))


class Cache:
    """Pools of shuffled blocks; whatever holds no token of a sequence is NaN, and so are the scales there."""

    def __init__(self, g, lens, Hkv, bs, kv8=False, spare=4, swapped=False, scales="powers"):
        self.lens, self.bs, B = lens, bs, len(lens)
        most = max(1, max(-(-n // bs) for n in lens)) + 1
        nb = B * most + spare
        self.table = torch.randperm(nb, generator=g)[: B * most].view(B, most)
        self.kv8 = kv8
        self.pools, self.scales, self.tokens = [], torch.full((nb, Hkv, 2, bs), NAN) if kv8 else None, []
        for at in range(2):
            pool = torch.full((nb, Hkv, bs, 128), NAN, dtype=torch.bfloat16)
            pool = torch.full(pool.shape, 0x7F, dtype=torch.uint8) if kv8 else pool
            held = []
            for b, n in enumerate(lens):
                x = (torch.randn((n, Hkv, 128), generator=g) * torch.exp(torch.randn((n, Hkv, 1), generator=g) * (0.3 if at == 0 else 1))).to(torch.bfloat16)
                if kv8:
                    codes, s = quantise_ref(x)
                    if scales == "any":
                        s = s * (torch.rand(s.shape, generator=g) + 0.5) * torch.where(torch.rand(s.shape, generator=g) < 0.1, 0.0, 1.0)
                        s = torch.where(torch.rand(s.shape, generator=g) < 0.1, -s, s)
                    held.append(codes.view(torch.float8_e4m3fn).to(F64) * s.to(F64)[..., None])
                else:
                    held.append(x)
                for i in range(-(-n // bs)):
                    m, blk = min(bs, n - i * bs), int(self.table[b, i])
                    rows = slice(i * bs, i * bs + m)
                    pool[blk, :, :m] = (codes if kv8 else x)[rows].transpose(0, 1)
                    if kv8:
                        self.scales[blk, :, at, :m] = s[rows].T
            self.tokens.append(held)
            self.pools.append(pool.view(torch.float8_e4m3fn) if kv8 else pool)
        self.swapped = swapped

    def on(self):
        got = []
        for p in self.pools:
            x = p.to(DEV)
            got.append(x.transpose(1, 2).contiguous().transpose(1, 2) if self.swapped else x)
        return (*got, None if self.scales is None else self.scales.to(DEV))

    def forget(self, b, first, last):
        """Tokens first .. last - 1 of sequence b are gone: whole blocks of them leave the table, the others' rows become NaN."""
        for i in range(self.table.shape[1]):
            a, z = max(first, i * self.bs), min(last, (i + 1) * self.bs)
            if z - a == self.bs:
                self.table[b, i] = [-1, 1 << 30, int(self.table[b, i])][i % 3]
                blk = int(self.table[b, i])
                if not 0 <= blk < len(self.pools[0]):
                    continue
            if a < z:
                blk = int(self.table[b, i])
                for p in self.pools:
                    if self.kv8:
                        p.view(torch.uint8)[blk, :, a - i * self.bs:z - i * self.bs] = 0x7F
                    else:
                        p[blk, :, a - i * self.bs:z - i * self.bs] = NAN
                if self.kv8:
                    self.scales[blk, :, :, a - i * self.bs:z - i * self.bs] = NAN


CHUNKS = [  # Hq, Hkv, queries, keys, block size, window, sinks
    (8, 2, [70, 0, 1, 300], [70, 5, 1, 300], 16, 0, 0), (32, 8, [1], [1], 64, 0, 0), (32, 8, [1], [2049], 64, 0, 0), (4, 4, [1] * 40, list(range(0, 400, 10)), 16, 0, 0),
    (8, 1, [4, 1, 7, 33], [500, 3000, 7, 5000], 32, 0, 0), (16, 1, [130], [1000], 8, 0, 0), (6, 2, [43, 100, 7], [30, 260, 3], 128, 0, 0),
    (12, 4, [512], [1700], 256, 0, 0), (7, 1, [18, 19], [700, 19], 512, 0, 0), (8, 8, [5, 0], [0, 0], 64, 0, 0),
    (8, 2, [1] * 9, [900, 0, 130, 257, 5000, 64, 128, 1, 2000], 64, 128, 4), (32, 2, [200, 33], [200, 1500], 16, 64, 129), (4, 4, [1], [9000], 32, 4096, 1),
    (8, 1, [64, 3], [2600, 1700], 128, 500, 0), (16, 1, [1, 1], [4000, 70], 256, 1, 1), (8, 2, [300], [5000], 8, 700, 20), (2, 1, [257], [3000], 64, 2 ** 31 - 1, 9),
    (8, 2, [3], [12000], 16, 3000, 3001), (8, 2, [300, 90], [5000, 200], 32, 1000, 4), (4, 4, [700], [900], 16, 65, 100), (5, 5, [1] * 3, [4097, 4096, 4095], 1024, 1024, 2),
]


@pytest.mark.parametrize("kv", ["bf16", "bf16_swapped", "e4m3", "e4m3_any"])
@pytest.mark.parametrize("Hq,Hkv,lq,lk,bs,window,sinks", CHUNKS, ids=str)
def test_chunk(Hq, Hkv, lq, lk, bs, window, sinks, kv):
    kv8 = kv.startswith("e4m3")
    if kv8 and bs < 16:
        pytest.skip("e4m3 pools: blocks of 16 and more")
    g = torch.Generator().manual_seed(73)
    cache = Cache(g, lk, Hkv, bs, kv8, swapped=kv == "bf16_swapped", scales="any" if kv == "e4m3_any" else "powers")
    c = cu(lq, first=1)
    q = torch.randn((c[-1] + 2, Hq, 128), generator=g).to(torch.bfloat16)
    # scales that are no powers of two: keys and values may be rounded to bf16, each element off by 2^-8 of it
    ref, tol, have = attend_ref(q, *cache.tokens, c, SCALE, window, sinks, kv_eps=2.0 ** -8 if kv == "e4m3_any" else 0.0)

    def call():
        wide = torch.full((len(lk), cache.table.shape[1] + 3), 1 << 29, dtype=torch.int32)  # rows further apart
        wide[:, :-3] = cache.table
        kp, vp, sc = cache.on()
        out = canvas(q)
        assert da.decode_attn_chunk(q.to(DEV), kp, vp, sc, wide.to(DEV)[:, :-3], i32(c), i32(lk), out, SCALE, window, sinks) is out
        return out

    out = call()
    check(out, ref, tol, have, kv)
    if window:  # what no query sees any more has been given to others
        for b in range(len(lq)):
            cache.forget(b, min(sinks, lk[b]), max(0, lk[b] - lq[b] - window + 1))
        again = call()
        check(again, ref, tol, have, "after the window has moved on")
        assert torch.equal(bits(again), bits(out))


@pytest.mark.parametrize("kv8", [False, True])
def test_chunk_is_read_then_prompt(kv8):
    """The same bits as the cache read back and decode_attn_prefill over it, where neither cuts the keys into parts."""
    g = torch.Generator().manual_seed(74)
    lq, lk = [300, 129, 512, 64], [300, 1000, 1300, 65]
    cache = Cache(g, lk, 8, 32, kv8)
    c, ck = cu(lq), cu(lk)
    q = torch.randn((c[-1], 32, 128), generator=g).to(torch.bfloat16).to(DEV)
    pools, t = cache.on(), cache.table.to(torch.int32).to(DEV)
    k, v = (torch.empty((ck[-1], 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    da.decode_attn_cache_read(*pools, t, i32(ck), k, v)
    a, b = torch.empty_like(q), torch.empty_like(q)
    da.decode_attn_prefill(q, k, v, i32(c), i32(ck), a, SCALE)
    da.decode_attn_chunk(q, *pools, t, i32(c), i32(lk), b, SCALE)
    assert torch.equal(bits(a), bits(b))
    assert da.decode_attn_last_device_error() == 0


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("bs", [16, 256])
def test_blocks_outside_the_pool(kv8, bs):
    """They read as zeros and are reported; so are lengths past the table's capacity, which end there."""
    g = torch.Generator().manual_seed(75)
    lk = [3 * bs, 2 * bs + 5]
    cache = Cache(g, lk, 2, bs, kv8)
    kp, vp, sc = cache.on()
    q = torch.randn((2, 8, 128), generator=g).to(torch.bfloat16)
    table = cache.table.clone()
    table[0, 1], table[1, 0] = -3, len(cache.pools[0])
    out = canvas(q)
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, table.to(torch.int32).to(DEV), i32([0, 1, 2]), i32(lk), out, SCALE)
    assert da.decode_attn_last_device_error() == 64
    for held in cache.tokens:
        held[0][bs:2 * bs] = 0
        held[1][:bs] = 0
    ref, tol, _ = attend_ref(q, *cache.tokens, [0, 1, 2], SCALE)
    assert_within(out.cpu(), ref, tol, "zeros")
    # a table of two entries each: sequence 0 ends with its second block
    for held in cache.tokens:
        held[0], held[1] = held[0][:2 * bs], held[1][:2 * bs]
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, table[:, :2].contiguous().to(torch.int32).to(DEV), i32([0, 1, 2]), i32([2 ** 31 - 1, 3 * bs]), out, SCALE)
    assert da.decode_attn_last_device_error() == 64
    ref, tol, _ = attend_ref(q, *cache.tokens, [0, 1, 2], SCALE)
    assert_within(out.cpu(), ref, tol, "capacity")


def test_scores_past_24_bits_and_negative_scales():
    """Scores that fp32 products part by whole powers of two: the largest keys share the row, in a window too; few rows and many."""
    g = torch.Generator().manual_seed(76)
    bs, lk, window, sinks = 16, 900, 300, 5
    for scale, lq in ((SCALE, 70), (-0.3, 70), (SCALE, 3), (-0.3, 2)):
        for size in (26, 40):
            cache = Cache(g, [lk], 1, bs)
            c = torch.randint(1, 256, (lk, 1, 1), generator=g).float()
            k = (c * 2.0 ** (size - size // 2 - 7)).expand(-1, -1, 128).to(torch.bfloat16)
            for i in range(-(-lk // bs)):
                rows = k[i * bs:(i + 1) * bs]
                cache.pools[0][int(cache.table[0, i]), :, :len(rows)] = rows.transpose(0, 1)
            q = torch.full((lq, 4, 128), 2.0 ** (size // 2)).to(torch.bfloat16)
            kp, vp, _ = cache.on()
            out = canvas(q)
            da.decode_attn_chunk(q.to(DEV), kp, vp, None, cache.table.to(torch.int32).to(DEV), i32([0, lq]), i32([lk]), out, scale, window, sinks)
            for r in sorted({0, 1, lq // 2, lq - 1}):
                i = r + lk - lq
                seen = torch.tensor([j for j in range(i + 1) if j > i - window or j < sinks])
                cs = c[seen, 0, 0]
                rows = cache.tokens[1][0][seen, 0].double()[cs == (cs.max() if scale > 0 else cs.min())]
                d = (out[r, 1].cpu().double() - rows.mean(0)).abs()
                assert bool((d <= 2.0 ** -8 * (rows.abs().mean(0) + rows.mean(0).abs())).all()), (scale, size, r)


def test_pool_past_32_bits():
    """Blocks whose elements lie past 2^32, of K, V, codes and scales."""
    g = torch.Generator().manual_seed(77)
    bs, Hkv = 128, 8
    nb = (1 << 32) // (Hkv * bs * 128) + 40
    for kv8 in (False, True):
        small = Cache(g, [700], Hkv, bs, kv8)
        n = len(small.pools[0])
        big = []
        for p in small.on():
            if p is not None:
                x = torch.empty((nb, *p.shape[1:]), dtype=p.dtype, device=DEV)
                x[nb - n:] = p
                big.append(x)
            else:
                big.append(None)
        q = torch.randn((40, 16, 128), generator=g).to(torch.bfloat16)
        out = canvas(q)
        da.decode_attn_chunk(q.to(DEV), *big, (small.table + nb - n).to(torch.int32).to(DEV), i32([0, 40]), i32([700]), out, SCALE)
        ref, tol, have = attend_ref(q, *small.tokens, [0, 40], SCALE)
        check(out, ref, tol, have, "far blocks")
        del big, x


@pytest.mark.parametrize("more", [0, 600])
@pytest.mark.parametrize("paged", [None, False, True])
def test_long_keys_from_far(paged, more):
    """More work items of one query tile than SMs, none cut into parts, keys that no cache holds yet: K and V tiles land late
    and out of step (None: packed keys; `more`: queries of one sequence besides the two of each)."""
    g = torch.Generator().manual_seed(80)
    B, H = 24, 8
    lk = torch.randint(2500, 4500, (B,), generator=g).tolist()
    c = cu([2] * (B - 1) + [2 + more])
    q = torch.randn((c[-1], H, 128), generator=g).to(torch.bfloat16)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    if paged is None:
        ck = cu(lk)
        k, v = (torch.randn((ck[-1], H, 128), generator=g).to(torch.bfloat16) for _ in range(2))
        tokens = [[x[a:b] for a, b in zip(ck, ck[1:])] for x in (k, v)]
        args = q.to(DEV), k.to(DEV), v.to(DEV), i32(c), i32(ck)
        run = lambda out: da.decode_attn_prefill(*args, out, SCALE)  # noqa: E731
    else:
        cache = Cache(g, lk, H, 64, paged)
        tokens = cache.tokens
        pools = cache.on()
        args = (q.to(DEV), *pools, cache.table.to(torch.int32).to(DEV), i32(c), i32(lk))
        run = lambda out: da.decode_attn_chunk(*args, out, SCALE)  # noqa: E731
    ref, tol, have = attend_ref(q, *tokens, c, SCALE)
    for i in range(5):
        out = canvas(q)
        flush.fill_(i)
        run(out)
        check(out, ref, tol, have, f"pass {i}")


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("scale", [0.0, 1e-42, -1.0, 3.0])
def test_scales_of_every_kind(scale, kv8):
    """0 gives every key the same weight; few rows and many."""
    g = torch.Generator().manual_seed(85)
    cache = Cache(g, [200, 333], 2, 16, kv8)
    for lq in (1, 120):
        q = torch.randn((2 * lq, 8, 128), generator=g).to(torch.bfloat16)
        out = canvas(q)
        da.decode_attn_chunk(q.to(DEV), *cache.on(), cache.table.to(torch.int32).to(DEV), i32([0, lq, 2 * lq]), i32([200, 333]), out, scale)
        ref, tol, have = attend_ref(q, *cache.tokens, [0, lq, 2 * lq], scale)
        check(out, ref, tol, have, "scale")


def test_offsets_of_any_kind():
    """Offsets that decrease or lie outside, negative lengths: nothing but rows of out is written, and well-formed sequences come out right."""
    g = torch.Generator().manual_seed(86)
    for kv8 in (False, True):
        for rows in (1, 40):
            cache = Cache(g, [300, 90, 200], 2, 16, kv8)
            T = 3 * rows + 4
            q = torch.randn((T, 4, 128), generator=g).to(torch.bfloat16)
            for c in ([-5, 2, 1, 10 ** 6], [3, 3, -1, 2], [2 ** 31 - 1, -2 ** 31, 5, 7], [0, T, 0, T]):
                big = torch.full((T + 2, 4, 128), 7.5, dtype=torch.bfloat16, device=DEV)
                da.decode_attn_chunk(q.to(DEV), *cache.on(), cache.table.to(torch.int32).to(DEV), i32(c), i32([300, -9, 200]), big[1:-1], SCALE)
                assert (big[0] == 7.5).all() and (big[-1] == 7.5).all()
                assert da.decode_attn_last_device_error() == 0
            out = canvas(q)
            c = [1, 1 + rows, 1 + rows, 1 + 2 * rows]
            da.decode_attn_chunk(q.to(DEV), *cache.on(), cache.table.to(torch.int32).to(DEV), i32(c), i32([300, -9, 200]), out, SCALE)
            held = [[x[0], x[1][:0], x[2]] for x in cache.tokens]
            check(out, *attend_ref(q, *held, c, SCALE), "sound")


def test_many_sequences():
    """1000 sequences of one query, and more queries than a table's row of work items."""
    g = torch.Generator().manual_seed(78)
    lk = torch.randint(0, 300, (1000,), generator=g).tolist()
    for kv8 in (False, True):
        cache = Cache(g, lk, 1, 16, kv8)
        c = cu([1] * 1000)
        q = torch.randn((1000, 4, 128), generator=g).to(torch.bfloat16)
        kp, vp, sc = cache.on()
        out = canvas(q)
        da.decode_attn_chunk(q.to(DEV), kp, vp, sc, cache.table.to(torch.int32).to(DEV), i32(c), i32(lk), out, SCALE)
        ref, tol, have = attend_ref(q, *cache.tokens, c, SCALE)
        check(out, ref, tol, have, "many")


@pytest.mark.parametrize("capacity,lq,lk", [(200_000, [70, 1, 0, 33, 90, 60, 64, 65], [900, 1, 300, 33, 2000, 777, 64, 1300]), (1_600_000, [150], [3000])], ids=str)
def test_tables_of_large_capacity(capacity, lq, lk):
    """A table whose capacity's tokens do not fit the workspace's part for them: sequences, or heads, a few at a time."""
    g = torch.Generator().manual_seed(84)
    cache = Cache(g, lk, 8, 16, True)
    wide = torch.full((len(lk), capacity // 16), -1, dtype=torch.int32)
    wide[:, :cache.table.shape[1]] = cache.table
    c = cu(lq, first=3)
    q = torch.randn((c[-1] + 2, 16, 128), generator=g).to(torch.bfloat16)
    kp, vp, sc = cache.on()
    out = canvas(q)
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, wide.to(DEV), i32(c), i32(lk), out, SCALE)
    ref, tol, have = attend_ref(q, *cache.tokens, c, SCALE)
    check(out, ref, tol, have, "parts")


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("G,lq,window,sinks", [(1, 1, 0, 0), (4, 2, 40, 3), (8, 1, 0, 0), (4, 4, 0, 0), (16, 1, 70, 1), (3, 5, 0, 0), (11, 2, 0, 0)], ids=str)
def test_many_short_items(G, lq, window, sinks, kv8):
    """Hundreds of sequences of up to 170 keys with 8 KV heads, none and one among them."""
    g = torch.Generator().manual_seed(81)
    lk = torch.randint(0, 171, (260,), generator=g).tolist()
    n = [min(lq, x) if i % 7 else lq for i, x in enumerate(lk)]  # some with more queries than keys
    n[5] = 0
    cache = Cache(g, lk, 8, 16, kv8)
    c = cu(n, first=2)
    q = torch.randn((c[-1] + 2, 8 * G, 128), generator=g).to(torch.bfloat16)
    kp, vp, sc = cache.on()
    out = canvas(q)
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, cache.table.to(torch.int32).to(DEV), i32(c), i32(lk), out, SCALE, window, sinks)
    ref, tol, have = attend_ref(q, *cache.tokens, c, SCALE, window, sinks)
    check(out, ref, tol, have, "short")


def v_scales_case(kind, bs, lk, Hkv, g):
    """Codes and scales of a cache whose V scales differ from token to token by far more than f16 holds."""
    nb = -(-lk // bs) + 2
    codes = [torch.randint(0, 256, (nb, Hkv, bs, 128), generator=g, dtype=torch.uint8) for _ in range(2)]
    for x in codes:
        x[(x & 0x7F) == 0x7F] = 0x38  # no NaN
    scales = torch.exp2(torch.randint(-9, -3, (nb, Hkv, 2, bs), generator=g).float())
    if kind == "spread":
        scales[:, :, 1] = torch.exp2(torch.randint(-60, 40, (nb, Hkv, bs), generator=g).float())
    elif kind == "zero_rows":  # zeros as decode_attn_cache_write leaves them, with a scale of 1, among small values
        zero = torch.rand((nb, Hkv, bs), generator=g) < 0.5
        zero[0] = True
        scales[:, :, 1] = torch.where(zero, 1.0, torch.exp2(torch.randint(-45, -40, (nb, Hkv, bs), generator=g).float()))
        codes[1][zero] = 0
    elif kind == "rising":  # larger and larger
        at = torch.arange(nb * bs).view(nb, 1, bs).expand(-1, Hkv, -1)
        scales[:, :, 1] = torch.exp2((at % 100).float() - 50)
    elif kind == "falling_behind_growing_scores":
        at = torch.arange(nb * bs).view(nb, 1, bs).expand(-1, Hkv, -1)
        scales[:, :, 1] = torch.exp2(20 - (at // 8 % 60).float())
        scales[:, :, 0] = torch.exp2((at * 6 / (nb * bs)).floor() - 8)
    return codes, scales


@pytest.mark.parametrize("kind", ["spread", "zero_rows", "rising", "falling_behind_growing_scores"])
@pytest.mark.parametrize("lq", [1, 4, 90])
def test_v_scales_of_every_size(kind, lq):
    """f16 weights are off by at most 2^-25 of the largest weight times V scale of the row's keys whose V is not all zero (and
    bf16 ones, where there are many rows, by 2^-8 of themselves)."""
    g = torch.Generator().manual_seed(82)
    bs, lk, Hkv, G = 16, 700, 2, 4
    codes, scales = v_scales_case(kind, bs, lk, Hkv, g)
    q = torch.randn((lq, Hkv * G, 128), generator=g).to(torch.bfloat16)
    t = torch.arange(codes[0].shape[0])[None].to(torch.int32)
    out = canvas(q)
    pools = [x.to(DEV).view(torch.float8_e4m3fn) for x in codes]
    da.decode_attn_chunk(q.to(DEV), *pools, scales.to(DEV), t.to(DEV), i32([0, lq]), i32([lk]), out, SCALE)
    flat = [x.view(torch.float8_e4m3fn).float().transpose(1, 2).reshape(-1, Hkv, 128)[:lk].to(F64) for x in codes]
    sc = scales.permute(0, 3, 1, 2).reshape(-1, Hkv, 2)[:lk].to(F64)
    k, v = flat[0] * sc[..., :1], flat[1] * sc[..., 1:]
    ref, tol, have = attend_ref(q, [k], [v], [0, lq], SCALE)
    for h in range(Hkv * G):  # the floor of the f16 weights
        j = h // G
        x = q[:, h].to(F64) @ k[:, j].T * SCALE
        x = x.masked_fill(torch.arange(lk)[None] > torch.arange(lq)[:, None] + lk - lq, -math.inf)
        p = torch.softmax(x, -1)
        some = (flat[1][:, j] != 0).any(-1)
        r = (p * torch.where(some, sc[:, j, 1], 0.0)).amax(-1, keepdim=True)
        tol[:, h] += 2.0 ** -25 * r * flat[1][:, j].abs().sum(0)[None]
    check(out, ref, tol, have, kind)


@pytest.mark.parametrize("power", [-120, -40, 40, 110])
def test_queries_of_every_size(power):
    """Rows of q around 2^power (f16 holds 2^-24 to 2^16), the scale making up for it; values in a row far apart."""
    g = torch.Generator().manual_seed(83)
    lk, Hkv, G = 300, 2, 4
    cache = Cache(g, [lk], Hkv, 16, True)
    q = torch.randn((2, Hkv * G, 128), generator=g) * torch.exp2(torch.randint(-12, 1, (2, Hkv * G, 128), generator=g).float())
    q = (q.double() * 2.0 ** power).to(torch.bfloat16)
    scale = SCALE * 2.0 ** -power
    kp, vp, sc = cache.on()
    out = canvas(q)
    da.decode_attn_chunk(q.to(DEV), kp, vp, sc, cache.table.to(torch.int32).to(DEV), i32([0, 2]), i32([lk]), out, scale)
    ref, tol, have = attend_ref(q, *cache.tokens, [0, 2], scale)
    check(out, ref, tol, have, "sizes")


@pytest.mark.parametrize("kv8", [False, True])
def test_captured_on_a_stream(kv8):
    """A step captured once and replayed with other queries and lengths on a stream of its own, an eager call between."""
    g = torch.Generator().manual_seed(79)
    lk = [1800, 40, 700]
    cache = Cache(g, lk, 2, 64, kv8)
    kp, vp, sc = cache.on()
    t = cache.table.to(torch.int32).to(DEV)
    q, lens, c = torch.zeros((6, 8, 128), dtype=torch.bfloat16, device=DEV), i32(lk), i32([0, 2, 4, 6])
    out = torch.zeros_like(q)
    run = lambda o: da.decode_attn_chunk(q, kp, vp, sc, t, c, lens, o, SCALE, 900, 3)  # noqa: E731
    run(out)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        run(out)
    for step in range(3):
        n = [max(2, x - 7 * step) for x in lk]
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        host = torch.randn(q.shape, generator=g).to(torch.bfloat16)
        q.copy_(host)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref, tol, have = attend_ref(host, [x[:m] for x, m in zip(cache.tokens[0], n)], [x[:m] for x, m in zip(cache.tokens[1], n)], [0, 2, 4, 6], SCALE, 900, 3)
        assert_within(out.cpu(), ref, tol, f"replay {step}")
        other = torch.zeros_like(q)
        run(other)
        torch.cuda.synchronize()
        assert torch.equal(bits(other), bits(out))
    assert da.decode_attn_last_device_error() == 0
