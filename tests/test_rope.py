"""decode_attn_rope and decode_attn_rope_cache_write: rows against the definition in 64 bits, pages bit for bit against
decode_attn_rope followed by decode_attn_cache_write, and every byte that is not theirs left as it was."""
import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import assert_within, places, quantise_ref
from rope_helpers import F64, angles, rope_f32, rope_ref, table
from test_cache import DEV, _library, bits, cu, i32, pools, tables  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-6


def dev(t):
    return None if t is None else t.to(DEV)


def fused_rows(g, T, Hq, Hkv, D):
    """q, k, v as a projection leaves them: views of one tensor of rows."""
    size = torch.exp(torch.randn((T, Hq + 2 * Hkv, 1), generator=g))
    x = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * size).to(torch.bfloat16)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def on_device(views):
    """The same views of one device tensor."""
    base = torch.cat(views, 1).to(DEV)
    at, got = 0, []
    for v in views:
        got.append(base[:, at:at + v.shape[1]])
        at += v.shape[1]
    return got


def weights(g, D, kind):
    if kind is None:
        return None, None
    return tuple(torch.exp(0.5 * torch.randn(D, generator=g)).to(kind) for _ in range(2))


def positions_of(g, T, P, A):
    if A == 0:
        return torch.randint(0, P, (T,), generator=g).to(torch.int32)
    return torch.randint(0, P, (A, T), generator=g).to(torch.int32)


ROPES = [  # T, Hq, Hkv, D, R, interleaved, axes (0: positions [T]), weights
    (1, 32, 8, 128, 128, False, 0, torch.bfloat16), (64, 32, 8, 128, 128, False, 0, None), (77, 8, 1, 128, 64, True, 0, torch.float32),
    (333, 6, 2, 128, 32, False, 3, torch.bfloat16), (129, 7, 7, 128, 128, True, 3, None), (50, 5, 1, 256, 256, False, 2, torch.float32),
    (1001, 16, 2, 256, 64, True, 0, torch.bfloat16), (19, 1, 1, 256, 192, False, 0, None), (40, 3, 1, 128, 8, False, 0, torch.bfloat16),
    (2050, 32, 8, 128, 72, True, 4, torch.bfloat16), (900, 12, 4, 128, 120, False, 1, None), (5, 128, 8, 128, 128, False, 0, torch.bfloat16),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,inter,A,wt", ROPES, ids=str)
def test_rope_rows(T, Hq, Hkv, D, R, inter, A, wt):
    g = torch.Generator().manual_seed(T)
    P = 5000
    q, k, _ = fused_rows(g, T, Hq, Hkv, D)
    tab, pos = table(P, R), positions_of(g, T, P, A)
    axes = torch.randint(0, A, (R // 2,), generator=g).to(torch.int32) if A else None
    qw, kw = weights(g, D, wt)
    dq, dk = on_device((q, k))
    qo = torch.full((T, Hq + 1, D), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :Hq]  # rows further apart
    ko = torch.full((T, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    more = dict(q_weight=dev(qw), k_weight=dev(kw), axes=dev(axes), eps=EPS, interleaved=inter)
    got = da.decode_attn_rope(dq, dk, tab.to(DEV), pos.to(DEV), qo, ko, **more)
    assert got[0] is qo and got[1] is ko
    cos, sin, _ = angles(tab, pos, axes)
    for name, x, y, w in (("q", q, qo, qw), ("k", k, ko, kw)):
        ref, tol = rope_ref(x, w, EPS, cos, sin, inter)
        assert_within(y.cpu(), ref, tol, name)
    # one without the other, and in place
    again = torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_rope(None, dk, tab.to(DEV), pos.to(DEV), None, again, **more)
    assert torch.equal(bits(again), bits(ko))
    kept = dk.clone()
    da.decode_attn_rope(dq, None, tab.to(DEV), pos.to(DEV), dq, None, **more)
    assert torch.equal(bits(dq.contiguous()), bits(qo.contiguous())) and torch.equal(dk, kept)
    assert da.decode_attn_last_device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
def test_positions_outside_the_table(inter):
    """They count as an angle of 0 and are reported; the other tokens are rotated as ever."""
    g = torch.Generator().manual_seed(3)
    q, k, _ = fused_rows(g, 6, 4, 2, 128)
    tab = table(100, 128)
    pos = torch.tensor([0, 99, 100, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
    da.decode_attn_rope(q.to(DEV), k.to(DEV), tab.to(DEV), pos.to(DEV), qo, ko, interleaved=inter)
    assert da.decode_attn_last_device_error() == 128 and da.decode_attn_last_device_error() == 0
    cos, sin, off = angles(tab, pos, None)
    assert off
    for x, y in ((q, qo), (k, ko)):
        ref, tol = rope_ref(x, None, EPS, cos, sin, inter)
        assert_within(y.cpu(), ref, tol, "rows")
        assert torch.equal(y.cpu()[2:], x[2:])
    axes = torch.tensor([0, 1, 2, -1] * 16, dtype=torch.int32)  # of two axes; the others are none
    pos2 = torch.stack([pos, pos.flip(0)])
    da.decode_attn_rope(q.to(DEV), None, tab.to(DEV), pos2.to(DEV), qo, None, axes=axes.to(DEV), interleaved=inter)
    assert da.decode_attn_last_device_error() == 128
    cos, sin, _ = angles(tab, pos2, axes)
    ref, tol = rope_ref(q, None, EPS, cos, sin, inter)
    assert_within(qo.cpu(), ref, tol, "axes")


def test_rows_keep_to_themselves():
    """NaN, infinities, zeros, the largest and the smallest values: other rows do not see them; a row of zeros stays zeros."""
    g = torch.Generator().manual_seed(4)
    T, H = 40, 8
    q, k, _ = fused_rows(g, T, H, 2, 128)
    q, k = q.clone(), k.clone()
    tab, pos = table(64, 128), torch.arange(T).to(torch.int32)
    qw, kw = weights(g, 128, torch.bfloat16)
    plain = [torch.empty(x.shape, dtype=torch.bfloat16, device=DEV) for x in (q, k)]
    odd = [torch.empty_like(t) for t in plain]
    args = tab.to(DEV), pos.to(DEV)
    da.decode_attn_rope(q.to(DEV), k.to(DEV), *args, *plain, q_weight=dev(qw), k_weight=dev(kw))
    q[3, 1, 5], q[7, 7, 127], q[8, 0], q[9, 2], k[0, 0, 0] = float("nan"), float("inf"), 0.0, 1e-30, float("-inf")
    da.decode_attn_rope(q.to(DEV), k.to(DEV), *args, *odd, q_weight=dev(qw), k_weight=dev(kw))
    touched = torch.zeros(T, H, dtype=torch.bool)
    for i, h in ((3, 1), (7, 7), (8, 0), (9, 2)):
        touched[i, h] = True
    assert torch.equal(bits(odd[0])[~touched], bits(plain[0])[~touched])
    assert torch.equal(bits(odd[1])[1:], bits(plain[1])[1:]) and torch.equal(bits(odd[1])[0, 1], bits(plain[1])[0, 1])
    assert odd[0][3, 1].isnan().all() and (odd[0][8, 0] == 0).all()
    assert odd[0][9, 2].float().abs().max() < 1e-25  # eps holds it down


APPENDS = [  # lengths, tokens before, block size, Hq, Hkv, D, R, interleaved, axes, weights
    ([1] * 5, [0, 7, 64, 1000, 15], 16, 32, 8, 128, 128, False, 0, None), ([1, 0, 300, 17], [0, 5, 33, 0], 16, 6, 2, 128, 64, True, 0, torch.float32),
    ([70, 3], [58, 0], 64, 8, 8, 128, 128, False, 3, torch.bfloat16), ([513], [0], 128, 4, 1, 128, 32, True, 2, None),
    ([9, 1, 1, 2], [3, 2, 1, 0], 8, 16, 1, 128, 128, False, 0, torch.bfloat16), ([1500, 900], [100, 1], 32, 12, 4, 128, 128, False, 0, None),
    ([37, 64], [11, 0], 16, 5, 1, 256, 256, False, 0, torch.bfloat16), ([200], [50], 256, 4, 4, 256, 64, True, 3, None),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n,before,bs,Hq,Hkv,D,R,inter,A,wt", APPENDS, ids=str)
def test_append(n, before, bs, Hq, Hkv, D, R, inter, A, wt, fp8):
    if fp8 and (D == 256 or bs < 16):
        pytest.skip("e4m3 pools: head dim 128, blocks of 16 and more")
    g = torch.Generator().manual_seed(len(n) + bs)
    lens = [a + b for a, b in zip(n, before)]
    c = cu(n, first=2)  # two rows of no sequence before the first, three behind the last
    T = c[-1] + 3
    q, k, v = fused_rows(g, T, Hq, Hkv, D)
    tab = table(max(lens) + 1, R)
    at = torch.zeros(T, dtype=torch.int32)
    for b in range(len(n)):
        at[c[b]:c[b + 1]] = torch.arange(before[b], lens[b])
    pos = positions_of(g, T, max(lens), A) if A else at
    axes = torch.randint(0, A, (R // 2,), generator=g).to(torch.int32) if A else None
    qw, kw = weights(g, D, wt)
    t, blocks = tables(lens, bs, g)
    pool, want = pools(blocks, Hkv, bs, D, fp8), pools(blocks, Hkv, bs, D, fp8)
    dq, dk, dv = on_device((q, k, v))
    more = dict(q_weight=dev(qw), k_weight=dev(kw), axes=dev(axes), eps=EPS, interleaved=inter)
    place = i32(c), t.to(torch.int32).to(DEV), i32(lens)
    qo = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    # the two calls that it replaces
    q2, k2 = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_rope(dq, dk, tab.to(DEV), pos.to(DEV), q2, k2, **more)
    da.decode_attn_cache_write(k2, dv, *place, *want)
    for given in ([pos.to(DEV)] if A else [None, pos.to(DEV)]):
        for x in pool:
            if x is not None:
                x.view(torch.uint8).copy_(pools(blocks, Hkv, bs, D, fp8)[0 if x is pool[0] else 1 if x is pool[1] else 2].view(torch.uint8))
        got = da.decode_attn_rope_cache_write(dq, dk, dv, tab.to(DEV), *place, qo, *pool, positions=given, **more)
        assert got is qo
        inside = torch.zeros(T, dtype=torch.bool)
        inside[c[0]:c[-1]] = True
        assert torch.equal(bits(qo)[inside], bits(q2)[inside]) and qo[~inside.to(DEV)].isnan().all()
        assert torch.equal(bits(pool[1]), bits(want[1]))
        if not fp8:
            assert torch.equal(bits(pool[0]), bits(want[0]))
            continue
        assert torch.equal(bits(pool[2])[:, :, 1], bits(want[2])[:, :, 1])
        cos, sin, _ = angles(tab, pos, axes)
        mine, scales = bits(pool[0]), pool[2].cpu()
        wrote = torch.zeros(mine.shape[:3], dtype=torch.bool)
        if wt is None:  # the codes of the fp32 values, bit for bit
            codes, s = quantise_ref(rope_f32(k, cos, sin, inter))
            for r, blk, row in places(t, c, lens, bs):
                assert torch.equal(mine[blk, :, row], codes[r]) and torch.equal(scales[blk, :, 0, row], s[r])
                wrote[blk, :, row] = True
        else:
            ref, tol = rope_ref(k, kw, EPS, cos, sin, inter, rounded=False)
            for r, blk, row in places(t, c, lens, bs):
                s = scales[blk, :, 0, row].to(F64)
                # the least power of two that holds the row, whose largest value is known within its bound
                size, off = ref[r].abs().amax(-1), tol[r].amax(-1)
                assert bool(((size - off <= 448 * s) & (size + off > 224 * s)).all())
                x = mine[blk, :, row].view(torch.float8_e4m3fn).float().to(F64) * s[:, None]
                assert_within(x, ref[r], tol[r] * (1 + 2.0 ** -4) + 2.0 ** -4 * ref[r].abs() + 2.0 ** -10 * s[:, None], "codes")
                wrote[blk, :, row] = True
        untouched = pools(blocks, Hkv, bs, D, fp8)
        assert torch.equal(mine[~wrote], bits(untouched[0])[~wrote])
        assert torch.equal(bits(pool[2])[:, :, 0][~wrote], bits(untouched[2])[:, :, 0][~wrote])
    assert da.decode_attn_last_device_error() == 0


def test_append_tokens_without_a_place():
    """Tokens before a sequence's first are neither written nor rotated into q_out; ones past the table, or of a block that
    is none, are reported and not written, their queries rotated."""
    g = torch.Generator().manual_seed(9)
    bs, H = 16, 2
    c, lens = cu([5, 4, 3]), [3, 34, 3]
    q, k, v = fused_rows(g, c[-1], 4, H, 128)
    t = torch.tensor([[0, 1], [2, 3], [-7, 900]])
    pool = pools(5, H, bs, 128, False)
    qo = torch.full((c[-1], 4, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    tab = table(40, 128)
    da.decode_attn_rope_cache_write(*on_device((q, k, v)), tab.to(DEV), i32(c), t.to(torch.int32).to(DEV), i32(lens), qo, *pool)
    assert da.decode_attn_last_device_error() == 64
    at = torch.tensor([-2, -1, 0, 1, 2, 30, 31, 32, 33, 0, 1, 2])
    cos, sin, _ = angles(tab, at.clamp_min(0), None)
    ref, tol = rope_ref(q, None, EPS, cos, sin, False)
    assert qo[:2].isnan().all()
    assert_within(qo.cpu()[2:], ref[2:], tol[2:], "q")
    untouched, wrote = pools(5, H, bs, 128, False), torch.zeros((5, H, bs), dtype=torch.bool)
    kr, kt = rope_ref(k, None, EPS, cos, sin, False)
    for row, blk, r in ((2, 0, 0), (3, 0, 1), (4, 0, 2), (5, 3, 14), (6, 3, 15)):
        assert_within(pool[0][blk, :, r].cpu(), kr[row], kt[row], "k")
        assert torch.equal(pool[1][blk, :, r].cpu(), v[row])
        wrote[blk, :, r] = True
    for x, y in zip(pool[:2], untouched[:2]):
        assert torch.equal(bits(x)[~wrote], bits(y)[~wrote])


def test_append_values_of_every_size():
    """Keys and values from the smallest bf16 numbers to the largest, infinities and NaN among them, without rotation (position
    0): codes and scales are decode_attn_cache_write's."""
    g = torch.Generator().manual_seed(10)
    T, H, bs = 254, 2, 16
    e = torch.arange(-127, 127).float()[:, None, None]
    k = (torch.randn((T, H, 128), generator=g) * torch.exp2(e)).to(torch.bfloat16)
    v = (torch.randn((T, H, 128), generator=g) * torch.exp2(-e)).to(torch.bfloat16)
    k[k == 0] = 2.0 ** -133  # (-0 and +0 add up to +0: zeros' signs are not kept)
    k[50, 0, 3], k[51, 1, 7], v[60, 0, 0], k[70], v[71, 1] = float("inf"), float("nan"), float("-inf"), 0.0, 0.0
    t, blocks = tables([T], bs, g)
    tab = table(T, 128)
    tab[:, :64], tab[:, 64:] = 1.0, 0.0
    for fp8 in (False, True):
        pool, want = pools(blocks, H, bs, 128, fp8), pools(blocks, H, bs, 128, fp8)
        place = i32([0, T]), t.to(torch.int32).to(DEV), i32([T])
        da.decode_attn_cache_write(k.to(DEV), v.to(DEV), *place, *want)
        da.decode_attn_rope_cache_write(None, k.to(DEV), v.to(DEV), tab.to(DEV), *place, None, *pool)
        keep = torch.ones(blocks, H, bs, 128, dtype=torch.bool)
        for i, h in ((50, 0), (51, 1)):  # inf * 0 is NaN in the pair's other dim, as the definition says
            keep[int(t[0, i // bs]), h, i % bs] = False
        assert torch.equal(bits(pool[0])[keep], bits(want[0])[keep]) and torch.equal(bits(pool[1]), bits(want[1]))
        if fp8:
            assert torch.equal(bits(pool[2])[:, :, 1], bits(want[2])[:, :, 1])
            rows = keep.all(-1)
            assert torch.equal(bits(pool[2])[:, :, 0][rows], bits(want[2])[:, :, 0][rows])


def test_append_captured_on_a_stream():
    """A step captured once and replayed with other tokens and lengths, on a stream of its own."""
    g = torch.Generator().manual_seed(11)
    B, H, bs = 6, 2, 16
    t, blocks = tables([64] * B, bs, g)
    tab = table(64, 128).to(DEV)
    q, k, v = (torch.zeros((B, h, 128), dtype=torch.bfloat16, device=DEV) for h in (8, H, H))
    lens, c, t = i32([1] * B), i32(list(range(B + 1))), t.to(torch.int32).to(DEV)
    pool, qo = pools(blocks, H, bs, 128, True), torch.zeros_like(q)
    call = lambda p, o: da.decode_attn_rope_cache_write(q, k, v, tab, c, t, lens, o, *p)  # noqa: E731
    call(pool, qo)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        call(pool, qo)
    for step in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        lens.copy_(torch.randint(1, 65, (B,), generator=g).to(torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, o2 = [x.clone() for x in pool], torch.zeros_like(q)
        call(want, o2)
        torch.cuda.synchronize()
        assert torch.equal(bits(qo), bits(o2)) and all(torch.equal(bits(a), bits(b)) for a, b in zip(pool, want))
        assert (qo != 0).any()
