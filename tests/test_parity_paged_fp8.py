"""decode_attn_only_paged_fp8 / decode_attn_fwd_paged_fp8 (a scale per token and KV head) against the formula in 64
bits, within the bounds of prompt_helpers."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import F64, assert_within, token_ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SCALE = 1 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _library():
    from decode_attention_output_gb300 import build

    build.build()
    da.load()
    torch.cuda.set_device(0)
    yield
    assert da.decode_attn_last_device_error() == 0


def case(B, Hq, Hkv, lens, bs, seed=0, spread=1.0, max_blocks=None, pow2=True):
    """q, pools with unused rows of garbage (NaN codes and scales), table, lens."""
    g = torch.Generator().manual_seed(seed)
    most = max_blocks or max(1, max(-(-n // bs) for n in lens))
    blocks = B * most + 2
    table = torch.randperm(blocks, generator=g)[: B * most].view(B, most)
    k, v = ((torch.randn((blocks, Hkv, bs, 128), generator=g) * 60).to(torch.float8_e4m3fn) for _ in range(2))
    size = torch.randn((blocks, Hkv, 2, bs), generator=g) * spread - 6
    scales = torch.exp2(torch.round(size) if pow2 else size).float()
    used = torch.zeros((blocks, bs), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(min(max(n, 0), most * bs)):
            used[table[b, t // bs], t % bs] = True
    for p in (k, v):
        p.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)
    scales.masked_fill_(~used[:, None, None, :], float("nan"))
    q = torch.randn((B, Hq, 128), generator=g).to(torch.bfloat16)
    return q, k, v, scales, table, list(lens)


def on(x):
    q, k, v, scales, table, lens = x
    return [q.to(DEV), k.to(DEV), v.to(DEV), scales.to(DEV), table.to(torch.int32).to(DEV),
            torch.tensor(lens, dtype=torch.int32, device=DEV)]


def check(x, what, scale=SCALE):
    ref, tol = token_ref(*x, scale)
    out = torch.full(x[0].shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_only_paged_fp8(*on(x), out, scale)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    assert_within(out.cpu(), ref, tol, what)
    return out, tol


CASES = [
    ("one_token", (1, 4, 1, [1], 16)),
    ("g4", (3, 8, 2, [320, 1, 129], 16)),
    ("zero_and_odd", (4, 16, 4, [0, 127, 128, 300], 32)),
    ("g8_bs64", (2, 16, 2, [224, 65], 64)),
    ("g16_bs128", (2, 32, 2, [256, 127], 128)),
    ("g12_bs32", (2, 24, 2, [500, 33], 32)),
    ("g1_bs256", (2, 4, 4, [300, 512], 256)),
    ("bs1024", (2, 4, 2, [1500, 700], 1024)),
    ("many", (40, 8, 1, [(i * 37) % 130 for i in range(40)], 16)),
    ("clusters_equal", (4, 32, 8, [2048] * 4, 64)),
    ("clusters_ragged", (8, 32, 8, [2048, 0, 1, 1500, 64, 2000, 777, 129], 16)),
]


@pytest.mark.parametrize("name,args", CASES, ids=[c[0] for c in CASES])
def test_parity(name, args):
    check(case(*args, seed=1), name)
    check(case(*args, seed=2, pow2=False), name + ", any scales")


@pytest.mark.parametrize("spread", [4.0, 12.0])
def test_scales_of_very_different_size(spread):
    """Values whose size differs by factors of thousands and more from token to token."""
    check(case(3, 16, 2, [700, 64, 3], 16, seed=3, spread=spread), f"spread {spread}")
    x = case(2, 8, 2, [400, 300], 32, seed=4)
    x[3][:, :, 1] *= torch.exp2(torch.linspace(-40, 40, x[3].shape[0]).round())[:, None, None]  # V
    check(x, "values from 2^-46 to 2^34")


def test_negative_scale_zero_scales_and_large_scores():
    x = case(2, 8, 2, [200, 150], 16, seed=5)
    check(x, "negative softmax scale", -0.05)
    check(x, "weights all alike", 0.0)
    check(x, "one weight only", 3.0)
    x[3][::2, :, 1] = 0.0  # every other block's values are zero
    check(x, "zero value scales")
    x[3][::3, :, 0] = 0.0
    check(x, "zero key scales")


@pytest.mark.parametrize("ctas", [1, 5, 300])
def test_split_counts(ctas):
    old = da.decode_attn_get_option("attn_ctas")
    da.decode_attn_set_option("attn_ctas", ctas)
    try:
        check(case(3, 16, 2, [640, 333, 17], 16, seed=6), f"{ctas} CTAs")
    finally:
        da.decode_attn_set_option("attn_ctas", old)


@pytest.mark.parametrize("Hq,Hkv", [(16, 1), (12, 1), (8, 1), (3, 1), (2, 2)])
@pytest.mark.parametrize("ctas", [0, 30, 500])
def test_sequences_in_many_parts(Hq, Hkv, ctas):
    """Ragged lengths on the flat grid: a long sequence's parts meet through L2, up to 70 and 500 of them."""
    old = da.decode_attn_get_option("attn_ctas")
    da.decode_attn_set_option("attn_ctas", ctas)
    try:
        check(case(3, Hq, Hkv, [9000, 5, 1300], 64, seed=14), f"{Hq} heads")
    finally:
        da.decode_attn_set_option("attn_ctas", old)


# (B, Hq, Hkv, length of each, capacity): how many CTAs a sequence gets, and whether its parts meet on chip
# or through L2, follows the common length and the capacity
EQUAL = [
    (1, 4, 1, 9000, 9000), (1, 16, 1, 700, 40000), (1, 2, 1, 2300, 40000), (1, 2, 1, 2305, 40000),  # one long sequence
    (2, 4, 2, 5000, 20000), (2, 4, 2, 129, 20000), (4, 8, 4, 4096, 4096), (6, 8, 2, 3000, 9000),
    (9, 6, 2, 3500, 3500), (25, 8, 2, 513, 513), (25, 2, 2, 1500, 1500),  # 18 and 50 sequences: no divisors of the SMs
    (48, 2, 2, 512, 512), (48, 4, 2, 700, 700), (32, 2, 2, 1, 2048), (5, 8, 8, 256, 256), (100, 2, 2, 200, 200),
    (3, 4, 2, 0, 2048),
]


@pytest.mark.parametrize("B,Hq,Hkv,n,most", EQUAL, ids=[f"{e[0]}x{e[2]}x{e[3]}" for e in EQUAL])
def test_equal_lengths(B, Hq, Hkv, n, most):
    x = case(B, Hq, Hkv, [n] * B, 64, seed=15, max_blocks=-(-most // 64))
    out, _ = check(x, "equal")
    again, _ = check(x, "equal again")
    assert torch.equal(out, again)  # nothing depends on which CTA is last
    one = list(x[5])
    one[-1] = max(0, n - 200)  # ragged now: the tiles split over every CTA
    check((*x[:5], one), "one shorter")


# (B, Hq, Hkv, lengths, capacity): ragged ones whose sequences keep CTAs of their own, and ones too uneven for it
RAGGED = [
    (24, 4, 4, [138 + 6 * b for b in range(24)], 300), (37, 2, 2, [147 + 4 * b for b in range(37)], 300),
    (13, 32, 8, [254 + 20 * b for b in range(13)], 512), (13, 32, 2, [106 + 3 * b for b in range(13)], 142),
    (5, 16, 8, [2900, 3000, 0, 2700, 3100], 3200), (24, 4, 1, [800 + 15 * b for b in range(24)], 1200),
    (24, 4, 1, [1, 0, 5000] * 8, 5000), (3, 16, 1, [9600, 11000, 12000], 12800), (38, 4, 4, [512, 1] * 19, 512),
    (60, 4, 2, [1 + 9 * b for b in range(60)], 600), (7, 8, 2, [0, 0, 700, 0, 0, 900, 0], 1024), (80, 4, 2, [300] * 79 + [7], 512),
]


@pytest.mark.parametrize("B,Hq,Hkv,lens,most", RAGGED, ids=[str(i) for i in range(len(RAGGED))])
def test_ragged_lengths(B, Hq, Hkv, lens, most):
    x = case(B, Hq, Hkv, lens, 32, seed=19, max_blocks=-(-most // 32))
    out, _ = check(x, "ragged")
    again, _ = check(x, "ragged again")
    assert torch.equal(out, again)


def test_captured_call_serves_short_long_equal_and_ragged_lengths():
    B, most = 4, 12000
    x = case(B, 8, 2, [most] * B, 64, seed=16)
    a = on(x)
    out = torch.empty(x[0].shape, dtype=torch.bfloat16, device=DEV)
    da.decode_attn_only_paged_fp8(*a, out, SCALE)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.decode_attn_only_paged_fp8(*a, out, SCALE)
    for n in ([most] * 4, [1] * 4, [2048] * 4, [2304] * 4, [2305] * 4, [6000, 1, 0, 3000], [0] * 4, [most, 1, 1, 1], [512] * 4):
        a[5].copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert da.decode_attn_last_device_error() == 0
        ref, tol = token_ref(*x[:5], n, SCALE)
        assert_within(out.cpu(), ref, tol, f"lengths {n}")


def test_token_major_pool_views_and_padded_table():
    x = case(2, 8, 2, [250, 100], 32, seed=7)
    out, _ = check(x, "plain")
    q, k, v, scales, table, lens = on(x)
    k2, v2 = (p.transpose(1, 2).contiguous().transpose(1, 2) for p in (k, v))
    wide = torch.zeros((*scales.shape[:2], 3, 64), dtype=torch.float32, device=DEV)
    wide[:, :, :2, 16:48] = scales
    big = torch.full((2, 20), 1 << 30, dtype=torch.int32, device=DEV)
    big[:, : table.shape[1]] = table
    out2 = torch.empty_like(out)
    da.decode_attn_only_paged_fp8(q, k2, v2, wide[:, :, :2, 16:48], big[:, : table.shape[1]], lens, out2, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


@pytest.mark.parametrize("bs", [16, 64, 256])
def test_where_the_pools_lie(bs):
    """K before V in memory, V before K, one interleaved allocation, different layouts of the two, one pool as both."""
    x = case(3, 8, 2, [250, 100, 1], bs, seed=13)
    out, _ = check(x, "plain")
    q, k, v, scales, table, lens = on(x)
    n = k.numel()
    both = torch.empty(2 * n, dtype=torch.uint8, device=DEV)
    wide = torch.empty((*k.shape[:2], 2, *k.shape[2:]), dtype=torch.uint8, device=DEV)
    flat = [both[i * n:(i + 1) * n].view(k.shape).view(torch.float8_e4m3fn) for i in range(2)]
    mixed = k.transpose(1, 2).contiguous().transpose(1, 2)
    for k2, v2 in (flat, flat[::-1], [wide[:, :, i].view(torch.float8_e4m3fn) for i in range(2)], (mixed, v)):
        k2.view(torch.uint8).copy_(k.view(torch.uint8))
        v2.view(torch.uint8).copy_(v.view(torch.uint8))
        out2 = torch.empty_like(out)
        da.decode_attn_only_paged_fp8(q, k2, v2, scales, table, lens, out2, SCALE)
        torch.cuda.synchronize()
        assert torch.equal(out, out2)
    check((x[0], x[1], x[1], *x[3:]), "one pool")
    assert da.decode_attn_last_device_error() == 0


def test_block_outside_the_pool_reads_as_zeros():
    x = case(2, 8, 2, [64, 64], 16, seed=8)
    x[4][1, 2] = x[1].shape[0] + 7
    ref, tol = token_ref(*x, SCALE)
    out = torch.empty(x[0].shape, dtype=torch.bfloat16, device=DEV)
    da.decode_attn_only_paged_fp8(*on(x), out, SCALE)
    assert da.decode_attn_last_device_error() == 64
    assert_within(out.cpu(), ref, tol, "zeros")


def test_lengths_past_the_table_are_clamped():
    x = case(2, 8, 2, [96, 96], 32, seed=9)
    out, _ = check(x, "full")
    a = on(x)
    a[5] = torch.tensor([1 << 30, 97], dtype=torch.int32, device=DEV)
    out2 = torch.empty_like(out)
    da.decode_attn_only_paged_fp8(*a, out2, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


@pytest.mark.parametrize("B,N", [(1, 256), (5, 1032), (33, 512)])
def test_whole_step(B, N):
    Hq, Hkv = 16, 4
    x = case(B, Hq, Hkv, [(i * 97) % 400 + 1 for i in range(B)], 16, seed=10)
    ref, tol = token_ref(*x, SCALE)
    g = torch.Generator().manual_seed(11)
    w = (torch.randn((Hq * 128, N), generator=g) / math.sqrt(Hq * 128)).to(torch.bfloat16)
    out = torch.empty((B, N), dtype=torch.bfloat16, device=DEV)
    a = on(x)
    da.decode_attn_fwd_paged_fp8(*a, w.to(DEV), out, SCALE)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    ref, tol, w = ref.reshape(B, -1), tol.reshape(B, -1), w.to(F64)
    want = ref @ w
    # the attention's bound through W, K = 2048 products in fp32 (2^-23 of each partial sum), the output's bf16
    bound = tol @ w.abs() + Hq * 128 * 2.0 ** -23 * (ref.abs() @ w.abs()) + 2.0 ** -8 * want.abs()
    assert_within(out.cpu(), want, bound * 1.01, "step")


@pytest.mark.parametrize("B,n", [(1, 3000), (2, 512), (3, 512), (4, 256), (5, 500), (8, 512), (16, 300), (2, 9000)])
def test_whole_step_equal_lengths(B, n):
    Hq, Hkv, N = 16, 8, 264
    x = case(B, Hq, Hkv, [n] * B, 64, seed=17)
    ref, tol = token_ref(*x, SCALE)
    g = torch.Generator().manual_seed(18)
    w = (torch.randn((Hq * 128, N), generator=g) / math.sqrt(Hq * 128)).to(torch.bfloat16)
    out = torch.empty((B, N), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_fwd_paged_fp8(*on(x), w.to(DEV), out, SCALE)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    ref, tol, w = ref.reshape(B, -1), tol.reshape(B, -1), w.to(F64)
    want = ref @ w  # bounds as above
    bound = tol @ w.abs() + Hq * 128 * 2.0 ** -23 * (ref.abs() @ w.abs()) + 2.0 ** -8 * want.abs()
    assert_within(out.cpu(), want, bound * 1.01, "step")


def test_captured_and_other_stream():
    x = case(3, 32, 8, [900, 5, 400], 64, seed=12, max_blocks=16)
    a = on(x)
    out, tol = check(x, "eager")
    s = torch.cuda.Stream()
    out2 = torch.empty_like(out)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        da.decode_attn_only_paged_fp8(*a, out2, SCALE)
    s.synchronize()
    assert torch.equal(out, out2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.decode_attn_only_paged_fp8(*a, out2, SCALE)
    for n in ([900, 3, 17], [0, 5, 400]):  # shorter lengths: the rows that `case` filled
        a[5].copy_(torch.tensor(n, dtype=torch.int32))
        out2.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = token_ref(*x[:5], n, SCALE)
        assert_within(out2.cpu(), ref, tol, "replayed")


def test_empty_batch():
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16, device=DEV)
    kp = torch.zeros((4, 2, 16, 128), device=DEV).to(torch.float8_e4m3fn)
    sc = torch.ones((4, 2, 2, 16), device=DEV)
    da.decode_attn_only_paged_fp8(q, kp, kp, sc, torch.empty((0, 3), dtype=torch.int32, device=DEV),
                                  torch.empty((0,), dtype=torch.int32, device=DEV), q.clone(), 0.1)
    torch.cuda.synchronize()
