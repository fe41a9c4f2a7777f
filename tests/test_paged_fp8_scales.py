"""The paged e4m3 attention where the scales of V lie far apart: a token's share in the softmax's sum does not
depend on its V, whatever exponents stand beside it in the sequence (the writer's reach from -124 to 120)."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import F64, assert_within, bound, gather, softmax_rows, token_ref
from test_parity_paged_fp8 import DEV, SCALE, _library, case, check, on  # noqa: F401

pytestmark = pytest.mark.gpu


def two_tokens(a, at=1, n=2):
    """Tokens 0 and `at` of n with the same keys, so the same score, and V scales 2^a and 2^-a; the others' scores
    are far below and their V in between."""
    x = case(1, 8, 2, [n], 16, seed=21)
    q, k, v, scales, table, lens = x
    q[:] = q.abs()
    blocks = table[0, torch.arange(n) // 16]
    rows = torch.arange(n) % 16
    k[blocks, :, rows] = torch.full((n, 2, 128), -16.0).to(k.dtype)  # scores of -15 and less
    scales[blocks, :, 0, rows] = 2.0 ** -4
    scales[blocks, :, 1, rows] = 1.0
    v[blocks, :, rows] = torch.full((n, 2, 128), 3.0).to(v.dtype)
    for t, e in ((0, a), (at, -a)):
        k[blocks[t], :, rows[t]] = torch.full((2, 128), 1.0).to(k.dtype)
        v[blocks[t], :, rows[t]] = torch.full((2, 128), 448.0).to(v.dtype)
        scales[blocks[t], :, 1, rows[t]] = 2.0 ** e
    return x


@pytest.mark.parametrize("a", [30, 62, 64, 70, 100, 117, -64, -100, -117])
def test_two_tokens_of_equal_score(a):
    out, _ = check(two_tokens(a), f"2^{a} and 2^{-a}")
    want = 224.0 * 2.0 ** abs(a)  # half of the larger
    assert abs(out[0, 0, 0].item() / want - 1) <= 2.0 ** -7


@pytest.mark.parametrize("a", [64, -100])
@pytest.mark.parametrize("at,n", [(5, 6), (40, 41), (127, 128), (130, 400), (300, 400), (1990, 2000)],
                         ids=["one warp", "two warps", "one tile", "two tiles", "three tiles", "two CTAs"])
def test_tokens_that_meet_in_a_merge(a, at, n):
    check(two_tokens(a, at, n), f"token {at} of {n}")


@pytest.mark.parametrize("ctas", [0, 1, 7])
@pytest.mark.parametrize("lens", [[300, 1, 40], [1500] * 3, [4000, 129, 33], [4096] * 2], ids=str)
@pytest.mark.parametrize("most", [60, 119])
def test_random_exponents(lens, ctas, most):
    """V's exponents anywhere between -most and most, on one CTA, on few and in clusters."""
    old = da.decode_attn_get_option("attn_ctas")
    da.decode_attn_set_option("attn_ctas", ctas)
    try:
        for Hq in (4, 24):
            x = case(len(lens), Hq, 2, lens, 16, seed=22)
            g = torch.Generator().manual_seed(23)
            e = torch.randint(-most, most + 1, x[3][:, :, 1].shape, generator=g)
            x[3][:, :, 1] = torch.where(x[3][:, :, 1].isnan(), math.nan, torch.exp2(e.float()))
            check(x, f"exponents to {most}, {Hq} heads")
    finally:
        da.decode_attn_set_option("attn_ctas", old)


@pytest.mark.parametrize("e", [-126, -101, 101, 121, 126, 127])
@pytest.mark.parametrize("n", [1, 3, 700])
def test_all_scales_at_an_end_of_the_range(e, n):
    """Values up to 1.75 * 2^127 (no sum of them overflows on the way) and down to fp32's smallest normal scale."""
    x = case(2, 8, 2, [n, 1], 16, seed=24)
    x[2].copy_((x[2].float().nan_to_num(0).clamp(-1.75, 1.75) if e > 100 else x[2].float().nan_to_num(0)).to(x[2].dtype))
    x[3][:, :, 1] = torch.where(x[3][:, :, 1].isnan(), math.nan, 2.0 ** e)
    check(x, f"2^{e}")


def strict(x, scale=SCALE):
    """(reference, bound) as prompt_helpers.token_ref's, but what f16 weights lose at the small end is taken against the
    largest weight of a row of V that has a code other than 0. With y = log2 (weight) + floor(log2 V's scale), f16 weights
    are off by 2^-25 of their unit at most, and the unit lies 4 or more below the largest y (or 119 below the largest
    score, where that is more)."""
    q, k, v, scales, table, lens = x
    ref, tol = token_ref(*x, scale)
    B, Hq, _ = q.shape
    for b in range(B):
        L = lens[b]
        if L == 0:
            continue
        sc = gather(scales.transpose(2, 3).contiguous(), table, b, L).to(F64)
        code = gather(v.float(), table, b, L).to(F64)
        key, val = gather(k.float(), table, b, L).to(F64) * sc[..., :1], code * sc[..., 1:]
        for h in range(Hq):
            j = h // (Hq // k.shape[1])
            s = key[j] @ q[b, h].to(F64) * scale
            p = softmax_rows(s[None])[0]
            X = float((key[j].abs() @ q[b, h].to(F64).abs()).max()) * abs(scale)
            x2 = s / math.log(2)
            e = torch.frexp(sc[j, :, 1].abs())[1].to(F64) - 1
            some = (code[j].abs().sum(-1) > 0) & (sc[j, :, 1] != 0)
            top = (x2 + e)[some].max() if some.any() else torch.tensor(-math.inf, dtype=F64)
            unit = torch.maximum(top - 4, x2.max() - 119) - torch.logsumexp(s, 0) / math.log(2)
            tol[b, h] = bound(ref[b, h], p @ val[j].abs(), X, 2.0 ** -11, 2.0 ** -25 * code[j].abs().sum(0) * 2.0 ** unit)
    return ref, tol


def check_strict(x, what):
    ref, tol = strict(x)
    out = torch.full(x[0].shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_only_paged_fp8(*on(x), out, SCALE)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    assert_within(out.cpu(), ref, tol, what)


def zero_rows(x, b, tokens, up, code=0.0, scale=1.0):
    """Rows of V that hold zeros, with V's scale 1 (as the writer leaves them) and scores about `up` powers of two above
    the others'."""
    q, k, v, scales, table, lens = x
    bs = k.shape[2]
    for t in tokens:
        i, r = table[b, t // bs], t % bs
        size = q.float().abs().sum(-1).mean() * SCALE
        k[i, :, r] = torch.full((k.shape[1], 128), 16.0).to(k.dtype)
        scales[i, :, 0, r] = float(up * math.log(2) / size / 16)
        v.view(torch.uint8)[i, :, r] = 0
        if code:
            v[i, :, r] = torch.full((k.shape[1], 128), code).to(v.dtype)
        scales[i, :, 1, r] = scale


def small_values(B, Hq, lens, e, seed=25):
    x = case(B, Hq, 2, lens, 16, seed=seed)
    x[0].abs_()
    x[3][:, :, 1] = torch.where(x[3][:, :, 1].isnan(), math.nan, 2.0 ** e)
    return x


@pytest.mark.parametrize("e", [-7, -13, -20, -60])
@pytest.mark.parametrize("up", [10, 20, 40])
@pytest.mark.parametrize("Hq", [8, 32])
def test_zero_rows_do_not_set_the_reference(e, up, Hq):
    """A row of zeros with scale 1 and a score far above the others', beside ordinary rows of small scales: first, in the
    middle of a warp's tokens, alone in its warp, last, several, in every tile."""
    n = 1024
    for tokens in ([0], [13], [500], [n - 1], [3, 4, 40, 700], list(range(5, n, 50))):
        x = small_values(1, Hq, [n], e)
        zero_rows(x, 0, tokens, up)
        check_strict(x, f"{len(tokens)} from {tokens[0]}")
    x = small_values(2, Hq, [32, 2], e)
    zero_rows(x, 0, [0], up)
    zero_rows(x, 1, [1], up)
    check_strict(x, "short")


def test_zero_scales_minus_zeros_and_rows_of_nothing_else():
    x = small_values(3, 8, [700, 129, 20], -13)
    zero_rows(x, 0, [2, 300], 20, scale=0.0)  # a scale of 0 in place of codes of 0
    zero_rows(x, 1, list(range(129)), 3)  # no other rows at all: zeros
    check_strict(x, "zeros")
    x[2].view(torch.uint8)[x[2].view(torch.uint8) == 0] = 0x80  # -0
    check_strict(x, "minus zeros")


@pytest.mark.parametrize("code", [2.0 ** -9, 0.5, 448.0])
def test_rows_of_small_codes(code):
    """Rows whose codes are far below what their scale allows, with a dominating score."""
    x = small_values(2, 16, [600, 40], -10)
    zero_rows(x, 0, [1, 77, 411], 12, code=code)
    zero_rows(x, 1, [39], 12, code=code)
    check_strict(x, f"codes of {code}")


@pytest.mark.parametrize("small", [-10, -17, -21])
def test_small_queries_with_large_key_scales(small):
    """q enters the product as f16: exact from 2^-17 on, below it within 2^-25 of each element, so a score within
    2^-25 * scale * sum |k|, its weight by as large a factor, and the output by twice that of its mean magnitude."""
    x = case(2, 8, 2, [300, 77], 16, seed=26)
    q, k, v, scales, table, lens = x
    g = torch.Generator().manual_seed(27)
    size = 2.0 ** small * (1 + torch.rand(q.shape, generator=g))
    q.copy_((size * torch.sign(torch.randn(q.shape, generator=g))).to(torch.bfloat16))
    scales[:, :, 0] *= 2.0 ** -small
    ref, tol = token_ref(*x, SCALE)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    da.decode_attn_only_paged_fp8(*on(x), out, SCALE)
    torch.cuda.synchronize()
    for b, L in enumerate(lens):
        sc = gather(scales.transpose(2, 3).contiguous(), table, b, L).to(F64)
        key, val = gather(k.float(), table, b, L).to(F64) * sc[..., :1], gather(v.float(), table, b, L).to(F64) * sc[..., 1:]
        for h in range(8):
            off = 0.0 if small >= -17 else 2.0 ** -25 * SCALE * key[h // 4].abs().sum(-1).max().item()
            p = softmax_rows((key[h // 4] @ q[b, h].to(F64) * SCALE)[None])[0]
            tol[b, h] += 2 * math.expm1(off) * (p @ val[h // 4].abs())
    assert_within(out.cpu(), ref, tol, f"q of 2^{small}")


@pytest.mark.parametrize("size", [10, 20, 26, 29, 31, 40, 60, 110])
@pytest.mark.parametrize("e", [-60, -13, 0, 40, 100])
def test_scores_past_24_bits(size, e):
    """Scores scale * 2^size * c_j, the c_j whole numbers up to 255, so the keys with the largest one share the row: their
    V rows' mean, in warps, tiles and CTAs of their own. Their weights are powers of two; the sums are fp32."""
    for lens, Hq, ctas in (([300, 1, 40], 8, 0), ([4000, 129], 24, 0), ([2000] * 2, 8, 7)):
        x = case(len(lens), Hq, 2, lens, 16, seed=28)
        q, k, v, scales, table, _ = x
        g = torch.Generator().manual_seed(29)
        sign = torch.where(torch.rand((len(lens), Hq, 1), generator=g) < 0.5, -1.0, 1.0)
        q.copy_(sign.expand(-1, -1, 128))
        k.copy_(torch.ones(k.shape).to(k.dtype))
        c = torch.randint(1, 256, scales[:, :, 0].shape, generator=g).float()
        scales[:, :, 0] = c * 2.0 ** (size - 7)
        scales[:, :, 1] = 2.0 ** e
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        old = da.decode_attn_get_option("attn_ctas")
        da.decode_attn_set_option("attn_ctas", ctas)
        try:
            da.decode_attn_only_paged_fp8(*on(x), out, SCALE)
        finally:
            da.decode_attn_set_option("attn_ctas", old)
        torch.cuda.synchronize()
        got = out.cpu().to(F64)
        for b, L in enumerate(lens):
            cs, code = gather(c[..., None], table, b, L)[..., 0], gather(v.float(), table, b, L).to(F64)
            for h in range(Hq):
                j = h // (Hq // 2)
                top = cs[j].max() if sign[b, h, 0] > 0 else cs[j].min()
                rows = code[j][cs[j] == top] * 2.0 ** e
                ref, size_of = rows.mean(0), rows.abs().mean(0)
                # (at size 10 the next whole number has 2^-130 of the weight)
                assert bool(((got[b, h] - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size_of).all()), (lens, b, h)
