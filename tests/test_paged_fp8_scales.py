"""The paged e4m3 attention where the scales of V lie far apart: a token's share in the softmax's sum does not
depend on its V, whatever exponents stand beside it in the sequence (the writer's reach from -124 to 120)."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from test_parity_paged_fp8 import DEV, _library, case, check  # noqa: F401

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
