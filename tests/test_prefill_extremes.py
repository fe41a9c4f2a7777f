"""The prompt attention where scores are far larger than any model's: the largest one's V row comes out, and a scale
of 0 gives the mean whatever the products are."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from test_parity_paged_fp8 import DEV, _library  # noqa: F401

pytestmark = pytest.mark.gpu


def run(q, k, v, cu_q, cu_k, scale):
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(cu_q, dtype=torch.int32, device=DEV),
                           torch.tensor(cu_k, dtype=torch.int32, device=DEV), out, scale)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    return out.cpu().float()


@pytest.mark.parametrize("size", [20, 26, 31, 34, 40, 60, 110])
@pytest.mark.parametrize("scale", [1 / math.sqrt(128), -0.3, 1.7])
@pytest.mark.parametrize("lq,lk", [([300, 1], [300, 77]), ([130], [700]), ([3], [4000])], ids=str)
def test_scores_past_24_bits(size, scale, lq, lk):
    """Scores scale * 2^size * c_j, the c_j whole numbers up to 255 that fp32 sums hold exactly: the keys with the
    largest one share the row (smaller ones have 2^-1000 of its weight and less). Weights are bf16, off by 2^-9 of
    themselves against the unrounded sum, and so is the output's rounding."""
    Hq, Hkv = 8, 2
    g = torch.Generator().manual_seed(51)
    cu_q, cu_k = ([0] + torch.tensor(n).cumsum(0).tolist() for n in (lq, lk))
    half = size // 2
    q = torch.full((cu_q[-1], Hq, 128), 2.0 ** half)
    sign = torch.where(torch.rand((cu_q[-1], Hq, 1), generator=g) < 0.5, -1.0, 1.0)  # some rows: all scores below 0
    c = torch.randint(1, 256, (cu_k[-1], Hkv, 1), generator=g).float()
    k = (c * 2.0 ** (size - half - 7)).expand(-1, -1, 128)
    v = torch.randn((cu_k[-1], Hkv, 128), generator=g).to(torch.bfloat16)
    out = run((q * sign).to(torch.bfloat16), k.to(torch.bfloat16), v, cu_q, cu_k, scale)
    for b in range(len(lq)):
        for i in range(cu_q[b], cu_q[b + 1]):
            n = i - cu_q[b] + lk[b] - lq[b] + 1  # its keys
            for h in range(Hq):
                cs = c[cu_k[b]:cu_k[b] + n, h // 4, 0]
                top = cs.max() if sign[i, h, 0] * scale > 0 else cs.min()
                rows = v[cu_k[b]:cu_k[b] + n, h // 4].double()[cs == top]
                ref, size_of = rows.mean(0), rows.abs().mean(0)
                d = (out[i, h].double() - ref).abs()
                assert bool((d <= 2.0 ** -8 * size_of + 2.0 ** -8 * ref.abs()).all()), (b, i, h, d.max())


@pytest.mark.parametrize("power", [0, 10, 59])
def test_scale_of_zero_and_large_products(power):
    """Products up to 2^(2 * power + 7), times a scale of 0: the mean of the keys' V rows. (Weights 1 are exact in bf16;
    the sum of up to 300 of them and their V rows is fp32.)"""
    g = torch.Generator().manual_seed(52)
    q, k = (torch.randn((300, 2, 128), generator=g).sign() * 2.0 ** power * torch.randint(1, 3, (300, 2, 1), generator=g) for _ in range(2))
    v = torch.randn((300, 2, 128), generator=g).to(torch.bfloat16)
    out = run(q.to(torch.bfloat16), k.to(torch.bfloat16), v, [0, 300], [0, 300], 0.0)
    n = torch.arange(1, 301).double()[:, None, None]
    ref = v.double().cumsum(0) / n
    size = v.double().abs().cumsum(0) / n
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * size).all())
