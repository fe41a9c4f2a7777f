"""decode_attn_chunk over an e4m3 cache whose V scales lie as far apart as the entry point allows (2^-100 and up): where the
largest belongs to a key that some queries of a row group do not see, and where a weight above 1 (the softmax's maximum lags)
meets a scale near fp32's end."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from chunk_helpers import attend_ref, visible
from prompt_helpers import F64
from test_cache import DEV, _library, i32  # noqa: F401
from test_chunk import SCALE, canvas, check

pytestmark = pytest.mark.gpu


def far_case(kind, B, lk, Hkv, g):
    """Codes [2][B, Hkv, lk, 128] and scales [B, Hkv, 2, lk]; no value is past 2^124."""
    codes = torch.randint(0, 0x58, (2, B, Hkv, lk, 128), generator=g, dtype=torch.uint8)  # up to 15
    codes |= torch.randint(0, 2, codes.shape, generator=g, dtype=torch.uint8) << 7
    scales = torch.exp2(torch.randint(-9, -5, (B, Hkv, 2, lk), generator=g).float())
    if kind == "last":  # the last key's is 2^130 times the others'
        scales[:, :, 1] = 2.0 ** -60
        scales[:, :, 1, -1] = 2.0 ** 70
    elif kind == "ends":  # the least and the largest that decode_attn_cache_write's rule and the header meet
        scales[:, :, 1] = 2.0 ** -100
        scales[:, :, 1, -1] = -(2.0 ** 120)
    elif kind == "growing":  # each key's larger than the one before
        scales[:, :, 1] = torch.exp2(torch.linspace(-100, 120, lk).floor())
    elif kind == "lag":  # late keys with weights of 2^7.5 against the maximum so far, the last one's codes at e4m3's lower end
        codes[0] = 0x38  # 1
        scales[:, :, 0] = 0.5
        scales[:, :, 0, -(lk // 9):] = 123 / 128
        scales[:, :, 1] = 1.0
        scales[:, :, 1, -1] = 1.75 * 2.0 ** 126
        codes[1, :, :, -1] &= 0x83  # subnormal: up to 3 * 2^-9; 2^7.5 times its value is 2^127
    return codes, scales


@pytest.mark.parametrize("kind", ["last", "ends", "growing", "lag"])
@pytest.mark.parametrize("B,lk,Hkv,lq", [(1, 700, 2, 2), (1, 9000, 2, 4), (260, 100, 2, 3), (1, 700, 2, 90)], ids=str)
def test_v_scales_far_apart(kind, B, lk, Hkv, lq):
    """Bounds as for any cache; f16 weights are off by 2^-25 of the row's largest product of weight and scale."""
    g = torch.Generator().manual_seed(606)
    G, bs = 4, 16
    codes, scales = far_case(kind, B, lk, Hkv, g)
    most = -(-lk // bs)
    pools = torch.zeros((2, B * most, Hkv, bs, 128), dtype=torch.uint8)
    sc = torch.ones((B * most, Hkv, 2, bs))
    at = torch.arange(lk)
    for b in range(B):
        blk, row = b * most + at // bs, at % bs
        for i in range(2):
            pools[i][blk, :, row] = codes[i, b].transpose(0, 1)
        sc[blk, :, :, row] = scales[b].permute(2, 0, 1)
    q = torch.ones((B * lq, Hkv * G, 128)) if kind == "lag" else torch.randn((B * lq, Hkv * G, 128), generator=g)
    q = q.to(torch.bfloat16)
    table = torch.arange(B * most, dtype=torch.int32).view(B, most)
    cu = [b * lq for b in range(B + 1)]
    out = canvas(q)
    da.decode_attn_chunk(q.to(DEV), *(p.to(DEV).view(torch.float8_e4m3fn) for p in pools), sc.to(DEV), table.to(DEV), i32(cu), i32([lk] * B),
                         out, SCALE)
    code = [x.view(torch.float8_e4m3fn).float().to(F64) for x in codes]
    few = range(0, B, 37)  # sequences that are looked at
    for b in few:
        rows = slice(b * lq, b * lq + lq)
        k, v = (code[i][b] * scales[b, :, i].to(F64)[..., None] for i in range(2))
        ref, tol, _ = attend_ref(q[rows], [k.transpose(0, 1)], [v.transpose(0, 1)], [0, lq], SCALE)
        for h in range(Hkv * G):
            j = h // G
            x = (q[rows, h].to(F64) @ k[j].T * SCALE).masked_fill(~visible(lq, lk, 0, 0), -math.inf)
            some = (code[1][b, j] != 0).any(-1)
            r = (torch.softmax(x, -1) * torch.where(some, scales[b, j, 1].abs().to(F64), 0.0)).amax(-1, keepdim=True)
            tol[:, h] += 2.0 ** -25 * r * code[1][b, j].abs().sum(0)[None]
        check(out[rows], ref, tol, torch.ones(lq, dtype=torch.bool), f"{kind}, sequence {b}")
