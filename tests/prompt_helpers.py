"""64-bit references of the prompt attention, the paged cache's writing and reading, and the attention over a
paged e4m3 cache, from their definitions, with the bounds that the kernels' roundings give.

Bounds, per output element, with p the exact weights, A = sum_j p_j |v_j| and X = max_j of scale * sum_d |q_d k_jd|
(both computed here in 64 bits):
  * the output's rounding to bf16: 2^-8 |ref|
  * a weight's rounding before P.V: bf16 2^-8 of it (prompt attention), f16 2^-11 (e4m3 caches), so that much of A;
    f16 weights below 2^-14 of the reference are off by at most 2^-25 of it instead (`floor` below)
  * a score: 128 products summed in fp32 (each partial sum off by 2^-23 of it at most, truncation included) and
    scaled twice, so its weight by a factor within 128 * 2^-23 * X + 2^-20 (the exponential's own error is 2^-22);
    numerator and sum take it both: twice that of A
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
LN2 = math.log(2.0)


def bound(ref, A, X, weight_eps, floor=0.0):
    return 2.0 ** -8 * ref.abs() + (weight_eps + 2 * (X * 2.0 ** -16 + 2.0 ** -20)) * A * 1.01 + floor + 1e-30


def softmax_rows(x):
    """Softmax of the rows of x; zeros where every entry is -inf."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isneginf(top), torch.zeros_like(top), top))
    s = p.sum(-1, keepdim=True)
    return torch.where(s > 0, p / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(p))


def prefill_ref(q, k, v, cu_q, cu_k, scale):
    """(reference, bound, rows of a sequence) for CPU tensors q [Tq, Hq, D], k and v [Tk, Hkv, D]."""
    Tq, Hq, D = q.shape
    G = Hq // k.shape[1]
    ref, tol = torch.zeros((Tq, Hq, D), dtype=F64), torch.zeros((Tq, Hq, D), dtype=F64)
    have = torch.zeros(Tq, dtype=torch.bool)
    for b in range(len(cu_q) - 1):
        Lq, Lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        rows = slice(cu_q[b], cu_q[b + 1])
        have[rows] = True
        if Lq == 0 or Lk == 0:
            continue
        ok = torch.arange(Lk)[None, :] <= torch.arange(Lq)[:, None] + Lk - Lq
        for h in range(Hq):
            qd, kd = q[rows, h].to(F64), k[cu_k[b]:cu_k[b + 1], h // G].to(F64)
            vd = v[cu_k[b]:cu_k[b + 1], h // G].to(F64)
            x = (qd @ kd.T * scale).masked_fill(~ok, -math.inf)
            p = softmax_rows(x)
            ref[rows, h] = p @ vd
            X = (qd.abs() @ kd.abs().T * abs(scale)).masked_fill(~ok, 0.0).amax(-1, keepdim=True)
            tol[rows, h] = bound(ref[rows, h], p @ vd.abs(), X, 2.0 ** -8)
    return ref, tol, have


def quantise_ref(x):
    """(codes as uint8, scales fp32) of the rows of a bf16 tensor, from the definition in 64 bits."""
    d = x.to(F64)
    size = torch.where(torch.isfinite(d), d.abs(), torch.zeros_like(d)).amax(-1)
    e = torch.full(size.shape, -124.0, dtype=F64)
    for cand in range(120, -125, -1):  # the least e whose range holds the row
        e = torch.where(size <= 448.0 * 2.0 ** cand, torch.full_like(e, float(cand)), e)
    e = torch.where(size == 0, torch.zeros_like(e), e)
    scale = torch.tensor([2.0 ** i for i in range(-124, 121)], dtype=F64)[(e + 124).long()]
    top = torch.where(e == 120, 240.0, 448.0).to(F64)[..., None]  # 256 * 2^120 would be no bf16 value
    y = torch.minimum(torch.maximum(d / scale[..., None], -top), top)  # NaN stays NaN
    return y.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8), scale.to(torch.float32)


def places(table, cu, seq_lens, bs):
    """[(packed row, block, row in the block)] of the new tokens (seq_lens None: the first tokens)."""
    got = []
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            pos = i + (0 if seq_lens is None else seq_lens[b] - n)
            if 0 <= pos < table.shape[1] * bs:
                got.append((cu[b] + i, int(table[b, pos // bs]), pos % bs))
    return got


def gather(pages, table, b, L):
    """The first L tokens of sequence b, [Hkv, L, D], out of a CPU pool [num_blocks, Hkv, bs, D]; a block outside
    the pool is zeros."""
    bs = pages.shape[2]
    if L == 0:
        return pages[0][:, :0]
    blocks = [pages[i] if 0 <= i < pages.shape[0] else torch.zeros_like(pages[0])
              for i in table[b, : -(-L // bs)].tolist()]
    return torch.cat(blocks, 1)[:, :L]


def token_ref(q, k_pages, v_pages, scales, table, lens, scale):
    """(reference, bound) of the attention of one token per sequence over a paged e4m3 cache (CPU tensors)."""
    B, Hq, D = q.shape
    Hkv = k_pages.shape[1]
    ref, tol = torch.zeros((B, Hq, D), dtype=F64), torch.zeros((B, Hq, D), dtype=F64)
    kf, vf = k_pages.to(torch.float32), v_pages.to(torch.float32)
    cap = table.shape[1] * k_pages.shape[2]
    for b in range(B):
        L = min(max(int(lens[b]), 0), cap)
        if L == 0:
            continue
        sc = gather(scales.transpose(2, 3).contiguous(), table, b, L).to(F64)  # [Hkv, L, 2]
        code = gather(vf, table, b, L).to(F64)
        k, v = gather(kf, table, b, L).to(F64) * sc[..., :1], code * sc[..., 1:]
        for h in range(Hq):
            j = h // (Hq // Hkv)
            x = k[j] @ q[b, h].to(F64) * scale
            p = softmax_rows(x[None])[0]
            ref[b, h] = p @ v[j]
            X = float((k[j].abs() @ q[b, h].to(F64).abs()).max()) * abs(scale)
            # f16 weights are taken against the largest 2^(x + e) of the row, V's scale being 2^e times 1 to 2
            e = torch.where(sc[j, :, 1] > 0, torch.frexp(sc[j, :, 1])[1].to(F64) - 1, torch.zeros_like(x))
            r = (x / LN2 + e).max()
            floor = 2.0 ** -25 * code[j].abs().sum(0) * torch.exp(r * LN2 - torch.logsumexp(x, 0))
            tol[b, h] = bound(ref[b, h], p @ v[j].abs(), X, 2.0 ** -11, floor)
    return ref, tol


def assert_within(got, ref, tol, what):
    d = (got.to(F64) - ref).abs()
    assert torch.isfinite(got.to(F64)).all(), f"{what}: non-finite values"
    if d.numel() == 0:
        return 0.0
    r = torch.where(d > 0, d / tol, torch.zeros_like(d))  # rows without a token: exactly 0
    worst = r.max().item()
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound at {divmod(int(r.argmax()), d.shape[-1])}"
    return worst
