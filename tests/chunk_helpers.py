"""The attention of packed queries in 64 bits, with a window and first tokens that stay visible, with the bound of
prompt_helpers (weights rounded to bf16 before P.V)."""
from __future__ import annotations

import math

import torch

from prompt_helpers import F64, bound, softmax_rows


def visible(lq, lk, window, sinks):
    """[lq, lk]: does the query at position i = r + lk - lq see key j?"""
    i, j = torch.arange(lq)[:, None] + lk - lq, torch.arange(lk)[None]
    ok = j <= i
    return ok & ((j > i - window) | (j < sinks)) if window else ok


def attend_ref(q, keys, values, cu, scale, window=0, sinks=0, rows=None, kv_eps=0.0):
    """(reference, bound, rows of a sequence) for q [Tq, Hq, D]; keys[b] and values[b] [Lk, Hkv, D] (CPU). Keys that no query
    sees may hold anything. `rows`: only these queries of each sequence (a list of indices). `kv_eps`: how far a key's or value's
    elements may be off, relative to them: scores by X kv_eps, numerator and sum by that factor each, values by theirs."""
    Tq, Hq, D = q.shape
    ref, tol = torch.zeros((Tq, Hq, D), dtype=F64), torch.zeros((Tq, Hq, D), dtype=F64)
    have = torch.zeros(Tq, dtype=torch.bool)
    for b in range(len(cu) - 1):
        lq, lk = cu[b + 1] - cu[b], keys[b].shape[0]
        pick = [r for r in (range(lq) if rows is None else rows) if r < lq]
        if not pick:
            continue
        at = cu[b] + torch.tensor(pick)
        have[at] = True
        if lk == 0:
            continue
        ok = visible(lq, lk, window, sinks)[torch.tensor(pick)]
        seen = ok.any(0)
        G = Hq // keys[b].shape[1]
        for j in range(keys[b].shape[1]):
            kd = torch.where(seen[:, None], keys[b][:, j].to(F64), 0.0)
            vd = torch.where(seen[:, None], values[b][:, j].to(F64), 0.0)
            for h in range(j * G, j * G + G):
                qd = q[at, h].to(F64)
                x = (qd @ kd.T * scale).masked_fill(~ok, -math.inf)
                p = softmax_rows(x)
                o = p @ vd
                X = (qd.abs() @ kd.abs().T * abs(scale)).masked_fill(~ok, 0.0).amax(-1, keepdim=True)
                ref[at, h] = o
                tol[at, h] = bound(o, p @ vd.abs(), X, 2.0 ** -8) + (2 * torch.expm1(X * kv_eps) + kv_eps) * (p @ vd.abs()) * 1.01
    return ref, tol, have
