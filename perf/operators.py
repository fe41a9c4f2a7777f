"""What a server does around one decode step, as measurable cases: the attention of whole prompts, the writing of their keys
and values into a paged cache with 8-bit codes, reading cached tokens back, and one new token's attention over that cache.

Each case's `op` names the operator; `run` computes it in elementary torch operations, or (with `own`) through
decode_attention_output_gb300. Layouts:

  q [Tq, Hq, 128], k / v [Tk, Hkv, 128] bf16: packed tokens; sequence b is rows cu[b] .. cu[b + 1]
  pages [num_blocks, Hkv, block_size, 128] e4m3; scales [num_blocks, Hkv, 2, block_size] fp32 (K's, then V's)
  table [B, max_blocks] int32: the blocks of each sequence in token order; lens [B] int32: its tokens
"""
import math

import torch

own = False

D = 128


# ---------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a chat turn's short prompt, alone: latency
        dict(name="prompt_77", op="prefill", Hq=32, Hkv=8, B=1, lo=77, hi=77, prefix=0, seed=1),
        # a batch of prompts of very different lengths, packed (a length of 1 among them)
        dict(name="prompts_ragged", op="prefill", Hq=32, Hkv=8, B=16, lo=1, hi=2048, prefix=0, seed=2),
        # chunks of 512 tokens of prompts whose first 7.5k tokens are cached
        dict(name="prompt_chunks", op="prefill", Hq=32, Hkv=8, B=4, lo=509, hi=512, prefix=7680, seed=3),
        # one long prompt of a model with 64 query heads
        dict(name="prompt_8k", op="prefill", Hq=64, Hkv=8, B=1, lo=8192, hi=8192, prefix=0, seed=4),
        # one decode step's new token of each of 64 sequences
        dict(name="write_step", op="write", Hkv=8, B=64, lo=1, hi=1, prefix=1000, bs=64, seed=5),
        # prompts written after their attention
        dict(name="write_prompts", op="write", Hkv=8, B=16, lo=1500, hi=4099, prefix=3, bs=16, seed=6),
        # the cached beginnings of four prompts, for the attention of their next chunk
        dict(name="read_prefixes", op="read", Hkv=8, B=4, lo=1, hi=2100, bs=16, seed=7),
        # a batch of long prefixes shared with earlier requests
        dict(name="read_long", op="read", Hkv=8, B=32, lo=4000, hi=8192, bs=64, seed=8),
        # one sequence of 2k tokens: latency
        dict(name="token_b1_2k", op="token", Hq=32, Hkv=8, B=1, lo=2048, hi=2048, bs=64, N=0, seed=9),
        # a small serving batch with its output projection
        dict(name="step_b8_8k", op="token", Hq=32, Hkv=8, B=8, lo=8192, hi=8192, bs=64, N=4096, seed=10),
        # ragged lengths, small blocks
        dict(name="token_b32_ragged", op="token", Hq=32, Hkv=8, B=32, lo=512, hi=32768, bs=16, N=0, seed=11),
        # a large serving batch of a model with 64 query heads
        dict(name="token_b64_16k", op="token", Hq=64, Hkv=8, B=64, lo=16384, hi=16384, bs=128, N=0, seed=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    c = dict(op=rng.choice(["prefill", "prefill", "write", "read", "token", "token"]), seed=rng.randrange(1 << 20))
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    c["B"] = log_int(1, 64)
    if c["op"] == "prefill":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
        c["B"] = log_int(1, 24)
        c["prefix"] = rng.choice([0, 0, log_int(1, 6000)])
        most = 1 << 32  # scores of the padded batch: at most those of prompt_8k
        c["hi"] = log_int(1, 4096)
        while c["B"] * c["Hq"] * c["hi"] * (c["hi"] + c["prefix"]) > most:
            c["hi"] = c["hi"] // 2
    elif c["op"] == "token":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
        c["bs"] = rng.choice([16, 32, 64, 128, 256])
        c["N"] = rng.choice([0, 0, 8 * log_int(8, 512)])
        c["hi"] = log_int(1, (1 << 20) // (c["B"] * (c["Hq"] // c["Hkv"])))
    else:
        c["bs"] = rng.choice([16, 32, 64, 128])
        c["hi"] = log_int(1, (1 << 18) // c["B"])
        if c["op"] == "write":
            c["hi"] = min(c["hi"], 4099)
            c["prefix"] = log_int(1, 2000)
    c["lo"] = rng.choice([1, c["hi"], max(1, c["hi"] // 2)])
    return c


def _lengths(c):
    """The sequences' lengths (new tokens for prefill and write), the longest and the shortest asked for among them."""
    g = torch.Generator().manual_seed(c["seed"])
    n = torch.randint(c["lo"], c["hi"] + 1, (c["B"],), generator=g).tolist()
    n[0] = c["hi"]
    n[-1] = c["lo"] if c["B"] > 1 else c["hi"]
    return n


def _kv_lengths(c):
    """Tokens of each sequence in all: the new ones behind `prefix` earlier ones (a few more or less by sequence)."""
    p = c.get("prefix", 0)
    return [n + (p + (i * 37) % 91 if p else 0) for i, n in enumerate(_lengths(c))]


# ------------------------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape, mult=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(mult).to(torch.bfloat16)


def _cu(n):
    return torch.tensor([0] + list(torch.tensor(n, dtype=torch.int64).cumsum(0)), dtype=torch.int32, device="cuda")


def _pool(c, lens, g, fill):
    """A pool of shuffled blocks (a few spare), its table and, with `fill`, codes and scales of cached tokens."""
    bs, most = c["bs"], max(-(-n // c["bs"]) for n in lens)
    blocks = len(lens) * most + 5
    table = torch.randperm(blocks, generator=g, device="cuda")[: len(lens) * most].view(len(lens), most).to(torch.int32)
    shape = (blocks, c["Hkv"], bs, D)
    k, v = (torch.zeros(shape, device="cuda", dtype=torch.float8_e4m3fn) for _ in range(2))
    scales = torch.ones((blocks, c["Hkv"], 2, bs), device="cuda", dtype=torch.float32)
    if fill:
        # rows of a cache: codes whose largest fills the range, a power-of-two scale for each that varies from token to token
        for pages, at, mult in ((k, 0, 1.0), (v, 1, 1.0)):
            step = max(1, (1 << 27) // (c["Hkv"] * bs * D))
            for i in range(0, blocks, step):
                j = min(blocks, i + step)
                x = torch.randn((j - i, *shape[1:]), generator=g, device="cuda", dtype=torch.float32).mul_(mult)
                x.mul_(torch.exp2(torch.randint(-2, 2, x.shape[:3], generator=g, device="cuda").float())[..., None])
                codes, s = _quantised(x)
                pages[i:j] = codes
                scales[i:j, :, at] = s
    return k, v, scales, table


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + c["seed"])
    s = dict(op=c["op"], scale=1.0 / math.sqrt(D))
    n, lens = _lengths(c), _kv_lengths(c)
    if c["op"] == "prefill":
        s.update(cu_q=_cu(n), cu_k=_cu(lens), most_q=max(n), most_k=max(lens))
        s["q"] = _randn(g, sum(n), c["Hq"], D)
        s["k"], s["v"] = _randn(g, sum(lens), c["Hkv"], D), _randn(g, sum(lens), c["Hkv"], D)
        s["out"] = torch.zeros_like(s["q"])
    elif c["op"] == "write":
        s.update(cu=_cu(n), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        # keys and values whose size differs from token to token and from head to head
        size = torch.exp(torch.randn((sum(n), c["Hkv"], 1), generator=g, device="cuda"))
        s["k"], s["v"] = ((_randn(g, sum(n), c["Hkv"], D).float() * size).to(torch.bfloat16) for _ in range(2))
        s["k_pages"], s["v_pages"], s["scales"], s["table"] = _pool(c, lens, g, False)
    elif c["op"] == "read":
        s.update(cu=_cu(n))
        s["k_pages"], s["v_pages"], s["scales"], s["table"] = _pool(c, n, g, True)
        s["k"], s["v"] = (torch.zeros((sum(n), c["Hkv"], D), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    else:
        s.update(lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        s["k_pages"], s["v_pages"], s["scales"], s["table"] = _pool(c, lens, g, True)
        s["q"] = _randn(g, c["B"], c["Hq"], D)
        s["w"] = _randn(g, c["Hq"] * D, c["N"], mult=1.0 / math.sqrt(c["Hq"] * D)) if c["N"] else None
        s["out"] = torch.zeros((c["B"], c["N"]) if c["N"] else (c["B"], c["Hq"], D), device="cuda", dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------------------------------------------ the operators
def run(state):
    s = state
    if own:
        return _own(s)
    return {"prefill": _prefill, "write": _write, "read": _read, "token": _token}[s["op"]](s)


def _own(s):
    import decode_attention_output_gb300 as da

    if s["op"] == "prefill":
        return da.decode_attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["scale"])
    if s["op"] == "write":
        da.decode_attn_cache_write(s["k"], s["v"], s["cu"], s["table"], s["lens"], s["k_pages"], s["v_pages"], s["scales"])
        return s["k_pages"], s["v_pages"], s["scales"]
    if s["op"] == "read":
        da.decode_attn_cache_read(s["k_pages"], s["v_pages"], s["scales"], s["table"], s["cu"], s["k"], s["v"])
        return s["k"], s["v"]
    args = s["q"], s["k_pages"], s["v_pages"], s["scales"], s["table"], s["lens"]
    if s["w"] is not None:
        return da.decode_attn_fwd_paged_fp8(*args, s["w"], s["out"], s["scale"])
    return da.decode_attn_only_paged_fp8(*args, s["out"], s["scale"])


def _rows(cu, most):
    """Rows of each sequence in the packed order, padded to [B, most], and which of them it has."""
    i = torch.arange(most, device=cu.device)
    have = i < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + i).long(), have


def _weights(x, mask):
    """Softmax over the last dimension of what the mask leaves; zeros where it leaves nothing."""
    x = x.masked_fill(~mask, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _prefill(s):
    rq, hq = _rows(s["cu_q"], s["most_q"])
    rk, hk = _rows(s["cu_k"], s["most_k"])
    Hq, Hkv = s["q"].shape[1], s["k"].shape[1]
    G, B = Hq // Hkv, len(rq)
    q = s["q"][rq.clamp_max(len(s["q"]) - 1)].float().view(B, -1, Hkv, G, D).permute(0, 2, 3, 1, 4)
    k, v = (s[n][rk.clamp_max(len(s["k"]) - 1)].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))
    more = (s["cu_k"].diff() - s["cu_q"].diff())[:, None, None]
    ok = torch.arange(s["most_k"], device=q.device) <= torch.arange(s["most_q"], device=q.device)[:, None] + more
    ok = (ok & hk[:, None])[:, None, None]
    o = _weights((q * s["scale"]) @ k.transpose(-1, -2), ok) @ v.masked_fill(~hk[:, None, None, :, None], 0.0)
    s["out"][rq[hq]] = o.permute(0, 3, 1, 2, 4).reshape(B, -1, Hq, D)[hq].to(torch.bfloat16)
    return s["out"]


def _quantised(x):
    """(e4m3 codes, power-of-two scale) of the rows of x: the least scale under which the row's largest value fits."""
    x = x.float()
    part, e = torch.frexp(x.abs().amax(-1))
    e = (e - 8 - (part <= 0.875).int()).clamp(-124, 120).int()
    scale = torch.where(part == 0, 1.0, ((e + 127) << 23).view(torch.float32))  # 2^e, exactly
    top = torch.where(e == 120, 240.0, 448.0)[..., None]  # larger codes times 2^120 are no bf16 values
    return (x / scale[..., None]).clamp(-top, top).to(torch.float8_e4m3fn), scale


def _places(s, rows, have, first, bs):
    """(block, row in the block) of the tokens first[b], first[b] + 1, ... that each sequence has."""
    pos = first[:, None] + torch.arange(rows.shape[1], device=rows.device)
    b, i = torch.nonzero(have, as_tuple=True)
    pos = pos[b, i].long()
    return s["table"][b, pos // bs].long(), pos % bs


def _write(s):
    bs = s["k_pages"].shape[2]
    n = s["cu"].diff()
    rows, have = _rows(s["cu"], s["table"].shape[1] * bs)
    block, row = _places(s, rows, have, s["lens"] - n, bs)
    for at, (x, pages) in enumerate(((s["k"], s["k_pages"]), (s["v"], s["v_pages"]))):
        codes, scale = _quantised(x[: len(block)])
        pages.view(torch.uint8)[block, :, row] = codes.view(torch.uint8)
        s["scales"][block, :, at, row] = scale
    return s["k_pages"], s["v_pages"], s["scales"]


def _read(s):
    bs = s["k_pages"].shape[2]
    rows, have = _rows(s["cu"], s["table"].shape[1] * bs)
    block, row = _places(s, rows, have, torch.zeros_like(s["cu"][1:]), bs)
    for at, (out, pages) in enumerate(((s["k"], s["k_pages"]), (s["v"], s["v_pages"]))):
        codes = pages.view(torch.uint8)[block, :, row].view(torch.float8_e4m3fn).float()
        out[: len(block)] = (codes * s["scales"][block, :, at, row][..., None]).to(torch.bfloat16)
    return s["k"], s["v"]


def _token(s):
    B, Hq, _ = s["q"].shape
    Hkv, bs = s["k_pages"].shape[1:3]
    most = s["table"].shape[1] * bs
    at = s["table"].long()
    # [B, Hkv, tokens, D]: codes times their scales
    k, v = ((pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["scales"][at, :, i][..., None]).transpose(1, 2)
            .reshape(B, Hkv, most, D) for i, pages in ((0, s["k_pages"]), (1, s["v_pages"])))
    have = torch.arange(most, device=at.device) < s["lens"][:, None]
    x = (s["q"].float() * s["scale"]).view(B, Hkv, Hq // Hkv, D) @ k.transpose(-1, -2)
    o = _weights(x, have[:, None, None]) @ v.masked_fill(~have[:, None, :, None], 0.0)
    o = o.reshape(B, Hq, D).to(torch.bfloat16)  # the step's own intermediate type
    s["out"].copy_(o if s["w"] is None else o.view(B, -1).float() @ s["w"].float())
    return s["out"]


def work(case):
    c = case
    n, lens = _lengths(c), _kv_lengths(c)
    if c["op"] == "prefill":
        pairs = sum(m * (L - m) + m * (m + 1) // 2 for m, L in zip(n, lens))
        return {"bytes": 4 * D * (sum(n) * c["Hq"] + sum(lens) * c["Hkv"]), "flops": 4 * D * c["Hq"] * pairs}
    if c["op"] == "token":
        return {"bytes": sum(lens) * c["Hkv"] * 2 * (D + 4) + 2 * c["B"] * c["Hq"] * D + 2 * c["Hq"] * D * c["N"]
                + 2 * c["B"] * (c["N"] or c["Hq"] * D),
                "flops": 4 * D * c["Hq"] * sum(lens) + 2 * c["B"] * c["Hq"] * D * c["N"]}
    rows = 2 * sum(n) * c["Hkv"]  # of K and of V: bf16 on one side, codes and a scale on the other
    return {"bytes": rows * (3 * D + 4), "flops": rows * 2 * D}


# --------------------------------------------------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    return {"prefill": _exact_prefill, "write": _exact_write, "read": _exact_read, "token": _exact_token}[s["op"]](s)


def _exact_prefill(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cq, ck, G = s["cu_q"].tolist(), s["cu_k"].tolist(), s["q"].shape[1] // s["k"].shape[1]
    for b in range(len(cq) - 1):
        m, L = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for h in range(s["q"].shape[1]):
            k, v = (s[x][ck[b]:ck[b + 1], h // G].double() for x in ("k", "v"))
            x = s["q"][cq[b]:cq[b + 1], h].double() @ k.T * s["scale"]
            x = x + torch.full((m, L), -math.inf, dtype=torch.float64, device="cuda").triu_(L - m + 1)
            out[cq[b]:cq[b + 1], h] = torch.softmax(x, -1) @ v
    return out


def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x in 64 bits rounded to the nearest e4m3 value, ties to the even one (all are below 448 here)."""
    unit = _power(torch.frexp(x.abs().clamp_min(2.0 ** -6))[1] - 4)
    return torch.round(x / unit) * unit


def _exact_write(s):
    k, v, scales = (s[x].double() if x == "scales" else s[x].float().double() for x in ("k_pages", "v_pages", "scales"))
    bs, cu, lens, table = s["k_pages"].shape[2], s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    block, row = [], []
    for b in range(len(lens)):
        for pos in range(lens[b] - (cu[b + 1] - cu[b]), lens[b]):
            block.append(table[b][pos // bs])
            row.append(pos % bs)
    block, row = torch.tensor(block, device="cuda"), torch.tensor(row, device="cuda")
    for at, (x, pages) in enumerate(((s["k"].double(), k), (s["v"].double(), v))):
        size = x.abs().amax(-1)
        part, e = torch.frexp(size / 448.0)
        scale = torch.where(size == 0, 1.0, _power((e - (part == 0.5).int()).clamp(-124, 120)))
        pages[block, :, row] = _e4m3(x / scale[..., None])
        scales[block, :, at, row] = scale
    return k, v, scales


def _exact_read(s):
    got = []
    bs, cu, table = s["k_pages"].shape[2], s["cu"].tolist(), s["table"].long()
    for at, pages in enumerate((s["k_pages"], s["v_pages"])):
        rows = []
        for b in range(len(cu) - 1):
            L = cu[b + 1] - cu[b]
            own_blocks = table[b, : -(-L // bs)]
            x = torch.stack([pages[i] for i in own_blocks.tolist()])
            x = x.float().double() * s["scales"][own_blocks, :, at].double()[..., None]
            rows.append(x.transpose(1, 2).reshape(-1, *x.shape[1:2], D)[:L])
        got.append(torch.cat(rows))
    return got[0], got[1]


def _exact_token(s):
    B, Hq, _ = s["q"].shape
    Hkv, bs = s["k_pages"].shape[1:3]
    o = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        blocks = s["table"][b, : -(-L // bs)].tolist()
        k, v = (torch.stack([pages[i].float().double() * s["scales"][i, :, at].double()[..., None] for i in blocks], 1)
                .reshape(Hkv, -1, D)[:, :L] for at, pages in ((0, s["k_pages"]), (1, s["v_pages"])))
        x = torch.einsum("hgd,htd->hgt", s["q"][b].double().view(Hkv, -1, D), k) * s["scale"]
        o[b] = torch.einsum("hgt,htd->hgd", torch.softmax(x, -1), v).reshape(Hq, D)
    # the attention's result is bf16 in the operator's definition before the projection takes it
    return o if s["w"] is None else o.to(torch.bfloat16).double().view(B, -1) @ s["w"].double()
