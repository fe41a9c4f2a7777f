"""What happens to a step's new tokens between their projection and their attention's result, as measurable cases: the norms
and the position rotation of their queries and keys, the same on the way into a paged cache, their attention over that cache
(one token or many), and prompts whose attention is limited to a window and a few first tokens.

Each case's `op` names the operator; `run` computes it in elementary torch operations, or (with `own`) through
decode_attention_output_gb300. Layouts:

  q [T, Hq, D], k / v [T, Hkv, D] bf16: packed tokens; sequence b is rows cu[b] .. cu[b + 1], the last of its lens[b] tokens
  table [rows, R] fp32: cos, then sin, of the R / 2 pairs' angles at each position; axes [R / 2] int32: a pair's position axis
  pages [num_blocks, Hkv, block_size, D] bf16, or e4m3 with scales [num_blocks, Hkv, 2, block_size] fp32 (K's, then V's)
  blocks [B, max_blocks] int32: the blocks of each sequence in token order; lens [B] int32: its tokens

A query at position p sees keys p - window + 1 .. p and the first `sinks` ones (window 0: keys 0 .. p).
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's queries and keys, one per sequence of a batch: latency
        dict(name="rope_step", op="rope", Hq=32, Hkv=8, D=128, T=64, R=128, axes=1, norm=True, pairs="halves", seed=1),
        # prompts with images: positions of three axes (time, height, width)
        dict(name="rope_images", op="rope", Hq=32, Hkv=8, D=128, T=8191, R=128, axes=3, norm=True, pairs="halves", seed=2),
        # a decode step's new tokens into the e4m3 cache that its attention reads
        dict(name="append_step", op="append", Hq=32, Hkv=8, D=128, B=64, lo=1, hi=1, prefix=1000, bs=64, kv="e4m3", R=128,
             axes=1, norm=False, pairs="halves", seed=3),
        # chunks of four prompts, half of a head's dims rotated, neighbouring dims paired
        dict(name="append_chunks", op="append", Hq=32, Hkv=8, D=128, B=4, lo=509, hi=512, prefix=7680, bs=16, kv="e4m3", R=64,
             axes=1, norm=False, pairs="neighbours", seed=4),
        # whole prompts of very different lengths, normed, into a bf16 cache
        dict(name="append_prompts", op="append", Hq=32, Hkv=8, D=128, B=16, lo=1500, hi=4099, prefix=3, bs=16, kv="bf16",
             R=128, axes=1, norm=True, pairs="halves", seed=5),
        # one sequence's next token: latency
        dict(name="chunk_b1_2k", op="chunk", Hq=32, Hkv=8, B=1, lo=1, hi=1, prefix=2048, bs=64, kv="bf16", window=0, sinks=0, seed=6),
        # four drafted tokens of each of 32 sequences, checked in one pass
        dict(name="chunk_drafts", op="chunk", Hq=32, Hkv=8, B=32, lo=4, hi=4, prefix=8192, bs=64, kv="bf16", window=0, sinks=0, seed=7),
        # the next 512 tokens of four prompts whose first 7.5k are cached, in 8-bit codes
        dict(name="chunk_prompts", op="chunk", Hq=32, Hkv=8, B=4, lo=509, hi=512, prefix=7680, bs=64, kv="e4m3", window=0,
             sinks=0, seed=8),
        # a long document's next 2k tokens, model with 64 query heads
        dict(name="chunk_long", op="chunk", Hq=64, Hkv=8, B=1, lo=2048, hi=2048, prefix=14336, bs=16, kv="bf16", window=0, sinks=0, seed=9),
        # a serving batch's next tokens over long caches, of which each sees the last 4096 and the first 4
        dict(name="window_step", op="chunk", Hq=32, Hkv=8, B=32, lo=1, hi=1, prefix=32000, bs=64, kv="e4m3", window=4096, sinks=4, seed=10),
        # packed prompts of very different lengths, a window of odd size
        dict(name="window_ragged", op="window", Hq=32, Hkv=8, B=16, lo=1, hi=2048, prefix=0, window=777, sinks=1, seed=11),
        # one long prompt, a window of 1024 and four first tokens
        dict(name="window_16k", op="window", Hq=64, Hkv=8, B=1, lo=16384, hi=16384, prefix=0, window=1024, sinks=4, seed=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    c = dict(op=rng.choice(["rope", "append", "append", "chunk", "chunk", "window"]), seed=rng.randrange(1 << 20))
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    if c["op"] in ("rope", "append"):
        c["D"] = rng.choice([128, 128, 256])
        c["R"] = c["D"] // rng.choice([1, 1, 2, 4])
        c["axes"] = rng.choice([1, 1, 2, 3])
        c["norm"] = rng.choice([True, False])
        c["pairs"] = rng.choice(["halves", "halves", "neighbours"])
    if c["op"] == "rope":
        c["T"] = log_int(1, 300000 // c["Hq"])
        return c
    c["B"] = log_int(1, 64)
    most = {"append": 1 << 20, "chunk": 1 << 33, "window": 1 << 33}[c["op"]]
    if c["op"] == "append":
        c["hi"] = log_int(1, max(1, min(4099, most // (c["B"] * c["Hq"]))))
        c["prefix"] = log_int(1, 2000)
        # a row's scale is the power of two above its largest value: sums of a norm in another order could move it across
        # one, so normed keys go to bf16 pools here
        c["kv"] = "bf16" if c["norm"] or c["D"] == 256 else "e4m3"
    else:
        c["hi"] = rng.choice([1, 1, log_int(1, 8), log_int(1, 2048), log_int(1, 2048)])
        if c["op"] == "window":
            c["hi"] = log_int(1, 4096)
        c["prefix"] = rng.choice([0, log_int(1, 16000), log_int(1, 16000)])
        c["window"] = log_int(1, 8192) if c["op"] == "window" else rng.choice([0, 0, log_int(1, 8192)])
        c["sinks"] = rng.choice([0, 1, 4, log_int(1, 300)]) if c["window"] else 0
        c["kv"] = rng.choice(["bf16", "e4m3"])
        # scores of the padded batch, tokens of the cache and products: at most those of the largest listed cases
        while (c["B"] * c["Hq"] * c["hi"] * (c["hi"] + c["prefix"]) > most // 4 or c["B"] * c["Hkv"] * (c["hi"] + c["prefix"]) > 1 << 21
               or c["B"] * c["Hq"] * c["hi"] * min(c["window"] + c["sinks"] if c["window"] else 1 << 30, c["hi"] + c["prefix"]) > 1 << 30):
            if c["B"] > 1:
                c["B"] //= 2
            else:
                c["hi"] = max(1, c["hi"] // 2)
    c["lo"] = rng.choice([1, c["hi"], max(1, c["hi"] // 2)])
    if c["op"] != "window":
        c["bs"] = rng.choice([16, 32, 64, 128, 256])
    return c


def _lengths(c):
    """The sequences' new tokens, the longest and the shortest asked for among them."""
    g = torch.Generator().manual_seed(c["seed"])
    n = torch.randint(c["lo"], c["hi"] + 1, (c["B"],), generator=g).tolist()
    n[0] = c["hi"]
    n[-1] = c["lo"] if c["B"] > 1 else c["hi"]
    return n


def _totals(c):
    """Tokens of each sequence in all: the new ones behind `prefix` earlier ones (a few more or less by sequence)."""
    return [n + (c["prefix"] + (i * 37) % 91 if c["prefix"] else 0) for i, n in enumerate(_lengths(c))]


# ------------------------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(n):
    return _i32([0] + list(torch.tensor(n, dtype=torch.int64).cumsum(0)))


def _blocks(c, totals, g):
    """(the sequences' blocks, shuffled over the pool; blocks of the pool: a few spare)"""
    most = max(-(-n // c["bs"]) for n in totals)
    blocks = len(totals) * most + 5
    return torch.randperm(blocks, generator=g, device="cuda")[: len(totals) * most].view(len(totals), most).to(torch.int32), blocks


def _filled(c, blocks, g):
    """Pools of cached tokens. e4m3: codes whose largest fills the range, a power-of-two scale that varies from row to row."""
    shape = (blocks, c["Hkv"], c["bs"], 128)
    if c["kv"] == "bf16":
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16), torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16), None
    pools, scales = [], torch.ones((blocks, c["Hkv"], 2, c["bs"]), device="cuda", dtype=torch.float32)
    for at in range(2):
        pages = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
        step = max(1, (1 << 27) // (c["Hkv"] * c["bs"] * 128))
        for i in range(0, blocks, step):
            j = min(blocks, i + step)
            x = torch.randn((j - i, *shape[1:]), generator=g, device="cuda", dtype=torch.float32)
            x.mul_(torch.exp2(torch.randint(-2, 2, x.shape[:3], generator=g, device="cuda").float())[..., None])
            pages[i:j], scales[i:j, :, at] = _quantised(x)
        pools.append(pages)
    return pools[0], pools[1], scales


def _rotation(c, T, rows, pos, g):
    """The table (its angles in 64 bits), the axis of each pair and each token's positions, as far as a program needs them."""
    half = c["R"] // 2
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * 500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    s = dict(table=torch.cat([angle.cos(), angle.sin()], 1).float(), axes=None, pos=pos)
    if c["axes"] > 1:
        # a token's place in time, and where it lies in a picture
        s["axes"] = (torch.arange(half, device="cuda") * c["axes"] // half).to(torch.int32)
        s["pos"] = torch.stack([pos] + [torch.randint(0, min(rows, 200), (T,), generator=g, device="cuda").to(torch.int32) for _ in range(c["axes"] - 1)])
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + c["seed"])
    s = dict(op=c["op"], Hq=c["Hq"], Hkv=c["Hkv"], scale=1.0 / math.sqrt(128), window=c.get("window", 0), sinks=c.get("sinks", 0))
    if c["op"] == "rope":
        T, D = c["T"], c["D"]
        pos = torch.randint(0, 32768, (T,), generator=g, device="cuda").to(torch.int32)
        s.update(_rotation(c, T, 32768, pos, g))
        s.update(q=_randn(g, T, c["Hq"], D), k=_randn(g, T, c["Hkv"], D))
        s.update(q_out=torch.zeros_like(s["q"]), k_out=torch.zeros_like(s["k"]))
    else:
        n, totals = _lengths(c), _totals(c)
        T = sum(n)
        s.update(cu=_cu(n), lens=_i32(totals), most=max(n), most_k=max(totals), q=_randn(g, T, c["Hq"], c.get("D", 128)))
    if c["op"] == "append":
        D = c["D"]
        # the tokens' places in their sequences: what the call takes for their positions where it gets none
        place = torch.cat([torch.arange(L - m, L) for m, L in zip(n, totals)]).to(torch.int32).cuda()
        s.update(_rotation(c, T, max(totals) + 100, place, g), place=place)
        size = torch.exp(torch.randn((T, c["Hkv"], 1), generator=g, device="cuda"))
        s["k"], s["v"] = ((_randn(g, T, c["Hkv"], D).float() * size).to(torch.bfloat16) for _ in range(2))
        s["q_out"] = torch.zeros_like(s["q"])
        s["blocks"], blocks = _blocks(c, totals, g)
        kind = torch.bfloat16 if c["kv"] == "bf16" else torch.float8_e4m3fn
        s["k_pages"], s["v_pages"] = (torch.zeros((blocks, c["Hkv"], c["bs"], D), device="cuda", dtype=kind) for _ in range(2))
        s["scales"] = torch.ones((blocks, c["Hkv"], 2, c["bs"]), device="cuda") if c["kv"] == "e4m3" else None
    if c["op"] in ("rope", "append"):
        s.update(pairs=c["pairs"], q_weight=None, k_weight=None)
        if c["norm"]:
            s["q_weight"], s["k_weight"] = (torch.exp(0.3 * torch.randn(c["D"], generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    elif c["op"] == "chunk":
        s["blocks"], blocks = _blocks(c, totals, g)
        s["k_pages"], s["v_pages"], s["scales"] = _filled(c, blocks, g)
        s["out"] = torch.zeros_like(s["q"])
    elif c["op"] == "window":
        s["cu_k"] = _cu(totals)
        s.update(k=_randn(g, sum(totals), c["Hkv"], 128), v=_randn(g, sum(totals), c["Hkv"], 128), out=torch.zeros_like(s["q"]))
    return s


# ------------------------------------------------------------------------------------------------------ the operators
def run(state):
    s = state
    if own:
        return _own(s)
    return {"rope": _rope, "append": _append, "chunk": _chunk, "window": _window}[s["op"]](s)


def _own(s):
    import decode_attention_output_gb300 as da

    if s["op"] == "chunk":
        return da.decode_attn_chunk(s["q"], s["k_pages"], s["v_pages"], s["scales"], s["blocks"], s["cu"], s["lens"], s["out"], s["scale"],
                                    window=s["window"], sinks=s["sinks"])
    if s["op"] == "window":
        return da.decode_attn_prefill_window(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], s["out"], s["scale"], s["window"], s["sinks"])
    more = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], axes=s["axes"], eps=EPS, interleaved=s["pairs"] == "neighbours")
    if s["op"] == "rope":
        return da.decode_attn_rope(s["q"], s["k"], s["table"], s["pos"], s["q_out"], s["k_out"], **more)
    da.decode_attn_rope_cache_write(s["q"], s["k"], s["v"], s["table"], s["cu"], s["blocks"], s["lens"], s["q_out"], s["k_pages"], s["v_pages"],
                                    s["scales"], positions=None if s["axes"] is None else s["pos"], **more)
    return s["q_out"], s["k_pages"], s["v_pages"], s["scales"]


def _turned(s, x, weight):
    """x [T, H, D], normed (with `weight`) and rotated, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    R = s["table"].shape[1]
    pair = torch.arange(R // 2, device=x.device)
    at = s["pos"].long()[:, None] if s["axes"] is None else s["pos"].long().T[:, s["axes"].long()]
    cos, sin = s["table"][at, pair][:, None], s["table"][at, R // 2 + pair][:, None]
    if s["pairs"] == "halves":
        a, b = x[..., : R // 2], x[..., R // 2: R]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., R:]], -1)


def _rope(s):
    s["q_out"].copy_(_turned(s, s["q"], s["q_weight"]))
    s["k_out"].copy_(_turned(s, s["k"], s["k_weight"]))
    return s["q_out"], s["k_out"]


def _quantised(x):
    """(e4m3 codes, power-of-two scale) of the rows of x: the least scale under which the row's largest value fits."""
    x = x.float()
    part, e = torch.frexp(x.abs().amax(-1))
    e = (e - 8 - (part <= 0.875).int()).clamp(-124, 120).int()
    scale = torch.where(part == 0, 1.0, ((e + 127) << 23).view(torch.float32))  # 2^e, exactly
    top = torch.where(e == 120, 240.0, 448.0)[..., None]  # larger codes times 2^120 are no bf16 values
    return (x / scale[..., None]).clamp(-top, top).to(torch.float8_e4m3fn), scale


def _rows(cu, most):
    """Rows of each sequence in the packed order, padded to [B, most], and which of them it has."""
    i = torch.arange(most, device=cu.device)
    have = i < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + i).long(), have


def _append(s):
    s["q_out"].copy_(_turned(s, s["q"], s["q_weight"]))
    bs = s["k_pages"].shape[2]
    b = _rows(s["cu"], s["most"])[1].nonzero()[:, 0]  # the sequence of each token
    place = s["place"].long()
    block, row = s["blocks"][b, place // bs].long(), place % bs
    k = _turned(s, s["k"], s["k_weight"])
    if s["scales"] is None:
        s["k_pages"][block, :, row] = k.to(torch.bfloat16)
        s["v_pages"][block, :, row] = s["v"]
        return s["q_out"], s["k_pages"], s["v_pages"], None
    (kc, ks), (vc, vs) = _quantised(k), _quantised(s["v"])
    s["k_pages"].view(torch.uint8)[block, :, row] = kc.view(torch.uint8)
    s["v_pages"].view(torch.uint8)[block, :, row] = vc.view(torch.uint8)
    s["scales"][block, :, :, row] = torch.stack([ks, vs], -1)
    return s["q_out"], s["k_pages"], s["v_pages"], s["scales"]


def _attend(s, k, v, lens, most_k):
    """Attention of the packed queries over k and v [B, Hkv, most_k, 128] fp32."""
    rows, have = _rows(s["cu"], s["most"])
    B, G = len(rows), s["Hq"] // s["Hkv"]
    q = s["q"][rows.clamp_max(len(s["q"]) - 1)].float().view(B, -1, s["Hkv"], G, 128).permute(0, 2, 3, 1, 4).reshape(B, s["Hkv"], -1, 128)
    key = torch.arange(most_k, device=q.device)
    p = ((lens - s["cu"].diff())[:, None] + torch.arange(s["most"], device=q.device))[..., None]  # the queries' positions
    ok = (key <= p) & (key < lens[:, None, None])
    if s["window"]:
        ok &= (key > p - s["window"]) | (key < s["sinks"])
    x = ((q * s["scale"]) @ k.transpose(-1, -2)).view(B, s["Hkv"], G, -1, most_k)
    x = x.masked_fill_(~ok[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    x = x.div_(x.sum(-1, keepdim=True).clamp_min_(1e-30))
    o = x.view(B, s["Hkv"], -1, most_k) @ v.masked_fill((key >= lens[:, None])[:, None, :, None], 0.0)
    o = o.view(B, s["Hkv"], G, -1, 128).permute(0, 3, 1, 2, 4).reshape(B, -1, s["Hq"], 128)
    s["out"][rows[have]] = o[have].to(torch.bfloat16)
    return s["out"]


def _chunk(s):
    blocks, (B, most) = s["blocks"].long(), s["blocks"].shape
    most *= s["k_pages"].shape[2]

    def cached(pages, at):
        x = pages[blocks] if s["scales"] is None else pages.view(torch.uint8)[blocks].view(torch.float8_e4m3fn)
        x = x.float()
        if s["scales"] is not None:
            x = x.mul_(s["scales"][blocks, :, at][..., None])
        return x.transpose(1, 2).reshape(B, s["Hkv"], most, 128)

    return _attend(s, cached(s["k_pages"], 0), cached(s["v_pages"], 1), s["lens"], most)


def _window(s):
    rows, _ = _rows(s["cu_k"], s["most_k"])
    k, v = (s[n][rows.clamp_max(len(s[n]) - 1)].float().transpose(1, 2) for n in ("k", "v"))
    return _attend(s, k, v, s["lens"], s["most_k"])


def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["T"] * (c["Hq"] + c["Hkv"])
        return {"bytes": rows * c["D"] * 4 + c["T"] * (4 * c["R"] + 4 * c["axes"]), "flops": rows * (3 * c["R"] + 4 * c["D"] * c["norm"])}
    n, totals = _lengths(c), _totals(c)
    if c["op"] == "append":
        rows = sum(n) * c["Hkv"]
        kv = 2 * rows * (2 * c["D"] + (2 * c["D"] if c["kv"] == "bf16" else c["D"] + 4))
        return {"bytes": sum(n) * c["Hq"] * c["D"] * 4 + kv + sum(n) * 4 * c["R"], "flops": (rows + sum(n) * c["Hq"]) * (3 * c["R"] + 4 * c["D"] * c["norm"])}
    pairs = seen = 0
    W = c["window"] or 1 << 40
    for m, L in zip(n, totals):
        p = torch.arange(L - m, L)  # the queries' positions
        pairs += int((p + 1).clamp_max(W).sum() + (p + 1 - W).clamp(0, c["sinks"]).sum())
        first = max(0, L - m - W + 1)  # of the window of the chunk's first query
        seen += L - first + min(first, c["sinks"])
    return {"bytes": 4 * 128 * sum(n) * c["Hq"] + seen * c["Hkv"] * 2 * (256 if c["op"] == "window" or c["kv"] == "bf16" else 132),
            "flops": 4 * 128 * c["Hq"] * pairs}


# --------------------------------------------------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    w = work(case)
    if w["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _exact_turned(s, s["q"], s["q_weight"]), _exact_turned(s, s["k"], s["k_weight"])
    return _exact_append(s) if s["op"] == "append" else _exact_attend(s)


def _exact_turned(s, x, weight):
    """Each pair of dims as a complex number, times its angle's."""
    T, H, D = x.shape
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * weight.double()
    half = s["table"].shape[1] // 2
    turn = torch.empty((T, half), dtype=torch.complex128, device="cuda")
    for i in range(half):
        row = (s["pos"] if s["axes"] is None else s["pos"][int(s["axes"][i])]).long()
        turn[:, i] = torch.complex(s["table"][row, i].double(), s["table"][row, half + i].double())
    first, second = (slice(0, half), slice(half, 2 * half)) if s["pairs"] == "halves" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_append(s):
    k, v = _exact_turned(s, s["k"], s["k_weight"]), s["v"].double()
    bs, cu = s["k_pages"].shape[2], s["cu"].tolist()
    out = [torch.zeros(s["k_pages"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    scales = None if s["scales"] is None else torch.ones(s["scales"].shape, dtype=torch.float64, device="cuda")
    table = s["blocks"].long()
    for b, L in enumerate(s["lens"].tolist()):
        at = torch.arange(L - (cu[b + 1] - cu[b]), L, device="cuda")
        block, row = table[b][at // bs], at % bs
        for i, x in enumerate((k, v)):
            x = x[cu[b]:cu[b + 1]]
            if scales is not None:
                size = x.abs().amax(-1)
                e = torch.ceil(torch.log2(size / 448)).clamp(-124, 120)
                e = e + (size > 448 * torch.exp2(e)).double() - (size <= 448 * torch.exp2(e - 1)).double()
                scale = torch.where(size > 0, torch.exp2(e), 1.0)
                scales[block, :, i, row] = scale
                x = x / scale[..., None]  # codes before their rounding
            out[i][block, :, row] = x
    return _exact_turned(s, s["q"], s["q_weight"]), out[0], out[1], scales


def _exact_attend(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, G = s["cu"].tolist(), s["Hq"] // s["Hkv"]
    first = s["cu_k"].tolist() if s["op"] == "window" else None
    for b, L in enumerate(s["lens"].tolist()):
        m = cu[b + 1] - cu[b]
        i, j = torch.arange(L - m, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
        hidden = j > i
        if s["window"]:
            hidden = hidden | ((i - j >= s["window"]) & (j >= s["sinks"]))
        for h in range(s["Hkv"]):
            if first is None:
                bs = s["k_pages"].shape[2]
                own_blocks = s["blocks"][b, : -(-L // bs)].long()
                k, v = (torch.cat([(p[n, h].double() * (1.0 if s["scales"] is None else s["scales"][n, h, at].double()[:, None]))
                                   for n in own_blocks.tolist()])[:L] for at, p in enumerate((s["k_pages"], s["v_pages"])))
            else:
                k, v = (s[x][first[b]:first[b + 1], h].double() for x in ("k", "v"))
            for g in range(h * G, h * G + G):
                x = (s["q"][cu[b]:cu[b + 1], g].double() @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
                out[cu[b]:cu[b + 1], g] = torch.softmax(x, -1) @ v
    return out
