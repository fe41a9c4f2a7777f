"""decode_attn_prefill against the formula in 64 bits, at the lengths, groups, strides and masks where it can go
wrong, within the bounds of prompt_helpers."""
import math

import pytest
import torch

import decode_attention_output_gb300 as da
from prompt_helpers import assert_within, prefill_ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CANARY = 0x7FA5  # a bf16 NaN the kernels never write


@pytest.fixture(scope="module", autouse=True)
def _library():
    from decode_attention_output_gb300 import build

    build.build()
    da.load()
    torch.cuda.set_device(0)
    yield
    assert da.decode_attn_last_device_error() == 0


def cu(lengths, first=0):
    c = [first]
    for n in lengths:
        c.append(c[-1] + n)
    return c


def inputs(lq, lk, Hq, Hkv, seed=0, first=0, spare=0, k_mult=1.0):
    g = torch.Generator().manual_seed(seed)
    cq, ck = cu(lq, first), cu(lk, first)
    Tq, Tk = cq[-1] + spare, ck[-1] + spare
    q = torch.randn((Tq, Hq, 128), generator=g).to(torch.bfloat16)
    k = (torch.randn((Tk, Hkv, 128), generator=g) * k_mult).to(torch.bfloat16)
    v = torch.randn((Tk, Hkv, 128), generator=g).to(torch.bfloat16)
    return q, k, v, cq, ck


def offsets(c):
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def canaries(shape):
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    t.view(torch.int16).fill_(CANARY)
    return t


def check(q, k, v, cq, ck, scale, what, out=None, **kw):
    out = canaries(q.shape) if out is None else out
    da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck), out, scale, **kw)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    ref, tol, have = prefill_ref(q, k, v, cq, ck, scale)
    got = out.cpu()
    assert_within(got[have], ref[have], tol[have], what)
    assert (got[~have].contiguous().view(torch.int16) == CANARY).all(), f"{what}: rows of no sequence were written"
    return got


SCALE = 1 / math.sqrt(128)

LENGTHS = [  # (queries, tokens) of each sequence
    ([1], [1]),
    ([2], [2]),
    ([127], [127]),
    ([128], [128]),
    ([129], [129]),
    ([255, 1, 256, 257], [255, 1, 256, 257]),
    ([300, 0, 5, 64], [300, 0, 5, 64]),      # an empty sequence
    ([1, 7, 200], [500, 129, 777]),           # the last tokens of longer sequences
    ([9, 130, 70], [4, 0, 69]),               # fewer keys than queries, none at all
    ([0, 0], [3, 0]),
    ([640], [1300]),
    (list(range(40)), list(range(40))),       # more than 32 sequences
]


@pytest.mark.parametrize("lq,lk", LENGTHS, ids=[str(i) for i in range(len(LENGTHS))])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (8, 2), (2, 2)])
def test_lengths(lq, lk, Hq, Hkv):
    check(*inputs(lq, lk, Hq, Hkv, seed=1, first=3, spare=5), SCALE, f"{lq} {lk}")


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 12, 15, 16])
def test_groups(G):
    check(*inputs([150, 33, 1], [150, 170, 9], G, 1, seed=G), SCALE, f"group {G}")
    check(*inputs([65], [300], 3 * G, 3, seed=G), SCALE, f"group {G}, three KV heads")


def test_many_items():
    """More work items than SMs, so that a CTA takes several (and more than 64 sequences)."""
    g = torch.Generator().manual_seed(3)
    lq = torch.randint(0, 70, (90,), generator=g).tolist()
    lk = [n + int(torch.randint(0, 200, (1,), generator=g)) for n in lq]
    check(*inputs(lq, lk, 8, 4, seed=4), SCALE, "90 sequences")
    check(*inputs([1500, 700], [1500, 900], 16, 8, seed=5), SCALE, "two long ones")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 3.0])
def test_scales(scale):
    check(*inputs([140, 20], [140, 150], 8, 2, seed=6), scale, f"scale {scale}")


def test_growing_scores():
    """Keys that grow along the sequence move the running maximum in every tile, by a lot in some rows only."""
    q, k, v, cq, ck = inputs([700], [700], 4, 1, seed=7)
    k = (k.float() * torch.linspace(0, 8, 700)[:, None, None]).to(torch.bfloat16)
    check(q, k, v, cq, ck, SCALE, "growing keys")
    check(q, k.flip(0), v, cq, ck, SCALE, "shrinking keys")


def test_constant_values_come_back():
    """The weights of every row sum to one: values that are all the same bf16 number are the output."""
    q, k, v, cq, ck = inputs([333], [400], 8, 2, seed=8)
    v = torch.full_like(v, 1.625)
    out = check(q, k, v, cq, ck, SCALE, "constant values")
    assert (out.float() - 1.625).abs().max() <= 1.625 * 2.0 ** -7  # weights and output rounded to bf16


def test_strided_views():
    """q, k, v as slices of one projection's output [T, (Hq + 2 Hkv), 128], out with padded rows and heads."""
    T, Hq, Hkv = 210, 8, 2
    q, k, v, cq, ck = inputs([100, 110], [100, 110], Hq, Hkv, seed=9)
    qkv = torch.cat([q, k, v], 1).to(DEV)
    out = canaries((T, Hq + 1, 136))
    view = out[:, :Hq, :128]
    da.decode_attn_prefill(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], offsets(cq), offsets(ck), view, SCALE)
    torch.cuda.synchronize()
    ref, tol, _ = prefill_ref(q, k, v, cq, ck, SCALE)
    assert_within(view.cpu(), ref, tol, "views")
    assert (out[:, Hq].contiguous().view(torch.int16) == CANARY).all()
    assert (out[:, :, 128:].contiguous().view(torch.int16) == CANARY).all()
    # head-major tensors
    qh, kh, vh = (x.to(DEV).transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    out2 = torch.empty((Hq, T, 128), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    da.decode_attn_prefill(qh, kh, vh, offsets(cq), offsets(ck), out2, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out2, view)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_sequences_do_not_reach_a_row(bad):
    """NaN and infinities in a neighbour's rows, before and behind, and behind the last sequence."""
    q, k, v, cq, ck = inputs([60, 90, 77], [60, 200, 77], 4, 2, seed=10, spare=200)
    clean = check(q, k, v, cq, ck, SCALE, "clean")
    for t, c in ((q, cq), (k, ck), (v, ck)):
        t[:c[1]] = bad
        t[c[2]:] = bad
    out = canaries(q.shape)
    da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck), out, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu()[cq[1]:cq[2]], clean[cq[1]:cq[2]])


FEW_ROWS = [  # few query rows over many keys: the items are cut into parts and joined
    ([1], [5000], 8, 2),
    ([64], [4096], 4, 1),
    ([100], [2500], 16, 4),                   # the second item's rows end in different tiles
    ([5, 1, 33], [3001, 40, 2049], 8, 2),      # one of them too short to cut
    ([700], [640], 2, 1),                      # rows without a key beside rows with five tiles of them
    ([3, 0, 2], [6000, 0, 0], 12, 1),
    ([130], [1500], 3, 1),
]


@pytest.mark.parametrize("lq,lk,Hq,Hkv", FEW_ROWS, ids=[str(i) for i in range(len(FEW_ROWS))])
def test_few_rows_over_many_keys(lq, lk, Hq, Hkv):
    q, k, v, cq, ck = inputs(lq, lk, Hq, Hkv, seed=18, first=1, spare=140)
    out = check(q, k, v, cq, ck, SCALE, "few rows")
    check(q, (k.float() * torch.linspace(0, 6, len(k))[:, None, None]).to(torch.bfloat16), v, cq, ck, SCALE, "growing keys")
    check(q, k, v, cq, ck, -0.3, "negative scale")
    for t, c in ((q, cq), (k, ck), (v, ck)):  # what lies around the sequences does not matter
        t[:1] = float("nan")
        t[c[-1]:] = float("inf")
    again = canaries(q.shape)
    da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck), again, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(again.cpu()[cq[0]:cq[-1]], out[cq[0]:cq[-1]])


MIXED_CUT = [  # items of one call on both sides of the length from which they are cut (twelve tiles)
    ([1700], [1700], 4, 1),                    # a prompt: its first rows' items whole, the last ones cut
    ([2000], [1900], 2, 1),                    # and its first hundred rows without a key
    ([3, 3, 3, 3], [1408, 1409, 1536, 1537], 8, 2),
    ([1, 700, 1], [2900, 700, 1411], 4, 2),
]


@pytest.mark.parametrize("lq,lk,Hq,Hkv", MIXED_CUT, ids=[str(i) for i in range(len(MIXED_CUT))])
def test_whole_and_cut_items_in_one_call(lq, lk, Hq, Hkv):
    q, k, v, cq, ck = inputs(lq, lk, Hq, Hkv, seed=22, first=1, spare=3)
    check(q, k, v, cq, ck, SCALE, "whole and cut")
    check(q, (k.float() * torch.linspace(0, 6, len(k))[:, None, None]).to(torch.bfloat16), v, cq, ck, SCALE, "growing keys")


def test_few_rows_nan_in_the_sequence_reaches_its_rows():
    q, k, v, cq, ck = inputs([4, 4], [3000, 3000], 4, 1, seed=19)
    k[100] = float("nan")
    out = canaries(q.shape)
    da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck), out, SCALE)
    torch.cuda.synchronize()
    assert torch.isnan(out[:4]).all() and torch.isfinite(out[4:]).all()


def test_few_rows_with_offsets_of_any_kind_stay_inside():
    q, k, v, _, _ = inputs([30], [3000], 4, 1, seed=21)
    before = canaries((32, 4, 128))
    for cq, ck in (([20, 5, 30], [0, 3000, 10]), ([2 ** 31 - 1, -2 ** 31, 7], [-9, 1 << 30, 3]), ([0, 30, 0], [3000, 0, 3000])):
        out = before.clone()
        da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck), out[1:31], SCALE)
        torch.cuda.synchronize()
        assert da.decode_attn_last_device_error() == 0
        assert torch.equal(out[[0, 31]].view(torch.int16), before[[0, 31]].view(torch.int16))


def test_few_rows_captured_with_other_lengths():
    """The cut follows the lengths on the device: a captured call serves other ones."""
    q, k, v, cq, ck = inputs([6, 6], [2000, 2000], 8, 2, seed=20)
    dq, dk, dv, oq, ok = q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck)
    out = canaries(q.shape)
    da.decode_attn_prefill(dq, dk, dv, oq, ok, out, SCALE)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        da.decode_attn_prefill(dq, dk, dv, oq, ok, out, SCALE)
    for cq, ck in (([0, 1, 12], [0, 3900, 4000]), ([0, 12, 12], [0, 100, 4000]), ([0, 6, 12], [0, 2000, 4000])):
        oq.copy_(offsets(cq))
        ok.copy_(offsets(ck))
        graph.replay()
        torch.cuda.synchronize()
        ref, tol, _ = prefill_ref(q, k, v, cq, ck, SCALE)
        assert_within(out.cpu(), ref, tol, f"{cq} {ck}")


def test_many_short_sequences():
    """1000 sequences, most of them empty: far fewer work items than there could be."""
    lq = [0] * 1000
    for i in range(0, 1000, 37):
        lq[i] = 1 + i % 5
    lk = [n + (i % 3) * 7 if n else 0 for i, n in enumerate(lq)]
    check(*inputs(lq, lk, 8, 8, seed=16), SCALE, "short sequences")
    check(*inputs([1] * 1024, [1] * 1024, 2, 1, seed=17), SCALE, "1024 single tokens")


def test_offsets_are_clamped():
    """Offsets past the tokens end there; a sequence whose end lies before its start is empty."""
    q, k, v, _, _ = inputs([100], [100], 4, 2, seed=11)
    out = canaries(q.shape)
    da.decode_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), offsets([-5, 40, 30, 1 << 30]), offsets([0, 40, 40, 1 << 30]),
                           out, SCALE)
    torch.cuda.synchronize()
    assert da.decode_attn_last_device_error() == 0
    ref, tol, _ = prefill_ref(q, k, v, [0, 40], [0, 40], SCALE)
    assert_within(out.cpu()[:30], ref[:30], tol[:30], "first sequence")  # its last ten rows: the third one's too
    ref, tol, _ = prefill_ref(q[30:], k[40:], v[40:], [0, 70], [0, 60], SCALE)
    assert_within(out.cpu()[40:], ref[10:], tol[10:], "third sequence")


def test_other_stream_and_repeatable():
    q, k, v, cq, ck = inputs([500, 3], [500, 300], 8, 2, seed=12)
    s = torch.cuda.Stream()
    dq, dk, dv, oq, ok = q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck)
    outs = [torch.empty(q.shape, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        da.decode_attn_prefill(dq, dk, dv, oq, ok, outs[0], SCALE)
    da.decode_attn_prefill(dq, dk, dv, oq, ok, outs[1], SCALE, stream=s)
    s.synchronize()
    da.decode_attn_prefill(dq, dk, dv, oq, ok, outs[2], SCALE)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_captured_and_replayed():
    """One captured call serves new inputs and new lengths of the same packed size."""
    q, k, v, cq, ck = inputs([200, 100], [200, 100], 8, 2, seed=13)
    dq, dk, dv, oq, ok = q.to(DEV), k.to(DEV), v.to(DEV), offsets(cq), offsets(ck)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    da.decode_attn_prefill(dq, dk, dv, oq, ok, out, SCALE)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.decode_attn_prefill(dq, dk, dv, oq, ok, out, SCALE)
        da.decode_attn_prefill(dq, dk, dv, oq, ok, out, SCALE)
    q, k, v, cq, ck = inputs([37, 263], [37, 263], 8, 2, seed=14)
    for d, s in ((dq, q), (dk, k), (dv, v), (oq, offsets(cq)), (ok, offsets(ck))):
        d.copy_(s)
    out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    ref, tol, _ = prefill_ref(q, k, v, cq, ck, SCALE)
    assert_within(out.cpu(), ref, tol, "replayed")


def test_empty_calls():
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16, device=DEV)
    k = torch.empty((0, 2, 128), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_prefill(q, k, k, offsets([0, 0]), offsets([0, 0]), q.clone(), 1.0)
    da.decode_attn_prefill(q, k, k, offsets([0]), offsets([0]), q.clone(), 1.0)
    q = torch.ones((5, 8, 128), dtype=torch.bfloat16, device=DEV)  # queries, no tokens
    out = canaries(q.shape)
    da.decode_attn_prefill(q, k, k, offsets([0, 4]), offsets([0, 0]), out, 1.0)
    torch.cuda.synchronize()
    assert (out[:4] == 0).all() and (out[4].view(torch.int16) == CANARY).all()


def test_last_token_matches_the_decode_step():
    """The last query of a prompt is a decode step over the same tokens."""
    Hq, Hkv, L = 32, 8, 1000
    q, k, v, cq, ck = inputs([1] * 3, [L] * 3, Hq, Hkv, seed=15)
    out = check(q, k, v, cq, ck, SCALE, "single queries")
    kc, vc = (x.view(3, L, Hkv, 128).transpose(1, 2).contiguous().to(DEV) for x in (k, v))
    lens = torch.full((3,), L, dtype=torch.int32, device=DEV)
    dec = torch.empty((3, Hq, 128), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_only(q.to(DEV), kc, vc, lens, dec, SCALE)
    torch.cuda.synchronize()
    _, tol, _ = prefill_ref(q, k, v, cq, ck, SCALE)
    assert_within(dec.cpu(), out.double(), 2 * tol, "decode step")
