"""The workspace of decode_attn_chunk: what is held after calls of growing size, shares of a call where it may not be as large as
the call would like, and the refusal where not even one head of one sequence fits."""
import pytest
import torch

import decode_attention_output_gb300 as da
from chunk_helpers import attend_ref
from test_cache import DEV, _library, bits, cu, i32  # noqa: F401
from test_chunk import SCALE, Cache, canvas, check

pytestmark = pytest.mark.gpu

DA_ERR_NOMEM = -7
MIB = 1 << 20


@pytest.fixture
def fresh():
    torch.cuda.synchronize()
    da.decode_attn_release()
    yield
    da.decode_attn_set_option("workspace_mib", 0)
    torch.cuda.synchronize()
    da.decode_attn_release()


def wide_call(capacity, lq, lk, Hq, Hkv, kv8=True, seed=71, window=0, sinks=0):
    """A call whose tables have `capacity` tokens of each sequence; (run, what it has to give)."""
    g = torch.Generator().manual_seed(seed)
    cache = Cache(g, lk, Hkv, 16, kv8)
    table = torch.full((len(lk), capacity // 16), -1, dtype=torch.int32)
    table[:, :cache.table.shape[1]] = cache.table
    c = cu(lq, first=2)
    q = torch.randn((c[-1] + 3, Hq, 128), generator=g).to(torch.bfloat16)
    args = q.to(DEV), *cache.on(), table.to(DEV), i32(c), i32(lk)
    return (lambda out: da.decode_attn_chunk(*args, out, SCALE, window, sinks)), q, attend_ref(q, *cache.tokens, c, SCALE, window, sinks)


def held():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free, total = torch.cuda.mem_get_info()
    return total - free


def test_calls_of_growing_size_hold_twice_the_largest_at_most(fresh):
    """Tokens of 480 MiB laid out, then of 500 (and 9 for parts of items): both fit a block of 512, and nothing larger is taken."""
    for mib in (480, 500):  # a KB for each token, K and V of two heads
        run, q, want = wide_call(mib * 1024, [60], [300], 8, 2)
        out = canvas(q)
        if mib == 480:
            before = held()
        run(out)
        check(out, *want, str(mib))
    more = held() - before
    assert more <= 2 * 512 * MIB, f"{more / MIB:.0f} MiB held"


CASES = [  # capacity, queries, keys, Hq, Hkv, window, sinks
    (40_000, [70, 1, 0, 33, 90], [900, 1, 300, 33, 2000], 16, 8, 0, 0),
    (40_000, [150], [3000], 16, 8, 0, 0), (40_000, [150], [3000], 16, 8, 300, 4),
    (20_000, [400] + [1] * 30, [900] + [37 * i for i in range(30)], 16, 8, 0, 0),  # of few rows too, by the kernel for those
]


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("capacity,lq,lk,Hq,Hkv,window,sinks", CASES, ids=str)
def test_shares_where_the_workspace_is_small(fresh, capacity, lq, lk, Hq, Hkv, window, sinks, kv8):
    """All sequences at once, some, one with all heads or some heads: the same results within their roundings, and again
    from a graph captured under the same limit; a block is never larger than the limit."""
    run, q, want = wide_call(capacity, lq, lk, Hq, Hkv, kv8, window=window, sinks=sinks)
    for mib in (0, 500, 200, 100, 40):
        da.decode_attn_release()
        da.decode_attn_set_option("workspace_mib", mib)
        out, before = canvas(q), held()
        run(out)
        if mib:
            assert held() - before <= (mib + 32) * MIB, f"a block past the limit of {mib}"
        check(out, *want, f"{mib} MiB")
        if mib in (0, 100):
            again, graph = canvas(q), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                run(again)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(bits(again), bits(out))
            del graph


def test_no_room_for_one_head(fresh):
    """Refused before anything is launched: by the option, and by the device for more than it has (half a TiB of one head's)."""
    run, q, want = wide_call(40_000, [150], [3000], 16, 8)
    out = canvas(q)
    da.decode_attn_set_option("workspace_mib", 15)
    with pytest.raises(da.DecodeAttnError) as e:
        run(out)
    assert e.value.code == DA_ERR_NOMEM and (out == 7.5).all()
    da.decode_attn_set_option("workspace_mib", 0)
    huge, q_huge, _ = wide_call(1 << 30, [40], [100], 4, 2)
    out = canvas(q_huge)
    before = held()
    for _ in range(2):
        with pytest.raises(da.DecodeAttnError) as e:
            huge(out)
        assert e.value.code == DA_ERR_NOMEM and (out == 7.5).all()
    assert held() - before <= 64 * MIB
    out = canvas(q)
    run(out)  # as if nothing had been
    check(out, *want, "after the refusals")


def test_a_capture_does_not_take_smaller_shares(fresh):
    """A first call during a capture is refused as for the other entry points, whatever a smaller share would need."""
    small, q_small, _ = wide_call(1024, [60], [300], 8, 2)
    small(canvas(q_small))
    run, q, want = wide_call(100_000, [150], [3000], 16, 8)
    out, status = canvas(q), None
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        torch.zeros((8,), device=DEV)  # (something in the graph)
        try:
            run(out)
        except da.DecodeAttnError as e:
            status = e.code
    assert status == DA_ERR_NOMEM
    run(out)
    check(out, *want, "eager")
