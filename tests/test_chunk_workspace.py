"""The workspace of decode_attn_chunk: what is held after calls of growing size."""
import pytest
import torch

import decode_attention_output_gb300 as da
from chunk_helpers import attend_ref
from test_cache import DEV, _library, cu, i32  # noqa: F401
from test_chunk import SCALE, Cache, canvas, check

pytestmark = pytest.mark.gpu

MIB = 1 << 20


@pytest.fixture
def fresh():
    torch.cuda.synchronize()
    da.decode_attn_release()
    yield
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
