"""Two host threads that call on one stream: a call of several launches (tokens laid out and their attention, parts of items and their
join, the attention and its projection) is not mixed with the other thread's, whose scratch is the same workspace."""
import threading

import pytest
import torch

import decode_attention_output_gb300 as da
from test_cache import DEV, _library, bits, cu, i32  # noqa: F401
from test_chunk import SCALE, Cache, canvas

pytestmark = pytest.mark.gpu

CALLS = 200


def chunk(seed, lq, lk, kv8, bs):
    g = torch.Generator().manual_seed(seed)
    cache = Cache(g, lk, 2, bs, kv8)
    c = cu(lq)
    q = torch.randn((c[-1], 8, 128), generator=g).to(torch.bfloat16)
    args = q.to(DEV), *cache.on(), cache.table.to(torch.int32).to(DEV), i32(c), i32(lk)
    return canvas(q), lambda out: da.decode_attn_chunk(*args, out, SCALE)


def prompt(seed, lq, lk):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((n, h, 128), generator=g).to(torch.bfloat16).to(DEV) for n, h in ((lq, 8), (lk, 2), (lk, 2)))
    c = i32([0, lq]), i32([0, lk])
    return canvas(q), lambda out: da.decode_attn_prefill_window(q, k, v, *c, out, SCALE, 5000, 2)


def step(seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(s, generator=g).to(torch.bfloat16).to(DEV) for s in ((4, 8, 128), (4, 2, 900, 128), (4, 2, 900, 128)))
    w = (torch.randn((1024, 256), generator=g) / 32).to(torch.bfloat16).to(DEV)
    lens = i32([900, 1, 300, 777])
    return torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV), lambda out: da.decode_attn_fwd(q, k, v, lens, w, out, SCALE)


PAIRS = {
    "laid_out": lambda: (chunk(1, [60, 40], [900, 300], True, 16), chunk(2, [60, 40], [900, 300], True, 16)),
    "laid_out_and_tokens": lambda: (chunk(3, [70], [2500], False, 16), chunk(4, [1, 1], [3000, 900], True, 64)),
    "parts": lambda: (prompt(5, 40, 4000), prompt(6, 40, 4000)),
    "parts_and_step": lambda: (prompt(7, 40, 4000), step(8)),
    "steps": lambda: (step(9), step(10)),
}


@pytest.mark.parametrize("name", sorted(PAIRS))
def test_two_threads_on_one_stream(name):
    calls = PAIRS[name]()
    want, outs = [], []
    for out, run in calls:
        run(out)
        want.append(out.clone())
        outs.append([torch.zeros_like(out) for _ in range(CALLS)])
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def work(i):
        try:
            torch.cuda.set_device(0)
            start.wait()
            for out in outs[i]:
                calls[i][1](out)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for i in range(2):
        wrong = sum(not torch.equal(bits(o), bits(want[i])) for o in outs[i])
        assert wrong == 0, f"{wrong} of {CALLS} results of thread {i} differ"
    assert da.decode_attn_last_device_error() == 0
