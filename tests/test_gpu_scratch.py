"""The library-owned scratch under graph capture: a graph's buffer outlives its being outgrown, and goes back once the
graph is destroyed."""
import gc
import time

import pytest
import torch

import plain_select as plain
from gpu_util import DEV
from paged_kv_gqa_06_gb300 import binding

pytestmark = pytest.mark.gpu

STEP = 32768                    # blocks: 2 * 32 heads of 524288 logits, 134 MB


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.init()


def make(width, seed=0):
    """A decode with totals of two short sequences whose tables are `width` blocks wide: the scratch goes by the width."""
    gen = torch.Generator().manual_seed(seed)
    lens = [100, 37]
    tables, k, v = plain.caches(lens, 8, 128, gen, DEV, 2.0)
    wide = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    wide[:, :tables.shape[1]] = tables
    return dict(q=torch.randn(2, 32, 128, generator=gen).to(torch.bfloat16).to(DEV), k=k, v=v, tables=wide,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), out=torch.zeros(2, 32, 128, device=DEV),
                totals=torch.zeros(2, 8, 128, device=DEV))


def decode(a):
    binding.forge_paged_gqa_decode_weights(a["q"], a["k"], a["v"], a["tables"], a["lens"], 0.1, a["out"], a["totals"])


def held():
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return total - free - torch.cuda.memory_reserved()


def capture(a, stream):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        decode(a)
    return g


def check(a, seed=0):
    want = make(a["tables"].shape[1], seed)
    ref, bound, tot, tb = plain.weights(want["q"], want["k"], want["v"], want["tables"], want["lens"], 0.1, want["out"],
                                        want["totals"])
    assert ((a["out"].double() - ref).abs() <= bound).all() and ((a["totals"].double() - tot).abs() <= tb).all()


def test_scratch_goes_back_when_its_graphs_are_destroyed():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    small = make(16)
    with torch.cuda.stream(s):
        decode(small)
    before = held()
    for i in range(1, 6):
        a = make(STEP * i)
        with torch.cuda.stream(s):
            decode(a)           # grows
        s.synchronize()
        a["totals"].zero_()
        torch.cuda.synchronize()
        g = capture(a, s)
        g.replay()
        torch.cuda.synchronize()
        check(a)
        del g, a
        gc.collect()
    for _ in range(20):         # the last captures' destruction may reach the library a little later
        with torch.cuda.stream(s):
            decode(small)
        now = held() - before
        if now < 7 * 2 ** 27:
            break
        time.sleep(0.1)
    # the last buffer, 5 * 134 MB and the split partials; all five together are 15 * 134 MB
    assert now < 7 * 2 ** 27, f"{now >> 20} MiB held"
    assert binding.forge_paged_get_device_error() == 0


def test_graphs_of_one_buffer_keep_it_while_one_lives():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls = [make(64, seed) for seed in (1, 2)]
    for a in calls:
        with torch.cuda.stream(s):
            decode(a)
        s.synchronize()
        a["totals"].zero_()
    torch.cuda.synchronize()
    graphs = [capture(a, s) for a in calls]
    with torch.cuda.stream(s):
        decode(make(STEP))      # outgrows the graphs' buffer
    del graphs[0]
    gc.collect()
    time.sleep(0.2)
    for _ in range(3):
        big = make(STEP)
        with torch.cuda.stream(s):
            decode(big)
        s.synchronize()
        filler = [torch.full((1 << 20,), 7.0, device=DEV) for _ in range(16)]   # in memory that was given back, if any
        calls[1]["totals"].zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        torch.cuda.synchronize()
        check(calls[1], 2)
        assert all((x == 7.0).all() for x in filler)
    assert binding.forge_paged_get_device_error() == 0
