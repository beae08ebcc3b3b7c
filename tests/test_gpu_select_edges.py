"""The operators that choose among cached tokens at the ends of their ranges: totals of no columns, lists read again from
L2, tables far wider than the lengths, cut work of many sequences, infinities and odd scales in the decode with totals,
and what follows a call whose sequences are all empty."""
import math

import pytest
import torch

import plain_select as plain
from gpu_util import DEV
from paged_kv_gqa_06_gb300 import binding
from test_gpu_evict import check_select, clean, decode, i32, make, totals_of, within
from test_gpu_tree import check as check_tree
from test_gpu_tree import make as make_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.init()


def test_totals_of_no_columns_are_reported():
    """A sequence longer than the totals is recorded whatever their length, 0 too."""
    a = make([40, 9], 2, 4, 64, torch.float32, seed=1)
    ref, bound, _, _ = plain.weights(a["q"], a["k"], a["v"], a["tables"], a["lens"], a["scale"], a["out"], a["totals"])
    a["totals"] = torch.empty(2, 2, 0, device=DEV)
    decode(a)
    assert binding.forge_paged_get_device_error() == 2
    within(a["out"], ref, bound)
    kept, n = i32([[[3, 20, 35]] * 2, [[1, 2, 8]] * 2]), i32([3, 3])
    want = plain.compact(a["k"].cpu(), a["v"].cpu(), a["tables"].cpu(), a["lens"].cpu(), kept.cpu(), n.cpu(), None, None)
    binding.forge_paged_kv_compact(a["k"], a["v"], a["tables"], a["lens"], kept, n, weights=a["totals"])
    assert binding.forge_paged_get_device_error() == 2
    assert torch.equal(a["k"].cpu().view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(a["v"].cpu().view(torch.int16), want[1].view(torch.int16))
    a["lens"].zero_()                # nothing is longer than no columns
    n.zero_()
    decode(a)
    binding.forge_paged_kv_compact(a["k"], a["v"], a["tables"], a["lens"], kept, n, weights=a["totals"])
    clean()


# ---------------------------------------------------------------- lists and tables

@pytest.mark.parametrize("kind", ["plain", "ties", "same"])
def test_lists_longer_than_a_cluster_holds(kind):
    """More than 16 * 8192 positions: keys are read again from L2, and a thread's run is longer than 32."""
    L = 16 * 8192 + 70001
    x = totals_of(kind, (1, 2, (L + 3) // 4 * 4), 1)
    check_select(x, [L], L // 2, 5, 1000)
    check_select(x, [L], 77, 1, 2)


def test_a_list_just_past_what_a_cluster_holds():
    for L in (16 * 8192 + 5, 16 * 8192 + 6, 16 * 8192 + 16 * 1024):
        check_select(totals_of("near", (1, 1, (L + 3) // 4 * 4), L), [L], 5000, 3, 2)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_cut_trees_of_many_sequences(out_dtype):
    """More sequences than a warp, long enough to be cut, with empty ones among them."""
    lens = [700 + 37 * i % 900 for i in range(70)]
    nodes = [(3 * i) % 11 for i in range(70)]
    check_tree(make_tree(lens, nodes, 2, 4, 64, out_dtype, seed=2))


def wider(tables, width):
    t = torch.full((tables.shape[0], width), -1, dtype=torch.int32, device=DEV)
    t[:, :tables.shape[1]] = tables
    return t


@pytest.mark.parametrize("lens,nodes", [([600, 33, 1, 290], [9, 20, 1, 40]), ([20], [4])])
def test_trees_in_tables_far_wider_than_the_lengths(lens, nodes):
    a = make_tree(lens, nodes, 2, 4, 128, torch.bfloat16, seed=3)
    a["tables"] = wider(a["tables"], 4096)
    check_tree(a)


@pytest.mark.parametrize("lens", [[600, 33, 1, 290, 0, 1100], [20]])
def test_totals_in_tables_far_wider_than_the_lengths(lens):
    a = make(lens, 2, 4, 128, torch.float32, seed=4, S=65536)
    before = a["totals"].clone()
    a["tables"] = wider(a["tables"], 4096)
    ref, bound, tot, tb = plain.weights(a["q"], a["k"], a["v"], a["tables"], a["lens"], a["scale"], a["out"], a["totals"])
    decode(a)
    clean()
    within(a["out"], ref, bound)
    within(a["totals"], tot, tb)
    for b, L in enumerate(lens):
        assert torch.equal(a["totals"][b, :, L:], before[b, :, L:])
    kept, n = torch.full((len(lens), 2, 64), -5, dtype=torch.int32, device=DEV), i32([-5] * len(lens))
    binding.forge_paged_evict_select(a["totals"], a["lens"], 64, 4, 16, kept, n)
    clean()
    want = plain.select(a["totals"], lens, 64, 4, 16)
    for b in range(len(lens)):
        assert [kept[b, g, :n[b]].tolist() for g in range(2)] == want[b]


# ---------------------------------------------------------------- decode with totals: values

@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
@pytest.mark.parametrize("G", [1, 8])
def test_totals_at_odd_scales(scale, G):
    a = make([700, 33, 1], 2, G, 64, torch.float32, seed=5)
    a["scale"] = scale
    ref, bound, tot, tb = plain.weights(a["q"], a["k"], a["v"], a["tables"], a["lens"], scale, a["out"], a["totals"])
    decode(a)
    clean()
    within(a["out"], ref, bound)
    within(a["totals"], tot, tb)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("pos", [5, 650])
def test_a_bad_value_stays_in_its_dim(bad, pos):
    """An infinity or NaN of V reaches its own dim of its own KV head, and no total."""
    a = make([700, 33], 2, 4, 128, torch.float32, seed=6)
    ref, bound, tot, tb = plain.weights(a["q"], a["k"], a["v"], a["tables"], a["lens"], a["scale"], a["out"], a["totals"])
    a["v"][int(a["tables"][0, pos // 16]), 1, pos % 16, 3] = bad
    decode(a)
    clean()
    within(a["totals"], tot, tb)
    hit = torch.zeros_like(a["out"], dtype=torch.bool)
    hit[0, 4:8, 3] = True
    got = a["out"].double()
    assert not got[hit].isfinite().any()
    assert ((got - ref).abs()[~hit] <= bound[~hit]).all()


def test_what_follows_empty_sequences_waits_for_the_decode():
    """Sequences that are all empty leave the totals' grid nothing to do; a copy behind the call must still find the
    decode's zeros, in an output that has held something else until then."""
    big = make([4000] * 40, 4, 4, 128, torch.float32, seed=12)
    a = make([0] * 40, 4, 4, 128, torch.float32, seed=11, S=2048)
    outs = [torch.full_like(a["out"], 7.25) for _ in range(20)]
    seen = [torch.empty_like(a["out"]) for _ in outs]
    totals = a["totals"].clone()
    torch.cuda.synchronize()
    for out, copy in zip(outs, seen):
        decode(big)
        a["out"] = out
        decode(a)
        copy.copy_(out)
    clean()
    assert all((x == 0).all() for x in seen) and torch.equal(a["totals"], totals)


def test_lengths_that_a_selection_has_just_written():
    """kept_lens as the lengths of the calls right behind the selection and the move, which start while these run: every
    call must see this step's lengths, not those of the step before."""
    lens = [700, 120, 333, 64, 1024, 15]
    a = make(lens, 4, 4, 128, torch.float32, seed=7, S=1024)
    budgets, sets = [64, 700, 200, 31, 1000], []
    k0, v0, t0 = a["k"].clone(), a["v"].clone(), a["totals"].clone()
    kept = torch.zeros(6, 4, 1024, dtype=torch.int32, device=DEV)
    n = torch.zeros(6, dtype=torch.int32, device=DEV)
    tree_out = torch.zeros(12, 16, 128, device=DEV)
    tree_q = a["q"].repeat_interleave(2, dim=0)
    start, mask = i32(range(0, 13, 2)), torch.tensor([[1], [3]] * 6, dtype=torch.int64, device=DEV)

    def step(budget, wait):
        out = torch.empty_like(a["out"])
        for x, y in ((a["k"], k0), (a["v"], v0), (a["totals"], t0)):
            x.copy_(y)
        calls = [lambda: binding.forge_paged_evict_select(a["totals"], a["lens"], budget, 4, 16, kept, n),
                 lambda: binding.forge_paged_kv_compact(a["k"], a["v"], a["tables"], a["lens"], kept, n, weights=a["totals"]),
                 lambda: binding.forge_paged_gqa_decode(a["q"], a["k"], a["v"], a["tables"], n, a["scale"], out),
                 lambda: binding.forge_paged_tree_attention(tree_q, a["k"], a["v"], a["tables"], n, start, mask, a["scale"],
                                                            tree_out),
                 lambda: binding.forge_paged_gqa_decode_weights(a["q"], a["k"], a["v"], a["tables"], n, a["scale"], a["out"],
                                                                a["totals"])]
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()
        return [x.clone() for x in (out, tree_out, a["out"], a["totals"], n)]

    for budget in budgets:
        sets.append(step(budget, True))
        assert sets[-1][4].tolist() == [min(L, budget) for L in lens]
    for _ in range(20):
        for budget, want in zip(budgets, sets):
            got = step(budget, False)
            for x, y in zip(got, want):
                assert torch.equal(x, y)
    clean()
