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
