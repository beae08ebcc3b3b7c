"""Argument checks of the operators that choose among cached tokens, beside those of test_select_cpu.py."""
import pytest
import torch

from paged_kv_gqa_06_gb300 import binding
from test_abi_cpu import BF16, F32, I32, I64, _desc
from test_select_cpu import DEC, MOVE, TREE, _dec, _move, _select, _tree


@pytest.fixture(scope="module")
def lib():
    from paged_kv_gqa_06_gb300 import build
    build.build()
    return binding.load_library()


# Overlapping rows of an output hold whatever was written last.
@pytest.mark.parametrize("shape,call,base,strides", [
    ([6, 8, 64], _tree, TREE, [(0, 64), (512, 0), (512, 60), (64, 64), (64, 380), (508, 64)]),
    ([2, 8, 64], _dec, DEC, [(0, 64), (512, 0), (512, 60), (64, 64), (64, 124), (508, 64)]),
])
def test_outputs_with_overlapping_rows_are_refused(lib, shape, call, base, strides):
    for a, b in strides:
        assert call(lib, {**base, "out": _desc(shape, F32, stride=[a, b, 1])}) == -3, (a, b)
    if torch.cuda.is_available():
        return                     # these descriptors hold no device memory
    # rows side by side, in either order
    for a, b in ((512, 64), (64, 64 * shape[0]), (1024, 128), (520, 64)):
        assert call(lib, {**base, "out": _desc(shape, F32, stride=[a, b, 1])}) != -3, (a, b)


def test_a_single_column_has_any_inner_stride(lib):
    """The stride of a dimension of one element says nothing (a transposed row, a sliced column)."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; these descriptors hold no device memory")
    one = _desc([2, 3, 1], I32, stride=[3, 1, 7])
    assert _select(lib, budget=1, sink=0, recent=0, kept=one) == -6
    assert _select(lib, budget=1, sink=0, recent=0, kept=_desc([2, 3, 1], I32, stride=[1, 2, 2])) == -6
    table = _desc([2, 1], I32, stride=[1, 2])
    assert _tree(lib, {**TREE, "bt": table}) == -6
    assert _tree(lib, {**TREE, "mask": _desc([6, 1], I64, stride=[1, 6])}) == -6
    single = dict(bt=_desc([1, 4], I32), cl=_desc([1], I32, stride=[5]), qs=_desc([2], I32))
    assert _tree(lib, {**TREE, **single}) == -6
    assert _move(lib, {**MOVE, "bt": table, "kept": _desc([2, 2, 1], I32, stride=[2, 1, 9])}) == -6
    # two columns still have to be neighbours
    assert _select(lib, budget=2, sink=0, recent=0, kept=_desc([2, 3, 2], I32, stride=[12, 4, 2])) == -3
    assert _tree(lib, {**TREE, "bt": _desc([2, 2], I32, stride=[4, 2])}) == -3
    assert _move(lib, {**MOVE, "bt": _desc([2, 2], I32, stride=[4, 2])}) == -3
