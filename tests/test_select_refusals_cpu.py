"""Argument checks of the operators that choose among cached tokens, beside those of test_select_cpu.py."""
import pytest

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
    # rows side by side, in either order
    for a, b in ((512, 64), (64, 64 * shape[0]), (1024, 128), (520, 64)):
        assert call(lib, {**base, "out": _desc(shape, F32, stride=[a, b, 1])}) != -3, (a, b)
