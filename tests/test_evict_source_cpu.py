"""What the compaction and selection kernels' sources promise where a GPU test could not show a breach: bounds that the
compiler checks, and memory orderings that hold by rule and not by luck."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_06_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def constants(text):
    return {n: int(v) for n, v in re.findall(r"^constexpr int (k\w+) = (\d+);", text, re.M)}


def ring_overwritten(ring, block, stages, per):
    """Whether an address ring entry is overwritten while a thread may still need it.  Before round r + 1's barrier a
    fast thread translates rows, `block` at a time, until those of round r + stages are there; a slow thread of the CTA
    may still write the rows of round r."""
    for r in range(8 * ring // per):
        translated = -(-(r + stages + 1) * per // block) * block
        if translated - r * per > ring:
            return True
    return False


@pytest.mark.parametrize("stages", [2, 3, 4, 5, 6])
@pytest.mark.parametrize("block", [256, 512, 1024])
@pytest.mark.parametrize("rows", [32, 64, 100, 113, 128])
def test_the_address_rings_assertion_refuses_what_overwrites_rows_in_flight(stages, block, rows):
    text = source("evict.cu")
    held = re.search(r"static_assert\((kMoveRing[^,]*),", text).group(1)
    for ring in (1024, 2048):
        names = dict(constants(text), kMoveRing=ring, kMoveBlock=block, kMoveStages=stages, kMoveRows=rows)
        if any(ring_overwritten(ring, block, stages, per) for per in range(1, rows + 1)):
            assert not eval(held, {}, names)


def test_the_address_ring_as_built_is_long_enough():
    c = constants(source("evict.cu"))
    assert not any(ring_overwritten(c["kMoveRing"], c["kMoveBlock"], c["kMoveStages"], per)
                   for per in range(1, c["kMoveRows"] + 1))


def function(text, name):
    """The text of a function from its name to the closing brace of its column."""
    at = re.search(r"^[^\n]*\b%s\([^;]*?\{\n" % name, text, re.M | re.S)
    return text[at.start(): text.index("\n}\n", at.end())]


@pytest.mark.parametrize("name", ["evict.cu", "tree.cu"])
def test_no_non_coherent_loads_where_the_writer_may_still_run(name):
    """These kernels start while the grid that writes their lengths, lists and totals may still run; a non-coherent load
    wants its data unwritten for as long as the kernel lives."""
    text = re.sub(r"//[^\n]*", "", source(name))
    assert "__ldg(" not in text and ".nc" not in text and "__restrict__" not in text


def test_the_decodes_length_is_no_non_coherent_load():
    """Lengths may be the kept_lens of a selection that is still running when the decode starts."""
    assert "__ldg(" not in function(source("decode.cu"), "checked_length")


def test_what_the_totals_read_ahead_goes_past_l1():
    """accumulate_weights reads lengths and totals before its wait: past L1, which may hold older lines."""
    text = source("evict.cu")
    ahead = function(text, "accumulate_weights_kernel").split("griddep_wait();  // the decode")[0]
    assert "__ldcg(" in ahead and "length_of<true>" in ahead


def test_selections_last_barrier_orders_its_reads():
    """A CTA reads the counts of its cluster's others; its arrival at the barrier that lets them leave must order those
    reads, which a relaxed one does not."""
    text = function(source("evict.cu"), "evict_select_kernel")
    assert "cluster_arrive_relaxed" not in text
    reads = text.index("cluster_read_int(&sh.counts[1], r)")
    assert reads < text.index("cluster_arrive();") < text.index("cluster_wait();")
