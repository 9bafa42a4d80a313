"""Places in the rings of the 4-bit kernels are handed back by what was loaded from them.

A warp barrier alone does not do: a load whose result is needed last can then come after the hand-back and see what is
brought into its place next, where that is quick and the other operands are late. Which loads come late is the compiler's
choice, so that running a build says nothing about the next one; the sources are looked at instead.
"""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "sparse_attention_indexer_lt_gb300" / "csrc"


def text(name):
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


@pytest.mark.parametrize("name", ["lt_kv4_prefill.cuh", "lt_w4_many.cu"])
def test_arrivals_of_readers_go_by_what_they_have_read(name):
    code = text(name)
    given = re.findall(r"\barrive\((&sh->\w+_empty\[[^\]]*\][^)]*)\)", code)  # (mma_commit is a call of its own)
    assert given
    for where in given:
        m = re.search(r"\] \+ (\w+)$", where)
        assert m, f"{name}: {where}"
        assert re.search(r"uint32_t " + m[1] + r" = zero_of\([^;]*, p\.zero\);", code), f"{name}: {m[1]}"


@pytest.mark.parametrize("name,first", [("lt_kv4_rows.cuh", r"bring\(s, pos\[s\], page\[s\], 0\)"), ("lt_w4_linear.cu", r"bring\(s, 0\)")])
def test_copies_into_a_place_that_was_read_go_by_what_was_read(name, first):
    code = text(name)
    calls = re.findall(r"\bbring\([^;{]*\);", code)
    later = [c for c in calls if not re.match(first, c)]
    assert len(later) == len(calls) - 1 and later
    assert all(re.search(r"zero_of\(.*, p\.zero\)\);$", c) for c in later), later
    assert re.search(r"const uint32_t (tile_at|at) = [^;]* \+ zero;", code)
