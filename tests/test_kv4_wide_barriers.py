"""The barriers of the 4-bit cache's tcgen05 attention kernel (kv4_wide.cu), proved on the model of its warps in
test_kv8_wide_barriers.py (CPU): the roles, waits and arrivals are the same, the depths and counts are read from this source.
The number of tokens of a page that the copy warp leaves for the converters goes with the page's ring entry."""
import os
import re

import pytest

import test_kv8_wide_barriers as M

SRC = os.path.join(os.path.dirname(M.SRC), "kv4_wide.cu")


def _source():
    return re.sub(r"//[^\n]*", "", open(SRC).read())


@pytest.mark.parametrize("vec", [True, False])
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("runs", M.RUNS, ids=str)
def test_no_wait_can_be_overtaken(runs, fp32, vec):
    bad = M.wide_model(_source(), runs, fp32, vec).check()
    assert not bad, bad[:5]


def test_the_roles_wait_and_arrive_as_in_the_model(monkeypatch):
    """The same sequence of waits, arrivals, commits and rings as the kernel that the model was written for."""
    steps = r"wait\(&bar\.\w+\[[^\]]*\]|wait\(&bar\.\w+|wait\(v \? [^,]*|mbar_arrive\([^;]*|tc_commit\([^;]*|mbar_expect_tx\(&[^,]*|Turn<\w+> [^;]*|tc_mma<[^;]*"
    mine, other = (re.findall(steps, x) for x in (_source(), M._source()))
    assert mine == other
    monkeypatch.setattr(M, "SRC", SRC)
    M.test_the_source_uses_the_depths_of_the_model()
    body = _source().split("k_kv4_wide(w4a8_kv4_cache c")[1]
    assert 0 < body.index("griddep_enter();") < body.index("tcgen05.alloc")


def test_the_token_counts_go_with_the_ring():
    text = _source()
    write, arrive = text.index("held[e.i] ="), text.index("mbar_expect_tx(&bar.code_full[e.i]")
    assert text.index("wait(&bar.code_empty[e.i]") < write < arrive
    read = text.index("= held[e.i];")
    assert text.index("wait(&bar.code_full[e.i], e.ph)") < read < text.index("mbar_arrive(&bar.code_empty[e.i])")
    assert text.count("held[") == 2
