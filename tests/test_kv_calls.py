"""Page ownership: calls and sizes beside those of test_kv_cache.py, with the same model."""
import pytest

import persistent_moe_decode_sm_gb300 as mk
from kv_model import NO_PAGES, PAGE_OOB, Refused
from test_kv_cache import Pair, start

gpu = pytest.mark.gpu


def status(p):
    with pytest.raises(mk.MkError) as e:
        p.cache.sync()
    return e.value.code


@gpu
@pytest.mark.parametrize("name, a, b", [
    ("fork", [9, 0], [1, 2]),                       # a row that is not there; a page that is not held
    ("fork", [0, 0, 0], [2, 2, 3]),                 # the same row twice; the page
    ("resize", [9, 0], [5, 3]), ("resize", [1, 1, 0], [5, 5, 3]),
    ("resize", [9, 1], [5, 16 * 40 + 1]),           # a row that is not there; a length behind the table
    ("copy_pages", [0, 0, 50], [5, 5, 6])])         # a target twice; a page behind the pool
def test_of_several_wrong_arguments_the_same_one_is_reported(name, a, b):
    """A wrong row number is met at once, a wrong page behind three loads: whichever comes
    first, the page is reported."""
    m = start(50, 6, 40, 16, [40])
    m.tables[0, 2] = 50
    p = Pair(m)
    for _ in range(5):
        getattr(p.cache, name)(p.i32(a), p.i32(b))
        assert status(p) == PAGE_OOB
    p.same()


def two_holders(pages):
    """Rows 0 and 1 end inside a page that both hold; `pages` in the pool, 3 of them held."""
    m = start(pages, 4, 6, 16, [40])
    m.fork([0], [1])
    m.resize([0, 1], [20, 20])                      # page 1 of both, shared by the fork
    assert m.tables[0, 1] == m.tables[1, 1] and (m.refs > 0).sum() == 2
    return m


def holders_count_as_they_were(run):
    """A last page with two holders is copied for each of them that grows, whatever the other
    one does in the same call."""
    m = two_holders(4)
    shared = int(m.tables[0, 1])
    assert run(m, [0, 1], [21, 21]) == 0            # two copies; the page gets free
    assert m.refs[shared] == 0 and shared not in m.tables[:2, :2]
    m = two_holders(4)
    assert run(m, [0, 1], [0, 21]) == 0             # one copy, the page is released by the other
    assert m.refs[shared] == 0 and m.tables[1, 1] != shared
    m = two_holders(4)
    m.refs[[p for p in range(4) if m.refs[p] == 0][0]] = 1     # a holder outside: one page is free
    assert run(m, [0, 1], [21, 21]) == NO_PAGES
    m.refs[[p for p in range(4) if m.refs[p] == 0][0]] = 1     # none is
    assert run(m, [0, 1], [0, 21]) == NO_PAGES
    assert run(m, [0], [0]) == 0                    # in a call of its own first
    assert run(m, [1], [21]) == 0 and m.tables[1, 1] == shared


def test_model_holders_count_as_they_were():
    def run(m, seqs, lens):
        try:
            m.resize(seqs, lens)
        except Refused as r:
            return r.code
        return 0

    holders_count_as_they_were(run)


@gpu
def test_holders_count_as_they_were():
    def run(m, seqs, lens):
        p = Pair(m)
        p.m = m                                     # the model goes along
        code = p.do("resize", seqs, lens)
        p.same()
        return code

    holders_count_as_they_were(run)
