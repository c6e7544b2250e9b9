"""Page ownership: calls and sizes beside those of test_kv_cache.py, with the same model."""
import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
from kv_model import INVALID_ARG, NO_PAGES, PAGE_OOB, Refused
from test_kv_cache import Pair, sound, start

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


def big(rows, entries, extra=0, lens=None, seed=0):
    """A model of `rows` sequences, and as many empty rows, in a pool that has room for all."""
    rng = np.random.default_rng(seed)
    lens = [int(rng.integers(0, entries * 16 + 1)) for _ in range(rows)] if lens is None else lens
    pages = 2 * sum(-(-n // 16) for n in lens) + 2 * rows + extra
    return start(pages, 2 * rows, entries, 16, lens, seed, page_bytes=16, pools=2)


def traffic(m, seed):
    """Forks (first ones and repeated ones), beams, growth, frees and compaction."""
    rng = np.random.default_rng(seed)
    p, S = Pair(m), len(m.lens)
    half = S // 2
    cap = m.tables.shape[1] * m.P
    p.do("fork", rng.integers(0, half, half), np.arange(half, S))
    p.same()
    p.do("fork", rng.integers(0, S, S), rng.permutation(S))
    p.same()
    sound(m)
    some = rng.permutation(S)[:half + half // 2]
    p.do("resize", some, np.minimum(cap, m.lens[some] + rng.integers(0, 20, len(some))))
    p.same()
    p.do("resize", some[::2], rng.integers(0, 2, len(some[::2])) * m.lens[some[::2]] // 2)
    p.same()
    sound(m)
    p.compact()
    p.same()
    sound(m)
    assert (p.m.refs[:int((p.m.refs > 0).sum())] > 0).all()
    bad = np.arange(S)
    bad[-1] = 0                                     # the last row number twice
    assert p.do("fork", np.arange(S), bad) == INVALID_ARG
    assert p.do("resize", bad, np.zeros(S, int)) == INVALID_ARG
    p.same()


@gpu
@pytest.mark.parametrize("rows, entries, extra", [
    (120, 30, 0), (150, 30, 0), (300, 30, 0),       # on both sides of the larger launch
    (700, 6, 0),                                    # more rows than a block has threads
    (1500, 3, 0), (9, 700, 0), (20, 1000, 0),
    (3, 9, 17000), (3, 9, 36000), (3, 9, 70000),    # large pools
    (2, 2, 2 ** 18)])
def test_large_calls(rows, entries, extra):
    traffic(big(rows, entries, extra, seed=rows), rows + extra)


@gpu
@pytest.mark.parametrize("free", [0, 1])
def test_out_of_pages_in_a_large_call(free):
    """300 forks of a partly filled page, with the pages for all of them and for one less."""
    m = start(1 + 300 - 1 + free, 301, 40, 16, [7], page_bytes=16, pools=1)
    p = Pair(m)
    assert p.do("fork", [0] * 300, np.arange(1, 301)) == (0 if free else NO_PAGES)
    p.same()


@gpu
@pytest.mark.parametrize("pages, pairs", [(12000, 4096), (12000, 4097), (12000, 6000),
                                          (2 ** 18, 100), (2 ** 18 + 1, 100), (300000, 9000)])
def test_copies_of_many_pages(pages, pairs):
    """One kernel up to 4096 pairs and 2^18 pages, a plan and a move beyond; with its refusals."""
    rng = np.random.default_rng(pairs)
    order = rng.permutation(pages)
    p = Pair(start(pages, 1, 1, 16, [], page_bytes=16, pools=2))
    src, dst = order[:pairs].copy(), order[pairs:2 * pairs].copy()
    src[5] = dst[5]                                 # the same page: nothing to do
    src[7] = src[8]                                 # one source, two targets
    assert p.do("copy_pages", src, dst) == 0
    p.same()
    for a, b, code in ((src, np.append(dst[:-1], dst[0]), INVALID_ARG),
                       (np.append(src[:-1], dst[0]), dst, INVALID_ARG),
                       (np.append(src[:-1], pages), dst, PAGE_OOB),
                       (src, np.append(dst[:-1], -1), PAGE_OOB)):
        assert p.do("copy_pages", a, b) == code
        p.same()
