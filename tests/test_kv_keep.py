"""Picked tokens of a sequence move together (mk_kv_keep), against a plain model, bit for bit."""
import ctypes

import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
from kv_model import INVALID_ARG, PAGE_OOB, KvModel, Refused
from test_kv_cache import Pair, start

gpu = pytest.mark.gpu


def keep(m, seqs, starts, offsets, picks, heads):
    """The call's definition on a KvModel, one token at a time.  Raises Refused."""
    n = len(seqs)
    ok = all(0 <= s < len(m.lens) for s in seqs) and len(set(map(int, seqs))) == n
    ok = ok and offsets[0] == 0 and offsets[-1] <= len(picks) and all(a <= b for a, b in zip(offsets, offsets[1:]))
    if not ok:
        raise Refused(INVALID_ARG)
    codes, moves = [], []
    for i, s in enumerate(seqs):
        mine = [int(p) for p in picks[offsets[i]:offsets[i + 1]]]
        for j, p in enumerate(mine):
            if p <= (mine[j - 1] if j else -1):
                codes.append(INVALID_ARG)
            elif starts[i] < 0 or m.lens[s] > m.cap or starts[i] + p >= m.lens[s]:
                codes.append(PAGE_OOB)
            elif p >= j:
                src, dst = int(starts[i]) + p, int(starts[i]) + j
                rows = [int(m.tables[s, x // m.P]) for x in (src, dst)]
                if any(not 0 <= r < len(m.refs) or m.refs[r] < 1 for r in rows):
                    codes.append(PAGE_OOB)
                elif m.refs[rows[1]] > 1 and p != j:
                    codes.append(INVALID_ARG)
                else:
                    moves.append((rows[0], src % m.P, rows[1], dst % m.P))
    if codes:
        raise Refused(max(codes))
    pools, pages, size = m.pool.shape
    view = m.pool.reshape(pools, pages, heads, m.P, size // heads // m.P)
    old = view.copy()
    for sp, ss, dp, ds in moves:
        view[:, dp, :, ds] = old[:, sp, :, ss]


class Both(Pair):
    def keep(self, seqs, starts, offsets, picks, heads):
        code = 0
        try:
            keep(self.m, seqs, starts, offsets, picks, heads)
        except Refused as e:
            code = e.code
        self.cache.keep(self.i32(seqs), self.i32(starts), self.i32(offsets), self.i32(picks), heads)
        try:
            self.cache.sync()
            got = 0
        except mk.MkError as e:
            got = e.code
        assert got == code
        self.same()
        return code

    def same(self):
        for p, want in zip(self.pools, self.m.pool):
            assert np.array_equal(p.cpu().numpy(), want)
        for t, want in ((self.tables, self.m.tables), (self.lens, self.m.lens), (self.refs, self.m.refs)):
            assert np.array_equal(t.cpu().numpy(), want)


def both(pages, seqs, width, P, lens, heads=2, row=32, pools=3, seed=0):
    return Both(start(pages, seqs, width, P, lens, seed, heads * P * row, pools))


def random_picks(rng, n, drafted, most):
    offsets, picks = [0], []
    for i in range(n):
        k = int(rng.integers(0, min(most, drafted[i]) + 1))
        picks += sorted(rng.choice(drafted[i], k, replace=False).tolist())
        offsets.append(len(picks))
    return offsets, picks


# ------------------------------------------------------------------------- without a GPU


def test_model():
    m = start(6, 2, 3, 4, [10, 5], page_bytes=2 * 4 * 16)
    row = m.pool.reshape(3, 6, 2, 4, 16)
    at = lambda pos: row[:, m.tables[0, pos // 4], :, pos % 4].copy()
    want = [at(p) for p in (3, 5, 6, 9)]
    keep(m, [0], [3], [0, 4], [0, 2, 3, 6], 2)
    for pos, w in zip((3, 4, 5, 6), want):
        assert np.array_equal(at(pos), w)


def test_null_and_host_arguments():
    L = mk.lib()
    assert L.mk_kv_keep(None, 1, 0x1000, 0x1000, 0x1000, 1, 0x1000, 1) == mk.MK_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ on a GPU


@gpu
@pytest.mark.parametrize("P", [1, 3, 16])
@pytest.mark.parametrize("picks", [[0], [0, 1, 2], [0, 2, 3, 7], [5], [1, 2, 3, 4, 5, 6, 7], [],
                                   list(range(0, 30, 2)), list(range(3, 30))])
def test_one_sequence(P, picks):
    """Paths of every length against pages, some of whose tokens are sources and targets both."""
    for at in (0, 7, 16):
        b = both(60, 2, 50, P, [at + 30, 3])
        assert b.keep([0], [at], [0, len(picks)], picks, 2) == 0


@gpu
@pytest.mark.parametrize("heads, row, pools", [(1, 16, 1), (2, 64, 3), (4, 256, 16), (3, 48, 5), (8, 128, 2)])
def test_shapes_of_a_page(heads, row, pools):
    rng = np.random.default_rng(heads)
    lens = [60, 25, 44, 0, 33]
    b = both(40, 5, 8, 16, lens, heads, row, pools)
    drafted = [20, 5, 9, 0, 33]
    offsets, picks = random_picks(rng, 5, drafted, 9)
    assert b.keep([0, 1, 2, 3, 4], [L - d for L, d in zip(lens, drafted)], offsets, picks, heads) == 0
    # and in another order, some of them
    offsets, picks = random_picks(rng, 2, [33, 9], 33)
    assert b.keep([4, 2], [0, 35], offsets, picks, heads) == 0


@gpu
@pytest.mark.parametrize("n, most", [(1024, 2), (1025, 2), (128, 16), (300, 60), (2000, 40), (3, 900)])
def test_both_sides_of_the_single_kernel(n, most):
    """Up to 1024 sequences and 2048 picks in one kernel, more behind a plan."""
    rng = np.random.default_rng(n)
    drafted = [most] * n if most < 100 else [1000, 900, 40]
    lens = [int(rng.integers(0, 5)) + d for d in drafted]
    b = both(sum(-(-L // 16) for L in lens) + 3, n, 70, 16, lens, 1, 16, 2)
    seqs = rng.permutation(n)
    offsets, picks = [0], []
    for s in seqs:
        k = int(rng.integers(0, drafted[s] + 1))
        picks += sorted(rng.choice(drafted[s], k, replace=False).tolist())
        offsets.append(len(picks))
    assert b.keep(seqs, [lens[s] - drafted[s] for s in seqs], offsets, picks, 1) == 0


@gpu
def test_behind_a_fork_and_before_a_resize():
    """The round of a drafter: grow, keep, set the next length; the shared prompt stays."""
    b = both(80, 4, 20, 16, [37], 2, 32, 4)
    b.do("fork", [0, 0, 0], [1, 2, 3])
    rng = np.random.default_rng(5)
    for _ in range(6):
        lens = b.m.lens.copy()
        b.do("resize", [0, 1, 2, 3], lens + 12)
        offsets, picks = random_picks(rng, 4, [12] * 4, 5)
        assert b.keep([0, 1, 2, 3], lens, offsets, picks, 2) == 0
        b.do("resize", [0, 1, 2, 3], lens + np.diff(offsets))
    b.same()


WRONG = [
    (([0, 9], [4, 4], [0, 1, 2], [0, 1]), INVALID_ARG),          # no such sequence
    (([0, -1], [4, 4], [0, 1, 2], [0, 1]), INVALID_ARG),
    (([1, 1], [4, 4], [0, 1, 2], [0, 1]), INVALID_ARG),          # twice
    (([0, 1], [4, 4], [1, 1, 2], [0, 1]), INVALID_ARG),          # offsets
    (([0, 1], [4, 4], [0, 2, 1], [0, 1]), INVALID_ARG),
    (([0, 1], [4, 4], [0, 1, 3], [0, 1]), INVALID_ARG),
    (([0, 1], [4, 4], [0, -5, 2], [0, 1]), INVALID_ARG),
    (([0, 1], [4, 4], [0, 2, 4], [0, 3, 2, 2]), INVALID_ARG),    # picks that do not rise
    (([0, 1], [4, 4], [0, 2, 4], [5, 3, 0, 2]), INVALID_ARG),
    (([0, 1], [4, 4], [0, 2, 4], [-1, 3, 0, 2]), INVALID_ARG),
    (([0, 1], [4, 4], [0, 3, 4], [5, -3, 0, 2]), INVALID_ARG),
    (([0, 1], [4, -1], [0, 2, 4], [0, 3, 0, 2]), PAGE_OOB),      # places
    (([0, 1], [4, 4], [0, 2, 4], [0, 36, 0, 2]), PAGE_OOB),
    (([0, 1], [4, 2 ** 31 - 3], [0, 2, 4], [0, 3, 0, 2 ** 31 - 1]), PAGE_OOB),
    (([0, 2], [4, 0], [0, 2, 3], [0, 3, 0]), PAGE_OOB),          # an empty sequence
    (([0, 1], [4, -1], [0, 2, 4], [3, 3, 0, 2]), PAGE_OOB),      # the larger of two
]


@gpu
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("call, code", WRONG)
def test_refused_calls_change_nothing(many, call, code):
    """In one kernel and (with picks enough behind the last offset) behind a plan."""
    b = both(20, 4, 8, 16, [40, 40, 0, 20])
    seqs, starts, offsets, picks = call
    if many:
        if offsets[-1] > len(picks):
            offsets = offsets[:-1] + [5000]
        picks = picks + [0] * 3000
    assert b.keep(seqs, starts, offsets, picks, 2) == code
    assert b.keep([0, 3], [4, 0], [0, 2, 4], [0, 3, 1, 2], 2) == 0


@gpu
@pytest.mark.parametrize("many", [False, True])
def test_pages_of_other_holders_and_wild_entries(many):
    junk = [0] * 3000 if many else []
    b = both(20, 4, 8, 16, [40, 0, 0, 20])
    b.do("fork", [0], [1])
    # the first two pages are shared: what stays in place or moves within the last is fine
    assert b.keep([0], [30], [0, 1], [0] + junk, 2) == 0
    assert b.keep([0], [32], [0, 2], [1, 4] + junk, 2) == 0
    assert b.keep([1], [30], [0, 2], [0, 4] + junk, 2) == INVALID_ARG
    assert b.keep([1], [32], [0, 2], [0, 4] + junk, 2) == 0
    for bad in (-1, 20, 10 ** 6):
        b = both(20, 4, 8, 16, [40, 0, 0, 20])
        b.m.tables[0, 1] = bad
        b.tables.copy_(b.t.from_numpy(b.m.tables))
        assert b.keep([0, 3], [10, 0], [0, 2, 4], [0, 10, 1, 2] + junk, 2) == PAGE_OOB
        assert b.keep([3], [0], [0, 2], [1, 2] + junk, 2) == 0


@gpu
@pytest.mark.parametrize("many", [False, True])
def test_a_refused_call_holds_up_the_next(many):
    junk = [0] * 3000 if many else []
    b = both(20, 4, 8, 16, [40, 30, 0, 20])
    i = b.i32
    b.cache.fork(i([0, 9]), i([2, 3]))                           # refused
    b.cache.keep(i([0]), i([4]), i([0, 2]), i([1, 2] + junk), 2)
    with pytest.raises(mk.MkError):
        b.cache.sync()
    b.same()
    b.cache.keep(i([0]), i([4]), i([0, 2]), i([2, 2] + junk), 2)
    b.cache.resize(i([1]), i([0]))
    b.cache.keep(i([0]), i([4]), i([0, 2]), i([1, 2] + junk), 2)
    with pytest.raises(mk.MkError) as e:
        b.cache.sync()
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    b.same()


@gpu
def test_host_arguments():
    b = both(20, 4, 8, 16, [40, 30, 0, 20])
    i, c = b.i32, b.cache
    s, st, off, p = i([0]), i([4]), i([0, 2]), i([1, 2])
    for heads in (0, -1, 3, 4):                     # 4: rows of 16 bytes, which is fine
        if heads == 4:
            c.keep(s, st, off, p, heads)
            c.sync()
            continue
        with pytest.raises(mk.MkError) as e:
            c.keep(s, st, off, p, heads)
        assert e.value.code == mk.MK_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="n_kv_heads"):
        c.keep(s, st, off, p)
    for bad in ((s, i([4, 4]), off, p), (s, st, i([0]), p)):
        with pytest.raises(ValueError):
            c.keep(*bad, 2)
    for k in range(4):
        args = [s, st, off, p]
        args[k] = args[k].long()
        with pytest.raises(TypeError):
            c.keep(*args, 2)
    L = mk.lib()
    good = [c.handle, 1, s.data_ptr(), st.data_ptr(), off.data_ptr(), 2, p.data_ptr(), 2]
    for k, v in ((1, -1), (1, 5), (2, None), (3, None), (4, None), (5, -1), (6, None), (4, off.data_ptr() + 2)):
        assert L.mk_kv_keep(*(good[:k] + [v] + good[k + 1:])) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_keep(*(good[:1] + [0] + good[2:])) == mk.MK_OK
    c.sync()


@gpu
def test_four_dimensional_pools_name_their_heads():
    import torch

    k = torch.arange(6 * 2 * 16 * 32, device="cuda").to(torch.bfloat16).view(6, 2, 16, 32)
    want = k.clone()
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tables, lens, refs = t([3, 1, -1], [2, -1, -1]), t(20, 9), t(0, 1, 1, 1, 0, 0)
    c = mk.KvCache([k], tables, lens, refs, 16)
    c.keep(t(0), t(14), t(0, 3), t(1, 3, 5))
    c.sync()
    for to, fro in ((14, 15), (15, 17), (16, 19)):
        want[(3, 1)[to // 16], :, to % 16] = want[(3, 1)[fro // 16], :, fro % 16]
    assert torch.equal(k, want)


@gpu
def test_pages_behind_two_to_the_32():
    import torch

    pages = (1 << 32) // (2 * 16 * 128 * 2) + 900            # 8 KB a page
    pool = torch.zeros(pages, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tables, lens = t([pages - 1, pages - 800]), t(30)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[[pages - 1, pages - 800]] = 1
    rows = torch.randn(30, 2, 128, device="cuda").to(torch.bfloat16)
    for i in range(30):
        pool[(pages - 1, pages - 800)[i // 16], :, i % 16] = rows[i]
    c = mk.KvCache([pool], tables, lens, refs, 16)
    c.keep(t(0), t(10), t(0, 4), t(1, 4, 9, 19))
    c.sync()
    want = rows.clone()
    want[10:14] = rows[[11, 14, 19, 29]]
    for i in range(30):
        assert torch.equal(pool[(pages - 1, pages - 800)[i // 16], :, i % 16], want[i])


@gpu
def test_captured_calls_follow_their_tensors():
    import torch

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        m = start(30, 4, 8, 16, [40, 30, 0, 60], 0, 2 * 16 * 32, 3)
        b = Both(m, stream)
        args = [b.i32([0, 3]), b.i32([4, 40]), b.i32([0, 3, 5]), b.i32([1, 4, 9, 0, 19])]
        b.cache.keep(*args, 2)
        keep(m, [0, 3], [4, 40], [0, 3, 5], [1, 4, 9, 0, 19], 2)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            b.cache.keep(*args, 2)
        for seqs, starts, offsets, picks in (([1, 0], [0, 20], [0, 2, 5], [3, 20, 0, 7, 15]),
                                             ([3, 2], [1, 0], [0, 5, 5], [0, 1, 30, 31, 58])):
            for a, v in zip(args, (seqs, starts, offsets, picks)):
                a.copy_(b.i32(v))
            graph.replay()
            b.cache.sync()
            keep(m, seqs, starts, offsets, picks, 2)
            b.same()
