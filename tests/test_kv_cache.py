"""Page ownership of the paged cache: fork, resize, copy and compact.

The GPU tests compare tables, lengths, holders and every pool's bytes with the
plain model in kv_model.py; everything is a whole number, so equality is exact.
Refusals of host arguments and the model itself are checked without a GPU."""
import ctypes

import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
from kv_model import INVALID_ARG, NO_PAGES, PAGE_OOB, KvModel, Refused

gpu = pytest.mark.gpu


def start(pages, seqs, width, P, lens, seed=0, page_bytes=64, pools=3):
    """A model with `lens` tokens in shuffled pages."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(pages)
    tables = np.full((seqs, width), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    L = np.zeros(seqs, np.int32)
    at = 0
    for i, n in enumerate(lens):
        k = -(-n // P)
        tables[i, :k] = order[at:at + k]
        refs[order[at:at + k]] += 1
        L[i] = n
        at += k
    pool = rng.integers(0, 256, (pools, pages, page_bytes), dtype=np.uint8)
    return KvModel(pool, tables, L, refs, P)


def sound(m):
    """Holders equal the table rows that hold each page."""
    count = np.zeros(len(m.refs), np.int32)
    for i, L in enumerate(m.lens):
        used = m.used(L)
        np.add.at(count, m.tables[i, :used], 1)
        assert (m.tables[i, used:] == -1).all()
    assert (count == m.refs).all()


# ------------------------------------------------------------------------- without a GPU


def test_model_fork_shares_full_pages_and_copies_the_partial_one():
    m = start(10, 3, 4, 4, [10])
    row = m.tables[0].copy()
    content = m.pool[:, row[2]].copy()
    m.fork([0, 0], [1, 2])
    sound(m)
    assert (m.tables[1, :2] == row[:2]).all() and (m.tables[2, :2] == row[:2]).all()
    last = [m.tables[i, 2] for i in range(3)]
    assert len(set(last)) == 3
    for p in last:
        assert (m.pool[:, p] == content).all()
    m.resize([0, 1, 2], [0, 0, 0])
    sound(m)
    assert not m.refs.any()


def test_model_copies_a_shared_partial_page_before_it_grows():
    m = start(10, 2, 4, 4, [8])
    m.fork([0], [1])
    m.resize([1], [6])           # ends inside a page that sequence 0 holds too
    m.resize([1], [7])
    sound(m)
    assert m.tables[1, 1] != m.tables[0, 1]


def desc(**over):
    pools = (ctypes.c_void_p * 2)(0x10000, 0x20000)
    a = dict(n_pools=2, num_pages=8, page_size=16, n_seqs=4, max_pages_per_seq=8, page_bytes=64,
             pools=pools, page_tables=0x1000, seq_lens=0x2000, page_refs=0x3000)
    a.update(over)
    return mk.mk_kv_desc(*[a[f[0]] for f in mk.mk_kv_desc._fields_])


@pytest.mark.parametrize("over, code", [
    (dict(n_pools=0), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(n_seqs=0), 1),
    (dict(max_pages_per_seq=0), 1), (dict(page_bytes=24), 1), (dict(page_bytes=0), 1),
    (dict(pools=None), 1), (dict(pools=(ctypes.c_void_p * 2)(0x10000, 0x20008)), 1),
    (dict(pools=(ctypes.c_void_p * 2)(0x10000, None)), 1), (dict(page_tables=None), 1),
    (dict(seq_lens=0x2002), 1), (dict(page_refs=None), 1),
    (dict(n_pools=513), 8), (dict(num_pages=(1 << 21) + 1), 8), (dict(n_seqs=65537), 8),
    (dict(page_size=1 << 20, max_pages_per_seq=1 << 12), 8)])
def test_create_refuses(over, code):
    h = ctypes.c_void_p()
    d = desc(**over)
    assert mk.lib().mk_kv_create(ctypes.byref(d), None, ctypes.byref(h)) == code
    assert not h.value


def test_null_handles_are_refused():
    L = mk.lib()
    for call in (L.mk_kv_copy_pages, L.mk_kv_fork, L.mk_kv_resize):
        assert call(None, 1, 0x1000, 0x1000) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_compact(None, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_sync(None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_create(None, None, None) == mk.MK_ERR_INVALID_ARG
    L.mk_kv_destroy(None)
    assert mk.status_string(mk.MK_ERR_NO_PAGES) not in ("", "unknown status")


# ------------------------------------------------------------------------------ on a GPU


class Pair:
    """The library's cache and the model, side by side."""

    def __init__(self, model, stream=None):
        import torch

        self.t, self.m = torch, model
        self.pools = [torch.from_numpy(p.copy()).cuda() for p in model.pool]
        self.tables = torch.from_numpy(model.tables.copy()).cuda()
        self.lens = torch.from_numpy(model.lens.copy()).cuda()
        self.refs = torch.from_numpy(model.refs.copy()).cuda()
        torch.cuda.synchronize()
        self.cache = mk.KvCache(self.pools, self.tables, self.lens, self.refs, model.P, stream)

    def i32(self, v):
        return self.t.tensor(np.asarray(v, np.int32), device="cuda")

    def do(self, name, a, b):
        """Runs a call on both sides; a refusal has to be the same on both."""
        code = 0
        try:
            getattr(self.m, name)(a, b)
        except Refused as r:
            code = r.code
        getattr(self.cache, name)(self.i32(a), self.i32(b))
        if code:
            with pytest.raises(mk.MkError) as e:
                self.cache.sync()
            assert e.value.code == code
        return code

    def same(self):
        self.cache.sync()
        assert (self.lens.cpu().numpy() == self.m.lens).all()
        assert (self.tables.cpu().numpy() == self.m.tables).all()
        assert (self.refs.cpu().numpy() == self.m.refs).all()
        for got, want in zip(self.pools, self.m.pool):
            assert (got.cpu().numpy() == want).all()

    def compact(self, want_map=True):
        page_map = self.t.full_like(self.refs, -7) if want_map else None
        self.cache.compact(page_map)
        want = self.m.compact()
        if want_map:
            assert (page_map.cpu().numpy() == want).all()


@gpu
@pytest.mark.parametrize("page_bytes", [16, 48, 4096, 4112, 16384])
def test_copy_pages(page_bytes):
    p = Pair(start(40, 1, 1, 16, [], page_bytes=page_bytes, pools=5))
    p.do("copy_pages", [3, 3, 9, 20], [0, 39, 9, 21])
    p.same()
    p.do("copy_pages", [7], [8])
    p.same()


@gpu
@pytest.mark.parametrize("P, lens", [(1, [5]), (4, [0]), (4, [4]), (4, [7]), (16, [1]), (16, [160]),
                                     (16, [4097]), (7, [30, 0, 14, 1])])
def test_fork_one_to_many(P, lens):
    n = len(lens)
    p = Pair(start(600, n + 5, -(-max(lens + [1]) // P) + 1, P, lens))
    p.do("fork", [0] * 5, list(range(n, n + 5)))
    p.same()
    # again onto the same rows: what they held is released first
    p.do("fork", [n - 1] * 5, list(range(n, n + 5)))
    p.same()
    sound(p.m)


@gpu
def test_fork_permutes_beams():
    p = Pair(start(200, 6, 9, 16, [70, 64, 33, 128, 1, 16]))
    p.do("fork", [1, 2, 0, 3, 0, 4], [0, 1, 2, 3, 4, 5])
    p.same()
    p.do("fork", [5, 5, 5, 5, 5, 5], [0, 1, 2, 3, 4, 5])
    p.same()
    sound(p.m)


@gpu
def test_resize_grows_shrinks_and_copies_on_write():
    p = Pair(start(300, 5, 20, 16, [70, 64, 33, 0, 1]))
    p.do("resize", [0, 1, 2, 3, 4], [71, 65, 0, 300, 320])
    p.same()
    p.do("fork", [4], [2])
    p.do("resize", [2, 4], [37, 37])     # both end inside a page that both hold
    p.same()
    p.do("resize", [4, 2], [38, 60])     # both take a copy, the page gets free
    p.same()
    p.do("resize", [0, 1, 2, 3, 4], [0] * 5)
    p.same()
    assert not p.m.refs.any()


@gpu
@pytest.mark.parametrize("seed", range(5))
def test_random_traffic(seed):
    rng = np.random.default_rng(100 + seed)
    P, S, W, N = [(16, 12, 30, 150), (4, 40, 200, 1500), (1, 3, 64, 100), (32, 70, 6, 5000),
                  (16, 12, 30, 60)][seed]
    p = Pair(start(N, S, W, P, [], seed, page_bytes=[128, 16, 4112, 48, 32][seed]))
    refused = 0
    for step in range(60):
        kind = rng.integers(0, 10)
        n = int(rng.integers(1, S + 1))
        rows = rng.permutation(S)[:n]
        if kind < 5:
            refused += p.do("resize", rows, rng.integers(0, W * P + 1, n) // (1 + rng.integers(0, 6))) != 0
        elif kind < 9:
            refused += p.do("fork", rng.integers(0, S, n), rows) != 0
        else:
            p.compact(step % 2 == 0)
        p.same()
        sound(p.m)
    assert seed != 4 or refused            # the small pool runs out on the way


@gpu
@pytest.mark.parametrize("pages, lens", [(1, [3]), (5000, [1, 17, 16 * 900, 40]), (37, [100, 0, 30]),
                                         (64, [16 * 64])])
def test_compact(pages, lens):
    p = Pair(start(pages, len(lens) + 1, 1000, 16, lens, seed=3))
    p.compact()
    p.same()
    held = int((p.m.refs > 0).sum())
    assert (p.m.refs[:held] > 0).all()
    p.compact(False)                       # nothing left to move
    p.same()


@gpu
def test_compact_moves_pages_that_others_hold():
    m = start(50, 2, 4, 16, [30])
    m.refs[40] += 2                        # a holder outside the tables
    p = Pair(m)
    p.compact()
    p.same()


@gpu
@pytest.mark.parametrize("name, a, b, code", [
    ("copy_pages", [0, 1], [5, 5], INVALID_ARG), ("copy_pages", [0, 1], [1, 6], INVALID_ARG),
    ("copy_pages", [0], [50], PAGE_OOB), ("copy_pages", [-1], [3], PAGE_OOB),
    ("fork", [0, 0], [2, 2], INVALID_ARG), ("fork", [0], [4], INVALID_ARG),
    ("fork", [-1], [2], INVALID_ARG), ("resize", [1, 1], [5, 6], INVALID_ARG),
    ("resize", [4], [5], INVALID_ARG), ("resize", [1], [-1], PAGE_OOB),
    ("resize", [1], [16 * 40 + 1], PAGE_OOB), ("resize", [2, 3], [640, 640], NO_PAGES)])
def test_refused_on_the_device(name, a, b, code):
    p = Pair(start(50, 4, 40, 16, [40, 100, 0, 0]))
    assert p.do(name, a, b) == code
    p.same()
    p.do("resize", [2], [33])              # the status was taken: calls work again
    p.same()


@gpu
def test_out_of_pages_for_a_fork_changes_nothing():
    p = Pair(start(3, 4, 4, 16, [40]))
    assert p.do("fork", [0], [1]) == NO_PAGES
    p.same()


@gpu
@pytest.mark.parametrize("entry", [-1, 50, 49, 2 ** 30])
def test_table_entries_are_checked(entry):
    m = start(50, 3, 4, 16, [40])
    m.refs[49] = 0 if 49 not in m.tables[0, :3] else m.refs[49]
    if 49 in m.tables[0, :3]:
        pytest.skip("page 49 is held in this draw")
    m.tables[0, 1] = entry
    for call in ("fork", "resize", "compact"):
        p = Pair(m)
        if call == "compact":
            p.cache.compact()
            with pytest.raises(mk.MkError) as e:
                p.cache.sync()
            assert e.value.code == PAGE_OOB
        else:
            a, b = ([0], [1]) if call == "fork" else ([0], [0])
            assert p.do(call, a, b) == PAGE_OOB
        p.same()


@gpu
def test_calls_behind_a_refused_one_change_nothing_until_sync():
    p = Pair(start(50, 4, 40, 16, [40]))
    p.cache.resize(p.i32([1]), p.i32([-5]))
    p.cache.resize(p.i32([1]), p.i32([64]))
    p.cache.fork(p.i32([0]), p.i32([2]))
    p.cache.copy_pages(p.i32([0]), p.i32([1]))
    p.cache.compact()
    with pytest.raises(mk.MkError) as e:
        p.cache.sync()
    assert e.value.code == PAGE_OOB
    p.same()


@gpu
def test_host_arguments_are_checked():
    import torch

    p = Pair(start(50, 4, 40, 16, [40]))
    one, two = p.i32([0]), p.i32([1, 2])
    with pytest.raises(ValueError):
        p.cache.fork(one, two)
    with pytest.raises(TypeError):
        p.cache.fork(one.long(), one)
    with pytest.raises(ValueError):
        p.cache.fork(one.cpu(), one)
    with pytest.raises(ValueError):
        p.cache.resize(p.i32([0, 1, 2, 3])[::2], two)
    with pytest.raises(mk.MkError):
        p.cache.fork(p.i32([0] * 5), p.i32([0, 1, 2, 3, 0]))   # more than there are sequences
    with pytest.raises(ValueError):
        p.cache.compact(torch.zeros(3, dtype=torch.int32, device="cuda"))
    p.cache.fork(p.i32([]), p.i32([]))                         # nothing to do
    p.same()


@gpu
def test_on_a_stream_and_replayed_from_a_graph():
    import torch

    st = torch.cuda.Stream()
    p = Pair(start(400, 8, 40, 16, [200, 100]), stream=st)
    src, dst = p.i32([0, 0, 1]), p.i32([2, 3, 4])
    seqs, lens = p.i32([0, 1, 2, 3, 4]), p.i32([210, 101, 240, 201, 16])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        p.cache.fork(src, dst)
        p.cache.resize(seqs, lens)
    torch.cuda.synchronize()
    p.same()                                # capturing ran nothing
    for new in ([210, 101, 240, 201, 16], [300, 5, 0, 640, 17]):
        with torch.cuda.stream(st):
            lens.copy_(p.i32(new))
            g.replay()
        st.synchronize()
        p.m.fork([0, 0, 1], [2, 3, 4])
        p.m.resize([0, 1, 2, 3, 4], new)
        p.same()


@gpu
def test_two_caches_of_one_shape_do_not_share_a_workspace():
    import torch

    a, b = (Pair(start(400, 8, 40, 16, [200, 100], seed=s), stream=torch.cuda.Stream()) for s in (1, 2))
    for step in range(20):
        for p in (a, b):
            p.do("fork", [step % 2, 1 - step % 2], [2 + step % 3, 5])
            p.do("resize", [2 + step % 3, 0], [150 + step, 200 + step])
    a.same()
    b.same()


@gpu
def test_holders_behind_two_billion_bytes():
    """Pools whose later pages lie past 2^32 bytes."""
    import torch

    pages, size = 70000, 65536                # 4.6 GB a pool
    pool = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    pool[69998] = 7
    pool[3] = 9
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = mk.KvCache([pool], torch.full((1, 1), -1, **i32), torch.zeros(1, **i32),
                       torch.zeros(pages, **i32), 16)
    cache.copy_pages(torch.tensor([69998, 3], **i32), torch.tensor([2, 69999], **i32))
    cache.sync()
    assert bool((pool[2] == 7).all()) and bool((pool[69999] == 9).all())
