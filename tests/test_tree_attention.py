"""Attention for drafted trees (mk_tree_attention) against its definition in 64 bits.

The arithmetic is that of mk_prefix_attention over the keys that a token sees, so the bounds are
those of test_prefix_attention.py, whose batches these are."""
import ctypes
import math

import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
from test_prefix_attention import Case

gpu = pytest.mark.gpu


def random_parents(rng, n, near=4, roots=0.05):
    return [-1 if i == 0 or rng.random() < roots else int(rng.integers(max(0, i - near), i)) for i in range(n)]


class Tree(Case):
    """bits: "tree" (each sequence's tokens form a random tree), or a function (rng, T) -> [T][T]."""

    def __init__(self, groups, *how, bits="tree", words=None, junk=False, **more):
        super().__init__(groups, *how, **more)
        rng = np.random.default_rng(more.get("seed", 0) + 17)
        words = words or max(1, -(-max(self.T + [1]) // 32))
        full = rng.integers(0, 2, (self.n_tokens, words * 32)) if junk else np.zeros((self.n_tokens, words * 32), int)
        self.seen = []
        for b, T in enumerate(self.T):
            if bits == "tree":
                parents = random_parents(rng, T, near=int(rng.choice([1, 3, max(1, T)])))
                m = np.zeros((T, T), int)
                for i, p in enumerate(parents):
                    if p >= 0:
                        m[i] = m[p]
                    m[i, i] = 1
            else:
                m = np.asarray(bits(rng, T), int)
            rows = full[self.off[b]:self.off[b + 1]]
            lower = np.tril(np.ones((T, T), int))
            # what lies above the diagonal does not count: junk there, and behind the T bits
            rows[:, :T] = np.where(lower, m, rows[:, :T])
            self.seen.append(m * lower)
        self.tree = np.packbits(full.astype(np.uint8), axis=1, bitorder="little").view(np.int32).copy()

    def exact(self):
        G = self.Hq // self.Hkv
        k, v, q = (x.double().numpy() for x in (self.k, self.v, self.q))
        out = np.zeros((self.n_tokens, self.Hq, self.D))
        A, lse = np.zeros_like(out), np.full((self.n_tokens, self.Hq), -np.inf)
        E = np.zeros((self.n_tokens, self.Hq))
        scale = self.scale or 1.0 / math.sqrt(self.D)
        for b, L in enumerate(self.lens):
            K = k[self.rows[b]].transpose(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, :L]
            V = v[self.rows[b]].transpose(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, :L]
            T = self.T[b]
            for t in range(T):
                at = np.array([p for p in range(L) if p < L - T or self.seen[b][t, p - L + T]], int)
                if not len(at):
                    continue
                row = int(self.off[b]) + t
                for h in range(self.Hq):
                    s = K[h // G, at] @ q[row, h] * scale
                    m = s.max()
                    p = np.exp(s - m)
                    out[row, h] = p @ V[h // G, at] / p.sum()
                    A[row, h] = p @ np.abs(V[h // G, at]) / p.sum()
                    lse[row, h] = m + math.log(p.sum())
                    E[row, h] = (np.abs(K[h // G, at]) @ np.abs(q[row, h])).max() * scale * self.D * 2.0 ** -23
        return out, lse, A, E

    def run(self, d=None, **how):
        t = self.t
        d = d or self.device()
        a, b = self.attention(d, **how)
        out = t.full(d["q"].shape, 123.0, dtype=t.bfloat16, device="cuda")
        lse = t.full(d["q"].shape[:2], 123.0, dtype=t.float32, device="cuda")
        a.run(0, b, d["q"], out, lse, tree=d.get("tree", t.from_numpy(self.tree).cuda()))
        a.sync()
        a.close()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()


HEADS = [(2, 2, 64), (6, 2, 32), (16, 4, 64), (32, 4, 128), (3, 1, 128), (64, 1, 32)]


@gpu
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("P", [16, 48, 64])
def test_heads_and_page_sizes(heads, P):
    """Trees of several sizes, with contexts that end inside pages and at their ends."""
    Tree([(0, [(2 * P + 5, 5), (40, 40), (100, 17), (P, 1), (70, 33)])], heads, P).check(grouped=False)


@gpu
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("context", [0, 5, 127, 128, 140])
def test_sizes_of_one_tree(T, context):
    """The tree's words against the tiles of 128 keys at every offset that matters."""
    Tree([(0, [(context + T, T)])], (8, 2, 64), seed=T + context).check()


@gpu
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 2, 128), (6, 2, 32)])
def test_trees_behind_a_shared_prefix(heads):
    Tree([(160, [(24, 24), (9, 7), (70, 64), (33, 1)]), (0, [(20, 4)]), (33, [(50, 12), (12, 12)])], heads).check()
    c = Tree([(160, [(24, 24), (9, 7), (70, 64), (33, 1)])], heads)
    c.check(grouped=False)


@gpu
def test_trees_that_reach_into_the_shared_pages():
    """More tokens than the sequence has of its own."""
    Tree([(64, [(2, 10), (5, 30), (1, 1)]), (32, [(0, 32), (0, 1)])], (4, 2, 64)).check()


@gpu
@pytest.mark.parametrize("heads", [(4, 2, 64), (32, 4, 128)])
@pytest.mark.parametrize("junk", [False, True])
def test_any_bits(heads, junk):
    """Random bits: rows that do not see themselves, rows without a bit; what lies above the
    diagonal and behind the tokens does not count."""
    some = lambda r, T: r.integers(0, 2, (T, T)) * (r.random((T, 1)) < 0.7)
    Tree([(0, [(90, 40), (33, 33), (300, 129), (20, 1)])], heads, bits=some, words=9, junk=junk).check()


@gpu
def test_rows_that_see_nothing():
    """No context and no bit, beside others; more tokens than the sequence; empty sequences."""
    none = lambda r, T: np.zeros((T, T))
    Tree([(0, [(12, 12), (40, 8), (0, 3), (5, 5)])], (4, 2, 64), bits=none, extra_rows=3).check()
    some = lambda r, T: np.eye(T) * (np.arange(T) % 3 > 0)[:, None]
    Tree([(0, [(150, 150), (4, 9), (16, 16)])], (8, 1, 64), bits=some).check()
    Tree([(0, [(0, 1), (3, 9), (0, 0), (40, 2)])], (4, 2, 64), extra_rows=7).check()


@gpu
@pytest.mark.parametrize("heads", [(4, 2, 64), (32, 4, 128), (6, 2, 32)])
def test_all_bits_are_the_plain_call(heads):
    """Bit for bit: each token sees all before it."""
    c = Tree([(300, [(90, 40), (33, 33), (200, 129), (1, 1)]), (0, [(700, 5)])], heads,
             bits=lambda r, T: np.ones((T, T)), words=6, junk=True)
    out, lse = c.run()
    plain, plain_lse = Case.run(c)
    assert np.array_equal(out, plain) and np.array_equal(lse, plain_lse)
    again = c.run()
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


@gpu
def test_single_tokens_and_rows_behind_them():
    """One token a sequence without offsets; its bit says whether it sees itself."""
    c = Tree([(64, [(9, 1), (100, 1), (17, 1)])], (16, 2, 64), bits=lambda r, T: [[r.integers(0, 2)]], seed=2)
    want = c.exact()
    c.check(want=want, offsets=False)
    c.check(want=want, offsets=True)
    Tree([(48, [(5, 1), (9, 6)])], (4, 2, 64), extra_rows=70).check()


@gpu
def test_what_lies_behind_a_length_does_not_matter():
    c = Tree([(40, [(9, 3), (100, 50)]), (0, [(5, 3), (33, 33)])], (4, 2, 64))
    want = c.exact()
    used = np.zeros(c.k.shape[0], bool)
    for r in c.rows:
        used[r] = True
    for x, bad in ((c.k, float("nan")), (c.v, float("inf"))):
        x[~used] = bad
        for b, L in enumerate(c.lens):
            if L % 16:
                x[c.rows[b][L // 16], :, L % 16:] = bad
    c.tables[c.tables < 0] = 2 ** 30
    c.check(want=want)


def hiding(rng, T):
    """Any bits, and tokens that none sees."""
    m = np.tril(rng.random((T, T)) < 0.7)
    m[:, rng.random(T) < 0.3] = 0
    return m


SPOILT = [([(0, [(90, 40), (33, 33), (300, 129), (20, 1)])], heads) for heads in HEADS] + [
    ([(304, [(90, 40), (33, 33), (200, 129), (1, 1)]), (0, [(700, 5)])], (32, 4, 128)),   # behind shared pages
    ([(0, [(9000, 50)]), (2000, [(50, 20), (40, 20)])], (16, 2, 64)),                     # cut over the SMs
    ([(0, [(400, 150), (700, 170)])], (8, 8, 32)),                                        # many blocks of the join
    ([(0, [(12, 12), (150, 150), (4, 9), (0, 3), (16, 16)])], (4, 2, 64))]                # no context, no place


@gpu
@pytest.mark.parametrize("groups, heads", SPOILT)
def test_what_lies_at_hidden_tokens_does_not_matter(groups, heads):
    """K and V of tokens that no row sees are infinite or NaN, in some columns or all."""
    c = Tree(groups, heads, bits=hiding, words=6, seed=5)
    want, rng, n = c.exact(), np.random.default_rng(6), 0
    for b, (L, T) in enumerate(zip(c.lens, c.T)):
        for u in range(T):
            place = L - T + u
            if place < 0 or c.seen[b][:, u].any():
                continue
            page, slot, n = c.rows[b][place // 16], place % 16, n + 1
            c.k[page, :, slot] = float(rng.choice([np.nan, np.inf]))
            columns = rng.random(c.D) < rng.choice([0.05, 0.5, 1.0])
            c.v[page, :, slot, c.t.from_numpy(columns)] = float(rng.choice([np.nan, np.inf, -np.inf]))
    assert n > 0
    c.check(want=want)
    first, again = c.run(), c.run()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@gpu
@pytest.mark.parametrize("groups, heads", SPOILT[1:5] + SPOILT[6:9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_spoilt_token_stays_in_its_branch(groups, heads, bad):
    """A column of V of one drafted token in three: rows that see it have no number there, all else is as before."""
    c = Tree(groups, heads, seed=7)
    want, (out, lse) = c.exact(), c.run()
    spoilt, column = np.zeros(out.shape[0], bool), c.D // 3
    for b, (L, T) in enumerate(zip(c.lens, c.T)):
        for u in range(1, T, 3):
            place = L - T + u
            c.v[c.rows[b][place // 16], :, place % 16, column] = bad
            spoilt[c.off[b]:c.off[b + 1]] |= c.seen[b][:, u].astype(bool)
    assert spoilt.any() and not spoilt.all()
    got, got_lse = c.run()
    assert np.array_equal(got_lse, lse)
    rest = np.arange(c.D) != column
    assert np.array_equal(got[..., rest], out[..., rest])
    assert not np.isfinite(got[spoilt][..., column]).any()
    got[spoilt, :, column] = out[spoilt, :, column]
    c.check(got=(got, got_lse), want=want)


@gpu
def test_rising_scores_among_the_tokens():
    """The last keys, which the tree hides from most rows, have the largest scores."""
    c = Tree([(0, [(500, 200)])], (16, 2, 64), scale=1.0)
    c.q[:] = 1.0
    n = len(c.rows[0]) * 16
    ramp = c.t.linspace(0.0, 6.0, n).view(-1, 1, 16, 1).expand(-1, 2, 16, 64)
    c.k[c.rows[0]] = (ramp + 0.1 * c.k[c.rows[0]].float()).to(c.t.bfloat16)
    c.check()


@gpu
def test_long_contexts_cut_over_the_sms():
    Tree([(0, [(9000, 48), (5000, 64)])], (8, 1, 128)).check(grouped=False)


@gpu
@pytest.mark.parametrize("seed", range(8))
def test_random_batches(seed):
    rng = np.random.default_rng(seed)
    groups = []
    for _ in range(int(rng.integers(1, 4))):
        seqs = []
        for _ in range(int(rng.integers(1, 7))):
            T = int(rng.choice([0, 1, 3, 16, 40, 90]))
            seqs.append((T + int(rng.integers(0, 200)), T))
        groups.append((int(rng.integers(0, 400)), seqs))
    heads = [(2, 2, 64), (6, 2, 32), (16, 4, 64), (16, 2, 128)][seed % 4]
    Tree(groups, heads, P=int(rng.choice([16, 32, 64])), seed=seed, extra_rows=int(rng.integers(0, 4))).check()


# ---- what is refused, and calls in captured graphs


def test_null_handles_and_words():
    L, b = mk.lib(), mk.mk_attn_batch(1, 1, 0, 1, 16, 16, None, None, None)
    for handle, words, tree in ((None, 1, 16), (None, 0, 16), (None, 1 << 16, 16), (None, 1, 18), (None, 1, None)):
        assert L.mk_tree_attention(handle, 0, ctypes.byref(b), tree, words, 16, 64, 16, None) == mk.MK_ERR_INVALID_ARG


def test_tree_rows():
    tree, depths = mk.tree_rows([[-1, 0, 0, 1, -1], [], [-1] + list(range(39))])
    assert tree.shape == (45, 2) and depths.tolist()[:5] == [0, 1, 1, 2, 0]
    assert tree[:5].tolist() == [[1, 0], [3, 0], [5, 0], [11, 0], [16, 0]]
    assert depths[-1] == 39 and tree[-1].tolist() == [-1, 255]
    for bad in ([[0]], [[-1, 1]], [[-1, -2]]):
        with pytest.raises(ValueError):
            mk.tree_rows(bad)
    assert mk.tree_rows([])[0].shape == (0, 1)


@gpu
def test_longer_trees_than_their_rows_write_nothing():
    c = Tree([(0, [(90, 33), (20, 5)])], (4, 2, 64))
    t, d = c.t, c.device()
    a, b = c.attention(d)
    out = t.full(d["q"].shape, 123.0, dtype=t.bfloat16, device="cuda")
    narrow = t.from_numpy(c.tree[:, :1].copy()).cuda()
    a.run(0, b, d["q"], out, tree=narrow)
    with pytest.raises(mk.MkError) as e:
        a.sync()
    assert e.value.code == mk.MK_ERR_INVALID_ARG and (out == 123.0).all()
    lse = t.empty(d["q"].shape[:2], device="cuda")
    a.run(0, b, d["q"], out, lse, tree=t.from_numpy(c.tree).cuda())
    a.sync()
    c.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))


@gpu
def test_wrong_trees_are_refused():
    c = Tree([(0, [(90, 33), (20, 5)])], (4, 2, 64))
    t, d = c.t, c.device()
    a, b = c.attention(d)
    tree, out = t.from_numpy(c.tree).cuda(), t.zeros_like(d["q"])
    for bad, error in ((tree.long(), TypeError), (tree[:-1], ValueError), (tree.t().contiguous().t(), ValueError),
                       (tree.cpu(), ValueError), (tree[0], ValueError)):
        with pytest.raises(error):
            a.run(0, b, d["q"], out, tree=bad)
    over = out.view(t.int32).view(-1)[:tree.numel()].view(tree.shape)
    with pytest.raises(mk.MkError):
        a.run(0, b, d["q"], out, tree=over)
    lse = t.zeros(d["q"].shape[:2], device="cuda")
    with pytest.raises(mk.MkError):
        a.run(0, b, d["q"], out, lse, tree=lse.view(t.int32).view(-1)[:tree.numel()].view(tree.shape))
    a.sync()
    assert (out == 0).all()


@gpu
def test_a_captured_call_follows_its_tree():
    c = Tree([(100, [(24, 24), (9, 9)]), (0, [(70, 33)])], (16, 2, 64))
    other = Tree([(100, [(24, 24), (9, 9)]), (0, [(70, 33)])], (16, 2, 64), bits=lambda r, T: r.integers(0, 2, (T, T)))
    t = c.t
    stream = t.cuda.Stream()
    with t.cuda.stream(stream):
        d = c.device()
        a, b = c.attention(d, stream=stream)
        tree, out = t.from_numpy(c.tree).cuda(), t.empty_like(d["q"])
        lse = t.empty(d["q"].shape[:2], device="cuda")
        a.run(0, b, d["q"], out, lse, tree=tree)
        stream.synchronize()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=stream):
            a.run(0, b, d["q"], out, lse, tree=tree)
        for x in (other, c):
            tree.copy_(t.from_numpy(x.tree))
            graph.replay()
            a.sync()
            x.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))
