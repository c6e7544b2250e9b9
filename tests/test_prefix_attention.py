"""Attention over shared pages against its definition in 64 bits.

Tolerance, per element.  With u = 2^-8 (half a step of bf16 relative to the
value) and A = sum_j p_j |v_j| / sum_j p_j:

- the result is rounded to bf16: u |exact|;
- each probability is rounded to bf16 before the product with V: u A (calls with few
  results keep the rest of that rounding and are far better; the bound holds for all);
- a score is a sum of D products in 32 bits, off by at most
  E = 2^-23 D scale max_j sum_d |q_d k_jd| (2^-23: a chopped sum), which moves
  each probability by the factor e^E and the result by at most 2 E A;
- 2^-15 A covers second-order terms, the exponential (2^-22) and the 32-bit sums.

The logarithm of the sum moves by at most E, plus 2^-18 for the exponential, the
sum and the logarithm, plus its own rounding 2^-23 |lse|.
"""
import ctypes
import math

import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk

gpu = pytest.mark.gpu


class Case:
    """A paged batch: groups of (prefix tokens, [(own tokens, query tokens), ...])."""

    def __init__(self, groups, heads=(4, 2, 64), P=16, seed=0, spare=3, extra_rows=0, offsets=None,
                 scale=None):
        import torch

        self.t = torch
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D = heads
        self.P, self.scale = P, scale
        lens, self.T, self.prefix, starts, rows = [], [], [], [0], []
        count = sum(-(-(p + o) // P) for p, ss in groups for o, _ in ss) + sum(
            -(-p // P) for p, _ in groups) + spare
        order = [int(i) for i in rng.permutation(count)]
        for prefix, seqs in groups:
            shared = [order.pop() for _ in range(prefix // P)]
            for own, T in seqs:
                used = -(-(prefix + own) // P)
                rows.append(shared + [order.pop() for _ in range(used - len(shared))])
                lens.append(prefix + own)
                self.T.append(T)
            self.prefix.append(prefix)
            starts.append(len(lens))
        wide = max([len(r) for r in rows] + [1]) + 1
        self.rows, self.lens, self.starts = rows, lens, starts
        self.tables = np.array([r + [-1] * (wide - len(r)) for r in rows], np.int32)
        self.off = np.concatenate([[0], np.cumsum(self.T)]).astype(np.int32)
        self.n_tokens = int(self.off[-1]) + extra_rows
        shape = (count, self.Hkv, P, self.D)
        self.k = torch.randn(shape, generator=g).to(torch.bfloat16)
        self.v = torch.randn(shape, generator=g).to(torch.bfloat16)
        # a partly filled prefix page has the same contents in every sequence
        for gi, (prefix, _) in enumerate(groups):
            if prefix % P:
                j, n = prefix // P, prefix % P
                first = rows[starts[gi]][j]
                for b in range(starts[gi] + 1, starts[gi + 1]):
                    self.k[rows[b][j], :, :n] = self.k[first, :, :n]
                    self.v[rows[b][j], :, :n] = self.v[first, :, :n]
        self.q = (2.0 * torch.randn(self.n_tokens, self.Hq, self.D, generator=g)).to(torch.bfloat16)

    def single(self):
        return all(t == 1 for t in self.T) and self.n_tokens == len(self.T)

    def exact(self):
        """(out, lse, A, E) in 64 bits, one sequence, token and head at a time."""
        G = self.Hq // self.Hkv
        k, v, q = (x.double().numpy() for x in (self.k, self.v, self.q))
        out = np.zeros((self.n_tokens, self.Hq, self.D))
        A, lse = np.zeros_like(out), np.full((self.n_tokens, self.Hq), -np.inf)
        E = np.zeros((self.n_tokens, self.Hq))
        scale = self.scale or 1.0 / math.sqrt(self.D)
        for b, L in enumerate(self.lens):
            K = k[self.rows[b]].transpose(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, :L]
            V = v[self.rows[b]].transpose(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, :L]
            for t in range(self.T[b]):
                n = max(0, L - self.T[b] + t + 1)
                if n == 0:
                    continue
                row = int(self.off[b]) + t
                for h in range(self.Hq):
                    s = K[h // G, :n] @ q[row, h] * scale
                    m = s.max()
                    p = np.exp(s - m)
                    out[row, h] = p @ V[h // G, :n] / p.sum()
                    A[row, h] = p @ np.abs(V[h // G, :n]) / p.sum()
                    lse[row, h] = m + math.log(p.sum())
                    E[row, h] = (np.abs(K[h // G, :n]) @ np.abs(q[row, h])).max() * scale * self.D * 2.0 ** -23
        return out, lse, A, E

    def device(self, **over):
        t = self.t
        d = {"q": self.q.cuda(), "k": self.k.cuda(), "v": self.v.cuda(),
             "tables": t.from_numpy(self.tables.copy()).cuda(),
             "lens": t.tensor(self.lens, dtype=t.int32).cuda(),
             "off": t.from_numpy(self.off).cuda(),
             "starts": t.tensor(self.starts, dtype=t.int32).cuda(),
             "prefix": t.tensor(self.prefix, dtype=t.int32).cuda()}
        d.update(over)
        return d

    def attention(self, d, grouped=True, stream=None, offsets=None):
        a = mk.PrefixAttention(self.Hq, self.Hkv, self.D, self.P, [(d["k"], d["v"])],
                               max_tokens=max(1, self.n_tokens), scale=self.scale, stream=stream)
        with_offsets = (not self.single()) if offsets is None else offsets
        b = a.batch(d["tables"], d["lens"], q_offsets=d["off"] if with_offsets else None,
                    group_starts=d["starts"] if grouped else None,
                    prefix_lens=d["prefix"] if grouped else None,
                    n_tokens=self.n_tokens)
        return a, b

    def run(self, d=None, **how):
        t = self.t
        d = d or self.device()
        a, b = self.attention(d, **how)
        out = t.full(d["q"].shape, 123.0, dtype=t.bfloat16, device="cuda")
        lse = t.full(d["q"].shape[:2], 123.0, dtype=t.float32, device="cuda")
        a.run(0, b, d["q"], out, lse)
        a.sync()
        a.close()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def check(self, got=None, want=None, **how):
        out, lse = got or self.run(**how)
        eo, el, A, E = want or self.exact()
        n = int(self.off[-1])
        assert (out[n:] == 123.0).all() and (lse[n:] == 123.0).all()
        out, lse, eo, el, A, E = out[:n], lse[:n], eo[:n], el[:n], A[:n], E[:n]
        empty = np.isneginf(el)
        assert (out[empty] == 0.0).all() and np.isneginf(lse[empty]).all()
        ok = ~empty
        assert np.isfinite(out).all() and np.isfinite(lse[ok]).all()
        tol = 2.0 ** -8 * np.abs(eo) + (2.0 ** -8 + 2.0 ** -15 + 2.0 * E[..., None]) * A
        worst = np.max(np.abs(out - eo)[ok] / tol[ok]) if ok.any() else 0.0
        assert worst <= 1.0, worst
        ltol = E[ok] + 2.0 ** -18 + 2.0 ** -23 * np.abs(el[ok])
        assert (np.abs(lse[ok] - el[ok]) <= ltol).all(), np.max(np.abs(lse[ok] - el[ok]))


HEADS = [(2, 2, 64), (4, 2, 64), (6, 2, 32), (16, 4, 64), (32, 4, 128), (3, 1, 128), (64, 1, 32)]


@gpu
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("P", [16, 48, 64, 256])
def test_heads_and_page_sizes(heads, P):
    Case([(2 * P, [(5, 1), (P, 1), (2 * P + 3, 1)]), (0, [(1, 1), (P + 1, 1)])], heads, P).check()


@gpu
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 127, 128, 129, 255, 257, 640, 1000, 4099])
def test_lengths_of_one_sequence(length):
    Case([(0, [(length, 1)])], (8, 1, 64), seed=length).check()


@gpu
@pytest.mark.parametrize("prefix", [1, 15, 16, 31, 127, 128, 144, 160, 2047, 2048])
def test_prefix_lengths(prefix):
    Case([(prefix, [(1, 1), (16, 1), (20, 1), (140, 1)])], (16, 2, 128), seed=prefix).check()


@gpu
@pytest.mark.parametrize("each", [1, 2, 15, 16, 17, 31, 32, 33, 40, 70])
def test_rows_of_a_group(each):
    """Rows (sequences times heads of a kv head) around the row tiles' edges."""
    Case([(300, [(1 + 7 * i % 50, 1) for i in range(each)])], (16, 2, 64), seed=each).check()


@gpu
@pytest.mark.parametrize("T", [[1, 2, 3], [16, 1, 33], [64, 65, 7], [130, 1], [300], [5, 0, 9]])
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 2, 128), (6, 2, 32)])
def test_several_query_tokens(T, heads):
    Case([(160, [(max(1, t + 3 * i), t) for i, t in enumerate(T)]), (0, [(20, 4)])], heads,
         seed=len(T)).check()


@gpu
def test_queries_inside_the_prefix():
    """More query tokens than own tokens: they reach back into the shared pages."""
    c = Case([(64, [(2, 10), (5, 30), (1, 1)]), (32, [(0, 32), (0, 1)])], (4, 2, 64))
    c.check()


@gpu
def test_tokens_that_see_nothing():
    """Longer queries than the sequence, and empty sequences."""
    Case([(0, [(0, 1), (3, 9), (0, 0), (40, 2), (0, 5)])], (4, 2, 64), extra_rows=7).check()
    Case([(0, [(0, 1), (0, 1)])], (4, 2, 64)).check()


@gpu
def test_rows_behind_the_last_sequence_are_left():
    Case([(48, [(5, 1), (6, 2)])], (4, 2, 64), extra_rows=70).check()


@gpu
def test_shorter_sequences_than_the_prefix_says():
    c = Case([(0, [(40, 1), (70, 1), (20, 1)])], (4, 2, 64))
    # one group over rows that share their first page only in name: the same pages
    c.rows[1][:2], c.rows[2][:1] = c.rows[0][:2], c.rows[0][:1]
    for i, r in enumerate(c.rows):
        c.tables[i, :len(r)] = r
    c.prefix, c.starts = [32], [0, 3]
    c.check()


@gpu
def test_finished_sequences_inside_a_group():
    """Rows of length 0 with no pages, first in the group and within it."""
    c = Case([(64, [(10, 1), (7, 1), (33, 1), (9, 1)])], (4, 2, 64))
    for b in (0, 2):
        c.lens[b] = 0
        c.tables[b] = -1
    c.check()
    c = Case([(64, [(10, 0), (7, 3), (33, 0), (9, 2)])], (4, 2, 64))
    c.tables[0] = -1                       # no query tokens: not read
    c.check()


@gpu
def test_groups_change_nothing_but_the_order_of_sums():
    c = Case([(333, [(9, 1), (100, 1), (17, 1)]), (64, [(1, 1)]), (0, [(5, 1), (6, 1)])], (16, 2, 64))
    want = c.exact()
    c.check(want=want)
    c.check(want=want, grouped=False)
    c.check(want=want, offsets=True)


@gpu
def test_empty_groups_and_zero_prefixes():
    c = Case([(40, [(9, 1), (100, 1)]), (0, [(5, 1)])], (4, 2, 64))
    t = c.t
    d = c.device(starts=t.tensor([0, 0, 2, 2, 3], dtype=t.int32).cuda(),
                 prefix=t.tensor([77, 40, 5, 0], dtype=t.int32).cuda())
    c.check(c.run(d))


@gpu
def test_what_lies_behind_a_length_does_not_matter():
    """NaN and infinities behind the lengths, in spare pages, and wild page ids."""
    c = Case([(40, [(9, 1), (100, 1)]), (0, [(5, 3), (33, 1)])], (4, 2, 64))
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


@gpu
@pytest.mark.parametrize("scale", [1e-3, 0.5, 3.0])
def test_scales_and_peaked_scores(scale):
    Case([(200, [(30, 1), (129, 1)])], (4, 2, 64), scale=scale).check()


@gpu
@pytest.mark.parametrize("scale", [None, 1.0, 3.0])
@pytest.mark.parametrize("each", [1, 40])
def test_rising_scores_move_the_maximum(scale, each):
    """Every block of keys beats the last one, up to e^1152 over the row, so the reference of
    the softmax has to move along; with one row tile and with two."""
    c = Case([(0, [(1500, each)]), (256, [(700, 1), (20, 1)])], (16, 2, 64), scale=scale)
    t = c.t
    c.q[:] = 1.0
    for b, r in enumerate(c.rows):
        n = len(r) * 16
        ramp = t.linspace(0.0, 6.0, n).view(len(r), 1, 16, 1).expand(len(r), 2, 16, 64)
        if b == 2:
            continue                       # shares its first pages with sequence 1
        c.k[r] = (ramp + 0.1 * c.k[r].float()).to(t.bfloat16)
    c.check()


@gpu
def test_nan_in_a_query_stays_in_its_row():
    """One head of one token holds NaN: its row is NaN, the others are what they were."""
    for each in (3, 40):                   # singles, and a pair
        c = Case([(200, [(10 + i, 1) for i in range(each)])], (16, 2, 64))
        want = c.exact()
        c.q[1, 3, 5] = float("nan")
        out, lse = c.run()
        assert np.isnan(out[1, 3]).all() and np.isnan(lse[1, 3])
        out[1, 3], lse[1, 3] = want[0][1, 3], want[1][1, 3]
        c.check((out, lse), want)


@gpu
def test_q_inside_a_fused_projection():
    c = Case([(48, [(5, 1), (20, 1), (9, 1)])], (4, 2, 64))
    t = c.t
    wide = t.zeros(3, (4 + 2 * 2) * 64, dtype=t.bfloat16, device="cuda")
    wide[:, :256] = c.q.view(3, 256).cuda()
    c.check(c.run(c.device(q=wide[:, :256].view(3, 4, 64))))


@gpu
def test_same_call_same_bits():
    c = Case([(1024, [(30 + i, 1) for i in range(40)])], (32, 4, 128))
    a, b = c.run(), c.run()
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


@gpu
def test_long_caches():
    Case([(9000, [(700, 1), (1, 1), (0, 1)]), (5000, [(10, 2), (20, 2)])], (8, 1, 128)).check()


@gpu
def test_pools_behind_two_to_the_32():
    """Pages whose first byte lies past 2^32 bytes of the pool."""
    import torch

    Hkv, D, P, pages = 4, 128, 16, 300000              # 4.9 GB a pool
    k = torch.zeros(pages, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ids = [pages - 1, 0, pages - 7]
    g = torch.Generator().manual_seed(1)
    small_k, small_v = (torch.randn(3, Hkv, P, D, generator=g).to(torch.bfloat16) for _ in range(2))
    k[ids], v[ids] = small_k.cuda(), small_v.cuda()
    q = torch.randn(1, 8, D, generator=g).to(torch.bfloat16)
    a = mk.PrefixAttention(8, Hkv, D, P, [(k, v)], max_tokens=1)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = a.batch(torch.tensor([ids], **i32), torch.tensor([41], **i32))
    out = torch.empty(1, 8, D, dtype=torch.bfloat16, device="cuda")
    a.run(0, b, q.cuda(), out)
    a.sync()
    K = small_k.transpose(0, 1).reshape(Hkv, -1, D)[:, :41].double()
    V = small_v.transpose(0, 1).reshape(Hkv, -1, D)[:, :41].double()
    p = torch.softmax((q[0].view(Hkv, 2, D).double() @ K.transpose(1, 2)) / math.sqrt(D), -1)
    want, A = p @ V, p @ V.abs()
    diff = (out[0].cpu().double().view(Hkv, 2, D) - want).abs()
    assert bool((diff <= 2.0 ** -8 * want.abs() + 2.0 ** -8 * 1.01 * A).all())


@gpu
def test_captured_and_replayed_with_new_lengths():
    import torch

    c = Case([(64, [(40, 1), (60, 1)])], (4, 2, 64))
    d = c.device()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = c.attention(d, stream=st)
    out = torch.full(d["q"].shape, 123.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(d["q"].shape[:2], 123.0, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        a.run(0, b, d["q"], out, lse)
    for lens in ([104, 124], [65, 100], [64, 70], [1, 0]):
        with torch.cuda.stream(st):
            d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            g.replay()
        st.synchronize()
        a.sync()
        c.lens = lens
        c.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))


@gpu
def test_two_handles_at_once():
    import torch

    cases = [Case([(500, [(30 + i, 1) for i in range(20)])], (32, 4, 128), seed=s) for s in (1, 2)]
    runs = []
    for c in cases:
        d, st = c.device(), torch.cuda.Stream()
        torch.cuda.synchronize()
        out = torch.empty(d["q"].shape, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(d["q"].shape[:2], device="cuda")
        runs.append((d, out, lse) + c.attention(d, stream=st))
    torch.cuda.synchronize()
    for _ in range(30):
        for d, out, lse, a, b in runs:
            a.run(0, b, d["q"], out, lse)
    for c, (d, out, lse, a, b) in zip(cases, runs):
        a.sync()
        c.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))


@gpu
@pytest.mark.parametrize("what, value", [
    ("lens", [-1, 40]), ("lens", [40, 16 * 1000]), ("off", [1, 1, 2]), ("off", [0, 2, 1]),
    ("off", [0, 1, 9]), ("starts", [0, 1]), ("starts", [1, 2]), ("starts", [0, 3]),
    ("prefix", [-4])])
def test_wrong_device_arguments(what, value):
    c = Case([(32, [(5, 1), (8, 1)])], (4, 2, 64))
    t = c.t
    d = c.device(**{what: t.tensor(value, dtype=t.int32).cuda()})
    a, b = c.attention(d, offsets=True)
    out = t.full(d["q"].shape, 123.0, dtype=t.bfloat16, device="cuda")
    a.run(0, b, d["q"], out)
    with pytest.raises(mk.MkError) as e:
        a.sync()
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    assert bool((out == 123.0).all())
    d2 = c.device()
    c.check(c.run(d2))
    a.sync()                                # reported once


@gpu
@pytest.mark.parametrize("page", [-1, 10 ** 6, -2 ** 31])
def test_page_ids_are_checked(page):
    c = Case([(32, [(50, 1), (8, 1)])], (4, 2, 64))
    c.tables[0, 3] = page
    d = c.device()
    a, b = c.attention(d)
    out = c.t.empty_like(d["q"])
    a.run(0, b, d["q"], out)
    with pytest.raises(mk.MkError) as e:
        a.sync()
    assert e.value.code == mk.MK_ERR_PAGE_OOB
    eo, _, A, _ = c.exact()                  # the other sequence is not touched by it
    assert (np.abs(out[1].double().cpu().numpy() - eo[1])
            <= 2.0 ** -8 * np.abs(eo[1]) + 2.0 ** -8 * 1.01 * A[1]).all()


@gpu
def test_host_arguments_are_checked():
    c = Case([(32, [(5, 1), (8, 1)])], (4, 2, 64))
    d = c.device()
    a, b = c.attention(d)
    out = c.t.empty_like(d["q"])
    with pytest.raises(ValueError):
        a.run(0, b, d["q"][:1], out)
    with pytest.raises(ValueError):
        a.run(0, b, d["q"].transpose(0, 1).contiguous().transpose(0, 1), out)
    with pytest.raises(ValueError):
        a.run(0, b, d["q"].float(), out)
    with pytest.raises(TypeError):
        a.run(0, b, d["q"], out.float())
    with pytest.raises(mk.MkError):
        a.run(1, b, d["q"], out)
    with pytest.raises(ValueError):
        a.batch(d["tables"], d["lens"][:1])
    with pytest.raises(ValueError):
        a.batch(d["tables"], d["lens"], group_starts=d["starts"])
    with pytest.raises(TypeError):
        a.batch(d["tables"].long(), d["lens"])


@gpu
def test_a_refused_workspace_leaves_no_error_behind():
    """2^20 tokens of 1024 heads want 1.1 TB: MK_ERR_CUDA, and torch's next launches, which
    ask for the last error, work."""
    import torch

    pool = torch.zeros((1, 16, 16, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mk.MkError):
        mk.PrefixAttention(1024, 16, 128, 16, [(pool, pool)], max_tokens=1 << 20)
    assert int((pool + 1).sum().item()) == pool.numel()


# ------------------------------------------------------------------------- without a GPU


def _desc(**over):
    pools = (ctypes.c_void_p * 1)(0x10000)
    a = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16, num_pages=8, max_tokens=4,
             max_seqs=4, max_groups=4, n_layers=1, k_caches=pools, v_caches=pools, scale=0.0)
    a.update(over)
    return mk.mk_attn_desc(*[a[f[0]] for f in mk.mk_attn_desc._fields_])


@pytest.mark.parametrize("over, code", [
    (dict(n_q_heads=0), 1), (dict(n_q_heads=5), 1), (dict(head_dim=0), 1), (dict(max_tokens=0), 1),
    (dict(max_seqs=0), 1), (dict(max_groups=-1), 1), (dict(n_layers=0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(k_caches=None), 1),
    (dict(v_caches=(ctypes.c_void_p * 1)(0x10008)), 1), (dict(v_caches=(ctypes.c_void_p * 1)(None)), 1),
    (dict(head_dim=96), 8), (dict(page_size=8), 8), (dict(page_size=272), 8),
    (dict(n_q_heads=130, n_kv_heads=2), 8), (dict(max_tokens=(1 << 20) + 1), 8),
    (dict(max_seqs=1025), 8), (dict(max_groups=1025), 8), (dict(num_pages=1 << 30), 8)])
def test_create_refuses(over, code):
    h, d = ctypes.c_void_p(), _desc(**over)
    assert mk.lib().mk_attn_create(ctypes.byref(d), None, ctypes.byref(h)) == code
    assert not h.value


@pytest.mark.parametrize("scale, code", [(3e38, 1), (2e38, 8)])
def test_a_scale_beyond_32_bits_is_refused(scale, code):
    """Scores are multiplied by scale / ln 2, which has to be finite in fp32 (at most 3.4e38);
    a scale that passes gets as far as the head size, which is refused with another status."""
    h, d = ctypes.c_void_p(), _desc(scale=scale, head_dim=96)
    assert mk.lib().mk_attn_create(ctypes.byref(d), None, ctypes.byref(h)) == code


def test_null_handles_are_refused():
    L = mk.lib()
    assert L.mk_attn_create(None, None, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_prefix_attention(None, 0, None, None, 0, None, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_attn_sync(None) == mk.MK_ERR_INVALID_ARG
    L.mk_attn_destroy(None)


def test_the_definition_agrees_with_itself():
    """One visible key gives its V row; the case builder shares the prefix pages."""
    c = Case([(0, [(1, 1)]), (40, [(9, 1), (30, 1)])], (4, 2, 64))
    out, lse, _, _ = c.exact()
    want = c.v[c.rows[0][0], :, 0].double().numpy().repeat(2, axis=0)
    assert np.allclose(out[0], want)
    assert c.rows[1][:2] == c.rows[2][:2] and c.rows[1][2] != c.rows[2][2]
