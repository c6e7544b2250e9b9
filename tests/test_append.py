"""Appending normed and rotated keys and values (mk_append_tokens) against the definition in 64 bits.

Tolerance, per element of a turned pair (a, b) (after the norm) with magnitude m.  The cosine and
sine are off by the angle (2^-22: a 24-bit residue within pi / 4 times a rounded constant) and the
series (2^-23); with the rounded products and sum that is 2^-21 m (|a| + |b|).  The norm's factor
is off by the sum of squares (at most 13 roundings in a row, 2^-21), the root (2^-22) and two
products: below 2^-20 of a and b.  Together 2^-19 m (|a| + |b|), and the result's own rounding to
bf16, 2^-8 of the value.  v and dims behind the rotary part without a norm are copied bit for bit."""
import ctypes

import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk

gpu = pytest.mark.gpu


class Case:
    """seqs: [(cached tokens with the new ones, new tokens), ...]"""

    def __init__(self, seqs, heads=(4, 2, 64), P=16, rotary=None, interleaved=False, norm="", extra=0,
                 positions=None, seed=0, frequencies=None, base=10000.0, magnitude=1.0, eps=1e-6,
                 single=False, gap=0):
        import torch

        self.t = torch
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D = heads
        self.P, self.interleaved, self.base = P, interleaved, base
        self.R = self.D if rotary is None else rotary
        self.magnitude, self.eps, self.frequencies = magnitude, eps, frequencies
        self.lens, self.T = [s[0] for s in seqs], [s[1] for s in seqs]
        self.off = np.concatenate([[0], np.cumsum(self.T)]).astype(np.int32)
        self.n, self.single = int(self.off[-1]) + extra, single
        used = [-(-L // P) for L in self.lens]
        self.pages = sum(used) + 3
        order = rng.permutation(self.pages)
        wide = max(used + [1]) + 1
        self.tables = np.full((len(seqs), wide), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.tables[b, :u] = order[at:at + u]
            at += u
        shape = (self.pages, self.Hkv, P, self.D)
        self.k, self.v = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2))
        self.qkv = torch.randn(self.n, self.Hq + 2 * self.Hkv + gap, self.D, generator=g).to(torch.bfloat16)
        self.gq = (1 + 0.3 * torch.randn(self.D, generator=g)).to(torch.bfloat16) if "q" in norm else None
        self.gk = (1 + 0.3 * torch.randn(self.D, generator=g)).to(torch.bfloat16) if "k" in norm else None
        self.positions = None
        if positions is not None:
            self.positions = np.asarray(positions(rng, self.n), np.int32)

    def rates(self):
        if self.frequencies is not None:
            return np.asarray(self.frequencies, np.longdouble)
        return np.array([float(self.base) ** (-2.0 * i / self.R) for i in range(self.R // 2)], np.longdouble)

    def turned(self, x, gain, position):
        """(value, |a| + |b| of its pair) of heads x [heads][D] in 64 bits."""
        x = x.astype(np.float64)
        if gain is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(self.eps))) * gain
        i = np.arange(self.R // 2)
        a, b = (2 * i, 2 * i + 1) if self.interleaved else (i, i + self.R // 2)
        angle = np.longdouble(position) * self.rates()
        c, s = np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)
        m = np.float64(np.float32(self.magnitude))
        y, size = x.copy(), np.zeros_like(x) if gain is None else np.abs(x)
        y[:, a], y[:, b] = m * (x[:, a] * c - x[:, b] * s), m * (x[:, b] * c + x[:, a] * s)
        size[:, a] = size[:, b] = m * (np.abs(x[:, a]) + np.abs(x[:, b]))
        return y, size

    def device(self, **over):
        t = self.t
        d = {"qkv": self.qkv.cuda(), "k": self.k.cuda(), "v": self.v.cuda(),
             "tables": t.from_numpy(self.tables).cuda(), "lens": t.tensor(self.lens, dtype=t.int32).cuda(),
             "off": None if self.single else t.from_numpy(self.off).cuda(),
             "positions": None if self.positions is None else t.from_numpy(self.positions).cuda()}
        d.update(over)
        d["q_out"] = d.get("q_out", t.full((self.n, self.Hq, self.D), 123.0, dtype=t.bfloat16, device="cuda"))
        d["gq"] = None if self.gq is None else self.gq.cuda()
        d["gk"] = None if self.gk is None else self.gk.cuda()
        return d

    def handle(self, d, stream=None):
        return mk.KvAppend(self.Hq, self.Hkv, self.D, self.P, [(d["k"], d["v"])], rotary_dim=self.R,
                           interleaved=self.interleaved, rope_base=self.base, frequencies=self.frequencies,
                           magnitude=self.magnitude, norm_eps=self.eps, stream=stream)

    def parts(self, qkv):
        return qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:self.Hq + 2 * self.Hkv]

    def call(self, a, d, with_q=True):
        b = a.batch(d["tables"], d["lens"], q_offsets=d["off"], n_tokens=self.n)
        q, k, v = self.parts(d["qkv"])
        a.run(0, b, k, v, q=q if with_q else None, q_out=d["q_out"] if with_q else None,
              positions=d["positions"], q_norm=d["gq"], k_norm=d["gk"])
        return b

    def check(self, d=None, run=True, with_q=True, code=None, skip=()):
        """skip: tokens that are left out; code: the status that sync raises."""
        d = d or self.device()
        if run:
            a = self.handle(d)
            self.call(a, d, with_q)
            if code is None:
                a.sync()
            else:
                with pytest.raises(mk.MkError) as e:
                    a.sync()
                assert e.value.code == code
            a.sync()
            a.close()
        q0, k0, v0 = (x.float().numpy() for x in self.parts(self.qkv))
        q_out, kp, vp = (d[x].double().cpu().numpy() for x in ("q_out", "k", "v"))
        before_k, before_v = self.k.double().numpy(), self.v.double().numpy()
        fresh = np.ones((self.pages, self.P), bool)   # rows that no token goes to
        gq = None if self.gq is None else self.gq.double().numpy()
        gk = None if self.gk is None else self.gk.double().numpy()
        written = np.zeros(self.n, bool)
        for b, L in enumerate(self.lens):
            for i in range(self.T[b]):
                tok, place = int(self.off[b]) + i, L - self.T[b] + i
                if place < 0 or tok in skip:
                    continue
                written[tok] = True
                position = place if self.positions is None else int(self.positions[tok])
                page, slot = int(self.tables[b, place // self.P]), place % self.P
                if 0 <= page < self.pages:
                    fresh[page, slot] = False
                    want, size = self.turned(k0[tok], gk, position)
                    self.close(kp[page, :, slot], want, size)
                    assert np.array_equal(vp[page, :, slot], v0[tok])
                if with_q:
                    want, size = self.turned(q0[tok], gq, position)
                    self.close(q_out[tok], want, size)
        keep = np.repeat(fresh[:, None], self.Hkv, 1)
        assert np.array_equal(kp[keep], before_k[keep]) and np.array_equal(vp[keep], before_v[keep])
        if d["q_out"].data_ptr() != d["qkv"].data_ptr():
            assert (q_out[~written if with_q else slice(None)] == 123.0).all()

    @staticmethod
    def close(got, want, size):
        tol = 2.0 ** -19 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
        tol[size == 0] = 0.0
        assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


HEADS = [(4, 2, 64), (32, 4, 128), (6, 2, 32), (1, 1, 128), (5, 5, 64), (7, 1, 32)]


@gpu
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["", "qk"])
def test_ragged_sequences(heads, interleaved, norm):
    """New tokens from one to over a page, none at all, from an empty cache, across page ends."""
    Case([(40, 1), (17, 17), (33, 0), (16, 16), (0, 0), (100, 35), (3, 2)], heads, interleaved=interleaved,
         norm=norm, extra=3).check()


@gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("share", [0.0, 0.07, 0.25, 0.4, 0.5, 0.9, 1.0])
def test_part_of_the_head_turns(D, interleaved, share):
    """Each way to find a dim's partner; what does not turn is copied, or normed only."""
    R = 2 * round(D * share / 2)
    for norm in ("", "qk"):
        Case([(50, 9), (20, 3)], (3, 2, D), rotary=R, interleaved=interleaved, norm=norm, seed=R).check()


@gpu
@pytest.mark.parametrize("norm", ["q", "k"])
@pytest.mark.parametrize("P", [1, 5, 16, 64, 300])
def test_one_norm_and_page_sizes(norm, P):
    Case([(70, 33), (9, 9), (301, 2)], P=P, norm=norm).check()


@gpu
@pytest.mark.parametrize("heads", HEADS[:4])
def test_single_tokens(heads):
    """One token a sequence without offsets; empty rows of a padded batch are left out."""
    Case([(40, 1), (1, 1), (0, 1), (8000, 1), (16, 1), (17, 1), (0, 1)], heads, norm="qk", single=True).check()


@gpu
def test_single_tokens_at_other_positions():
    Case([(40, 1), (0, 1), (8000, 1), (16, 1)], (6, 2, 32), norm="q", single=True, rotary=20,
         positions=lambda r, n: r.integers(0, 100000, n)).check()


@gpu
def test_batches_of_the_attention_are_taken_with_their_groups():
    import torch

    c = Case([(40, 3), (33, 1)])
    d = c.device()
    attn = mk.PrefixAttention(4, 2, 64, 16, [(d["k"], d["v"])], max_tokens=c.n)
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    batch = attn.batch(d["tables"], d["lens"], q_offsets=d["off"], group_starts=t(0, 2), prefix_lens=t(32))
    a = c.handle(d)
    q, k, v = c.parts(d["qkv"])
    a.run(0, batch, k, v, q=q, q_out=d["q_out"])
    a.sync()
    c.check(d, run=False)


@gpu
def test_tokens_without_a_place_are_left_out():
    Case([(3, 7), (40, 2), (0, 4), (5, 5)], extra=2).check()


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_repeated_positions(interleaved):
    """Positions of a drafted tree, and as far as they go."""
    Case([(60, 24)], interleaved=interleaved, positions=lambda r, n: 36 + np.sort(r.integers(0, 6, n))).check()
    Case([(60, 24), (30, 8)], (2, 1, 128), interleaved=interleaved, norm="qk",
         positions=lambda r, n: r.integers(0, 2 ** 31, n)).check()
    Case([(40, 3)], interleaved=interleaved, positions=lambda r, n: [0, 2 ** 31 - 1, 262144]).check()


@gpu
def test_rates_and_magnitude():
    rates = mk.rope_frequencies(64, 500000.0, "parts", 8.0, 8192, 1.0, 4.0)
    Case([(9000, 30)], frequencies=rates, magnitude=1.2079).check()
    Case([(90, 30)], frequencies=[0.0, -0.5, 3.0, 100.25] + [1e-9] * 28, interleaved=True, magnitude=0.25).check()
    Case([(5000, 3)], (2, 2, 32), base=3.5).check()


@gpu
@pytest.mark.parametrize("scale, eps", [(0.0, 1e-6), (1e-30, 1e-6), (1e-20, 0.0), (1e15, 1e-6), (1.0, 100.0)])
def test_norm_of_small_and_large_heads(scale, eps):
    """All zeros, values whose squares vanish beside eps, squares near the ends of 32 bits."""
    c = Case([(40, 6)], norm="qk", eps=eps)
    # a scale of 1e-20: squares of 1e-40 keep few bits in 32, so only rows of equal size are compared
    c.qkv = (c.qkv.float().sign() if scale == 1e-20 else c.qkv.float()).mul(scale).to(c.t.bfloat16)
    if scale == 1e-20:
        d = c.device()
        a = c.handle(d)
        c.call(a, d)
        a.sync()
        assert c.t.isfinite(d["q_out"].float()).all()
        return
    c.check()


@gpu
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-35, 1e-6, 1e20])
@pytest.mark.parametrize("heads", [(4, 2, 64), (5, 3, 32), (2, 1, 128)])
def test_norm_over_the_whole_range(heads, eps):
    """Heads whose squares leave 32 bits at either end, each beside others that do not, and heads with both
    large and small values.  The scales by powers of two are exact, so the tolerance is the same; results
    below 2^-126 are rounded to steps of 2^-133."""
    c = Case([(40, 30)], heads, norm="qk", eps=eps, seed=8)
    t, rng = c.t, np.random.default_rng(8)
    sizes = [-132, -125, -100, -67, -60, -51, -49, 0, 49, 51, 57]
    if eps < 2.0 ** -100:
        sizes += [63, 64, 100, 124]
    size = 2.0 ** rng.choice(sizes, c.qkv.shape[:2])
    spread = 2.0 ** rng.choice([0, 0, -20, -45], c.qkv.shape)
    x = c.qkv.double() * t.from_numpy(size)[:, :, None] * t.from_numpy(np.where(rng.random(c.qkv.shape[:2] + (1,)) < 0.5, 1, spread))
    c.qkv = x.clamp(-3e38, 3e38).to(t.bfloat16)
    if eps == 0.0:  # no head of zeros: its norm is 0 / 0
        c.qkv[..., 0] = t.where((c.qkv == 0).all(-1), t.full((), 2.0 ** -133, dtype=t.bfloat16), c.qkv[..., 0])
    close = c.close
    c.close = lambda got, want, size: close(got, want, size + 2.0 ** -134 * 2.0 ** 19)
    c.check()


@gpu
@pytest.mark.parametrize("scale", [1e-20, 1e-30, 1e-38, 1e30])
def test_norm_without_eps_of_equal_sizes(scale):
    """A head of one size is its signs times the gain, at any size: of tiny heads K too."""
    c = Case([(40, 6)], norm="qk", eps=0.0)
    c.qkv = c.qkv.float().sign().mul(scale).to(c.t.bfloat16)
    c.check()


@gpu
def test_infinities_and_nan_stay_in_their_head():
    c = Case([(40, 4)], (4, 2, 64), rotary=32)
    c.qkv[0, 1, 3], c.qkv[2, 0, 50], c.qkv[3, 7, 5] = float("nan"), float("inf"), float("nan")
    d = c.device()
    a = c.handle(d)
    c.call(a, d)
    a.sync()
    q = d["q_out"].float().cpu()
    bad = ~c.t.isfinite(q)
    assert bad[0, 1, [3, 19]].all() and bad[2, 0, 50] and int(bad.sum()) == 3
    assert int((~c.t.isfinite(d["k"].float())).sum()) == 0
    assert int((~c.t.isfinite(d["v"].float())).sum()) == 1


@gpu
@pytest.mark.parametrize("heads", [(4, 2, 64), (3, 1, 128)])
def test_strides_and_in_place(heads):
    """Parts of one wide row, q turned in place, and an output with a stride of its own."""
    c = Case([(40, 9), (21, 21)], heads, norm="qk", gap=3)
    d = c.device()
    d["q_out"] = d["qkv"][:, :c.Hq]
    c.check(d)
    assert c.t.equal(d["qkv"][:, c.Hq:].cpu(), c.qkv[:, c.Hq:])
    d = c.device()
    wide = c.t.full((c.n, c.Hq + 2, c.D), 123.0, dtype=c.t.bfloat16, device="cuda")
    d["q_out"] = wide[:, 1:1 + c.Hq]
    c.check(d)
    assert (wide[:, 0] == 123.0).all() and (wide[:, -1] == 123.0).all()


@gpu
def test_keys_and_values_only():
    Case([(40, 9), (21, 21)], norm="k").check(with_q=False)
    c = Case([(40, 9), (21, 21)], (0, 2, 64))
    c.check(with_q=False)


@gpu
@pytest.mark.parametrize("n", [383, 1000, 1024])
def test_many_sequences(n):
    rng = np.random.default_rng(n)
    seqs = []
    for _ in range(n):
        t = int(rng.integers(0, 4))
        seqs.append((t + int(rng.integers(0, 40)), t))
    Case(seqs, (2, 1, 32), extra=5).check()


@gpu
@pytest.mark.parametrize("T", [1, 2, 7, 150, 1300])
def test_token_counts_on_both_sides_of_the_split(T):
    """Few tokens are cut into parts of their heads, many are not."""
    Case([(T + 5, T)], (32, 4, 128), norm="qk").check()
    Case([(T + 5, T)], (6, 2, 32), interleaved=True).check()


@gpu
def test_pool_offsets_past_32_bits():
    """The last pages of a pool of over 2^32 bytes."""
    import torch

    pages = (1 << 32) // (16 * 128 * 2 * 4) + 3000
    k = torch.zeros(pages, 4, 16, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([(20, 20)], (2, 4, 128))
    d = c.device(k=k, v=v)
    tables = np.array([[pages - 1, pages - 2900]], np.int32)
    d["tables"] = torch.from_numpy(tables).cuda()
    a = c.handle(d)
    c.call(a, d)
    a.sync()
    c.tables, (q0, k0, v0) = tables, c.parts(c.qkv)
    for i in range(20):
        page, slot = int(tables[0, i // 16]), i % 16
        want, size = c.turned(k0[i].float().numpy(), None, i)
        c.close(k[page, :, slot].double().cpu().numpy(), want, size)
        assert torch.equal(v[page, :, slot].cpu(), v0[i])
    assert int((v != 0).any(-1).any(1).sum()) == 20


# ---- what is refused, and calls in captured graphs and on other streams


def desc(**over):
    pools = (ctypes.c_void_p * 1)(0x10000)
    d = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16, num_pages=8, rotary_dim=64, interleaved=0,
             n_layers=1, k_caches=pools, v_caches=pools, frequencies=None, rope_base=10000.0, magnitude=0.0,
             norm_eps=1e-6)
    d.update(over)
    return mk.mk_append_desc(*[d[f[0]] for f in mk.mk_append_desc._fields_])


def create(d):
    h = ctypes.c_void_p()
    return mk.lib().mk_append_create(ctypes.byref(d) if d is not None else None, None, ctypes.byref(h))


@pytest.mark.parametrize("over", [
    dict(n_q_heads=-1), dict(n_kv_heads=0), dict(head_dim=0), dict(page_size=0), dict(num_pages=0),
    dict(n_layers=0), dict(rotary_dim=-2), dict(rotary_dim=3), dict(rotary_dim=66), dict(rope_base=0.0),
    dict(rope_base=-1.0), dict(rope_base=float("nan")), dict(rope_base=float("inf")),
    dict(magnitude=-1.0), dict(magnitude=float("nan")), dict(magnitude=float("inf")), dict(norm_eps=-1e-6),
    dict(norm_eps=float("nan")), dict(k_caches=None), dict(v_caches=(ctypes.c_void_p * 1)(0x10008)),
    dict(k_caches=(ctypes.c_void_p * 1)(None)),
    dict(frequencies=(ctypes.c_double * 32)(*[float("nan")] * 32))])
def test_create_refuses(over):
    assert create(desc(**over)) == mk.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(head_dim=96, rotary_dim=0), dict(head_dim=256), dict(n_q_heads=2048)])
def test_create_does_not_support(over):
    assert create(desc(**over)) == mk.MK_ERR_UNSUPPORTED


def test_null_handles():
    L = mk.lib()
    assert create(None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_append_create(ctypes.byref(desc()), None, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_append_tokens(None, 0, None, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_append_sync(None) == mk.MK_ERR_INVALID_ARG
    L.mk_append_destroy(None)


def test_rates_helper():
    plain = mk.rope_frequencies(8, 10000.0)
    assert plain == [10000.0 ** (-i / 4) for i in range(4)]
    assert mk.rope_frequencies(8, 10000.0, "linear", 4.0) == [f / 4.0 for f in plain]
    grown = mk.rope_frequencies(8, 10000.0, "base", 4.0)
    assert grown[0] == 1.0 and abs(grown[-1] * 4.0 / plain[-1] - 1.0) < 1e-12
    parts = mk.rope_frequencies(8, 10000.0, "parts", 4.0, 400)
    turns = [400 * f / (2 * np.pi) for f in plain]       # 63.7, 6.4, 0.64, 0.064
    assert parts[:2] == plain[:2] and turns[2] < 1.0 and np.allclose(parts[2:], [f / 4 for f in plain[2:]])
    mid = mk.rope_frequencies(8, 10000.0, "parts", 4.0, 400, low=1.0, high=11.0)
    kept = (turns[1] - 1.0) / 10.0
    assert abs(mid[1] - plain[1] * (kept + (1 - kept) / 4)) < 1e-15
    assert mk.rope_frequencies(0) == []
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, scaling="wide"),
                dict(rotary_dim=8, scaling="parts"), dict(rotary_dim=2, scaling="base"),
                dict(rotary_dim=8, factor=-1.0),
                dict(rotary_dim=8, scaling="parts", old_context=10, low=2.0, high=2.0)):
        with pytest.raises(ValueError):
            mk.rope_frequencies(**bad)


def test_binding_checks_without_a_gpu():
    import torch

    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mk.KvAppend(4, 2, 64, 16, [(pool, pool)])
    with pytest.raises(ValueError, match="magnitude"):
        mk.KvAppend(4, 2, 64, 16, [(pool, pool)], magnitude=1e-60)
    with pytest.raises(ValueError, match="frequencies"):
        mk.KvAppend(4, 2, 64, 16, [(pool, pool)], frequencies=[1.0])
    with pytest.raises(ValueError, match="no layers"):
        mk.KvAppend(4, 2, 64, 16, [])


@pytest.mark.parametrize("kind", ["KvAppend", "PrefixAttention"])
def test_batches_of_another_device_are_refused(kind):
    import torch

    a = getattr(mk, kind).__new__(getattr(mk, kind))
    a.handle, a.device, a.heads, a.kv_heads, a.head_dim, a._index = None, torch.device("cpu"), 1, 1, 32, -1
    a._bf16, a._int32, a.max_tokens = torch.bfloat16, torch.int32, 2
    b = a.batch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    a.device = torch.device("cuda", 1)
    x = torch.zeros(2, 1, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="the batch is on cpu, not on cuda:1"):
        a.run(0, b, x, x)


@gpu
def test_the_binding_refuses_wrong_tensors():
    c = Case([(40, 9), (21, 21)])
    t, d = c.t, c.device()
    a = c.handle(d)
    b = a.batch(d["tables"], d["lens"], q_offsets=d["off"], n_tokens=c.n)
    q, k, v = c.parts(d["qkv"])
    o = d["q_out"]
    wrong = [dict(k=k[:5]), dict(v=v.float()), dict(k=k.cpu()), dict(q=q), dict(q_out=o),
             dict(q=q, q_out=o[:, :1]), dict(k=k.transpose(1, 2)), dict(positions=d["lens"]),
             dict(q_norm=t.ones(32, dtype=t.bfloat16, device="cuda"))]
    for w in wrong:
        with pytest.raises(ValueError):
            a.run(0, b, **{**dict(k=k, v=v), **w})
    with pytest.raises(TypeError):
        a.run(0, b, k, v, positions=t.zeros(c.n, dtype=t.int64, device="cuda"))
    with pytest.raises(ValueError):
        a.batch(d["tables"], d["lens"], q_offsets=d["off"])
    with pytest.raises(mk.MkError) as e:
        a.run(1, b, k, v)
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    a.sync()
    assert t.equal(d["k"].cpu(), c.k) and t.equal(d["v"].cpu(), c.v)


@gpu
def test_the_library_refuses_wrong_rows():
    c = Case([(40, 9), (21, 21)])
    d = c.device()
    a = c.handle(d)
    b = a.batch(d["tables"], d["lens"], q_offsets=d["off"], n_tokens=c.n)
    q, k, v = c.parts(d["qkv"])
    wide, wq, wkv = d["qkv"].stride(0), c.Hq * c.D, c.Hkv * c.D

    def rows(**over):
        r = dict(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), q_out=d["q_out"].data_ptr(), q_stride=wide,
                 k_stride=wide, v_stride=wide, q_out_stride=wq, q_norm=None, k_norm=None, positions=None)
        r.update(over)
        return mk.lib().mk_append_tokens(a.handle, 0, ctypes.byref(b),
                                         ctypes.byref(mk.mk_append_rows(*[r[f[0]] for f in mk.mk_append_rows._fields_])))

    for over in (dict(k=None), dict(v=None), dict(q_out=None), dict(q=None), dict(k=k.data_ptr() + 2),
                 dict(q_stride=wide + 4), dict(k_stride=wkv - 8), dict(q_out_stride=wq - 8), dict(v_stride=1 << 39),
                 dict(q_norm=d["qkv"].data_ptr() + 8), dict(positions=d["lens"].data_ptr() + 2),
                 # q_out over q with another stride, over k, over v
                 dict(q_out=q.data_ptr()), dict(q_out=q.data_ptr() + 2 * wq, q_out_stride=wide),
                 dict(q_out=v.data_ptr(), q_out_stride=wide),
                 dict(q_out=q.data_ptr() + 16, q_out_stride=wide)):
        assert rows(**over) == mk.MK_ERR_INVALID_ARG, over
    many = mk.mk_attn_batch(1025, 1025, 0, 1, 16, 16, None, None, None)
    assert mk.lib().mk_append_tokens(a.handle, 0, ctypes.byref(many), ctypes.byref(mk.mk_append_rows())) == mk.MK_ERR_BATCH
    empty = mk.mk_attn_batch(0, 0, 0, 1, None, None, None, None, None)
    assert mk.lib().mk_append_tokens(a.handle, 0, ctypes.byref(empty), ctypes.byref(mk.mk_append_rows())) == mk.MK_OK
    a.sync()
    assert c.t.equal(d["k"].cpu(), c.k) and (d["q_out"] == 123.0).all()


@gpu
@pytest.mark.parametrize("what, value", [("off", [1, 9, 30]), ("off", [0, 9, 8]), ("off", [0, 9, 31]),
                                         ("off", [0, -1, 30]), ("lens", [-1, 21]), ("lens", [40, 10 ** 6])])
def test_wrong_offsets_and_lengths_write_nothing(what, value):
    c = Case([(40, 9), (21, 21)], norm="qk")
    t = c.t
    d = c.device(**{what: t.tensor(value, dtype=t.int32, device="cuda")})
    a = c.handle(d)
    c.call(a, d)
    with pytest.raises(mk.MkError) as e:
        a.sync()
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    assert t.equal(d["k"].cpu(), c.k) and t.equal(d["v"].cpu(), c.v) and (d["q_out"] == 123.0).all()
    d = c.device()
    c.check(d)                                   # another handle; and this one goes on
    a.sync()


@gpu
@pytest.mark.parametrize("page", [-1, 10 ** 6, "last"])
def test_a_wrong_page_is_not_written(page):
    c = Case([(40, 9), (21, 21)])
    c.tables[0, 2] = c.pages if page == "last" else page       # places 32 to 39
    c.check(code=mk.MK_ERR_PAGE_OOB)


@gpu
def test_negative_positions_are_left_out():
    c = Case([(40, 9), (21, 21)], positions=lambda r, n: np.where(np.arange(n) % 7 == 3, -5, np.arange(n)))
    c.check(code=mk.MK_ERR_INVALID_ARG, skip=set(range(3, 30, 7)))


@gpu
def test_captured_calls_follow_their_tensors():
    """Two handles captured into one graph; lengths, tables and rows change between replays."""
    import torch

    c = Case([(40, 9), (21, 21)], norm="qk", positions=lambda r, n: r.integers(0, 5000, n))
    other = Case([(33, 12), (21, 18)], norm="qk", positions=lambda r, n: r.integers(0, 5000, n), seed=9)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        d, e = c.device(), c.device()
        e["gq"], e["gk"] = d["gq"], d["gk"]
        a, b = c.handle(d, stream=stream), c.handle(e, stream=stream)
        keep = [c.call(a, d), c.call(b, e)]
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            keep += [c.call(a, d), c.call(b, e)]
            assert mk.lib().mk_append_sync(a.handle) == mk.MK_ERR_INVALID_ARG
        other.gq, other.gk = c.gq, c.gk
        wide = np.full_like(c.tables, -1)
        other.tables = np.concatenate([other.tables, wide], 1)[:, :c.tables.shape[1]]
        other.pages, other.k, other.v = c.pages, c.k, c.v
        for x in (d, e):
            for name, t in (("qkv", other.qkv), ("k", c.k), ("v", c.v), ("tables", torch.from_numpy(other.tables)),
                            ("lens", torch.tensor(other.lens, dtype=torch.int32)), ("off", torch.from_numpy(other.off)),
                            ("positions", torch.from_numpy(other.positions))):
                x[name].copy_(t)
            x["q_out"].fill_(123.0)
        graph.replay()
        a.sync(), b.sync()
        stream.synchronize()
        other.check(d, run=False)
        other.check(e, run=False)


@gpu
def test_another_stream_than_the_current_one():
    import torch

    c = Case([(40, 9), (21, 21)], norm="qk")
    d = c.device()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = c.handle(d, stream=side)
    c.call(a, d)
    a.sync()
    c.check(d, run=False)
