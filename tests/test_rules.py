"""Penalties, biases and masks on logits (mk_rules_apply).

The definition rounds each step to 32 bits by itself, so the results equal numpy's float32, step
by step, bit for bit.  Against the formula in 64 bits: at most five steps round (division or
product; frequency times count; two differences; bias), each by 2^-24 of a value no larger than
the sum of the terms' magnitudes: 5 * 2^-24, taken as 2^-21, of that sum.  A step whose result lies
below 2^-126 rounds by half of the smallest step, 2^-150, instead: 5 * 2^-150 are below 2^-147.  Where
the sum passes 2^127 a step may go to infinity, which the formula does not: there only the steps count."""
import ctypes

import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk

gpu = pytest.mark.gpu


class Case:
    """rows: (history or None to share the row's before, prompt, path, biases {id: b}, mask row)."""

    def __init__(self, vocab, n, seed=0, bf16=False, history=40, share=1, path=0, bias=0, masks=0, rules=True,
                 pad=False, stride=None, kinds="rpf"):
        import torch

        self.t, self.V, self.n, self.bf16 = torch, vocab, n, bf16
        rng = np.random.default_rng(seed)
        x = torch.from_numpy(rng.normal(0, 3, (n, vocab)).astype(np.float32))
        self.x = x.to(torch.bfloat16) if bf16 else x
        self.stride = stride or vocab
        word = lambda k: (rng.random(k) ** 3 * vocab).astype(np.int32)
        self.tokens = self.ranges = self.prompt = None
        self.off = self.path = self.boff = self.bids = self.bias = None
        self.rep = self.pres = self.freq = self.allowed = self.which = None
        if history is not None:
            self.ranges, tokens, at = np.zeros((n, 2), np.int32), [], 0
            for i in range(n):
                if i % share == 0:
                    k = int(rng.integers(0, history + 1))
                    tokens.append(word(k))
                    begin, at = at, at + k
                self.ranges[i] = begin, at
            self.tokens = np.concatenate(tokens + [word(1)])
            if pad:
                self.tokens[rng.random(len(self.tokens)) < 0.2] = rng.choice([-1, vocab, 2 ** 31 - 1, -2 ** 31])
            self.prompt = np.repeat(rng.integers(0, history + 5, n), 1).astype(np.int32)
            if share > 1:
                self.prompt = self.prompt[np.arange(n) // share * share]
        if path:
            k = rng.integers(0, path + 1, n)
            self.off = np.concatenate([[0], np.cumsum(k)]).astype(np.int32)
            self.path = word(max(1, int(k.sum())))
        if rules:
            self.rep = rng.uniform(0.5, 2.0, n).astype(np.float32) if "r" in kinds else None
            self.pres = rng.normal(0, 1, n).astype(np.float32) if "p" in kinds else None
            self.freq = rng.normal(0, 0.5, n).astype(np.float32) if "f" in kinds else None
        if bias:
            rows = [np.sort(rng.choice(vocab, int(rng.integers(0, min(bias, vocab) + 1)), replace=False)) for _ in range(n)]
            self.boff = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
            self.bids = np.concatenate(rows + [[0]]).astype(np.int32)
            self.bias = rng.normal(0, 4, len(self.bids)).astype(np.float32)
        if masks:
            bits = rng.random((masks, (vocab + 31) // 32 * 32)) < rng.random((masks, 1)) ** 2
            self.allowed = np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()
            self.which = rng.integers(-1, masks, n).astype(np.int32)

    def parts(self, i):
        """(known, counts, bias, where it is, may) of row i."""
        known, c = np.zeros(self.V, bool), np.zeros(self.V, np.int64)
        b, has, may = np.zeros(self.V, np.float32), np.zeros(self.V, bool), np.ones(self.V, bool)
        if self.ranges is not None:
            h = self.tokens[self.ranges[i, 0]:self.ranges[i, 1]]
            p = 0 if self.prompt is None else int(self.prompt[i])
            ok = (h >= 0) & (h < self.V)
            known[h[ok]] = True
            np.add.at(c, h[p:][ok[p:]], 1)
        if self.off is not None:
            h = self.path[self.off[i]:self.off[i + 1]]
            h = h[(h >= 0) & (h < self.V)]
            known[h] = True
            np.add.at(c, h, 1)
        if self.boff is not None:
            ids = self.bids[self.boff[i]:self.boff[i + 1]]
            b[ids], has[ids] = self.bias[self.boff[i]:self.boff[i + 1]], True
        if self.allowed is not None:
            m = i if self.which is None else int(self.which[i])
            if m >= 0:
                may = np.unpackbits(self.allowed[m].view(np.uint8), bitorder="little")[:self.V].astype(bool)
        return known, c, b, has, may

    def want(self):
        """Rows in float32, step by step; tokens."""
        f32 = np.float32
        rows, tokens = [], []
        for i in range(self.n):
            x = self.x[i].float().numpy().copy()
            known, c, b, has, may = self.parts(i)
            r, p, f = (d if a is None else a[i] for a, d in ((self.rep, f32(1)), (self.pres, f32(0)), (self.freq, f32(0))))
            x64 = x.astype(np.float64)
            with np.errstate(all="ignore"):
                x = np.where(known, np.where(x > 0, x / r, x * r), x)
                x = np.where(c > 0, (x - f * c.astype(f32)) - p, x)
                x = np.where(has, x + b, x)
                # and the formula in 64 bits
                y = np.where(known, np.where(x64 > 0, x64 / r, x64 * r), x64)
                size = np.abs(y) + np.where(c > 0, np.abs(f) * c + np.abs(p), 0) + np.abs(b)
                y = y - np.where(c > 0, np.float64(f) * c + p, 0) + np.where(has, b, 0)
                fine = np.isfinite(y) & (size < 2.0 ** 127)
                assert (np.abs(x - y)[fine] <= 2.0 ** -21 * size[fine] + 2.0 ** -147).all()
            x = np.where(may, x, f32(-np.inf)).astype(f32)
            rows.append(x)
            z = np.where(np.isnan(x), -np.inf, x)
            tokens.append(int(np.argmax(z)) if z.max() > -np.inf else -1)
        return np.stack(rows), np.array(tokens, np.int32)

    def gpu(self, v):
        return None if v is None else self.t.from_numpy(np.ascontiguousarray(v)).cuda()

    def handle(self, stream=None):
        return mk.TokenRules(self.V, self.n, stream=stream)

    def batch(self, rules, **over):
        d = dict(tokens=self.tokens, ranges=self.ranges, prompt_lens=self.prompt, path_offsets=self.off,
                 path_tokens=self.path, repetition=self.rep, presence=self.pres, frequency=self.freq,
                 bias_offsets=self.boff, bias_tokens=self.bids, bias=self.bias, allowed=self.allowed,
                 allowed_rows=self.which)
        d.update(over)
        return rules.batch(self.n, **{k: self.gpu(v) for k, v in d.items()})

    def logits(self):
        wide = self.t.full((self.n, self.stride), 55.0, dtype=self.x.dtype, device="cuda")
        wide[:, :self.V] = self.x.cuda()
        return wide[:, :self.V]

    def check(self, what="both", skip=(), code=None, **over):
        rules = self.handle()
        b, x = self.batch(rules, **over), self.logits()
        out = self.t.full((self.n, self.V), 77.0, device="cuda") if what in ("both", "out") else None
        tok = self.t.full((self.n,), -9, dtype=self.t.int32, device="cuda") if what in ("both", "tokens", "in place") else None
        if what == "in place":
            out = x
        rules.run(b, x, out=out, tokens=tok)
        if code is None:
            rules.sync()
        else:
            with pytest.raises(mk.MkError) as e:
                rules.sync()
            assert e.value.code == code
        rules.sync()
        rows, tokens = self.want()
        keep = np.array([i not in skip for i in range(self.n)])
        if out is not None:
            got = out.float().cpu().numpy()
            assert np.array_equal(got[keep].view(np.int32)[~np.isnan(rows[keep])], rows[keep].view(np.int32)[~np.isnan(rows[keep])])
            assert np.array_equal(np.isnan(got[keep]), np.isnan(rows[keep]))
            assert (got[~keep] == 77.0).all()
        if tok is not None:
            assert np.array_equal(tok.cpu().numpy()[keep], tokens[keep])
            assert (tok.cpu().numpy()[~keep] == -9).all()
        return rows, tokens


VOCABS = [1, 2, 31, 33, 300, 1023, 1024, 1025, 4096, 8191, 8192, 8193, 32000, 50001]


@gpu
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("bf16", [False, True])
def test_vocabularies(vocab, bf16):
    """On both sides of the slices, and not a multiple of anything."""
    Case(vocab, 5, vocab, bf16, history=60, path=4, bias=9, masks=3).check()
    Case(vocab, 2, vocab, bf16, history=5, bias=2, masks=2).check("tokens")


@gpu
@pytest.mark.parametrize("n", [1, 2, 17, 151, 160, 700])
def test_rows(n):
    """Few rows (small slices) and many (blocks go on from row to row and slice to slice)."""
    Case(9000, n, n, history=30, share=3, path=3, bias=5, masks=4).check()


@gpu
@pytest.mark.parametrize("how", [dict(), dict(history=None), dict(history=None, bias=7), dict(history=None, masks=2),
                                 dict(history=None, path=6), dict(rules=False), dict(kinds="r"), dict(kinds="p", bias=3),
                                 dict(kinds="f", path=3), dict(masks=5), dict(bias=300)])
@pytest.mark.parametrize("what", ["both", "out", "tokens", "in place"])
def test_rules_alone_and_together(how, what):
    Case(5000, 6, 3, **how).check(what)


@gpu
def test_the_full_vocabulary_and_long_histories():
    Case(152064, 9, 1, history=20000, share=4, path=8, bias=100, masks=4).check()
    Case(152064, 8, 2, True, history=9000, bias=50).check()


@gpu
@pytest.mark.parametrize("stride", [4096, 4100, 4097])
@pytest.mark.parametrize("vocab", [4093, 4096])
@pytest.mark.parametrize("bf16", [False, True])
def test_strides(vocab, stride, bf16):
    if stride >= vocab:
        Case(vocab, 4, 5, bf16, stride=stride, masks=2).check()
        Case(vocab, 4, 5, bf16, stride=stride, masks=2).check("tokens")


@gpu
@pytest.mark.parametrize("vocab, bf16", [(9000, False), (9000, True), (9001, False), (9001, True)])
@pytest.mark.parametrize("what", ["both", "out", "tokens", "in place"])
def test_many_rows(vocab, bf16, what):
    """Enough rows for the largest slices, whose tokens with a word are listed."""
    if bf16 and what == "in place":
        return
    Case(vocab, 360, 40, bf16, history=400, share=5, path=4, bias=30, masks=6).check(what)
    Case(vocab, 330, 41, bf16, history=None, bias=3).check(what)
    Case(vocab, 330, 42, bf16, history=30, share=2).check(what)


@gpu
def test_dense_rows():
    """More biases than a block's threads, paths longer than that, and a history that has most tokens."""
    Case(3000, 3, 43, history=9000, path=700, bias=3000, masks=2).check()
    Case(9000, 320, 44, history=9000, share=40, path=700, bias=1500, masks=2).check()


@gpu
def test_penalties_over_the_whole_range():
    """The quotient is rounded once everywhere: near the ends, at zero, with and without a remainder."""
    for seed in range(4):
        c = Case(20000, 4, seed, history=60000, kinds="r")
        rng = np.random.default_rng(seed)
        e = rng.integers(-149, 128, (4, 20000)) if seed % 2 else rng.integers(-20, 20, (4, 20000))
        c.x = c.t.from_numpy(np.ldexp(rng.uniform(-2, 2, (4, 20000)), e).astype(np.float32))
        c.x[:, ::97] = 0.0
        c.rep = np.float32([[1e-38, 1e38, 3.0, np.inf], [0.1, 7.0, 1e-3, 1.0 / 3], [1.2, 1.1, 1.7, 1.3],
                            [2.0 ** -30, 2.0 ** 30, 2.0 ** -29, 1.0000001]][seed])
        c.check()


@gpu
def test_the_largest_vocabulary():
    c = Case(1 << 24, 1, 45, history=50, bias=10)
    c.check()


@gpu
def test_padding_ids_and_masks_by_row():
    Case(700, 12, 6, history=50, share=2, pad=True, path=5).check()
    c = Case(700, 6, 7, masks=9)
    c.which = None
    c.check()


@gpu
def test_a_prompt_that_is_all_or_none_of_the_history():
    c = Case(400, 5, 8, history=90)
    c.prompt[:] = [0, 10 ** 6, 1, 2 ** 31 - 1, 3]
    c.check()
    c.prompt = None
    c.check()


@gpu
@pytest.mark.parametrize("bf16", [False, True])
def test_ties_infinities_and_nan(bf16):
    c = Case(9000, 9, 9, bf16, history=None, rules=False, masks=3)
    t, nan, inf = c.t, float("nan"), float("inf")
    c.which[:] = -1
    c.x[0] = 1.5                                   # all alike: the lowest
    c.x[1] = -inf                                  # nothing
    c.x[2] = nan
    c.x[3, 10:] = nan
    c.x[4, [8200, 40]] = inf
    c.x[5] = -0.0
    c.x[5, 8500] = 0.0                             # no larger than -0.0
    c.which[6] = 1
    c.allowed[1] = 0                               # a mask that leaves nothing
    c.which[7], c.allowed[2, :] = 2, 0
    c.allowed[2, 8999 // 32] = 1 << (8999 % 32)    # and one that leaves the last token
    c.x[8, :] = -inf
    c.x[8, 4000] = -3e38
    rows, tokens = c.check()
    assert tokens[0] == 0 and tokens[1] == -1 and tokens[2] == -1 and tokens[5] == 0
    assert tokens[4] == 40 and tokens[6] == -1 and tokens[7] == 8999 and tokens[8] == 4000
    c.check("tokens")


@gpu
def test_infinite_logits_under_penalties():
    c = Case(300, 3, 10, history=200, bias=40, masks=2)
    c.x[0, ::3], c.x[1, ::2], c.x[2, ::5] = float("inf"), float("-inf"), float("nan")
    c.check()


@gpu
def test_empty_arrays_and_rows():
    """No token anywhere, though ranges, paths and biases are given; a bias of -inf forbids."""
    c = Case(3000, 4, 46, history=0, masks=2)
    c.tokens = np.zeros(0, np.int32)
    c.off, c.path = np.zeros(5, np.int32), np.zeros(0, np.int32)
    c.boff, c.bids, c.bias = np.zeros(5, np.int32), np.zeros(0, np.int32), np.zeros(0, np.float32)
    c.check()
    c = Case(3000, 2, 47, history=9, bias=40)
    c.bias[:] = -np.inf
    rows, tokens = c.check()
    assert np.isneginf(rows).sum() >= 1 and (tokens >= 0).all()


@gpu
@pytest.mark.parametrize("rows", [3, 340])
def test_no_masks_and_rows_that_take_none(rows):
    """No grammar is active: allowed has no rows, and none is asked for; one that is asked for is reported."""
    c = Case(9000, rows, 48, bias=5)
    c.which = np.full(rows, -1, np.int32)
    none = np.zeros((0, (9000 + 31) // 32), np.int32)
    c.check(allowed=none)
    c.which[1] = 0
    c.check(allowed=none, skip={1}, code=mk.MK_ERR_INVALID_ARG)


@gpu
def test_counts_of_one_token():
    """A history of one token over and over: 30000 atomics on one word."""
    c = Case(2000, 3, 11, history=30000)
    c.tokens[:] = 1234
    c.check()


@gpu
def test_same_call_same_bits_and_no_state_between_calls():
    c = Case(20000, 30, 12, history=300, share=5, path=4, bias=20, masks=3)
    rules, rows, tokens = c.handle(), *c.want()
    b, x = c.batch(rules), c.logits()
    for _ in range(4):
        out, tok = c.t.empty(c.n, c.V, device="cuda"), c.t.empty(c.n, dtype=c.t.int32, device="cuda")
        rules.run(b, x, out=out, tokens=tok)
        rules.sync()
        assert np.array_equal(out.cpu().numpy(), rows) and np.array_equal(tok.cpu().numpy(), tokens)


@gpu
@pytest.mark.parametrize("seed", range(12))
def test_random_calls(seed):
    rng = np.random.default_rng(100 + seed)
    Case(int(rng.integers(1, 30000)), int(rng.integers(1, 60)), seed, bool(rng.integers(2)),
         history=[None, 0, 7, 500][rng.integers(4)], share=int(rng.integers(1, 9)), path=int(rng.integers(0, 9)),
         bias=int(rng.integers(0, 60)), masks=int(rng.integers(0, 6)), rules=bool(rng.integers(2)),
         pad=bool(rng.integers(2))).check(["both", "tokens", "out"][rng.integers(3)])


# ---- what is refused


WRONG = [("ranges", (1, 0), -1), ("ranges", (1, 1), 10 ** 6), ("ranges", (1, 0), 10 ** 6), ("prompt", 1, -1),
         ("off", 2, 10 ** 6), ("off", 1, -1), ("boff", 2, 10 ** 6), ("rep", 1, 0.0), ("rep", 1, -1.0),
         ("rep", 1, float("nan")), ("which", 1, 3), ("which", 1, 2 ** 31 - 1)]


@gpu
@pytest.mark.parametrize("rows", [6, 340])
@pytest.mark.parametrize("name, at, value", WRONG)
def test_wrong_rows_are_not_written(name, at, value, rows):
    """The other rows are right; offsets belong to the rows on both their sides."""
    c = Case(9000, rows, 13, path=4, bias=6, masks=3)
    a = getattr(c, name)
    good = a.copy()
    a[at] = value
    wrong = {1} if not name.endswith("off") else {at - 1, at}
    if name == "off" and value == -1:
        wrong = {0, 1}
    bad = {n: getattr(c, m) for n, m in (("ranges", "ranges"), ("prompt_lens", "prompt"), ("path_offsets", "off"),
                                          ("bias_offsets", "boff"), ("repetition", "rep"), ("allowed_rows", "which"))
           if m == name}
    bad = {k: v.copy() for k, v in bad.items()}
    a[...] = good
    c.check(skip=wrong, code=mk.MK_ERR_INVALID_ARG, **bad)


@gpu
@pytest.mark.parametrize("rows", [4, 340])
@pytest.mark.parametrize("ids", [[5, 5, 7], [7, 5, 9], [-1, 5, 7], [5, 7, 9000], [5, 2 ** 31 - 1, 7]])
def test_bias_tokens_that_do_not_rise(ids, rows):
    c = Case(9000, rows, 14, history=20, masks=2)
    c.boff = np.array([0, 2, 5, 5] + [7] * (rows - 3), np.int32)
    c.bids = np.array([1, 8999] + [3, 4, 5] + [0, 4000], np.int32)
    c.bias = np.arange(7).astype(np.float32)
    bad = c.bids.copy()
    bad[2:5] = ids
    c.check(skip={1}, code=mk.MK_ERR_INVALID_ARG, bias_tokens=bad)


def test_create_and_null_handles():
    L, h = mk.lib(), ctypes.c_void_p()
    for vocab, rows, code in ((0, 1, 1), (1, 0, 1), (-5, 1, 1), ((1 << 24) + 1, 1, 8), (1, (1 << 24) + 1, 8)):
        assert L.mk_rules_create(vocab, rows, None, ctypes.byref(h)) == code
    assert L.mk_rules_create(5, 5, None, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_rules_apply(None, None, None, 0, 0, None, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_rules_sync(None) == mk.MK_ERR_INVALID_ARG
    L.mk_rules_destroy(None)


def test_check_and_follow_of_null_handles():
    assert mk.lib().mk_rules_check(None, None, None, 0, 0, None, None) == mk.MK_ERR_INVALID_ARG
    assert mk.lib().mk_rules_follow(None, None, None, None) == mk.MK_ERR_INVALID_ARG


def binding(vocab=100):
    """A TokenRules over host tensors that makes no call into the library."""
    import torch

    r = mk.TokenRules.__new__(mk.TokenRules)
    r.handle, r.device, r.vocab = None, torch.device("cpu"), vocab
    r._f32, r._bf16, r._int32 = torch.float32, torch.bfloat16, torch.int32
    return r


def test_the_binding_checks_batches():
    import torch

    i, f = lambda *s: torch.zeros(s, dtype=torch.int32), lambda *s: torch.zeros(s)
    r = binding()
    r.batch(3)
    r.batch(3, tokens=i(9), ranges=i(3, 2), prompt_lens=i(3), repetition=f(3), allowed=i(2, 4), allowed_rows=i(3))
    for bad in (dict(tokens=i(9)), dict(ranges=i(3, 2)), dict(prompt_lens=i(3)), dict(path_offsets=i(4)),
                dict(bias_offsets=i(4), bias_tokens=i(5)), dict(allowed_rows=i(3)),
                dict(tokens=i(9), ranges=i(2, 2)), dict(tokens=i(9), ranges=i(3, 3)),
                dict(path_offsets=i(3), path_tokens=i(5)), dict(repetition=f(4)), dict(allowed=i(3, 3)),
                dict(allowed=i(2, 4)), dict(bias_offsets=i(4), bias_tokens=i(5), bias=f(6)),
                dict(tokens=i(18)[::2], ranges=i(3, 2))):
        with pytest.raises(ValueError):
            r.batch(3, **bad)
    for bad in (dict(repetition=i(3)), dict(tokens=i(9).long(), ranges=i(3, 2)), dict(presence=f(3).double())):
        with pytest.raises(TypeError):
            r.batch(3, **bad)


@pytest.mark.parametrize("vocab, device", [(64, "cpu"), (4096, "cpu"), (100, "cuda:1")])
def test_batches_of_other_rules_are_refused(vocab, device):
    """A mask of 100 tokens has 4 words; under 4096 tokens 128 would be read."""
    import torch

    a, b = binding(), binding(vocab)
    for r in (a, b):
        r._index, r.max_rows, r._lib = -1, 2, mk.lib()
    b.device = torch.device(device)
    batch = a.batch(2, allowed=torch.zeros(2, 4, dtype=torch.int32))
    logits, tokens = torch.zeros(2, vocab), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: b.run(batch, logits, tokens=tokens), lambda: b.check(batch, logits, tokens=tokens),
                 lambda: b.follow(batch, logits, tokens)):
        with pytest.raises(ValueError, match="made by rules"):
            call()


def decoder(monkeypatch, vocab=100, batch=2):
    """(a Decoder over host tensors whose step only counts, the counts)."""
    import types

    import torch

    steps = []
    d = mk.Decoder.__new__(mk.Decoder)
    d.ctx, d.dims, d.batch, d.stream = None, types.SimpleNamespace(vocab=vocab), batch, 0
    d.device = torch.device("cpu")
    monkeypatch.setattr(mk, "mk_decode_step", lambda *a: steps.append(a))
    return d, steps


@pytest.mark.parametrize("other", [64, 99, 101, 4096])
def test_a_step_refuses_rules_of_another_vocabulary(monkeypatch, other):
    """Before the step, which writes rows of its own vocabulary over the tensor that the rules look at."""
    import torch

    d, steps = decoder(monkeypatch)
    r = binding(other)
    r._index, r.max_rows, r.stream = -1, 2, 0
    with pytest.raises(ValueError, match="vocabulary"):
        d.decode_step(torch.zeros(2, dtype=torch.int32), torch.zeros(2, other), torch.zeros(2, dtype=torch.int32),
                      rules=(r, r.batch(2)))
    assert not steps


def test_a_step_refuses_rules_of_another_device(monkeypatch):
    import torch

    d, steps = decoder(monkeypatch)
    r = binding()
    r._index, r.max_rows, r.stream = -1, 2, 0
    d.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="the decoder on cuda:1"):
        d.decode_step(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 100), torch.zeros(2, dtype=torch.int32),
                      rules=(r, r.batch(2)))
    assert not steps


@gpu
def test_wrong_calls_are_refused():
    c = Case(4096, 4, 15)
    t, rules = c.t, c.handle()
    b, x = c.batch(rules), c.logits()
    out, tok = t.zeros(4, 4096, device="cuda"), t.zeros(4, dtype=t.int32, device="cuda")
    for bad in (dict(logits=x[:3]), dict(logits=x.half()), dict(logits=x.cpu()), dict(logits=x.t().contiguous().t()),
                dict(out=out[:, :5]), dict(out=out.half()), dict(tokens=tok.long()), dict(tokens=tok[:2])):
        with pytest.raises(ValueError):
            rules.run(b, **{**dict(logits=x, out=out, tokens=tok), **bad})
    flat = t.zeros(5 * 4096 + 8, device="cuda")
    wide = t.zeros(4, 4100, device="cuda")
    for over in (dict(logits=x), dict(logits=flat[:4 * 4096].view(4, 4096), out=flat[4:4 + 4 * 4096].view(4, 4096)),
                 dict(logits=wide[:, :4096], out=wide.view(-1)[:4 * 4096].view(4, 4096)),
                 dict(logits=flat.view(t.bfloat16)[:4 * 4096].view(4, 4096), out=flat[:4 * 4096].view(4, 4096))):
        with pytest.raises(mk.MkError) as e:
            rules.run(b, **over)
        assert e.value.code == mk.MK_ERR_INVALID_ARG
    big = rules.batch(5)
    with pytest.raises(mk.MkError) as e:
        rules.run(big, t.zeros(5, 4096, device="cuda"), tokens=t.zeros(5, dtype=t.int32, device="cuda"))
    assert e.value.code == mk.MK_ERR_BATCH
    none = rules.batch(0)
    rules.run(none, t.zeros(0, 4096, device="cuda"), tokens=t.zeros(0, dtype=t.int32, device="cuda"))
    rules.sync()
    assert (out == 0).all() and (tok == 0).all()


@gpu
def test_captured_calls_follow_their_tensors():
    """Two handles in one graph; histories, masks and logits change between replays."""
    import torch

    cases = [Case(9000, 6, 20 + k, history=50, path=3, bias=5, masks=3) for k in range(2)]
    size = max(len(c.tokens) for c in cases) + 5, max(len(c.path) for c in cases), max(len(c.bids) for c in cases)
    for c in cases:
        c.tokens = np.concatenate([c.tokens, np.zeros(size[0] - len(c.tokens), np.int32)])
        c.path = np.concatenate([c.path, np.zeros(size[1] - len(c.path), np.int32)])
        c.bids = np.concatenate([c.bids, np.zeros(size[2] - len(c.bids), np.int32)])
        c.bias = np.concatenate([c.bias, np.zeros(size[2] - len(c.bias), np.float32)])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        a, b = cases[0].handle(stream), cases[0].handle(stream)
        batches = [cases[0].batch(a), cases[0].batch(b)]
        x = cases[0].logits()
        outs = [(torch.empty(6, 9000, device="cuda"), torch.empty(6, dtype=torch.int32, device="cuda")) for _ in range(2)]
        for h, bt, (o, k) in zip((a, b), batches, outs):
            h.run(bt, x, out=o, tokens=k)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for h, bt, (o, k) in zip((a, b), batches, outs):
                h.run(bt, x, out=o, tokens=k)
        for c in cases[::-1]:
            arrays = (c.tokens, c.ranges, c.prompt, c.off, c.path, c.rep, c.pres, c.freq, c.boff, c.bids, c.bias,
                      c.allowed, c.which)
            for bt in batches:
                for t, v in zip(bt.keep, arrays):
                    t.copy_(torch.from_numpy(v))
            x.copy_(c.x)
            graph.replay()
            a.sync(), b.sync()
            rows, tokens = c.want()
            for o, k in outs:
                assert np.array_equal(o.cpu().numpy(), rows) and np.array_equal(k.cpu().numpy(), tokens)


@gpu
def test_another_stream_than_the_current_one():
    c = Case(5000, 4, 30, masks=2)
    side = c.t.cuda.Stream()
    rules = c.handle(side)
    b, x, tok = c.batch(rules), c.logits(), c.t.empty(4, dtype=c.t.int32, device="cuda")
    c.t.cuda.synchronize()
    rules.run(b, x, tokens=tok)
    rules.sync()
    assert np.array_equal(tok.cpu().numpy(), c.want()[1])
