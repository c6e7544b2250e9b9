"""Drafted decoding over the paged cache, all of its calls together as a server makes them.

A small model (two layers of attention, random weights) is decoded one token at a time with single
appends and plain attention, and in rounds that verify a tree of drafted tokens: resize, append at the
tokens' depths, tree attention, rules, keep, resize.  Both have to choose the same tokens and to leave
the same cache."""
import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
from test_cache_decode import DIMS, Shared, i32

pytestmark = pytest.mark.gpu

HEADS, KV, D, P, V, LAYERS, WIDTH = 8, 2, 64, 16, 5000, 2, 40


class Model:
    """h = embed(token); per layer h += attention(h W) Wo; logits = h E^T."""

    def __init__(self, seed=0):
        import torch

        self.t = torch
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        d = HEADS * D
        self.embed = rand(V, d).to(torch.bfloat16)
        self.w = [(rand(d, (HEADS + 2 * KV) * D) / d ** 0.5).to(torch.bfloat16) for _ in range(LAYERS)]
        self.wo = [(rand(d, d) / d ** 0.5).to(torch.bfloat16) for _ in range(LAYERS)]
        self.head = (rand(d, V) / 3.0).to(torch.bfloat16)
        # the first layer's projection of every token: a product over other rows may round otherwise
        self.first = self.embed @ self.w[0]
        self.gains = [(1 + 0.2 * rand(2, D)).to(torch.bfloat16) for _ in range(LAYERS)]


class Server:
    def __init__(self, model, seqs, pages):
        t = self.t = model.t
        self.m, self.n = model, seqs
        self.pools = [t.zeros(pages, KV, P, D, dtype=t.bfloat16, device="cuda") for _ in range(2 * LAYERS)]
        self.tables = t.full((seqs, WIDTH), -1, dtype=t.int32, device="cuda")
        self.lens = t.zeros(seqs, dtype=t.int32, device="cuda")
        self.refs = t.zeros(pages, dtype=t.int32, device="cuda")
        self.cache = mk.KvCache(self.pools, self.tables, self.lens, self.refs, P)
        layers = list(zip(self.pools[::2], self.pools[1::2]))
        self.append = mk.KvAppend(HEADS, KV, D, P, layers, rotary_dim=48, rope_base=5000.0)
        self.attn = mk.PrefixAttention(HEADS, KV, D, P, layers, max_tokens=2048)
        self.rules = mk.TokenRules(V, 2048)
        self.history = [[] for _ in range(seqs)]
        self.prompt = [0] * seqs

    def resize(self, lens):
        self.cache.resize(i32(range(self.n)), i32(lens))

    def forward(self, tokens, offsets, tree=None, positions=None):
        """Logits of the tokens, whose places the cache has already."""
        t = self.t
        n = len(tokens)
        ids = i32(tokens).long()
        h = self.m.embed[ids]
        off = None if offsets is None else i32(offsets)
        batch = self.attn.batch(self.tables, self.lens, q_offsets=off, n_tokens=n)
        q_out = t.empty(n, HEADS, D, dtype=t.bfloat16, device="cuda")
        out = t.empty_like(q_out)
        for l in range(LAYERS):
            qkv = (self.m.first[ids] if l == 0 else h @ self.m.w[l]).view(n, HEADS + 2 * KV, D)
            q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
            self.append.run(l, batch, k, v, q=q, q_out=q_out, positions=positions, q_norm=self.m.gains[l][0],
                            k_norm=self.m.gains[l][1])
            self.attn.run(l, batch, q_out, out, tree=tree)
            h = h + out.view(n, -1) @ self.m.wo[l]
        return h @ self.m.head

    def choose(self, logits, seq_of, paths):
        """Greedy tokens under the rules; paths: drafted tokens between a row and its history."""
        t, n = self.t, len(seq_of)
        begins = np.concatenate([[0], np.cumsum([len(x) for x in self.history])])
        batch = self.rules.batch(
            n, tokens=i32([x for h in self.history for x in h]),
            ranges=i32([[begins[b], begins[b + 1]] for b in seq_of]), prompt_lens=i32([self.prompt[b] for b in seq_of]),
            path_offsets=i32(np.concatenate([[0], np.cumsum([len(p) for p in paths])])),
            path_tokens=i32([x for p in paths for x in p] + [0]), repetition=t.full((n,), 1.3, device="cuda"),
            presence=t.full((n,), 0.5, device="cuda"), frequency=t.full((n,), 0.2, device="cuda"),
            bias_offsets=i32(2 * np.arange(n + 1)), bias_tokens=i32([7, 11] * n),
            bias=t.tensor([3.0, -3.0] * n, device="cuda"))
        tokens, ruled = t.empty(n, dtype=t.int32, device="cuda"), t.empty(n, V, device="cuda")
        self.rules.run(batch, logits, out=ruled, tokens=tokens)
        self.rules.sync()
        top = ruled.topk(2).values
        return tokens.tolist(), (top[:, 0] - top[:, 1]).tolist()

    def prompts(self, prompts):
        self.history, self.prompt = [list(p) for p in prompts], [len(p) for p in prompts]
        self.resize([len(p) for p in prompts])
        offsets = np.concatenate([[0], np.cumsum([len(p) for p in prompts])])
        logits = self.forward([x for p in prompts for x in p], offsets)
        last = [int(o) - 1 for o in offsets[1:]]
        return self.choose(logits[last], range(self.n), [[]] * self.n)

    def sync(self):
        for h in (self.cache, self.append, self.attn, self.rules):
            h.sync()


def sequential(model, prompts, steps):
    """(tokens, margins) of every sequence, one step at a time, and the server."""
    s = Server(model, len(prompts), 400)
    nxt, margin = s.prompts(prompts)
    made, margins = [[x] for x in nxt], [[m] for m in margin]
    for _ in range(steps):
        for b, x in enumerate(nxt):
            s.history[b].append(x)
        s.resize([len(h) for h in s.history])
        nxt, margin = s.choose(s.forward(nxt, None), range(s.n), [[]] * s.n)
        for b in range(s.n):
            made[b].append(nxt[b])
            margins[b].append(margin[b])
    s.sync()
    return made, margins, s


def draft(rng, last, truth, size):
    """(tokens, parents) of a tree that begins with the last chosen token and holds some of what follows
    in truth, among other branches."""
    tokens, parents, line, right = [last], [-1], 0, 0
    follow = int(rng.integers(0, 6))
    while len(tokens) < size:
        if right < follow and right < len(truth) and rng.random() < 0.5:
            tokens.append(truth[right])
            parents.append(line)
            line, right = len(tokens) - 1, right + 1
        else:
            tokens.append(int(rng.integers(0, V)))
            parents.append(int(rng.integers(max(0, len(tokens) - 6), len(tokens) - 1)))
    return tokens, parents


@pytest.mark.parametrize("seed", [0, 1])
def test_drafted_rounds_choose_the_tokens_of_single_steps(seed):
    rng = np.random.default_rng(seed)
    model = Model(seed)
    prompts = [rng.integers(0, V, k).tolist() for k in (5, 40, 33, 1, 16)]
    steps = 40
    truth, margins, seq = sequential(model, prompts, steps)
    s = Server(model, len(prompts), 400)
    nxt, _ = s.prompts(prompts)
    made = [[x] for x in nxt]
    n, rounds = s.n, 0
    accepted_in_all = 0
    while min(len(m) for m in made) < steps - 8:
        rounds += 1
        trees = [draft(rng, made[b][-1], truth[b][len(made[b]):], int(rng.integers(1, 25))) for b in range(n)]
        context = [len(h) for h in s.history]                   # cached tokens: all but the last chosen one
        s.resize([c + len(tr[0]) for c, tr in zip(context, trees)])
        tree, depth = mk.tree_rows([p for _, p in trees])
        offsets = np.concatenate([[0], np.cumsum([len(tr[0]) for tr in trees])])
        seq_of = [b for b in range(n) for _ in trees[b][0]]
        positions = i32(depth.numpy() + np.array([context[b] for b in seq_of]))
        logits = s.forward([x for tr in trees for x in tr[0]], offsets, tree=tree.cuda(), positions=positions)
        paths = []
        for tokens, parents in trees:
            for i in range(len(tokens)):
                p, j = [], i
                while j >= 0:
                    p.append(tokens[j])
                    j = parents[j]
                paths.append(p[::-1])
        chosen, _ = s.choose(logits, seq_of, paths)
        picks, off = [], [0]
        for b, (tokens, parents) in enumerate(trees):
            at, path = 0, [0]
            while True:                                         # walk down while a child is what was chosen
                want = chosen[offsets[b] + at]
                made[b].append(want)
                down = [i for i in range(at + 1, len(tokens)) if parents[i] == at and tokens[i] == want]
                if not down:
                    break
                at = down[0]
                path.append(at)
            s.history[b] += [tokens[i] for i in path]
            picks += path
            off.append(len(picks))
        accepted_in_all += len(picks) - n
        s.cache.keep(i32(range(n)), i32(context), i32(off), i32(picks))
        s.resize([len(h) for h in s.history])
    s.sync()
    assert accepted_in_all > rounds                             # the rounds did accept drafts
    for b in range(n):
        k = min(len(made[b]), len(truth[b]))
        clear = [i for i in range(k) if margins[b][i] < 0.05]   # a near tie may go either way, and then all differs
        k = min([k] + clear)
        assert made[b][:k] == truth[b][:k]
        # the cache: layer 0 follows from tokens and positions alone, so it is the same bit for bit
        common = min(k, len(s.history[b]) - len(prompts[b]), len(seq.history[b]) - len(prompts[b])) + len(prompts[b])
        for pool in range(2 * LAYERS):
            rows = []
            for server in (s, seq):
                table = server.tables[b].tolist()
                rows.append(server.t.stack([server.pools[pool][table[i // P], :, i % P] for i in range(common)]).float())
            if pool < 2:
                assert model.t.equal(rows[0], rows[1])
            else:
                # behind an attention: both round its result and their products to bf16 (2^-8 of
                # values of size 1 to 4, each in a sum over 512)
                assert (rows[0] - rows[1]).abs().max() < 0.1


def test_prompts_appended_here_are_decoded_by_the_step():
    """K rows that KvAppend rotates are those the decode step writes, but for flips of a last bit."""
    import torch

    s = Shared(20)
    s.step([0], [5])
    dims = DIMS
    qkv = s.dec.dump_qkv()
    H, KVH, HD = dims.n_q_heads, dims.n_kv_heads, dims.head_dim
    lens, tables = s.cache.read([0])
    names = [(f"l{l}.kpool", f"l{l}.vpool") for l in range(dims.n_layers)]
    mine = [(s.pools[a].clone(), s.pools[b].clone()) for a, b in names]
    page, slot = int(tables[0, 20 // 16]), 20 % 16
    for k, v in mine:
        k[page, :, slot], v[page, :, slot] = 0, 0
    app = mk.KvAppend(H, KVH, HD, 16, mine, rope_base=dims.rope_base)
    batch = app.batch(i32(tables), i32(lens))
    for l in range(dims.n_layers):
        row = torch.from_numpy(qkv[l].copy().view(np.int16)).cuda().view(torch.bfloat16).view(1, -1, HD)
        app.run(l, batch, row[:, H:H + KVH], row[:, H + KVH:])
    app.sync()
    differ = total = 0
    for (k, v), (a, b) in zip(mine, names):
        assert torch.equal(v, s.pools[b])
        x, y = k.view(torch.int16).int(), s.pools[a].view(torch.int16).int()
        assert int((x - y).abs().max()) <= 1
        differ, total = differ + int((x != y).sum()), total + KVH * HD
    assert differ <= max(2, total // 64)


@pytest.mark.parametrize("batch", [1, 3])
def test_a_step_with_rules_behind_it(batch):
    """decode_step(rules=): the logits under the rules and their greedy tokens, on the step's stream."""
    import torch

    s = Shared(20)
    seqs = list(range(batch))
    if batch > 1:
        s.cache.fork(i32([0] * (batch - 1)), i32(seqs[1:]))
    tokens = np.arange(3, 3 + batch, dtype=np.int32)
    p = s.private(seqs)
    plain, first = s.step(seqs, tokens)
    V = DIMS.vocab
    rules = mk.TokenRules(V, batch)
    allowed = torch.zeros(batch, (V + 31) // 32, dtype=torch.int32, device="cuda")
    allowed[:, 3], allowed[:, 9] = -1, 5
    b = rules.batch(batch, tokens=i32(np.concatenate([first, tokens])), ranges=i32([[0, 2 * batch]] * batch),
                    repetition=torch.full((batch,), 2.0, device="cuda"), allowed=allowed)
    logits = torch.zeros(batch, V, device="cuda")
    nxt = torch.zeros(batch, dtype=torch.int32, device="cuda")
    dec = p.make()
    dec.build_schedule(p.lens, p.tables)
    dec.decode_step(i32(tokens), logits, nxt, rules=(rules, b))
    dec.sync()
    want = plain.copy()
    seen = np.unique(np.concatenate([first, tokens]))
    want[:, seen] = np.where(want[:, seen] > 0, want[:, seen] / np.float32(2), want[:, seen] * np.float32(2))
    may = np.zeros(V, bool)
    may[96:128], may[288], may[290] = True, True, True
    want[:, ~may] = -np.inf
    assert np.array_equal(logits.cpu().numpy(), want)
    assert np.array_equal(nxt.cpu().numpy(), want.argmax(1))
    with pytest.raises(ValueError, match="out_logits"):
        dec.decode_step(i32(tokens), None, nxt, rules=(rules, b))
    for bad in (rules.batch(batch + 1), rules.batch(batch - 1)):
        with pytest.raises(ValueError, match="rows"):
            dec.decode_step(i32(tokens), logits, nxt, rules=(rules, bad))
    for out, to in ((logits.half(), nxt), (logits[:, :-1], nxt), (logits, nxt.long())):
        with pytest.raises(ValueError):
            dec.decode_step(i32(tokens), out, to, rules=(rules, b))
    dec.sync()
    assert dec.stats().steps == 1                               # refused before the step
    other = mk.TokenRules(V, batch, stream=torch.cuda.Stream())
    with pytest.raises(ValueError, match="stream"):
        dec.decode_step(i32(tokens), logits, nxt, rules=(other, b))


def test_a_step_is_refused_with_its_rules():
    """What the library refuses on the host is refused before the step, which cannot be taken back."""
    import torch

    s = Shared(20)
    s.cache.fork(i32([0, 0]), i32([1, 2]))
    p = s.private([0, 1, 2])
    dec = p.make()
    dec.build_schedule(p.lens, p.tables)
    V = DIMS.vocab
    logits, nxt = torch.full((3, V), 5.0, device="cuda"), torch.full((3,), -9, dtype=torch.int32, device="cuda")
    small, rules, closed = mk.TokenRules(V, 2), mk.TokenRules(V, 3), mk.TokenRules(V, 3)
    closed.close()
    long = rules.batch(3, tokens=i32([1, 2]), ranges=i32([[0, 2]] * 3))
    long.n_tokens = 2 ** 29
    drafted = rules.batch(3, path_offsets=i32([0] * 4), path_tokens=i32([1]))
    drafted.n_path = 2 ** 31 - 1
    lost = rules.batch(3, prompt_lens=i32([0] * 3), tokens=i32([1, 2]), ranges=i32([[0, 2]] * 3))
    lost.ranges = None
    for r, b, code in ((small, small.batch(3), mk.MK_ERR_BATCH), (rules, long, mk.MK_ERR_UNSUPPORTED),
                       (rules, drafted, mk.MK_ERR_UNSUPPORTED), (rules, lost, mk.MK_ERR_INVALID_ARG),
                       (closed, rules.batch(3), mk.MK_ERR_INVALID_ARG)):
        with pytest.raises(mk.MkError) as e:
            dec.decode_step(i32([3, 4, 5]), logits, nxt, rules=(r, b))
        assert e.value.code == code
    dec.sync()
    assert dec.stats().steps == 0
    assert (logits == 5.0).all() and (nxt == -9).all()


@pytest.mark.parametrize("wrong", ["repetition", "mask", "bias"])
def test_a_row_whose_rules_are_wrong_has_no_token(wrong):
    """Not the step's own, which the rules never saw; the decoder's sync() raises, once; the step behind it is
    right again."""
    import torch

    s = Shared(20)
    s.cache.fork(i32([0, 0]), i32([1, 2]))
    seqs, tokens = [0, 1, 2], np.array([3, 4, 5], np.int32)
    p = s.private(seqs)
    plain, first = s.step(seqs, tokens)
    V = DIMS.vocab
    rules = mk.TokenRules(V, 5)
    repetition = torch.full((3,), 2.0, device="cuda")
    allowed = torch.zeros(1, (V + 31) // 32, dtype=torch.int32, device="cuda")
    allowed[0, 3] = -1                                           # 96 to 127
    which, ids = i32([-1, 0, 0]), i32([7, 9, 11, 100, 101, 102])
    b = rules.batch(3, repetition=repetition, allowed=allowed, allowed_rows=which, bias_offsets=i32([0, 2, 4, 6]),
                    bias_tokens=ids, bias=torch.zeros(6, device="cuda"))
    logits, nxt = torch.zeros(3, V, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    dec = p.make()
    dec.build_schedule(p.lens, p.tables)
    if wrong == "repetition":
        repetition[1] = 0.0
    elif wrong == "mask":
        which[1] = 1
    else:
        ids[2] = 100
    dec.decode_step(i32(tokens), logits, nxt, rules=(rules, b))
    with pytest.raises(mk.MkError) as e:
        dec.sync()
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    dec.sync()
    rules.sync()
    masked = plain.copy()
    masked[:, :96], masked[:, 128:] = -np.inf, -np.inf
    got = logits.cpu().numpy()
    assert nxt.tolist() == [int(first[0]), -1, int(masked[2].argmax())]
    assert np.array_equal(got[:2], plain[:2]) and np.array_equal(got[2], masked[2])
    repetition[1], which[1], ids[2] = 2.0, 0, 11
    dec.build_schedule(p.lens, p.tables)
    dec.decode_step(i32(tokens), logits, nxt, rules=(rules, b))
    dec.sync()
    assert nxt.tolist() == [int(first[0])] + [int(x) for x in masked[1:].argmax(1)]


def test_rules_that_are_gone_do_not_matter_to_sync():
    import torch

    s = Shared(20)
    p = s.private([0])
    dec = p.make()
    dec.build_schedule(p.lens, p.tables)
    logits, nxt = torch.zeros(1, DIMS.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for close in (True, False):
        rules = mk.TokenRules(DIMS.vocab, 1)
        dec.decode_step(i32([3]), logits, nxt, rules=(rules, rules.batch(1)))
        if close:
            rules.close()
        else:
            del rules
        dec.sync()
    assert int(nxt) == int(logits.argmax())
