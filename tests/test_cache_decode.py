"""The paged-cache calls around the decode step, together, as a sampler uses them (GPU).

One prompt is forked into samples, the samples grow and decode with mk_decode_step,
some finish, the pool is compacted, and decoding goes on.  The step's arithmetic
depends on the lengths (they cut its attention) and on its decoder's history (the
experts seen weigh the cut), but not on which physical pages hold a sequence; so
with a new decoder for each step on both sides every logit has to be the same, bit
for bit, as with private contiguous copies of the cache.  The
attention of the step (dumped per layer) is compared with mk_prefix_attention over
the same shared pages."""
import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
import synth
from bf16util import to_f32, ulp

pytestmark = pytest.mark.gpu

DIMS = synth.TINY
P = DIMS.page_size


class Private:
    """The same sequences with pages of their own, copied whole."""

    def __init__(self, weights, pools, lens, tables, room):
        import torch

        n, width = len(lens), -(-(max(lens) + room) // P)
        self.torch, self.lens = torch, list(lens)
        self.tables = np.arange(n * width, dtype=np.int32).reshape(n, width)
        tensors = dict(weights)
        for name, pool in pools.items():
            t = torch.zeros((n * width,) + tuple(pool.shape[1:]), dtype=pool.dtype, device="cuda")
            for b, L in enumerate(lens):
                k = -(-L // P)
                t[self.tables[b, :k].tolist()] = pool[tables[b, :k].tolist()]
            tensors[name] = t
        self.make = lambda: mk.Decoder(DIMS, tensors, n * width, width, n)

    def step(self, tokens):
        dec = self.make()
        dec.build_schedule(self.lens, self.tables)
        self.lens = [L + 1 for L in self.lens]
        return step(dec, tokens)


def step(dec, tokens):
    import torch

    n = len(tokens)
    tok = torch.tensor(np.asarray(tokens, np.int32), device="cuda")
    logits = torch.zeros(n, DIMS.vocab, device="cuda")
    nxt = torch.zeros(n, dtype=torch.int32, device="cuda")
    dec.decode_step(tok, logits, nxt)
    dec.sync()
    return logits.cpu().numpy(), nxt.cpu().numpy()


def i32(v):
    import torch

    return torch.tensor(np.asarray(v, np.int32), device="cuda")


class Shared:
    def __init__(self, prompt, rows=8, pages=64, width=12):
        import torch

        inp = synth.device_inputs(DIMS, [pages * P], 0)      # weights, and pools of `pages` pages
        names = [f"l{l}.{k}" for l in range(DIMS.n_layers) for k in ("kpool", "vpool")]
        shape = (pages, DIMS.n_kv_heads, P, DIMS.head_dim)
        self.pools = {n: inp.tensors[n].view(torch.bfloat16).view(shape) for n in names}
        self.weights = {n: t for n, t in inp.tensors.items() if n not in self.pools}
        tables = np.full((rows, width), -1, np.int32)
        used = -(-prompt // P)
        order = np.random.default_rng(3).permutation(pages)[:used]
        tables[0, :used] = order
        refs = np.zeros(pages, np.int32)
        refs[order] = 1
        lens = np.zeros(rows, np.int32)
        lens[0] = prompt
        self.cache = mk.KvCache([self.pools[n] for n in names], i32(tables), i32(lens), i32(refs), P)
        self.make = lambda: mk.Decoder(DIMS, {**self.weights, **self.pools}, pages, width, rows)

    def private(self, seqs, room=16):
        lens, tables = self.cache.read(seqs)
        return Private(self.weights, self.pools, [int(x) for x in lens], tables, room)

    def step(self, seqs, tokens):
        """The next token of each sequence: its page first, then the step."""
        lens, _ = self.cache.read(seqs)
        self.cache.resize(i32(seqs), i32(lens + 1))
        self.dec = self.make()
        self.dec.schedule_cache(self.cache, seqs)
        return step(self.dec, tokens)


def rope(x, pos):
    """Rotate-half RoPE of bf16 rows [heads][D] at a position, rounded to bf16 (as bits)."""
    import torch

    half = DIMS.head_dim // 2
    a = pos * 10000.0 ** (-2.0 * np.arange(half) / DIMS.head_dim)
    c, s = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    lo, hi = x[:, :half], x[:, half:]
    y = np.concatenate([lo * c - hi * s, hi * c + lo * s], 1).astype(np.float32)
    return torch.from_numpy(y).to(torch.bfloat16)


def attention_agrees(s, seqs, prompt):
    """The step's attention output of every layer against mk_prefix_attention."""
    import torch

    lens, tables = s.cache.read(seqs)
    qkv, o = s.dec.dump_qkv(), s.dec.dump_o()
    H, D = DIMS.n_q_heads, DIMS.head_dim
    layers = [(s.pools[f"l{l}.kpool"], s.pools[f"l{l}.vpool"]) for l in range(DIMS.n_layers)]
    attn = mk.PrefixAttention(H, DIMS.n_kv_heads, D, P, layers, max_tokens=len(seqs))
    batch = attn.batch(i32(tables), i32(lens), group_starts=i32([0, len(seqs)]),
                       prefix_lens=i32([prompt]))
    for l in range(DIMS.n_layers):
        q = torch.stack([rope(to_f32(qkv[l, b, :H * D]).reshape(H, D), int(lens[b]) - 1)
                         for b in range(len(seqs))]).cuda()
        out = torch.empty_like(q)
        attn.run(l, batch, q, out)
        attn.sync()
        got = out.float().cpu().numpy().reshape(len(seqs), H * D)
        want = to_f32(o[l]).astype(np.float64)
        rms = np.sqrt(np.mean(want * want, -1, keepdims=True))
        # both round to bf16 (one flip each, two ulps), probabilities in bf16 on this side, and a
        # flipped bit of q moves a whole head (2^-5 of the row's rms: harness.layer_check)
        assert (np.abs(got - want) <= 2.0 * ulp(want) + 2.0 ** -5 * rms).all(), l


@pytest.mark.parametrize("prompt", [37, 48, 5])
def test_samples_of_one_prompt(prompt):
    s = Shared(prompt)
    seqs = [0, 1, 2, 3, 4]
    s.cache.fork(i32([0] * 4), i32([1, 2, 3, 4]))
    lens, tables = s.cache.read(seqs)
    full = prompt // P
    assert (tables[:, :full] == tables[0, :full]).all()
    p = s.private(seqs)
    tokens = np.array([3, 700, 41, 9, 512], np.int32)
    for _ in range(14):
        a, na = s.step(seqs, tokens)
        b, nb = p.step(tokens)
        assert np.array_equal(a, b) and np.array_equal(na, nb)
        attention_agrees(s, seqs, prompt)
        tokens = na
    # two samples finish, one is forked again, the rest moves together
    s.cache.resize(i32([1, 4]), i32([0, 0]))
    s.cache.fork(i32([2, 0]), i32([5, 6]))
    s.cache.compact()
    s.cache.sync()
    refs = s.cache.page_refs.cpu().numpy()
    held = int((refs > 0).sum())
    assert (refs[:held] > 0).all() and held < len(refs)
    seqs, tokens = [0, 2, 3, 5, 6], np.array([17, 1000, 8, 77, 300], np.int32)
    p = s.private(seqs)
    for _ in range(6):
        a, na = s.step(seqs, tokens)
        b, nb = p.step(tokens)
        assert np.array_equal(a, b) and np.array_equal(na, nb)
        attention_agrees(s, seqs, prompt // P * P)
        tokens = na


def test_beams_of_one_prompt():
    """Beams follow one another each step; each step's logits equal private copies' logits."""
    s = Shared(21)
    seqs = [0, 1, 2, 3]
    s.cache.fork(i32([0] * 3), i32([1, 2, 3]))
    tokens = np.array([1, 2, 3, 4], np.int32)
    rng = np.random.default_rng(0)
    for _ in range(12):
        parents = rng.integers(0, 4, 4)
        s.cache.fork(i32(parents), i32(seqs))
        p = s.private(seqs)
        a, na = s.step(seqs, tokens[parents])
        b, nb = p.step(tokens[parents])
        assert np.array_equal(a, b) and np.array_equal(na, nb)
        tokens = na + rng.integers(0, 3, 4).astype(np.int32)


def test_schedule_cache_checks_the_tables_width():
    s = Shared(20)
    other = mk.Decoder(DIMS, {**s.weights, **s.pools}, 64, 9, 4)
    with pytest.raises(ValueError):
        other.schedule_cache(s.cache, [0])
