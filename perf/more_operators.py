"""One round of drafted decoding over the paged cache: measured cases, plain forms and exact values.

Keys and values of prompts and drafts are normed, rotated and appended to the pages (append), a tree of drafted
tokens attends to them (tree), penalties, biases and grammar masks are put on the logits and the greedy tokens chosen
(rules), and the rows of the accepted path move together (keep).  The cache is the decode step's: per layer a K and a
V pool [pages][kv heads][page size][head dim] in bf16, and table rows of page ids.
"""
import math
import random

import numpy as np
import torch

own = False

# (layers, q heads, kv heads, head dim, vocabulary): the framework's tiny, mid and full models and its odd test shape
MODELS = {"tiny": (2, 4, 2, 64, 1024), "odd": (2, 6, 2, 32, 300), "mid": (8, 16, 4, 64, 32000),
          "full": (48, 32, 4, 128, 152064)}


def listed():
    return [
        # a decode step of eight long sequences: latency counts
        {"name": "append_step", "op": "append", "model": "full", "page": 16, "seqs": 8, "tokens": 1, "cached": 131072,
         "norm": True, "interleaved": False, "rotary": 128, "tree": False, "factor": 8.0},
        # drafted trees of many sequences, positions by depth; half of a head turns, neighbours paired
        {"name": "append_drafts", "op": "append", "model": "mid", "page": 16, "seqs": 64, "tokens": 24, "cached": 4000,
         "norm": False, "interleaved": True, "rotary": 32, "tree": True, "factor": 1.0},
        # ragged prompts of the full-scale model, all tokens at once
        {"name": "append_prompts", "op": "append", "model": "full", "page": 16, "seqs": 8, "tokens": 4000, "cached": 0,
         "norm": True, "interleaved": False, "rotary": 128, "tree": False, "factor": 1.0},
        # one small tree over a short context: latency counts
        {"name": "tree_small", "op": "tree", "model": "mid", "page": 16, "groups": 0, "seqs": 1, "prefix": 0,
         "context": 600, "nodes": 16},
        # eight ragged sequences of the full model's heads, a tree of up to 64 tokens each
        {"name": "tree_batch", "op": "tree", "model": "full", "page": 16, "groups": 0, "seqs": 8, "prefix": 0,
         "context": 8192, "nodes": 64},
        # two prompts with eight samples each, small trees
        {"name": "tree_samples", "op": "tree", "model": "full", "page": 16, "groups": 2, "seqs": 16, "prefix": 16384,
         "context": 300, "nodes": 24},
        # two very long contexts
        {"name": "tree_long", "op": "tree", "model": "full", "page": 16, "groups": 0, "seqs": 2, "prefix": 0,
         "context": 131072, "nodes": 48},
        # one sequence of the mid model, logits of one step: latency counts
        {"name": "rules_one", "op": "rules", "vocab": 32000, "seqs": 1, "nodes": 1, "history": 300, "half": False,
         "bias": 20, "masks": 1},
        # a decode step of eight sequences at the full vocabulary
        {"name": "rules_step", "op": "rules", "vocab": 152064, "seqs": 8, "nodes": 1, "history": 8192, "half": False,
         "bias": 100, "masks": 6},
        # all tokens of eight drafted trees, the sequences' histories shared by their tokens
        {"name": "rules_tree", "op": "rules", "vocab": 152064, "seqs": 8, "nodes": 48, "history": 8192, "half": True,
         "bias": 100, "masks": 40},
        # the accepted paths of a few sequences of the mid model: latency counts
        {"name": "keep_few", "op": "keep", "model": "mid", "page": 16, "seqs": 4, "cached": 500, "nodes": 16, "depth": 4},
        # a large batch of the full model
        {"name": "keep_full", "op": "keep", "model": "full", "page": 16, "seqs": 64, "cached": 200, "nodes": 64,
         "depth": 8},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "rules", "keep"])
    model = rng.choice(["tiny", "odd", "mid", "full"])
    page = rng.choice([16, 16, 32, 64])
    if op == "append":
        c = {"op": op, "model": model, "page": page, "seqs": _log(rng, 1, 200), "cached": rng.choice([0, _log(rng, 1, 200000)]),
             "norm": rng.random() < 0.5, "interleaved": rng.random() < 0.4, "factor": rng.choice([1.0, 4.0, 8.0, 32.0])}
        c["tokens"] = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, max(2, 24000 // c["seqs"]))])
        dim = MODELS[model][3]
        c["rotary"] = rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        c["tree"] = 1 < c["tokens"] <= 64 and rng.random() < 0.6
        return c
    if op == "tree":
        c = {"op": op, "model": model, "page": page, "groups": rng.choice([0, 0, 1, 2, 3]), "seqs": _log(rng, 1, 48),
             "prefix": 0, "context": _log(rng, 1, 60000)}
        c["nodes"] = rng.choice([1, 5, 8, 16, 33, 64, _log(rng, 2, 300)])
        if c["groups"]:
            c["prefix"] = _log(rng, 1, 65536)
            c["seqs"] = c["groups"] * max(1, c["seqs"] // c["groups"])
        c["context"] = max(1, min(c["context"], 200000 // c["seqs"]))
        while c["nodes"] > 1 and c["seqs"] * c["nodes"] * MODELS[model][1] * (c["prefix"] + c["context"] + c["nodes"]) > 3e8:
            c["nodes"] = max(1, c["nodes"] // 2)
        return c
    if op == "rules":
        vocab = rng.choice([MODELS[model][4], _log(rng, 200, 150000)])
        c = {"op": op, "vocab": vocab, "seqs": _log(rng, 1, 32), "nodes": rng.choice([1, 1, _log(rng, 2, 64)]),
             "history": rng.choice([0, _log(rng, 1, 16000)]), "half": rng.random() < 0.5, "bias": rng.choice([0, _log(rng, 1, 120)]),
             "masks": rng.choice([0, rng.randint(1, 40)])}
        while c["nodes"] > 1 and c["seqs"] * c["nodes"] * vocab > 5e7:
            c["nodes"] = max(1, c["nodes"] // 2)
        return c
    c = {"op": op, "model": model, "page": page, "seqs": _log(rng, 1, 128), "cached": _log(rng, 1, 300), "nodes": _log(rng, 2, 100)}
    c["depth"] = rng.randint(1, min(c["nodes"], 9))
    layers, _, kv, dim, _ = MODELS[model]
    while c["seqs"] > 1 and c["seqs"] * (c["cached"] + c["nodes"] + 2 * page) * layers * kv * dim * 4 > 3e9:
        c["seqs"] //= 2
    return c


# ------------------------------------------------------------------------------------------------ inputs


class State:
    pass


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _parents(rng, n):
    """A drafted tree, parents first: each token's parent, -1 for those that follow the context itself."""
    near = rng.choice([2, 4, n])
    return [-1 if i == 0 or rng.random() < 0.02 else rng.randint(max(0, i - near), i - 1) for i in range(n)]


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _counts(most, n, key):
    """Ragged token counts of n sequences: the outputs' shape, so the same for every seed."""
    r = random.Random(key)
    return [r.randint(max(1, most // 2), most) for _ in range(n)]


def _frequencies(rotary, factor):
    """Turning rates of a context longer by `factor` than the 8192 positions of before: fast pairs keep theirs, slow
    ones take 1 / factor of it, those between 1 and 4 turns over the old context a blend."""
    f = 10000.0 ** (-2.0 * torch.arange(rotary // 2, dtype=torch.float64) / rotary)
    blend = ((f * 8192 / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
    return f if factor == 1.0 else f * (blend + (1.0 - blend) / factor)


def _prepare_append(case, seed):
    s = State()
    rng = random.Random(seed * 7919 + 3)
    _, s.hq, s.hkv, s.dim, _ = MODELS[case["model"]]
    P, n = case["page"], case["seqs"]
    s.P, s.rotary, s.interleaved = P, case["rotary"], case["interleaved"]
    s.counts = _counts(case["tokens"], n, case["tokens"])
    cached = [case["cached"] - rng.randint(0, case["cached"] // 2) for _ in range(n)]
    s.lens_list = [a + b for a, b in zip(cached, s.counts)]
    # pages of the new tokens; those cached before are not touched, and all named 0 here
    need = [(-(-L // P)) - c // P for L, c in zip(s.lens_list, cached)]
    total = sum(need) + 4
    order = list(range(1, total))
    rng.shuffle(order)
    wide = -(-(case["cached"] + case["tokens"]) // P) + 1
    tables = np.full((n, wide), -1, np.int32)
    at = 0
    for b in range(n):
        tables[b, :cached[b] // P] = 0
        tables[b, cached[b] // P:cached[b] // P + need[b]] = order[at:at + need[b]]
        at += need[b]
    s.tables = torch.from_numpy(tables).cuda()
    s.tables_np = tables
    s.lens = _ints(s.lens_list)
    offsets = [0]
    for t in s.counts:
        offsets.append(offsets[-1] + t)
    s.offsets_list = offsets
    s.offsets = _ints(offsets) if case["tokens"] > 1 else None
    s.positions = None
    if case["tree"]:
        s.positions_list = [c + d for c, t in zip(cached, s.counts) for d in _depths(_parents(rng, t))]
        s.positions = _ints(s.positions_list)
    else:
        s.positions_list = [c + i for c, t in zip(cached, s.counts) for i in range(t)]
    # as many pages for every seed: the pools are outputs
    pool = sum(-(-t // P) + 1 for t in s.counts) + 4
    g = torch.Generator("cuda").manual_seed(seed)
    shape = (pool, s.hkv, P, s.dim)
    s.k = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    s.v = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    # q, k and v side by side, as a fused projection leaves them
    s.qkv = torch.empty(offsets[-1], s.hq + 2 * s.hkv, s.dim, dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.0, generator=g)
    s.wq = s.wk = None
    if case["norm"]:
        s.wq = torch.empty(s.dim, dtype=torch.bfloat16, device="cuda").normal_(1.0, 0.2, generator=g)
        s.wk = torch.empty(s.dim, dtype=torch.bfloat16, device="cuda").normal_(1.0, 0.2, generator=g)
    s.freq = _frequencies(s.rotary, case["factor"])
    s.freq_gpu = s.freq.cuda()
    s.eps, s.magnitude = 1e-6, 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
    if own:
        import persistent_moe_decode_sm_gb300 as mk

        s.q_out = torch.empty(offsets[-1], s.hq, s.dim, dtype=torch.bfloat16, device="cuda")
        s.append = mk.KvAppend(s.hq, s.hkv, s.dim, P, [(s.k, s.v)], rotary_dim=s.rotary, interleaved=s.interleaved,
                               frequencies=s.freq.tolist(), magnitude=s.magnitude, norm_eps=s.eps)
        s.batch = s.append.batch(s.tables, s.lens, q_offsets=s.offsets, n_tokens=offsets[-1])
    return s


def _prepare_tree(case, seed):
    s = State()
    rng = random.Random(seed * 104729 + 7)
    _, s.hq, s.hkv, s.dim, _ = MODELS[case["model"]]
    P, n, groups = case["page"], case["seqs"], case["groups"]
    each = n // groups if groups else 1
    s.P = P
    s.counts = _counts(case["nodes"], n, case["nodes"])
    # the later groups share shorter prefixes
    prefix = [max(1, case["prefix"] >> (2 * i)) for i in range(groups)]
    before = [case["context"] - rng.randint(0, case["context"] // 4) for _ in range(n)]
    s.lens_list = [(prefix[i // each] if groups else 0) + before[i] + s.counts[i] for i in range(n)]
    used = [-(-L // P) for L in s.lens_list]
    shared = [L // P for L in prefix]
    total = sum(shared) + sum(used[i] - (shared[i // each] if groups else 0) for i in range(n)) + 3
    order = np.random.RandomState(rng.randrange(1 << 31)).permutation(total)
    heads, at = [], 0
    for k in shared:
        heads.append(order[at:at + k])
        at += k
    tables = np.full((n, max(used) + 2), -1, np.int32)
    for i in range(n):
        h = shared[i // each] if groups else 0
        if h:
            tables[i, :h] = heads[i // each]
        tables[i, h:used[i]] = order[at:at + used[i] - h]
        at += used[i] - h
    s.tables_np = tables
    s.tables, s.lens = torch.from_numpy(tables).cuda(), _ints(s.lens_list)
    s.offsets_list = [0]
    for t in s.counts:
        s.offsets_list.append(s.offsets_list[-1] + t)
    s.offsets = _ints(s.offsets_list)
    s.starts = _ints([i * each for i in range(groups + 1)]) if groups else None
    s.prefix_lens = _ints(prefix) if groups else None
    # what each token sees of its tree, a bit for each drafted token
    words = -(-case["nodes"] // 32)
    s.parents = [_parents(rng, t) for t in s.counts]
    bits = np.zeros((s.offsets_list[-1], words * 32), np.uint8)
    for b, parents in enumerate(s.parents):
        rows = bits[s.offsets_list[b]:s.offsets_list[b + 1]]
        for i, p in enumerate(parents):
            if p >= 0:
                rows[i] = rows[p]
            rows[i, i] = 1
    s.tree = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()
    g = torch.Generator("cuda").manual_seed(seed)
    shape = (total, s.hkv, P, s.dim)
    s.k = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    s.v = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    s.q = torch.empty(s.offsets_list[-1], s.hq, s.dim, dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.0, generator=g)
    if own:
        import persistent_moe_decode_sm_gb300 as mk

        s.out = torch.empty_like(s.q)
        s.lse = torch.empty(s.q.shape[:2], dtype=torch.float32, device="cuda")
        s.attn = mk.PrefixAttention(s.hq, s.hkv, s.dim, P, [(s.k, s.v)], max_tokens=s.offsets_list[-1])
        s.batch = s.attn.batch(s.tables, s.lens, q_offsets=s.offsets, group_starts=s.starts, prefix_lens=s.prefix_lens)
    return s


def _prepare_rules(case, seed):
    s = State()
    rng = random.Random(seed * 15485863 + 1)
    V, n = case["vocab"], case["seqs"] * case["nodes"]
    g = torch.Generator("cuda").manual_seed(seed)
    s.V, s.rows = V, n
    s.logits = torch.empty(n, V, dtype=torch.float32, device="cuda").normal_(0.0, 3.0, generator=g)
    if case["half"]:
        s.logits = s.logits.to(torch.bfloat16)

    def words(count):  # text: few words often, many seldom
        return (torch.rand(count, device="cuda", generator=g).double() ** 4 * V).to(torch.int32).clamp(max=V - 1)

    # a sequence's history, and what lies between it and a drafted token (the same lengths for every seed are not
    # needed: no output has their shape)
    s.ranges = s.tokens = s.path_offsets = s.path = s.prompt = None
    s.rep = s.pres = s.freq = None
    if case["history"]:
        lens = [case["history"] - rng.randint(0, case["history"] // 2) for _ in range(case["seqs"])]
        ends = np.cumsum([0] + lens)
        s.tokens = words(int(ends[-1]))
        s.ranges = _ints([[int(ends[b]), int(ends[b + 1])] for b in range(case["seqs"]) for _ in range(case["nodes"])])
        s.prompt = _ints([int(lens[b] * 0.4) for b in range(case["seqs"]) for _ in range(case["nodes"])])
        depth = [rng.randint(0, 8) if case["nodes"] > 1 else 0 for _ in range(n)]
        if case["nodes"] > 1:
            s.path_offsets = _ints(np.cumsum([0] + depth).tolist())
            s.path = words(max(1, sum(depth)))
        s.rep = 1.0 + 0.5 * torch.rand(n, device="cuda", generator=g)
        s.pres = torch.rand(n, device="cuda", generator=g)
        s.freq = 0.3 * torch.rand(n, device="cuda", generator=g)
    s.bias_offsets = s.bias_tokens = s.bias = None
    if case["bias"]:
        some = [rng.randint(0, min(case["bias"], V)) for _ in range(n)]
        ids = [sorted(rng.sample(range(V), k)) for k in some]
        s.bias_offsets = _ints(np.cumsum([0] + some).tolist())
        s.bias_tokens = _ints([i for row in ids for i in row] or [0])
        s.bias = torch.empty(max(1, sum(some)), device="cuda").normal_(0.0, 4.0, generator=g)
    s.allowed = s.allowed_rows = None
    if case["masks"]:
        # some grammars leave few tokens, some most
        bits = torch.rand(case["masks"], -(-V // 32) * 32, device="cuda", generator=g) < torch.rand(
            case["masks"], 1, device="cuda", generator=g) ** 3 + 0.002
        bits[:, :1] = True
        weights = (1 << torch.arange(31, device="cuda", dtype=torch.int64)).tolist() + [-(1 << 31)]
        s.allowed = (bits.view(case["masks"], -1, 32).long() * torch.tensor(weights, device="cuda")).sum(-1).to(torch.int32)
        s.allowed_rows = _ints([rng.randint(-1, case["masks"] - 1) for _ in range(n)])
    if own:
        import persistent_moe_decode_sm_gb300 as mk

        s.out = torch.empty(n, V, dtype=torch.float32, device="cuda")
        s.chosen = torch.empty(n, dtype=torch.int32, device="cuda")
        s.rules = mk.TokenRules(V, max_rows=n)
        s.batch = s.rules.batch(n, tokens=s.tokens, ranges=s.ranges, prompt_lens=s.prompt, path_offsets=s.path_offsets,
                                path_tokens=s.path, repetition=s.rep, presence=s.pres, frequency=s.freq,
                                bias_offsets=s.bias_offsets, bias_tokens=s.bias_tokens, bias=s.bias, allowed=s.allowed,
                                allowed_rows=s.allowed_rows)
    return s


def _prepare_keep(case, seed):
    s = State()
    rng = random.Random(seed * 32452843 + 9)
    layers, _, s.hkv, s.dim, _ = MODELS[case["model"]]
    P, n = case["page"], case["seqs"]
    s.P = P
    start = [case["cached"] - rng.randint(0, case["cached"] // 3) for _ in range(n)]
    picks, offsets = [], [0]
    for _ in range(n):
        # the accepted path of a tree: its first token, then some way down
        depth = rng.randint(1, case["depth"])
        picks += [0] + sorted(rng.sample(range(1, case["nodes"]), depth - 1))
        offsets.append(len(picks))
    per = -(-(case["cached"] + case["nodes"]) // P)
    order = np.random.RandomState(rng.randrange(1 << 31)).permutation(n * per + 2)
    tables = order[:n * per].reshape(n, per).astype(np.int32)
    used = [-(-(L + case["nodes"]) // P) for L in start]
    refs = np.zeros(n * per + 2, np.int32)
    for b in range(n):
        tables[b, used[b]:] = -1
        refs[tables[b, :used[b]]] = 1
    s.tables, s.refs = torch.from_numpy(tables).cuda(), torch.from_numpy(refs).cuda()
    s.lens = _ints([L + case["nodes"] for L in start])
    s.seqs, s.start, s.offsets, s.picks = _ints(list(range(n))), _ints(start), _ints(offsets), _ints(picks)
    s.which = _ints([b for b in range(n) for _ in range(offsets[b + 1] - offsets[b])])
    g = torch.Generator("cuda").manual_seed(seed)
    s.pool = torch.empty(2 * layers, n * per + 2, s.hkv, P, s.dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    if own:
        import persistent_moe_decode_sm_gb300 as mk

        s.cache = mk.KvCache(list(s.pool), s.tables, s.lens, s.refs, page_size=P)
    return s


def prepare(case, seed):
    s = {"append": _prepare_append, "tree": _prepare_tree, "rules": _prepare_rules, "keep": _prepare_keep}[case["op"]](case, seed)
    s.op = case["op"]
    return s


# ------------------------------------------------------------------------------------------------ one pass


def _norm(x, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _turn(x, cos, sin, rotary, interleaved):
    """x [tokens][heads][D] in 32 bits with its first `rotary` dims turned."""
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rotary // 2], r[..., rotary // 2:])
    c, s = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([c, s], -1).flatten(-2) if interleaved else torch.cat([c, s], -1)
    return torch.cat([r, x[..., rotary:]], -1)


def _append(s):
    q, k, v = s.qkv[:, :s.hq], s.qkv[:, s.hq:s.hq + s.hkv], s.qkv[:, s.hq + s.hkv:]
    if own:
        s.append.run(0, s.batch, k, v, q=q, q_out=s.q_out, positions=s.positions, q_norm=s.wq, k_norm=s.wk)
        return {"q": s.q_out, "k": s.k, "v": s.v}
    tokens = q.shape[0]
    if s.offsets is None:
        row, slot = torch.arange(tokens, device="cuda"), s.lens.long() - 1
    else:
        off = s.offsets.long()
        row = torch.bucketize(torch.arange(tokens, device="cuda"), off[1:], right=True)
        slot = s.lens.long()[row] - off[row + 1] + torch.arange(tokens, device="cuda")
    at = slot if s.positions is None else s.positions.long()
    angle = at[:, None, None].double() * s.freq_gpu
    cos, sin = (angle.cos() * s.magnitude).float(), (angle.sin() * s.magnitude).float()
    q, k = q.float(), k.float()
    if s.wq is not None:
        q, k = _norm(q, s.wq, s.eps), _norm(k, s.wk, s.eps)
    page = s.tables[row, slot // s.P].long()
    s.k[page, :, slot % s.P] = _turn(k, cos, sin, s.rotary, s.interleaved).to(torch.bfloat16)
    s.v[page, :, slot % s.P] = v
    return {"q": _turn(q, cos, sin, s.rotary, s.interleaved).to(torch.bfloat16), "k": s.k, "v": s.v}


def _tree(s):
    if own:
        s.attn.run(0, s.batch, s.q, s.out, s.lse, tree=s.tree)
        return {"out": s.out, "lse": s.lse}
    P, G, tokens = s.P, s.hq // s.hkv, s.q.shape[0]
    out = torch.empty(tokens, s.hq, s.dim, device="cuda")
    lse = torch.empty(tokens, s.hq, device="cuda")
    q = s.q.float() / math.sqrt(s.dim)
    bits = (s.tree[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1).flatten(1).bool()
    n, b0 = len(s.lens_list), 0
    while b0 < n:
        # some sequences at a time, padded to the longest: 4 GB of keys, values and scores
        b1 = b0 + 1
        while b1 < n:
            L, T = max(s.lens_list[b0:b1 + 1]), max(s.counts[b0:b1 + 1])
            if (b1 + 1 - b0) * L * (s.hkv * s.dim * 8 + T * s.hq * 8) > 4 << 30:
                break
            b1 += 1
        L, T, m = max(s.lens_list[b0:b1]), max(s.counts[b0:b1]), b1 - b0
        lens, count = s.lens[b0:b1].long(), s.offsets[b0 + 1:b1 + 1].long() - s.offsets[b0:b1].long()
        at = torch.arange(L, device="cuda")
        page = s.tables[b0:b1][:, at // P].clamp(min=0).long()
        there = (at[None] < lens[:, None])[:, :, None, None]
        k = s.k[page, :, at % P].float().masked_fill(~there, 0.0)
        v = s.v[page, :, at % P].float().masked_fill(~there, 0.0)
        t = torch.arange(T, device="cuda")
        live = t[None] < count[:, None]
        token = (s.offsets[b0:b1].long()[:, None] + t[None]).clamp(max=tokens - 1)
        drafted = at[None] - (lens - count)[:, None]  # number of the drafted token at a position
        seen = bits[token].gather(2, drafted.clamp(0, bits.shape[1] - 1)[:, None].expand(m, T, L))
        seen = torch.where(drafted[:, None] < 0, torch.ones_like(seen), seen & (drafted[:, None] <= t[None, :, None]))
        mine = q[token].view(m, T, s.hkv, G, s.dim).permute(0, 2, 1, 3, 4).reshape(m, s.hkv, T * G, s.dim)
        x = mine @ k.permute(0, 2, 3, 1)
        x = x.view(m, s.hkv, T, G, L).masked_fill(~seen[:, None, :, None], -math.inf)
        top = x.amax(-1, keepdim=True).clamp(min=-1e30)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        o = (p.view(m, s.hkv, T * G, L) @ v.permute(0, 2, 1, 3)).view(m, s.hkv, T, G, s.dim) / total
        z = top + torch.log(total)
        out[token[live]] = o.permute(0, 2, 1, 3, 4).reshape(m, T, s.hq, s.dim)[live]
        lse[token[live]] = z.permute(0, 2, 1, 3, 4).reshape(m, T, s.hq)[live]
        b0 = b1
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _rules(s):
    if own:
        s.rules.run(s.batch, s.logits, out=s.out, tokens=s.chosen)
        return {"logits": s.out, "tokens": s.chosen}
    V, n = s.V, s.rows
    x = s.logits.float()
    rows = torch.arange(n, device="cuda")
    if s.ranges is not None:
        count = torch.zeros(n * V, dtype=torch.int32, device="cuda")
        seen = torch.zeros(n * V, dtype=torch.bool, device="cuda")
        begin, length = s.ranges[:, 0].long(), (s.ranges[:, 1] - s.ranges[:, 0]).long()
        row = rows.repeat_interleave(length)
        j = torch.arange(row.numel(), device="cuda") - (length.cumsum(0) - length)[row]
        place = row * V + s.tokens[begin[row] + j].long()
        seen[place] = True
        made = place[j >= s.prompt.long()[row]]
        count.index_add_(0, made, torch.ones_like(made, dtype=torch.int32))
        if s.path is not None:
            length = (s.path_offsets[1:] - s.path_offsets[:-1]).long()
            row = rows.repeat_interleave(length)
            place = row * V + s.path[:row.numel()].long()
            seen[place] = True
            count.index_add_(0, place, torch.ones_like(place, dtype=torch.int32))
        count, seen = count.view(n, V), seen.view(n, V)
        x = torch.where(seen, torch.where(x > 0, x / s.rep[:, None], x * s.rep[:, None]), x)
        x = x - s.freq[:, None] * count.float()
        x = torch.where(count > 0, x - s.pres[:, None], x)
    if s.bias is not None:
        length = (s.bias_offsets[1:] - s.bias_offsets[:-1]).long()
        row = rows.repeat_interleave(length)
        x = x.index_put((row, s.bias_tokens[:row.numel()].long()), s.bias[:row.numel()], accumulate=True)
    if s.allowed is not None:
        ids = torch.arange(V, device="cuda")
        word = s.allowed[s.allowed_rows.clamp(min=0).long()][:, ids // 32]
        free = (word >> (ids % 32).int() & 1).bool() | (s.allowed_rows < 0)[:, None]
        x = x.masked_fill(~free, -math.inf)
    top, first = x.amax(-1, keepdim=True), torch.arange(V, device="cuda", dtype=torch.int32)
    chosen = torch.where(x == top, first, torch.full_like(first, V)).amin(-1)
    return {"logits": x, "tokens": torch.where(top[:, 0] > -math.inf, chosen, torch.full_like(chosen, -1))}


def _keep(s):
    if own:
        s.cache.keep(s.seqs, s.start, s.offsets, s.picks)
        return {"pool": s.pool.view(torch.int16)}
    b = s.which.long()
    to = torch.arange(b.numel(), device="cuda") - s.offsets.long()[b] + s.start.long()[b]
    fro = s.picks.long() + s.start.long()[b]
    row = s.seqs.long()[b]
    source = s.tables[row, fro // s.P].long()
    target = s.tables[row, to // s.P].long()
    s.pool[:, target, :, to % s.P] = s.pool[:, source, :, fro % s.P]
    return {"pool": s.pool.view(torch.int16)}


def run(s):
    return {"append": _append, "tree": _tree, "rules": _rules, "keep": _keep}[s.op](s)


# ------------------------------------------------------------------------------------------------ what it needs, and is


def work(case):
    if case["op"] == "rules":
        n, V = case["seqs"] * case["nodes"], case["vocab"]
        return {"bytes": n * (V * (6 if case["half"] else 8) + 4 * case["bias"]) + case["masks"] * V / 8
                + 3 * case["seqs"] * case["history"], "flops": 0}
    layers, hq, kv, dim, _ = MODELS[case["model"]]
    if case["op"] == "append":
        tokens = sum(_counts(case["tokens"], case["seqs"], case["tokens"]))
        return {"bytes": tokens * (hq + 2 * kv) * dim * 4, "flops": 0}
    if case["op"] == "tree":
        tokens = sum(_counts(case["nodes"], case["seqs"], case["nodes"]))
        prefix = [max(1, case["prefix"] >> (2 * i)) for i in range(case["groups"])]
        mine = case["seqs"] * case["context"] * 0.875
        seen = mine / case["seqs"] + (sum(prefix) / len(prefix) if prefix else 0) + 5
        return {"bytes": (sum(prefix) + mine + tokens) * kv * dim * 4 + tokens * hq * (dim * 4 + 4),
                "flops": 4 * dim * tokens * hq * seen}
    kept = case["seqs"] * (case["depth"] - 1) / 2
    return {"bytes": 2 * kept * layers * 2 * kv * dim * 2, "flops": 0}


def _exact_append(case, seed):
    """A head is a row of complex numbers, its rotary part, and the rest; turned by e^(i angle), one sequence at a time."""
    s = _prepare_append(case, seed)
    K, V = s.k.double(), s.v.double()
    Q = torch.empty(s.qkv.shape[0], s.hq, s.dim, dtype=torch.float64, device="cuda")
    even = torch.arange(s.rotary // 2, device="cuda")
    real, imag = (2 * even, 2 * even + 1) if s.interleaved else (even, even + s.rotary // 2)
    for b, L in enumerate(s.lens_list):
        lo, hi = s.offsets_list[b], s.offsets_list[b + 1]
        x = s.qkv[lo:hi].double()
        if s.wq is not None:
            scale = 1.0 / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / s.dim + s.eps)
            x[:, :s.hq] *= scale[:, :s.hq] * s.wq.double()
            x[:, s.hq:s.hq + s.hkv] *= scale[:, s.hq:s.hq + s.hkv] * s.wk.double()
        place = torch.tensor(s.positions_list[lo:hi], dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full((hi - lo, 1, s.rotary // 2), s.magnitude, dtype=torch.float64, device="cuda"),
                           place[:, None, None] * s.freq.cuda())
        qk = x[:, :s.hq + s.hkv]
        z = torch.complex(qk[..., real], qk[..., imag]) * turn
        qk[..., real], qk[..., imag] = z.real, z.imag
        Q[lo:hi] = x[:, :s.hq]
        slots = range(L - (hi - lo), L)
        pages = torch.tensor([int(s.tables_np[b, i // s.P]) for i in slots], device="cuda")
        inside = torch.tensor([i % s.P for i in slots], device="cuda")
        K[pages, :, inside] = x[:, s.hq:s.hq + s.hkv]
        V[pages, :, inside] = x[:, s.hq + s.hkv:]
    return {"q": Q, "k": K, "v": V}


def _exact_tree(case, seed):
    """Attention from its definition, one sequence and head at a time; a token's ancestors by walking up its parents."""
    s = _prepare_tree(case, seed)
    G = s.hq // s.hkv
    out = torch.empty(s.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s.q.shape[:2], dtype=torch.float64, device="cuda")
    for b, L in enumerate(s.lens_list):
        lo, hi = s.offsets_list[b], s.offsets_list[b + 1]
        T = hi - lo
        seen = np.zeros((T, L), bool)
        seen[:, :L - T] = True
        for t in range(T):
            i = t
            while i >= 0:
                seen[t, L - T + i] = True
                i = s.parents[b][i]
        hidden = torch.from_numpy(~seen).cuda()
        pages = torch.from_numpy(s.tables_np[b, :-(-L // s.P)].astype(np.int64)).cuda()
        for h in range(s.hkv):
            k = s.k[pages, h].reshape(-1, s.dim)[:L].double()
            v = s.v[pages, h].reshape(-1, s.dim)[:L].double()
            for i in range(h * G, (h + 1) * G):
                x = torch.matmul(s.q[lo:hi, i].double(), k.t()) / math.sqrt(s.dim)
                x[hidden] = -math.inf
                z = torch.logsumexp(x, dim=1)
                lse[lo:hi, i] = z
                out[lo:hi, i] = torch.matmul(torch.exp(x - z[:, None]), v)
    return {"out": out, "lse": lse}


def _exact_rules(case, seed):
    """One row at a time.  The chosen tokens are whole numbers and have no value of their own here."""
    s = _prepare_rules(case, seed)
    out = torch.empty(s.rows, s.V, dtype=torch.float64, device="cuda")
    for i in range(s.rows):
        x = s.logits[i].double()
        if s.ranges is not None:
            a, e = s.ranges[i].tolist()
            old, made = s.tokens[a:a + int(s.prompt[i])].long(), s.tokens[a + int(s.prompt[i]):e].long()
            if s.path is not None:
                made = torch.cat([made, s.path[int(s.path_offsets[i]):int(s.path_offsets[i + 1])].long()])
            c = torch.bincount(made, minlength=s.V)
            known = (torch.bincount(old, minlength=s.V) + c) > 0
            r = float(s.rep[i])
            x[known & (x > 0)] /= r
            x[known & (s.logits[i] <= 0)] *= r
            x -= float(s.freq[i]) * c
            x[c > 0] -= float(s.pres[i])
        if s.bias is not None:
            a, e = s.bias_offsets[i:i + 2].tolist()
            x[s.bias_tokens[a:e].long()] += s.bias[a:e].double()
        if s.allowed is not None and int(s.allowed_rows[i]) >= 0:
            row = s.allowed[int(s.allowed_rows[i])].cpu().numpy().view(np.uint8)
            x[torch.from_numpy(np.unpackbits(row, bitorder="little")[:s.V] == 0).cuda()] = -math.inf
        out[i] = x
    return {"logits": out, "tokens": None}


def exact(case, seed):
    """The operators from their definitions, in 64 bits.  keep moves rows and computes nothing."""
    if case["op"] == "keep":
        return None
    return {"append": _exact_append, "tree": _exact_tree, "rules": _exact_rules}[case["op"]](case, seed)
