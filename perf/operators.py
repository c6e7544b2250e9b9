"""The paged-cache operators and the shared-prefix attention: measured cases, plain forms and exact values.

A state is a paged KV cache as the decode step reads it: pools [pools][pages][kv heads][page size][head dim] in
bf16 (K and V of every layer), page tables, lengths, and how many tables hold each page.  The page operators'
results are whole numbers (tables, lengths, holders, and the pools' bits), so both sides have to be equal there.
"""
import math

import torch

own = False

# (layers, q heads, kv heads, head dim): the framework's tiny, mid and full models and its odd test shape
MODELS = {"tiny": (2, 4, 2, 64), "odd": (2, 6, 2, 32), "mid": (8, 16, 4, 64), "full": (48, 32, 4, 128)}


def listed():
    return [
        # a beam step of the mid model moves a few private pages
        {"name": "copy_beams", "op": "copy", "model": "mid", "page": 16, "pages": 1024, "count": 24},
        # a quarter of a full-scale pool is moved aside
        {"name": "copy_quarter", "op": "copy", "model": "full", "page": 16, "pages": 4096, "count": 1024},
        # one prompt of the mid model, four samples: latency counts
        {"name": "fork_samples_small", "op": "fork", "model": "mid", "page": 16, "pages": 512, "groups": 1, "each": 4,
         "longest": 2048, "beams": False},
        # eight ragged prompts of the full-scale model, eight samples each
        {"name": "fork_samples_full", "op": "fork", "model": "full", "page": 16, "pages": 8320, "groups": 8, "each": 8,
         "longest": 16384, "beams": False},
        # every sequence of a large batch takes a few draft tokens and gives them back
        {"name": "resize_draft", "op": "resize", "model": "mid", "page": 16, "pages": 8192, "seqs": 256, "longest": 400,
         "turnover": False},
        # long sequences finish, others of the same lengths are admitted
        {"name": "resize_turnover", "op": "resize", "model": "full", "page": 16, "pages": 6000, "seqs": 8,
         "longest": 10000, "turnover": True},
        # a small fragmented pool
        {"name": "compact_mid", "op": "compact", "model": "mid", "page": 16, "pages": 1000, "seqs": 16, "live": 0.35},
        # a full-scale pool, half of it live and scattered
        {"name": "compact_full", "op": "compact", "model": "full", "page": 16, "pages": 4096, "seqs": 64, "live": 0.5},
        # single tokens of a few samples over a short prompt: latency counts
        {"name": "attend_small", "op": "attend", "model": "mid", "page": 16, "groups": 1, "each": 4, "prefix": 480,
         "own_tokens": 24, "query": 1},
        # single tokens, 64 samples of one prompt at the full model's heads
        {"name": "attend_samples", "op": "attend", "model": "full", "page": 16, "groups": 1, "each": 64, "prefix": 8192,
         "own_tokens": 512, "query": 1},
        # single tokens over a very long shared context, and a second, smaller group
        {"name": "attend_long", "op": "attend", "model": "full", "page": 16, "groups": 2, "each": 8, "prefix": 131072,
         "own_tokens": 1000, "query": 1},
        # ragged questions after one long shared document, all their tokens at once
        {"name": "attend_questions", "op": "attend", "model": "full", "page": 16, "groups": 1, "each": 16,
         "prefix": 32768, "own_tokens": 500, "query": 400},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["copy", "fork", "resize", "compact", "attend", "attend"])
    model = rng.choice(["tiny", "odd", "mid", "full"])
    page = rng.choice([16, 16, 32, 64])
    if op == "attend":
        c = {"op": op, "model": model, "page": page, "groups": rng.randint(1, 3), "each": _log(rng, 1, 48),
             "prefix": _log(rng, 16, 65536), "own_tokens": _log(rng, 1, 600)}
        c["query"] = rng.choice([1, 1, 1, 4, 7, _log(rng, 2, 300)])
        heads = MODELS[model][1]
        while c["query"] > 1 and c["groups"] * c["each"] * c["query"] * heads * c["prefix"] > 4e9:
            c["query"] = max(1, c["query"] // 2)
        return c
    pages = _log(rng, 200, 4000 * 16 // page)
    c = {"op": op, "model": model, "page": page, "pages": pages}
    if op == "copy":
        c["count"] = _log(rng, 1, pages // 4)
    elif op == "fork":
        c["groups"], c["each"] = rng.randint(1, 6), _log(rng, 1, 12)
        spare = 2 * c["groups"] * (c["each"] + 1)
        c["longest"] = _log(rng, 1, max(2, (pages - spare) // c["groups"] * page))
        c["beams"] = rng.random() < 0.3
    elif op == "resize":
        c["turnover"] = rng.random() < 0.5
        c["seqs"] = _log(rng, 1, max(1, pages // 4))
        c["longest"] = _log(rng, 1, max(2, (pages // c["seqs"] - 2) * page))
    else:
        c["seqs"], c["live"] = _log(rng, 1, 64), round(rng.uniform(0.1, 0.9), 3)
    return c


# ------------------------------------------------------------------------------------------------ inputs


class State:
    pass


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _plan(case, seed):
    """Lengths, tables and holders of a case's sequences as lists, from the seed alone."""
    import random

    rng = random.Random(seed * 7919 + 11)
    P, N = case["page"], case["pages"]
    order = list(range(N))
    rng.shuffle(order)
    op = case["op"]
    if op == "fork":
        n = case["groups"]
        lens = [max(1, case["longest"] - rng.randint(0, max(1, case["longest"] // 3))) for _ in range(n)]
        lens += [0] * (n * case["each"])
    elif op == "resize":
        lens = [rng.randint(1, case["longest"]) for _ in range(case["seqs"])]
    elif op == "compact":
        left, lens = int(N * case["live"]), []
        for i in range(case["seqs"]):
            k = left // (case["seqs"] - i) if i + 1 < case["seqs"] else left
            left -= k
            lens.append(max(0, k * P - rng.randint(0, P - 1)))
    else:
        lens = [0]
    rows, at, refs = [], 0, [0] * N
    for L in lens:
        k = -(-L // P)
        rows.append(order[at:at + k])
        at += k
        for p in rows[-1]:
            refs[p] += 1
    return rng, order, lens, rows, refs


def _prepare_pages(case, seed):
    s = State()
    layers, _, kv, dim = MODELS[case["model"]]
    P, N = case["page"], case["pages"]
    g = torch.Generator("cuda").manual_seed(seed)
    s.pool = torch.empty(2 * layers, N, kv * P * dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    rng, order, lens, rows, refs = _plan(case, seed)
    s.P = P
    draft = [rng.randint(1, 8) for _ in lens]
    # as many table entries as the longest sequence of any seed can use
    wide = 1
    if "longest" in case:
        wide = -(-case["longest"] // P) + 1
    elif case["op"] == "compact":
        wide = int(N * case["live"]) // case["seqs"] + 2
    s.tables = _ints([r + [-1] * (wide - len(r)) for r in rows])
    s.lens, s.refs = _ints(lens), _ints(refs)
    if case["op"] == "copy":
        s.src, s.dst = _ints(order[:case["count"]]), _ints(order[case["count"]:2 * case["count"]])
    elif case["op"] == "fork":
        n, k = case["groups"], case["each"]
        if case["beams"]:
            # all the samples of a group exist already; every beam then follows a random one of its group
            own_rows = list(range(n * (k + 1)))
            s.dst = _ints(own_rows)
            s.first_src = _ints([i if i < n else (i - n) // k for i in own_rows])
            members = [[i] + [n + i * k + j for j in range(k)] for i in range(n)]
            s.src = _ints([rng.choice(members[i if i < n else (i - n) // k]) for i in own_rows])
        else:
            s.first_src = None
            s.src = _ints([i for i in range(n) for _ in range(k)])
            s.dst = _ints([n + i for i in range(n * k)])
    elif case["op"] == "resize":
        s.seqs = _ints(list(range(len(lens))))
        s.back = _ints(lens)
        s.there = _ints([0 if rng.random() < 0.7 else L for L in lens] if case["turnover"]
                        else [L + d for L, d in zip(lens, draft)])
    else:
        s.kept = (s.tables.clone(), s.refs.clone())
        s.page_map = torch.empty(N, dtype=torch.int32, device="cuda")
    if own:
        import persistent_moe_decode_sm_gb300 as mk

        s.cache = mk.KvCache(list(s.pool), s.tables, s.lens, s.refs, page_size=P)
    if case["op"] == "fork" and s.first_src is not None:
        _fork(s, s.first_src, s.dst)
    return s


def _prepare_attend(case, seed):
    import random

    s = State()
    rng = random.Random(seed * 104729 + 5)
    _, s.hq, s.hkv, s.dim = MODELS[case["model"]]
    P, n = case["page"], case["groups"] * case["each"]
    # the second and third groups share shorter prefixes; prefixes end where a page does or inside one
    s.prefix = [max(1, case["prefix"] >> (2 * i)) for i in range(case["groups"])]
    lengths = random.Random(case["query"])  # of the questions: the outputs' shape, the same for every seed
    s.query = [lengths.randint(max(1, case["query"] // 2), case["query"]) for _ in range(n)]
    extra = [rng.randint(0, case["own_tokens"]) for _ in range(n)]
    s.lens_list = [s.prefix[i // case["each"]] + max(extra[i], s.query[i]) for i in range(n)]
    used = [-(-L // P) for L in s.lens_list]
    shared = [L // P for L in s.prefix]
    total = sum(shared) + sum(used[i] - shared[i // case["each"]] for i in range(n)) + 3
    order = list(range(total))
    rng.shuffle(order)
    at, heads, rows = 0, [], []
    for k in shared:
        heads.append(order[at:at + k])
        at += k
    for i in range(n):
        k = used[i] - shared[i // case["each"]]
        rows.append(heads[i // case["each"]] + order[at:at + k])
        at += k
    wide = max(used) + 2
    s.rows = rows
    s.P, s.each = P, case["each"]
    s.tables = _ints([r + [-1] * (wide - len(r)) for r in rows])
    s.lens, s.prefix_lens = _ints(s.lens_list), _ints(s.prefix)
    s.starts = _ints([i * case["each"] for i in range(case["groups"] + 1)])
    offsets = [0]
    for t in s.query:
        offsets.append(offsets[-1] + t)
    s.offsets_list = offsets
    s.offsets = _ints(offsets) if case["query"] > 1 else None
    g = torch.Generator("cuda").manual_seed(seed)
    shape = (total, s.hkv, P, s.dim)
    s.k = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    s.v = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    s.q = torch.empty(offsets[-1], s.hq, s.dim, dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.0, generator=g)
    if own:
        import persistent_moe_decode_sm_gb300 as mk

        s.out = torch.empty_like(s.q)
        s.lse = torch.empty(offsets[-1], s.hq, dtype=torch.float32, device="cuda")
        s.attn = mk.PrefixAttention(s.hq, s.hkv, s.dim, P, [(s.k, s.v)], max_tokens=offsets[-1])
        s.batch = s.attn.batch(s.tables, s.lens, q_offsets=s.offsets, group_starts=s.starts,
                               prefix_lens=s.prefix_lens)
    return s


def prepare(case, seed):
    s = _prepare_attend(case, seed) if case["op"] == "attend" else _prepare_pages(case, seed)
    s.op = case["op"]
    return s


# ------------------------------------------------------------------------------------------------ one pass


def _fork(s, src, dst):
    if own:
        s.cache.fork(src, dst)
        return
    P, Mp = s.P, s.tables.shape[1]
    a, b = src.long(), dst.long()
    ls, ld, live = s.lens[a], s.lens[b], src != dst
    rows, old = s.tables[a], s.tables[b]
    j = torch.arange(Mp, device="cuda")[None]
    full = ls // P
    held = live[:, None] & (j < full[:, None])
    gone = live[:, None] & (j < ((ld + P - 1) // P)[:, None])
    after = s.refs.clone()
    after.index_add_(0, rows[held].long(), torch.ones_like(rows[held]))
    after.index_add_(0, old[gone].long(), -torch.ones_like(old[gone]))
    part = (live & (ls % P != 0)).nonzero()[:, 0]
    source = rows[part, full[part].long()].long()
    free = after == 0
    free[source] = False
    fresh = free.nonzero()[:part.numel(), 0]
    new = torch.where(j < full[:, None], rows, -torch.ones_like(rows))
    new[part, full[part].long()] = fresh.int()
    after[fresh] = 1
    s.tables[b] = torch.where(live[:, None], new, old)
    s.lens[b] = ls
    s.refs.copy_(after)
    s.pool[:, fresh] = s.pool[:, source]


def _resize(s, seqs, lens):
    if own:
        s.cache.resize(seqs, lens)
        return
    P, Mp = s.P, s.tables.shape[1]
    a = seqs.long()
    was, rows = s.lens[a], s.tables[a]
    u0, u1 = (was + P - 1) // P, (lens + P - 1) // P
    j = torch.arange(Mp, device="cuda")[None]
    gone = (j >= u1[:, None]) & (j < u0[:, None])
    after = s.refs.clone()
    after.index_add_(0, rows[gone].long(), -torch.ones_like(rows[gone]))
    last = rows.gather(1, (u0 - 1).clamp(min=0).long()[:, None])[:, 0]
    cow = (lens > was) & (was % P != 0) & (s.refs[last.clamp(min=0).long()] > 1)
    source = last[cow].long()
    after.index_add_(0, source, -torch.ones_like(last[cow]))
    free = after == 0
    free[source] = False
    wanted = ((j >= u0[:, None]) & (j < u1[:, None])) | (cow[:, None] & (j == u0[:, None] - 1))
    at = wanted.nonzero()
    fresh = free.nonzero()[:at.shape[0], 0]
    rows = torch.where(gone, -torch.ones_like(rows), rows)
    rows[at[:, 0], at[:, 1]] = fresh.int()
    after[fresh] = 1
    s.tables[a] = rows
    s.lens[a] = lens
    s.refs.copy_(after)
    target = rows.gather(1, (u0 - 1).clamp(min=0).long()[:, None])[:, 0][cow].long()
    s.pool[:, target] = s.pool[:, source]


def _compact(s):
    s.tables.copy_(s.kept[0])
    s.refs.copy_(s.kept[1])
    if own:
        s.cache.compact(s.page_map)
        return
    live = s.refs > 0
    ids = torch.arange(live.numel(), device="cuda")
    n = live.sum()
    holes, movers = (~live & (ids < n)).nonzero()[:, 0], (live & (ids >= n)).nonzero()[:, 0]
    to = torch.where(live, ids, -torch.ones_like(ids))
    to[movers] = holes
    s.page_map.copy_(to)
    s.tables.copy_(torch.where(s.tables >= 0, to[s.tables.clamp(min=0).long()].int(), s.tables))
    s.refs[holes] = s.refs[movers]
    s.refs[movers] = 0
    s.pool[:, holes] = s.pool[:, movers]


def _part(q, k, v, mask):
    """(max, sum, weighted sum) of softmax pieces: q [..., rows, D], k and v [..., keys, D] in fp32."""
    x = q @ k.transpose(-1, -2)
    if mask is not None:
        x = x.masked_fill(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-1e30))
    return m, p.sum(-1, keepdim=True), p @ v


def _attend(s):
    if own:
        s.attn.run(0, s.batch, s.q, s.out, s.lse)
        return {"out": s.out, "lse": s.lse}
    P, each, G = s.P, s.each, s.hq // s.hkv
    n, tokens = len(s.lens_list), s.q.shape[0]
    scale = 1.0 / math.sqrt(s.dim)
    # kv head, token, head of the group, D
    q = (s.q.float() * scale).view(tokens, s.hkv, G, s.dim).transpose(0, 1).contiguous()
    m = torch.full((s.hkv, tokens, G, 1), -math.inf, device="cuda")
    l, acc = torch.zeros_like(m), torch.zeros_like(q)
    # the shared pages, once for all rows of the group, 512 tokens at a time
    for g, length in enumerate(s.prefix):
        pages = s.tables[g * each, :length // P].long()
        if not pages.numel():
            continue
        k = s.k[pages].float().transpose(0, 1).reshape(s.hkv, -1, s.dim)
        v = s.v[pages].float().transpose(0, 1).reshape(s.hkv, -1, s.dim)
        low, high = s.offsets_list[g * each], s.offsets_list[(g + 1) * each]
        for t in range(low, high, 512):
            e = min(high, t + 512)
            a, b, c = _part(q[:, t:e].reshape(s.hkv, -1, s.dim), k, v, None)
            m[:, t:e], l[:, t:e], acc[:, t:e] = a.view(s.hkv, e - t, G, 1), b.view(s.hkv, e - t, G, 1), c.view(s.hkv, e - t, G, s.dim)
    # the sequences' own pages, padded to the longest
    lens = s.lens.long()
    begin = (s.prefix_lens // P * P).long().repeat_interleave(each)
    width = max(L - s.prefix[i // each] // P * P for i, L in enumerate(s.lens_list))
    at = begin[:, None] + torch.arange(width, device="cuda")[None]
    page = s.tables.gather(1, (at // P).clamp(max=s.tables.shape[1] - 1)).clamp(min=0).long()
    k = s.k[page, :, at % P].float().permute(0, 2, 1, 3)
    v = s.v[page, :, at % P].float().permute(0, 2, 1, 3)
    v = v.masked_fill((at >= lens[:, None])[:, None, :, None], 0.0)
    T = max(s.query)
    count = torch.tensor(s.query, device="cuda")
    t = torch.arange(T, device="cuda")
    there = t[None] < count[:, None]
    token = torch.tensor(s.offsets_list[:-1], device="cuda")[:, None] + t[None]
    token = token.clamp(max=tokens - 1)
    position = lens[:, None] - count[:, None] + t[None]
    mask = (at[:, None] <= position[:, :, None]) & (at < lens[:, None])[:, None]
    mine = q[:, token].transpose(0, 1).reshape(n, s.hkv, T * G, s.dim)
    a, b, c = _part(mine, k, v, mask[:, None, :, None].expand(n, 1, T, G, width).reshape(n, 1, T * G, width))

    def back(x):  # sequence, kv head, (token, head), . to kv head, token, head, .
        return x.view(n, s.hkv, T, G, -1).permute(0, 2, 1, 3, 4)[there].transpose(0, 1)

    a, b, c = back(a), back(b), back(c)
    top = torch.maximum(m, a)
    wm, wa = torch.exp(m - top), torch.exp(a - top)
    total = l * wm + b * wa
    out = (acc * wm + c * wa) / total
    return {"out": out.transpose(0, 1).reshape(tokens, s.hq, s.dim).to(torch.bfloat16),
            "lse": (top + torch.log(total)).transpose(0, 1).reshape(tokens, s.hq)}


def run(s):
    if s.op == "attend":
        return _attend(s)
    if s.op == "copy":
        if own:
            s.cache.copy_pages(s.src, s.dst)
        else:
            s.pool[:, s.dst.long()] = s.pool[:, s.src.long()]
        return {"pool": s.pool.view(torch.int16)}
    if s.op == "fork":
        _fork(s, s.src, s.dst)
    elif s.op == "resize":
        _resize(s, s.seqs, s.there)
        _resize(s, s.seqs, s.back)
    else:
        _compact(s)
    got = {"tables": s.tables, "lens": s.lens, "refs": s.refs, "pool": s.pool.view(torch.int16)}
    if s.op == "compact":
        got["page_map"] = s.page_map
    return got


# ------------------------------------------------------------------------------------------------ what it needs, and is


def work(case):
    layers, hq, kv, dim = MODELS[case["model"]]
    P = case["page"]
    if case["op"] == "attend":
        each, half = case["each"], 0.75 * case["query"] if case["query"] > 1 else 1
        tail = max(case["own_tokens"] / 2, half)
        keys = rows = pairs = 0.0
        for i in range(case["groups"]):
            prefix = max(1, case["prefix"] >> (2 * i))
            keys += prefix + each * tail
            rows += each * half * hq
            pairs += each * half * hq * (prefix + tail - half / 2)
        return {"bytes": keys * kv * dim * 4 + rows * (dim * 4 + 4), "flops": 4 * dim * pairs}
    page = kv * P * dim * 2 * 2 * layers
    if case["op"] == "copy":
        return {"bytes": 2 * case["count"] * page, "flops": 0}
    if case["op"] == "fork":
        n = case["groups"] * case["each"]
        return {"bytes": (case["groups"] + n) * page + 8 * n * max(1, case["longest"] // P) + 8 * case["pages"], "flops": 0}
    if case["op"] == "resize":
        return {"bytes": 2 * (12 * case["seqs"] + 8 * case["pages"]), "flops": 0}
    moves = case["pages"] * case["live"] * (1 - case["live"])
    return {"bytes": 2 * moves * page + 8 * case["pages"] * (1 + case["live"]), "flops": 0}


def exact(case, seed):
    """Attention from its definition, one sequence and kv head at a time, in 64 bits.  The page operators move and
    count whole numbers; they have no computed ones."""
    if case["op"] != "attend":
        return None
    s = _prepare_attend(case, seed)
    G = s.hq // s.hkv
    out = torch.empty(s.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s.q.shape[:2], dtype=torch.float64, device="cuda")
    for b, L in enumerate(s.lens_list):
        lo, hi = s.offsets_list[b], s.offsets_list[b + 1]
        pages = _ints(s.rows[b]).long()
        T = hi - lo
        seen = torch.arange(L, device="cuda")[None, :] <= (L - T + torch.arange(T, device="cuda"))[:, None]
        for h in range(s.hkv):
            k = s.k[pages, h].reshape(-1, s.dim)[:L].double()
            v = s.v[pages, h].reshape(-1, s.dim)[:L].double()
            for i in range(h * G, (h + 1) * G):
                x = torch.matmul(s.q[lo:hi, i].double(), k.t()) / math.sqrt(s.dim)
                x[~seen] = -math.inf
                z = torch.logsumexp(x, dim=1)
                lse[lo:hi, i] = z
                out[lo:hi, i] = torch.matmul(torch.exp(x - z[:, None]), v)
    return {"out": out, "lse": lse}
