"""mk_prefix_attention: calls that its documentation allows or refuses beside the plain ones."""
import time

import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
from test_prefix_attention import Case

gpu = pytest.mark.gpu


def refused(a, b, q, out, lse=None, code=mk.MK_ERR_INVALID_ARG):
    with pytest.raises(mk.MkError) as e:
        a.run(0, b, q, out, lse)
    assert e.value.code == code


@gpu
def test_results_over_the_queries_are_refused():
    """In place, and by a row; side by side in one buffer is fine."""
    c = Case([(32, [(5, 1), (8, 1), (3, 1)])], (4, 2, 64))
    t, d = c.t, c.device()
    a, b = c.attention(d)
    refused(a, b, d["q"], d["q"])
    both = t.zeros(7, 4, 64, dtype=t.bfloat16, device="cuda")
    both[:3] = d["q"]
    refused(a, b, both[:3], both[2:5])
    refused(a, b, both[:3], both[3:6], both.view(t.float32).view(-1)[:12].view(3, 4))
    refused(a, b, both[:3], both[3:6], both[3:].view(t.float32).view(-1)[:12].view(3, 4))
    lse = both[6:].view(t.float32).view(-1)[:12].view(3, 4)
    a.run(0, b, both[:3], both[3:6], lse)
    a.sync()
    c.check((both[3:6].double().cpu().numpy(), lse.double().cpu().numpy()))


def test_wait_limits_are_checked():
    L = mk.lib()
    assert L.mk_attn_set_wait_limit_ns(None, 5) == mk.MK_ERR_INVALID_ARG
    assert L.mk_attn_debug_poison_wait(None) == mk.MK_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("each, heads", [(3, (4, 2, 64)), (40, (32, 4, 128)), (70, (6, 2, 32))])
def test_a_wait_that_is_never_met_ends_the_call(each, heads):
    """The call ends with a status after the limit; the next one is right, on the same handle."""
    c = Case([(700, [(5 + i, 1) for i in range(each)])], heads)     # singles, and pairs
    t, d = c.t, c.device()
    a, b = c.attention(d)
    out = t.full(d["q"].shape, 123.0, dtype=t.bfloat16, device="cuda")
    lse = t.full(d["q"].shape[:2], 123.0, device="cuda")
    with pytest.raises(mk.MkError):
        a.set_wait_limit_ns(0)
    a.set_wait_limit_ns(100_000_000)
    assert mk.lib().mk_attn_debug_poison_wait(a.handle) == mk.MK_OK
    start = time.time()
    a.run(0, b, d["q"], out, lse)
    with pytest.raises(mk.MkError) as e:
        a.sync()
    assert e.value.code == mk.MK_ERR_DEVICE_TIMEOUT
    assert 0.1 <= time.time() - start < 10.0
    a.run(0, b, d["q"], out, lse)
    a.sync()
    c.check((out.double().cpu().numpy(), lse.double().cpu().numpy()))


@gpu
@pytest.mark.parametrize("order", [("page", "batch"), ("batch", "page"), ("time", "batch"),
                                   ("time", "page"), ("page", "fine", "time", "batch")])
def test_the_first_error_is_reported(order):
    c = Case([(32, [(50, 1), (8, 1)])], (4, 2, 64))
    t, d = c.t, c.device()
    a, fine = c.attention(d)
    wild = c.tables.copy()
    wild[0, 3] = 10 ** 6
    wild, wrong = t.from_numpy(wild).cuda(), t.tensor([-1, 40], dtype=t.int32).cuda()
    calls = {"fine": fine, "time": fine, "page": a.batch(wild, d["lens"]),
             "batch": a.batch(d["tables"], wrong)}
    codes = {"time": mk.MK_ERR_DEVICE_TIMEOUT, "page": mk.MK_ERR_PAGE_OOB,
             "batch": mk.MK_ERR_INVALID_ARG}
    out = t.empty_like(d["q"])
    a.set_wait_limit_ns(50_000_000)
    for _ in range(2):                     # taken once, so the second turn starts anew
        for name in order:
            if name == "time":
                mk.lib().mk_attn_debug_poison_wait(a.handle)
            a.run(0, calls[name], d["q"], out)
        with pytest.raises(mk.MkError) as e:
            a.sync()
        assert e.value.code == codes[order[0]]
        a.sync()


@gpu
def test_behind_page_calls_without_a_wait():
    """Pages move and tables change right before the attention reads them, on one stream."""
    c = Case([(300, [(40 + 7 * i, 1) for i in range(12)])], (8, 2, 64), P=16, spare=400)
    t = c.t
    n, want = c.k.shape[0], c.exact()
    rng = np.random.default_rng(0)
    i32 = dict(dtype=t.int32, device="cuda")
    kept = t.from_numpy(c.tables).cuda(), c.k.cuda(), c.v.cuda()
    refs = t.tensor(np.bincount(np.concatenate(c.rows), minlength=n), **i32)
    tables, k, v, holders = (x.clone() for x in kept + (refs,))
    lens = t.tensor(c.lens, **i32)
    cache = mk.KvCache([k, v], tables, lens, holders, 16)
    d = c.device(k=k, v=v, tables=tables, lens=lens)
    a, b = c.attention(d)
    outs = []
    for turn in range(6):
        tables.copy_(kept[0]), k.copy_(kept[1]), v.copy_(kept[2]), holders.copy_(refs)
        order = t.from_numpy(rng.permutation(n)).cuda()          # page p lies at order[p]
        k[order], v[order], holders[order] = kept[1], kept[2], refs
        tables.copy_(t.where(kept[0] < 0, kept[0], order[kept[0].clamp(min=0).long()].int()))
        out = t.empty_like(d["q"]), t.empty(d["q"].shape[:2], device="cuda")
        a.run(0, b, d["q"], *out)
        cache.compact()
        again = t.empty_like(d["q"]), t.empty(d["q"].shape[:2], device="cuda")
        a.run(0, b, d["q"], *again)
        outs += [out, again]
    a.sync()
    cache.sync()
    for out, lse in outs:
        c.check((out.double().cpu().numpy(), lse.double().cpu().numpy()), want)
    assert int((holders[:int((refs > 0).sum())] > 0).sum()) == int((refs > 0).sum())


@gpu
def test_one_head_may_have_any_head_stride():
    c = Case([(32, [(5, 1), (8, 1), (40, 1)])], (1, 1, 64))
    t = c.t
    wide = t.zeros(3, 200, dtype=t.bfloat16, device="cuda")
    q = wide.as_strided((3, 1, 64), (200, 7, 1))
    q.copy_(c.q)
    c.check(c.run(c.device(q=q)))
