"""mk_prefix_attention: calls that its documentation allows or refuses beside the plain ones."""
import time

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
