"""mk_prefix_attention: calls that its documentation allows or refuses beside the plain ones."""
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
