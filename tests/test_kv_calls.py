"""Page ownership: calls and sizes beside those of test_kv_cache.py, with the same model."""
import pytest

import persistent_moe_decode_sm_gb300 as mk
from kv_model import PAGE_OOB
from test_kv_cache import Pair, start

gpu = pytest.mark.gpu


def status(p):
    with pytest.raises(mk.MkError) as e:
        p.cache.sync()
    return e.value.code


@gpu
@pytest.mark.parametrize("name, a, b", [
    ("fork", [9, 0], [1, 2]),                       # a row that is not there; a page that is not held
    ("fork", [0, 0, 0], [2, 2, 3]),                 # the same row twice; the page
    ("resize", [9, 0], [5, 3]), ("resize", [1, 1, 0], [5, 5, 3]),
    ("resize", [9, 1], [5, 16 * 40 + 1]),           # a row that is not there; a length behind the table
    ("copy_pages", [0, 0, 50], [5, 5, 6])])         # a target twice; a page behind the pool
def test_of_several_wrong_arguments_the_same_one_is_reported(name, a, b):
    """A wrong row number is met at once, a wrong page behind three loads: whichever comes
    first, the page is reported."""
    m = start(50, 6, 40, 16, [40])
    m.tables[0, 2] = 50
    p = Pair(m)
    for _ in range(5):
        getattr(p.cache, name)(p.i32(a), p.i32(b))
        assert status(p) == PAGE_OOB
    p.same()
