"""Checks of the cache classes that come before any call into the library (no GPU)."""
import numpy as np
import pytest
import torch

import persistent_moe_decode_sm_gb300 as mk


def cache_of(lens, tables):
    """A KvCache over host tensors whose calls into the library do nothing."""
    c = mk.KvCache.__new__(mk.KvCache)
    c.handle = None
    c.seq_lens = torch.tensor(lens, dtype=torch.int32)
    c.page_tables = torch.tensor(tables, dtype=torch.int32)
    c.n_seqs, c.max_pages_per_seq = c.page_tables.shape
    c.sync = lambda: None
    return c


@pytest.mark.parametrize("rows", [[3], [0, 3], [-1], [0, -3], [2 ** 31]])
def test_read_refuses_rows_that_are_not_there(rows):
    """On the device an index behind the table would be an assertion in a kernel, and a
    negative one another sequence."""
    c = cache_of([5, 6, 7], [[0], [1], [2]])
    with pytest.raises(ValueError):
        c.read(rows)
    lens, tables = c.read([2, 0, 2])
    assert lens.tolist() == [7, 5, 7] and np.array_equal(tables, [[2], [0], [2]])


@pytest.mark.parametrize("scale", [1e-50, 0.0, -1.0, float("nan")])
def test_scales_that_are_no_positive_float_are_refused(scale):
    """1e-50 is 0 in 32 bits, which the library takes for 1 / sqrt(head_dim)."""
    pool = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="scale"):
        mk.PrefixAttention(1, 1, 64, 16, [(pool, pool)], max_tokens=1, scale=scale)


def test_a_schedule_over_another_page_size_is_refused():
    """A decoder of 16 tokens a page would read the rows of pages of 32 as its own."""
    dec = mk.Decoder.__new__(mk.Decoder)
    dec.ctx = None
    dec.cdims = mk.make_dims(2, 64, 4, 2, 64, 8, 2, 64, 64, 16, 4, 8, 1)
    dec.build_schedule = lambda lens, tables: None
    c = cache_of([5, 6, 7], [[0], [1], [2]])
    c.page_size = 16
    dec.schedule_cache(c, [0])
    c.page_size = 32
    with pytest.raises(ValueError, match="page size"):
        dec.schedule_cache(c, [0])
