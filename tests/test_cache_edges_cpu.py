"""Calls of the 8-bit cache at the edges of what it takes, without a GPU: each is answered before any
device work."""
import pytest

import sparse_mask_scaled_b200 as sp
from test_cache_cpu import D, HK, INVALID, PAGE, UNSUPPORTED, cache, call, desc


def empty_batch(name, c):
    """A call with no sequence: returns once its arguments have passed the checks."""
    c.batch = 0
    return call(name, c, desc((0, HK, 4, D), sp.SPATTN_BF16))


@pytest.mark.parametrize("name", ["write", "read", "attend"])
def test_a_table_may_hold_tokens_up_to_2_31_less_1024(name):
    # token numbers are 32-bit, and the kernels go on to the end of a step (up to 448 tokens and one more) behind them
    most = (2 ** 31 - 1024) // PAGE
    st, _ = empty_batch(name, cache(max_pages=most, table_stride=most))
    assert st == sp.SPATTN_OK
    st, msg = empty_batch(name, cache(max_pages=most + 1, table_stride=most + 1))
    assert st == UNSUPPORTED and "max_pages" in msg


@pytest.mark.parametrize("name", ["write", "read", "attend"])
@pytest.mark.parametrize("batch,m", [(0, 4), (3, 0), (0, 0)])
def test_calls_with_nothing_to_do(name, batch, m):
    # empty tensors have no address
    c = cache(batch=batch, page_table=None if batch == 0 else 0x300000)
    st, msg = call(name, c, desc((batch, HK, m, D), sp.SPATTN_BF16, data=None), lens=None if batch == 0 else 0x400000)
    assert st == sp.SPATTN_OK, msg
    # what they are is checked all the same
    assert call(name, c, desc((batch, HK, m, D), sp.SPATTN_I8, data=None))[0] == UNSUPPORTED
    assert call(name, c, desc((batch, HK, m, 2 * D), sp.SPATTN_BF16, data=None))[0] == INVALID


@pytest.mark.parametrize("name", ["write", "read", "attend"])
def test_addresses_are_needed_where_there_is_something_to_do(name):
    assert call(name, cache(page_table=None), desc((3, HK, 1, D), sp.SPATTN_BF16))[0] == INVALID
    assert call(name, cache(), desc((3, HK, 1, D), sp.SPATTN_BF16, data=None))[0] == INVALID
