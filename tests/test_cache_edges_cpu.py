"""Calls of the 8-bit cache at the edges of what it takes, without a GPU: each is answered before any
device work."""
import pytest

import sparse_mask_scaled_b200 as sp
from test_cache_cpu import D, HK, PAGE, UNSUPPORTED, cache, call, desc


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
