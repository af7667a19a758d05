"""What the Python calls of the 8-bit cache refuse by name, without a GPU."""
import pytest
import torch

import sparse_mask_scaled_b200 as sp


def make(B=2, Hk=2, page=16, d=32):
    table = torch.zeros((B, 3), dtype=torch.int32)
    return sp.Cache.empty(4, Hk, page, d, table, dtype=torch.int8)


def ints(n=2):
    return torch.zeros(n, dtype=torch.int32)


def test_a_cache_in_host_memory():
    c, x = make(), torch.zeros((2, 2, 1, 32))
    for call in (lambda: sp.spattn_cache_write(x, x, c), lambda: sp.spattn_cache_read(c, 1),
                 lambda: sp.spattn_fwd_cache(x, c, ints()), lambda: sp.spattn_cache_write(x, x, c, stream=0)):
        with pytest.raises(ValueError, match="cpu"):
            call()


@pytest.mark.parametrize("lse", [
    torch.zeros(7), torch.zeros(9), torch.zeros(8, dtype=torch.float64), torch.zeros(8, dtype=torch.bfloat16),
    torch.zeros((2, 4, 2))[..., 0], torch.zeros(8, device="meta"),
])
def test_an_lse_that_cannot_hold_the_rows(lse):
    c, q = make(), torch.zeros((2, 4, 1, 32))
    with pytest.raises(ValueError, match="lse"):
        sp.spattn_fwd_cache(q, c, ints(), lse=lse)


@pytest.mark.parametrize("lse", [torch.zeros(8), torch.zeros((2, 4, 1))])
def test_an_lse_of_the_right_size_passes(lse):
    with pytest.raises(ValueError, match="cpu"):        # on to the next refusal
        sp.spattn_fwd_cache(torch.zeros((2, 4, 1, 32)), make(), ints(), lse=lse)


@pytest.mark.parametrize("kw", [dict(window=2 ** 31), dict(window=2 ** 32 + 5), dict(window=-2 ** 31 - 1),
                                dict(n_global=2 ** 31), dict(n_global=2 ** 32), dict(window=1.5)])
def test_numbers_that_no_int32_holds(kw):
    # they went on as their low 32 bits: a window of 2^32 + 5 as one of 5
    with pytest.raises((ValueError, TypeError), match="window|n_global"):
        sp.spattn_fwd_cache(torch.zeros((2, 4, 1, 32)), make(), ints(), **kw)


@pytest.mark.parametrize("kw", [dict(window=2 ** 31 - 1), dict(window=-2 ** 31), dict(window=5, n_global=2 ** 31 - 1)])
def test_the_largest_numbers_pass(kw):
    with pytest.raises(ValueError, match="cpu"):        # on to the next refusal
        sp.spattn_fwd_cache(torch.zeros((2, 4, 1, 32)), make(), ints(), **kw)
