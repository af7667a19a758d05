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
