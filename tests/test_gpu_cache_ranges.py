"""Attention over the 8-bit cache where weights and V scales are small beside others: pages of zeros,
one token that outweighs all others, scales of many sizes, pages that are missing, on every kernel."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import cache_exact
import cache_reference as ref
from cache_reference import CODES

if torch.cuda.is_available():
    import sparse_mask_scaled_b200 as sp

REAL = {"bf16": torch.bfloat16, "f32": torch.float32}
# (H, Hk, m): one row, 24 rows and 130 rows a K/V head
ROWS = [(2, 2, 1), (8, 1, 3), (2, 2, 130)]


@pytest.fixture(autouse=True)
def no_device_error():
    sp.spattn_device_error()
    yield
    assert sp.spattn_device_error() == 0


def ints(v):
    return torch.tensor(v, dtype=torch.int32)


def dev_cache(codes, scales, table, dtype):
    return sp.Cache(codes[0].cuda().view(dtype), codes[1].cuda().view(dtype), scales[0].cuda(), scales[1].cuda(),
                    table.cuda())


def check(q, codes, scales, table, seqlen, dtype, used=None, gone=(), **kw):
    """used: the table that the call gets (`table`: the one without missing pages)."""
    cache = dev_cache(codes, scales, table if used is None else used, dtype)
    out, lse = sp.spattn_fwd_cache(q.cuda(), cache, ints(seqlen).cuda(), **kw)
    flags = sp.spattn_device_error()
    want, want_lse, tol, tol_lse = cache_exact.attend(q, codes, scales, table, seqlen, [q.shape[2]] * len(seqlen), dtype,
                                                      gone=gone, **kw)
    out, lse = out.double().cpu(), lse.double().cpu().view(want_lse.shape)
    some = ~torch.isneginf(want_lse)
    assert torch.equal(torch.isneginf(lse), ~some) and bool((out[~some] == 0).all())
    off = (out - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp(min=1e-300)).max())
    gap = (lse - want_lse).abs()[some]
    assert bool((gap <= tol_lse[some]).all()), float((gap / tol_lse[some]).max())
    return flags


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("size", [-14, -24, -30, 12])
def test_a_page_of_zeros_among_the_values(size, rows, code, real):
    """The zero page's tokens count in the sum of weights and leave the other pages' weights their bits,
    whether it comes first, in the middle or last."""
    (H, Hk, m), dtype, g = rows, CODES[code], torch.Generator().manual_seed(40 + size)
    n = [300, 290, 200]
    codes, scales, table = ref.make_cache(g, 3, Hk, 16, 64, n, dtype)
    scales[1].copy_(torch.where(torch.isnan(scales[1]), scales[1], 2.0 ** size * (1 + torch.rand(scales[1].shape, generator=g))))
    for b, slot in enumerate((0, 7, 12)):
        scales[1][table[b, slot]] = 0.0
    q = torch.randn((3, H, m, 64), generator=g).to(REAL[real])
    assert check(q, codes, scales, table, n, dtype) == 0


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
def test_values_that_are_all_zero(rows, real):
    (H, Hk, m), dtype, g = rows, torch.int8, torch.Generator().manual_seed(6)
    codes, scales, table = ref.make_cache(g, 1, Hk, 32, 32, [333], dtype)
    scales[1].fill_(0.0)
    assert check(torch.randn((1, H, m, 32), generator=g).to(REAL[real]), codes, scales, table, [333], dtype) == 0


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("rows", ROWS)
def test_value_scales_of_many_sizes(rows, code, real):
    (H, Hk, m), dtype, g = rows, CODES[code], torch.Generator().manual_seed(41)
    codes, scales, table = ref.make_cache(g, 2, Hk, 16, 128, [260, 190], dtype)
    s = scales[1]
    s.copy_(torch.where(torch.isnan(s), s, 2.0 ** torch.randint(-30, 11, s.shape, generator=g).float()))
    s[table[0, 3]] = 0.0
    s[table[1, 11], 0] = 0.0
    assert check(torch.randn((2, H, m, 128), generator=g).to(REAL[real]), codes, scales, table, [260, 190], dtype) == 0


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("at", [0, 4000])
def test_one_token_that_outweighs_all_others(at, rows, real):
    """Its value is zero, so that the result is what the small weights (2^-30.4 of its own) add up to."""
    (H, Hk, m), n, d, dtype = rows, 4200, 32, torch.int8
    table = torch.randperm(17, generator=torch.Generator().manual_seed(2)).int()[None, :]
    codes = [torch.zeros((17, Hk, 256, d), dtype=torch.int8) for _ in range(2)]
    codes[1].fill_(100)
    codes[0][table[0, at // 256], :, at % 256, 0] = 127
    codes[1][table[0, at // 256], :, at % 256] = 0
    scales = [torch.full((17, Hk), 1.0 / 127), torch.full((17, Hk), 2.0 ** -7)]
    q = torch.zeros((1, H, m, d), dtype=REAL[real])
    q[..., 0] = 1.0
    assert check(q, codes, scales, table, [n], dtype, scale=30.4 * math.log(2.0)) == 0


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
def test_tokens_that_outweigh_the_others_of_whole_sequences(rows, real):
    """As above with 448 heavy tokens, of a batch so large that a sequence is not shared out over the GPU:
    the light tokens meet the heavy ones' reference everywhere. The sequences share their pages."""
    (H, Hk, m), n, d, B, dtype = rows, 1500, 32, 320, torch.int8
    table = ints([[3, 0, 4, 1, 5, 2]])
    codes = [torch.zeros((6, Hk, 256, d), dtype=torch.int8) for _ in range(2)]
    codes[1].fill_(100)
    for j in range(448):
        codes[0][table[0, j // 256], :, j % 256, 0] = 127
        codes[1][table[0, j // 256], :, j % 256] = 0
    scales = [torch.full((6, Hk), 1.0 / 127), torch.full((6, Hk), 2.0 ** -7)]
    q = torch.zeros((1, H, m, d), dtype=REAL[real])
    q[..., 0] = 1.0
    kw = dict(scale=30.4 * math.log(2.0))
    want, want_lse, tol, tol_lse = cache_exact.attend(q, codes, scales, table, [n], [m], dtype, **kw)
    cache = dev_cache(codes, scales, table.expand(B, -1).contiguous(), dtype)
    out, lse = sp.spattn_fwd_cache(q.expand(B, -1, -1, -1).cuda(), cache, ints([n] * B).cuda(), **kw)
    off = (out.double().cpu() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    assert bool(((lse.double().cpu().view(B, H, m) - want_lse).abs() <= tol_lse).all())


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_fp32_queries_keep_their_bits(d, code):
    """The error of out in its norm, against twice what single roundings of a weight come to.

    In units u = 2^-24; a rounding by at most r u has a standard deviation of 0.58 r u, and errors of the weights
    that are independent move out by their standard deviation, since out itself is such a sum. A score (about 1
    in base e where the weights are large): d / 16 products in a row, each truncated by up to 2 u, on average u,
    of a sum that grows to the score: 0.6 u d / 16 in all, to one side. Two roundings of its factor: 1.2 u; of
    the exponent, below 4 where it counts: 0.8 u; the exponential (2^-22.5): 1.6 u; the weight times the rest of
    its scale and its second part: u; sums of 16 values, truncated twice, and of those sums: 1.5 u. The squares
    of the latter add up to less than 8 u^2. Accumulating all of P V in the products (8000 / 16 truncations to
    one side, shared among some pieces) or an exponent around 10 (4 u more) does not keep within this."""
    dtype, g = CODES[code], torch.Generator().manual_seed(50 + d)
    n, H = [8000, 5000], 8
    codes, scales, table = ref.make_cache(g, 2, H, 64, d, n, dtype)
    q = torch.randn((2, H, 1, d), generator=g)
    out, _ = sp.spattn_fwd_cache(q.cuda(), dev_cache(codes, scales, table, dtype), ints(n).cuda())
    off = norm = 0.0
    for b in range(2):
        k, v = (ref.tokens(c, s, table, b, n[b], dtype) for c, s in zip(codes, scales))
        want = torch.softmax(q[b].double() @ k.transpose(1, 2) / math.sqrt(d), -1) @ v
        off += float((out[b].double().cpu() - want).square().sum())
        norm += float(want.square().sum())
    assert math.sqrt(off / norm) <= 2 * 2.0 ** -24 * math.sqrt((0.6 * d / 16) ** 2 + 8), math.sqrt(off / norm)


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
def test_a_sequence_of_the_most_tokens(rows, real):
    """2^31 - 1024 tokens under a window, over eight pages again and again: the same as a short sequence that
    ends at the same place of the same page. The sequence beside it has fewer tokens than queries, and a
    window that reaches as far before its first token as an int does."""
    (H, Hk, m), dtype, g = rows, torch.int8, torch.Generator().manual_seed(46)
    n, short, page = 2 ** 31 - 1024, 5120, 256
    codes, scales, some = ref.make_cache(g, 1, Hk, page, 32, [8 * page], dtype)
    row = some[0, :8]
    table = row.repeat(n // page // 8 + 1)[None, :n // page].contiguous()
    q = torch.randn((1, H, m, 32), generator=g).to(REAL[real])
    kw = dict(window=700, n_global=40)
    cache = dev_cache(codes, scales, table, dtype)
    out, lse = sp.spattn_fwd_cache(q.cuda(), cache, ints([n]).cuda(), **kw)
    want, want_lse, tol, tol_lse = cache_exact.attend(q, codes, scales, row.repeat(3)[None, :], [short], [m], dtype, **kw)
    assert bool(((out.double().cpu() - want).abs() <= tol).all())
    assert bool(((lse.double().cpu().view(want_lse.shape) - want_lse).abs() <= tol_lse).all())
    assert check(q, codes, scales, row[None, :], [min(m, 5)], dtype, window=2 ** 31 - 1) == 0


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
def test_pages_that_are_missing(rows, real):
    (H, Hk, m), dtype, g = rows, torch.float8_e4m3fn, torch.Generator().manual_seed(43)
    codes, scales, table = ref.make_cache(g, 2, Hk, 16, 64, [330, 200], dtype)
    used = table.clone()
    used[0, 5], used[0, 20], used[1, 0] = 1 << 20, -7, -1
    q = torch.randn((2, H, m, 64), generator=g).to(REAL[real])
    assert check(q, codes, scales, table, [330, 200], dtype, used=used, gone={(0, 5), (0, 20), (1, 0)}) == 4


def test_the_status_of_each_cache_fault():
    table = ints([[0, 1]]).cuda()
    cache = sp.Cache.empty(2, 1, 16, 32, table, dtype=torch.int8)
    x = torch.ones((1, 1, 3, 32), device="cuda")
    sp.spattn_cache_write(x, x, cache, ints([30]).cuda())                 # behind the table
    assert sp.spattn_check_device_error() == sp.SPATTN_ERR_BAD_CACHE
    assert sp.spattn_check_device_error() == sp.SPATTN_OK
    x[0, 0, 1, 3] = math.inf
    sp.spattn_cache_write(x, x, cache)
    assert sp.spattn_check_device_error() == sp.SPATTN_ERR_BAD_CACHE
    assert sp.spattn_device_error() == 0
