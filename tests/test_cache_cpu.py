"""The 8-bit key/value cache without a GPU: argument checks reject bad calls before any device work,
in the C ABI and in the Python binding, and the tests' plain arithmetic is pinned."""
import ctypes
import math

import pytest
import torch

import cache_reference as ref
import sparse_mask_scaled_b200 as sp

PAGES, HK, PAGE, D, B = 7, 2, 16, 64, 3


def desc(shape, dtype, data=0x100000, stride=None, reserved=0):
    if stride is None:
        stride, acc = [0] * 4, 1
        for x in range(3, -1, -1):
            stride[x] = acc
            acc *= shape[x]
    return sp.spattn_tensor(data, dtype, reserved, tuple(shape), tuple(stride))


def cache(k=None, v=None, **kw):
    shape = (PAGES, HK, PAGE, D)
    a = dict(k_scale=0x200000, v_scale=0x200000, page_table=0x300000, batch=B, max_pages=5, table_stride=5)
    a.update(kw)
    k = k or desc(shape, sp.SPATTN_I8)
    return sp.spattn_cache(k, v or k, a["k_scale"], a["v_scale"], a["page_table"], a["batch"], a["max_pages"],
                           a["table_stride"])


def rows(heads=HK, m=4, d=D, dtype=sp.SPATTN_BF16, **kw):
    return desc((B, heads, m, d), dtype, **kw)


def call(name, c, x, y=None, lens=0x400000, qlen=None, window=-1, n_global=0, scale=0.1, lse=None):
    y = y or x
    before = sp.spattn_launch_count()
    if name == "write":
        st = sp.LIB.spattn_cache_write(ctypes.byref(x), ctypes.byref(y), ctypes.byref(c), lens, qlen, None)
    elif name == "read":
        st = sp.LIB.spattn_cache_read(ctypes.byref(c), lens, qlen, ctypes.byref(x), ctypes.byref(y), None)
    else:
        st = sp.LIB.spattn_fwd_cache(ctypes.byref(x), ctypes.byref(c), lens, qlen, window, n_global, scale,
                                     ctypes.byref(y), lse, None)
    assert sp.spattn_launch_count() == before
    return st, sp.spattn_last_error()


INVALID, UNSUPPORTED = sp.SPATTN_ERR_INVALID_ARG, sp.SPATTN_ERR_UNSUPPORTED
full = (PAGES, HK, PAGE, D)
BAD_CACHES = [
    (dict(k=desc(full, sp.SPATTN_BF16)), UNSUPPORTED, "dtype"),
    (dict(v=desc(full, sp.SPATTN_E4M3)), INVALID, "dtype"),
    (dict(v=desc((PAGES, HK, PAGE, 32), sp.SPATTN_I8)), INVALID, "shape"),
    (dict(k=desc((0, HK, PAGE, D), sp.SPATTN_I8)), INVALID, "shape"),
    (dict(k=desc((PAGES, HK, PAGE, 96), sp.SPATTN_I8)), UNSUPPORTED, "head dim"),
    (dict(k=desc((PAGES, HK, 24, D), sp.SPATTN_I8)), UNSUPPORTED, "page"),
    (dict(k=desc((PAGES, HK, 8, D), sp.SPATTN_I8)), UNSUPPORTED, "page"),
    (dict(k=desc((PAGES, HK, 512, D), sp.SPATTN_I8)), UNSUPPORTED, "page"),
    (dict(k=desc(full, sp.SPATTN_I8, data=None)), INVALID, "NULL"),
    (dict(k=desc(full, sp.SPATTN_I8, data=0x100008)), UNSUPPORTED, "aligned"),
    (dict(k=desc(full, sp.SPATTN_I8, stride=(HK * PAGE * D, PAGE * D, 2 * D, 2))), UNSUPPORTED, "stride 1"),
    (dict(k=desc(full, sp.SPATTN_I8, stride=(HK * PAGE * 72, PAGE * 72, 72, 1))), UNSUPPORTED, "stride"),
    (dict(k=desc(full, sp.SPATTN_I8, stride=(-HK * PAGE * D, PAGE * D, D, 1))), UNSUPPORTED, "stride"),
    (dict(k=desc(full, sp.SPATTN_I8, reserved=1)), INVALID, "reserved"),
    (dict(k_scale=None), INVALID, "k_scale"),
    (dict(v_scale=0x200002), INVALID, "v_scale"),
    (dict(page_table=None), INVALID, "page_table"),
    (dict(max_pages=0), INVALID, "max_pages"),
    (dict(batch=-1), INVALID, "batch"),
    (dict(table_stride=4), INVALID, "table_stride"),
    (dict(max_pages=1 << 28, table_stride=1 << 28), UNSUPPORTED, "max_pages"),
]


@pytest.mark.parametrize("name", ["write", "read", "attend"])
@pytest.mark.parametrize("kw,status,frag", BAD_CACHES)
def test_bad_caches_are_refused(name, kw, status, frag):
    st, msg = call(name, cache(**kw), rows())
    assert st == status and frag in msg


@pytest.mark.parametrize("name", ["write", "read", "attend"])
@pytest.mark.parametrize("x,kw,status,frag", [
    (rows(dtype=sp.SPATTN_I8), {}, UNSUPPORTED, "dtype"),
    (rows(dtype=5), {}, UNSUPPORTED, "dtype"),
    (rows(heads=3), {}, INVALID, ""),
    (rows(d=32), {}, INVALID, "shape"),
    (desc((B + 1, HK, 4, D), sp.SPATTN_BF16), {}, INVALID, "shape"),
    (rows(data=0x100004), {}, UNSUPPORTED, "aligned"),
    (rows(data=None), {}, INVALID, "NULL"),
    (rows(), dict(y=rows(dtype=sp.SPATTN_F32)), INVALID, "dtype"),
    (rows(), dict(y=rows(m=5)), INVALID, "shape"),
    (rows(), dict(lens=0x400002), INVALID, "aligned"),
    (rows(), dict(qlen=0x400001), INVALID, "aligned"),
])
def test_bad_rows_are_refused(name, x, kw, status, frag):
    st, msg = call(name, cache(), x, **kw)
    assert st == status and frag in msg


@pytest.mark.parametrize("kw,frag", [(dict(lens=None), "seqlen"), (dict(n_global=-1), "n_global"),
                                     (dict(scale=math.nan), "scale"), (dict(lse=0x500001), "lse")])
def test_bad_attention_arguments_are_refused(kw, frag):
    st, msg = call("attend", cache(), rows(heads=4), **kw)
    assert st == INVALID and frag in msg


def test_null_descriptors():
    x, c = rows(), cache()
    assert sp.LIB.spattn_cache_write(None, ctypes.byref(x), ctypes.byref(c), None, None, None) == INVALID
    assert sp.LIB.spattn_cache_read(None, None, None, ctypes.byref(x), ctypes.byref(x), None) == INVALID
    assert sp.LIB.spattn_fwd_cache(ctypes.byref(x), None, 0x400000, None, -1, 0, 0.1, ctypes.byref(x), None,
                                   None) == INVALID


def test_the_other_entry_points_do_not_take_codes():
    x = desc((1, 2, 16, 64), sp.SPATTN_I8)
    st = sp.LIB.spattn_fwd(ctypes.byref(x), ctypes.byref(x), ctypes.byref(x), 0x200000, 0x300000, 1, 10, None, None,
                           0.1, ctypes.byref(x), None, None)
    assert st == UNSUPPORTED
    with pytest.raises(ValueError):
        sp.tensor_desc(torch.zeros((1, 1, 1, 32), dtype=torch.int8))


def test_struct_layout():
    assert ctypes.sizeof(sp.spattn_cache) == 2 * 80 + 3 * 8 + 2 * 4 + 8


def _cache(**kw):
    a = dict(k=torch.zeros((4, 2, 16, 32), dtype=torch.int8), v=torch.zeros((4, 2, 16, 32), dtype=torch.int8),
             k_scale=torch.zeros((4, 2)), v_scale=torch.zeros((4, 2)), page_table=torch.zeros((2, 3), dtype=torch.int32))
    a.update(kw)
    return sp.Cache(**a)


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros((4, 2, 16), dtype=torch.int8)), dict(k=torch.zeros((4, 2, 16, 32))),
    dict(k_scale=torch.zeros((4, 3))), dict(v_scale=torch.zeros((4, 2), dtype=torch.float64)),
    dict(v_scale=torch.zeros((2, 4)).t()), dict(page_table=torch.zeros((2, 3), dtype=torch.int64)),
    dict(page_table=torch.zeros((3, 2), dtype=torch.int32).t()),
])
def test_binding_refuses_wrong_cache_tensors(kw):
    _cache()
    with pytest.raises(ValueError):
        _cache(**kw)


def test_binding_describes_views():
    pool = torch.zeros((4, 2, 16, 2, 32), dtype=torch.int8)       # pages, K / V, tokens, heads, d
    c = _cache(k=pool[:, 0].transpose(1, 2), v=pool[:, 1].transpose(1, 2))
    assert list(c.desc.k.stride) == [2048, 32, 64, 1] and list(c.desc.k.shape) == [4, 2, 16, 32]
    assert c.desc.v.data - c.desc.k.data == 1024
    assert (c.heads, c.page, c.d, c.batch, c.max_pages) == (2, 16, 32, 2, 3)


# ------------------------------------------------------------------ pins of the plain arithmetic
def test_int8_codes_by_hand():
    s = torch.tensor(0.5)
    x = torch.tensor([0.25, 0.75, -0.25, 63.5, 100.0, -100.0, math.nan, 0.26], dtype=torch.float64)
    # 0.5 and 1.5 are ties (to 0 and 2), the clipped ones are +-127
    assert ref.make_codes(x, s, torch.int8).tolist() == [0, 2, 0, 127, 127, -127, 0, 1]


def test_e4m3_codes_by_hand():
    x = torch.tensor([1.0, 1.0625, 1.1875, 448.0, 500.0, 2.0 ** -9, 2.0 ** -10, 0.0], dtype=torch.float64)
    got = ref.make_codes(x, torch.tensor(1.0), torch.float8_e4m3fn).view(torch.float8_e4m3fn).float()
    assert got.tolist() == [1.0, 1.0, 1.25, 448.0, 448.0, 2.0 ** -9, 0.0, 0.0]


def test_write_keeps_or_grows_a_scale():
    codes = torch.zeros((1, 1, 16, 32), dtype=torch.int8)
    scale, table = torch.zeros((1, 1)), torch.tensor([[0]], dtype=torch.int32)
    one = torch.full((1, 1, 1, 32), 127.0)
    ref.write(codes, scale, table, one, [0], [1], torch.int8)
    assert float(scale) == 1 and int(codes[0, 0, 0, 0]) == 127
    ref.write(codes, scale, table, one / 127, [1], [1], torch.int8)           # smaller: the scale stays
    assert float(scale) == 1 and int(codes[0, 0, 1, 0]) == 1
    ref.write(codes, scale, table, one * 2, [2], [1], torch.int8)             # larger: older codes are halved
    assert float(scale) == 2 and codes[0, 0, :3, 0].tolist() == [64, 0, 127]  # 63.5 and 0.5 tie to even
    ref.write(codes, scale, table, one, [0], [1], torch.int8)                 # first place again: a fresh scale
    assert float(scale) == 1


def test_attend_against_torch():
    g = torch.Generator().manual_seed(1)
    codes, scales, table = ref.make_cache(g, 1, 1, 16, 32, [20], torch.int8)
    q = torch.randn((1, 2, 20, 32), generator=g)
    out, lse, _, _ = ref.attend(q, codes, scales, table, [20], [20], torch.int8)
    k, v = (ref.tokens(c, s, table, 0, 20, torch.int8)[None] for c, s in zip(codes, scales))
    want = torch.nn.functional.scaled_dot_product_attention(q.double(), k.expand(1, 2, -1, -1), v.expand(1, 2, -1, -1),
                                                            is_causal=True)
    assert float((out - want).abs().max()) < 1e-12
    only, _, _, _ = ref.attend(q, codes, scales, table, [20], [20], torch.int8, window=0)
    assert float((only - v.expand(1, 2, -1, -1)).abs().max()) < 1e-12       # each token sees itself
