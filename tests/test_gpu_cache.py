"""The 8-bit key/value cache on the GPU against plain 64-bit arithmetic: writing, reading back,
attention of the last tokens, and the three together."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import cache_reference as ref
from cache_reference import CODES

if torch.cuda.is_available():
    import sparse_mask_scaled_b200 as sp

REAL = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev_cache(codes, scales, table, dtype):
    k, v = (c.cuda().view(dtype) if c.is_contiguous() else c.transpose(1, 2).cuda().view(dtype).transpose(1, 2)
            for c in codes)
    ks, vs = (s.cuda() for s in scales)
    return sp.Cache(k, v, ks, vs, table.cuda())


def raw(t):
    return t.view(torch.int8).cpu() if t.is_contiguous() else t.transpose(1, 2).view(torch.int8).transpose(1, 2).cpu()


def ints(v):
    return torch.tensor(v, dtype=torch.int32)


def same(a, b):
    """Equal, with NaN equal to NaN."""
    a, b = a.cpu(), b.cpu()
    return torch.equal(torch.isnan(a.float()), torch.isnan(b.float())) and torch.equal(a.float().nan_to_num(0), b.float().nan_to_num(0))


@pytest.fixture(autouse=True)
def no_device_error():
    sp.spattn_device_error()
    yield
    assert sp.spattn_device_error() == 0


# ------------------------------------------------------------------ write, read
WRITES = [
    # Hk, page, d, m, starts, lengths
    (3, 16, 32, 1, [0, 5, 15, 16, 31], [1, 1, 1, 1, 0]),
    (2, 64, 128, 70, [0, 63, 64, 1], [70, 2, 65, 64]),
    (1, 32, 64, 5, [27, 28, 0], [5, 4, 3]),
    (5, 128, 32, 300, [0, 100], [300, 29]),
    (2, 256, 128, 257, [255, 0, 256], [257, 256, 1]),
]


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_write_codes_and_scales_equal_the_definition(case, layout, real, code):
    Hk, page, d, m, start, length = WRITES[case]
    dtype, g = CODES[code], torch.Generator().manual_seed(case)
    B = len(start)
    # sequences hold `start` tokens; the table has room for the new ones
    codes, scales, table = ref.make_cache(g, B, Hk, page, d, [s + c for s, c in zip(start, length)], dtype, layout)
    new = [(torch.randn((B, Hk, m, d), generator=g) * torch.rand((B, Hk, 1, 1), generator=g) * 6).to(REAL[real])
           for _ in range(2)]
    cache = dev_cache(codes, scales, table, dtype)
    want_c, want_s = [c.clone() for c in codes], [s.clone() for s in scales]
    for c, s, x in zip(want_c, want_s, new):
        ref.write(c, s, table, x, start, length, dtype)
    args = (new[0].cuda(), new[1].cuda(), cache, ints(start).cuda(), ints(length).cuda())
    for _ in range(2):      # the second write of the same tokens changes nothing
        sp.spattn_cache_write(*args)
        for got, want in zip((cache.k, cache.v), want_c):
            assert torch.equal(raw(got), want)
        for got, want in zip((cache.k_scale, cache.v_scale), want_s):
            assert same(got, want)


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_tokens_written_one_by_one(code):
    """Every append may grow the page's scale and re-quantise what it holds."""
    dtype, g = CODES[code], torch.Generator().manual_seed(3)
    B, Hk, page, d, n = 2, 2, 16, 64, 35
    codes, scales, table = ref.make_cache(g, B, Hk, page, d, [n, n], dtype)
    cache = dev_cache(codes, scales, table, dtype)
    x = [torch.randn((B, Hk, n, d), generator=g) * torch.linspace(0.1, 4, n)[:, None] for _ in range(2)]
    for t in range(n):
        new = [y[:, :, t:t + 1].contiguous() for y in x]
        sp.spattn_cache_write(new[0].cuda(), new[1].cuda(), cache, ints([t, t]).cuda())
        for c, s, y in zip(codes, scales, new):
            ref.write(c, s, table, y, [t, t], [1, 1], dtype)
    for got, want in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), codes + scales):
        assert same(raw(got) if got.dtype == dtype else got, want)
    k, v = sp.spattn_cache_read(cache, n, dtype=torch.float32)
    # a value is off by at most half a code step at the page's final scale each time its page's scale
    # grew (at most page times): int8 s / 2 a time; e4m3 2^-4 |x| a time
    for got, want, s in zip((k, v), x, scales):
        step = s[table[:, :-(-n // page)].long()].repeat_interleave(page, 1)[:, :n].transpose(1, 2)[..., None]
        once = step / 2 if code == "i8" else 2.0 ** -4 * want.abs() + 2.0 ** -10 * step
        assert bool(((got.cpu() - want).abs() <= page * once + 1e-6).all())


def test_write_of_zeros_and_of_what_is_not_finite():
    dtype = torch.int8
    for dtype in CODES.values():
        table = ints([[0, 1]]).cuda()
        cache = sp.Cache.empty(2, 1, 16, 32, table, dtype=dtype)
        x = torch.zeros((1, 1, 16, 32))
        sp.spattn_cache_write(x.cuda(), x.cuda(), cache)
        assert float(cache.k_scale[0]) == 0 and not raw(cache.k).any()
        assert sp.spattn_device_error() == 0
        x[0, 0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 2.0])
        sp.spattn_cache_write(x.cuda(), x.cuda(), cache)
        k, _ = sp.spattn_cache_read(cache, 16, dtype=torch.float32)
        assert k[0, 0, 0, :4].tolist() == pytest.approx([2.0, -2.0, 0.0, 2.0], rel=2.0 ** -22)
        assert not k[0, 0, 1:].any()
        assert sp.spattn_device_error() == 8
        assert sp.spattn_check_device_error() == sp.SPATTN_OK


READS = [(2, 16, 32, 1, [0, 17], [1, 1]), (3, 64, 128, 200, [0, 63, 130], [200, 1, 0]), (1, 256, 64, 33, [250], [20])]


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("case", range(len(READS)))
def test_read_equals_the_definition(case, layout, real, code):
    Hk, page, d, m, start, length = READS[case]
    dtype, g = CODES[code], torch.Generator().manual_seed(10 + case)
    codes, scales, table = ref.make_cache(g, len(start), Hk, page, d, [s + c for s, c in zip(start, length)], dtype,
                                          layout)
    cache = dev_cache(codes, scales, table, dtype)
    k, v = sp.spattn_cache_read(cache, m, dtype=REAL[real], start=ints(start).cuda(), length=ints(length).cuda())
    for got, c, s in zip((k, v), codes, scales):
        want = torch.zeros(got.shape, dtype=torch.float64)
        for b in range(len(start)):
            want[b, :, :length[b]] = ref.tokens(c, s, table, b, start[b] + length[b], dtype)[:, start[b]:]
        assert torch.equal(got.cpu(), want.float().to(REAL[real]))


def test_strided_rows_and_rows_behind_the_last_sequence():
    """K and V as slices of a wider tensor, [batch, m, heads, d] in memory; what lies around them stays."""
    g = torch.Generator().manual_seed(5)
    B, Hk, m, d, page = 2, 3, 20, 64, 16
    table = ints([[3, 1], [0, 2]]).cuda()
    cache = sp.Cache.empty(5, Hk, page, d, table)
    wide = torch.randn((B, m, 2 * Hk + 1, d), generator=g).cuda()
    k, v = wide[:, :, :Hk].transpose(1, 2), wide[:, :, Hk:2 * Hk].transpose(1, 2)
    sp.spattn_cache_write(k, v, cache)
    plain = sp.Cache.empty(5, Hk, page, d, table)
    sp.spattn_cache_write(k.contiguous(), v.contiguous(), plain)
    assert torch.equal(raw(cache.k), raw(plain.k)) and torch.equal(raw(cache.v), raw(plain.v))
    assert not raw(cache.k)[4].any() and not raw(cache.k)[1, :, 4:].any()   # a page of nobody, places behind token 19
    back = torch.full((B, m, 2 * Hk + 1, d), 7.0, device="cuda")
    kb, vb = back[:, :, :Hk].transpose(1, 2), back[:, :, Hk:2 * Hk].transpose(1, 2)
    sp.spattn_cache_read(cache, m, k=kb, v=vb, dtype=torch.float32)
    k2, v2 = sp.spattn_cache_read(plain, m, dtype=torch.float32)
    assert torch.equal(kb, k2) and torch.equal(vb, v2) and bool((back[:, :, 2 * Hk] == 7).all())


# ------------------------------------------------------------------ attention
ATTEND = [
    # H, Hk, page, d, m, seqlens, qlens, window, n_global
    (4, 4, 16, 32, 1, [1, 2, 15, 16, 17, 0], None, -1, 0),
    (8, 2, 64, 128, 1, [63, 64, 65, 700], [1, 0, 1, 1], -1, 0),
    (12, 12, 32, 64, 1, [513, 31], None, 40, 5),
    (6, 2, 16, 64, 5, [5, 4, 130, 64], [5, 5, 3, 1], -1, 0),
    (16, 1, 128, 128, 1, [257], None, -1, 0),
    (5, 1, 256, 128, 7, [300, 7], None, 0, 0),
    (4, 4, 16, 128, 3, [200, 90, 3], [3, 2, 1], 17, 33),
    (14, 2, 64, 32, 9, [1000, 10], None, 64, 1),
    (4, 2, 64, 128, 150, [150, 400, 149], [150, 150, 100], -1, 0),
    (2, 1, 16, 64, 333, [700, 333], None, 100, 20),
    (8, 8, 32, 32, 64, [64, 65], None, 1 << 30, 0),
    (3, 3, 32, 128, 2, [2500, 2400, 1, 0], None, -1, 0),
]


def run_attend(case, code, real, layout="heads", scale=None):
    H, Hk, page, d, m, seqlen, qlen, window, n_global = ATTEND[case]
    dtype, g = CODES[code], torch.Generator().manual_seed(100 + case)
    B = len(seqlen)
    codes, scales, table = ref.make_cache(g, B, Hk, page, d, seqlen, dtype, layout)
    cache = dev_cache(codes, scales, table, dtype)
    q = (torch.randn((B, H, m, d), generator=g) * 2).to(REAL[real])
    out, lse = sp.spattn_fwd_cache(q.cuda(), cache, ints(seqlen).cuda(),
                                   qlen=None if qlen is None else ints(qlen).cuda(), window=window,
                                   n_global=n_global, scale=scale)
    want = ref.attend(q, codes, scales, table, seqlen, [m] * B if qlen is None else qlen, dtype, window, n_global,
                      scale)
    return out, lse, want


def assert_attend(out, lse, want):
    ref_out, ref_lse, tol, tol_lse = want
    out, lse = out.double().cpu(), lse.double().cpu().view(ref_lse.shape)
    assert torch.equal(torch.isneginf(lse), torch.isneginf(ref_lse))
    some = ~torch.isneginf(ref_lse)
    assert bool((out[~some] == 0).all())
    assert bool(((out - ref_out).abs() <= tol + 1e-30).all()), float(((out - ref_out).abs() / (tol + 1e-30)).max())
    gap = (lse - ref_lse).abs()[some]
    assert bool((gap <= tol_lse[some]).all()), float((gap / tol_lse[some]).max())


@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention_matches_the_definition(case, code, real):
    assert_attend(*run_attend(case, code, real))


@pytest.mark.parametrize("case", [1, 6, 8])
def test_attention_over_a_pool_with_tokens_before_heads(case):
    out, lse, want = run_attend(case, "e4m3", "bf16", layout="tokens")
    assert_attend(out, lse, want)
    again = run_attend(case, "e4m3", "bf16")
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_softmax_scales(scale):
    for case in (1, 8):
        assert_attend(*run_attend(case, "i8", "f32", scale=scale))


def test_scales_of_many_sizes_and_zero():
    """Pages whose scales differ by many powers of two, zeros among them; queries of many sizes."""
    g = torch.Generator().manual_seed(77)
    for code, real in (("i8", "f32"), ("e4m3", "bf16")):
        dtype = CODES[code]
        codes, scales, table = ref.make_cache(g, 2, 2, 16, 64, [230, 64], dtype)
        for s, low, high in ((scales[0], -30, -6), (scales[1], -40, 20)):
            s.copy_(torch.where(torch.isnan(s), s, 2.0 ** torch.randint(low, high, s.shape, generator=g).float()))
            s[table[0, 3]] = 0.0
            s[table[1, 1], 1] = 0.0
        cache = dev_cache(codes, scales, table, dtype)
        q = (torch.randn((2, 4, 3, 64), generator=g) * 10.0 ** torch.randint(-9, 1, (2, 4, 3, 1), generator=g)).to(REAL[real])
        q[0, 0, 0] = 0
        out, lse = sp.spattn_fwd_cache(q.cuda(), cache, ints([230, 64]).cuda())
        assert_attend(out, lse, ref.attend(q, codes, scales, table, [230, 64], [3, 3], dtype))


@pytest.mark.parametrize("m", [1, 130])
def test_large_scores_stay_finite(m):
    g = torch.Generator().manual_seed(8)
    codes, scales, table = ref.make_cache(g, 1, 1, 64, 64, [500], torch.int8)
    q = (torch.randn((1, 2, m, 64), generator=g) * 300).to(torch.bfloat16)
    cache = dev_cache(codes, scales, table, torch.int8)
    out, lse = sp.spattn_fwd_cache(q.cuda(), cache, ints([500]).cuda())
    assert_attend(out, lse, ref.attend(q, codes, scales, table, [500], [m], torch.int8))


def test_a_nan_query_spoils_its_own_row_only():
    for m in (4, 140):
        g = torch.Generator().manual_seed(9)
        codes, scales, table = ref.make_cache(g, 1, 1, 16, 32, [200], torch.int8)
        cache = dev_cache(codes, scales, table, torch.int8)
        q = torch.randn((1, 3, m, 32), generator=g).bfloat16()
        clean = sp.spattn_fwd_cache(q.cuda(), cache, ints([200]).cuda())
        q[0, 1, 2, 5] = math.nan
        out, lse = sp.spattn_fwd_cache(q.cuda(), cache, ints([200]).cuda())
        bad = torch.zeros((1, 3, m), dtype=torch.bool)
        bad[0, 1, 2] = True
        assert bool(out.cpu()[bad].isnan().all()) and bool(lse.view(1, 3, m).cpu()[bad].isnan().all())
        assert torch.equal(out.cpu()[~bad], clean[0].cpu()[~bad])
        assert torch.equal(lse.view(1, 3, m).cpu()[~bad], clean[1].view(1, 3, m).cpu()[~bad])


def test_strided_queries_and_outputs():
    g = torch.Generator().manual_seed(11)
    for m in (2, 150):
        codes, scales, table = ref.make_cache(g, 2, 2, 32, 64, [222, 150], torch.int8)
        cache = dev_cache(codes, scales, table, torch.int8)
        wide = torch.randn((2, m, 9, 64), generator=g).bfloat16().cuda()
        q = wide[:, :, 1:7].transpose(1, 2)                       # [B, 6, m, d], tokens before heads
        back = torch.full((2, m, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        out, lse = sp.spattn_fwd_cache(q, cache, ints([222, 150]).cuda(), out=back[:, :, 1:7].transpose(1, 2))
        plain, plain_lse = sp.spattn_fwd_cache(q.contiguous(), cache, ints([222, 150]).cuda())
        assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
        assert bool((back[:, :, 0] == 7).all()) and bool((back[:, :, 7] == 7).all())


def test_lengths_beyond_the_table_and_missing_pages():
    """Lengths are clamped to what the table holds; a page outside the pool is left out and flagged."""
    g = torch.Generator().manual_seed(12)
    for m in (1, 140):
        codes, scales, table = ref.make_cache(g, 2, 1, 16, 32, [160, 160], torch.int8)
        table = table[:, :10].contiguous()
        cache = dev_cache(codes, scales, table, torch.int8)
        q = torch.randn((2, 2, m, 32), generator=g).bfloat16()
        out, lse = sp.spattn_fwd_cache(q.cuda(), cache, ints([999, -4]).cuda(), qlen=ints([m + 9, m]).cuda())
        assert_attend(out, lse, ref.attend(q, codes, scales, table, [160, 0], [m, 0], torch.int8))
        assert sp.spattn_device_error() == 0
        gone = table.clone()
        gone[0, 4] = 1 << 20
        cache = dev_cache(codes, scales, gone, torch.int8)
        out, lse = sp.spattn_fwd_cache(q[:, :, :1].contiguous().cuda(), cache, ints([160, 160]).cuda())
        assert sp.spattn_device_error() == 4
        # what is left: the sequence without that page
        rest = torch.cat([table[:, :4], table[:, 5:]], 1)
        want = ref.attend(q[:1, :, :1], codes, scales, rest[:1], [144], [1], torch.int8)
        assert_attend(out[:1], lse.view(2, 2, 1)[:1], want)
        k, _ = sp.spattn_cache_read(cache, 80, dtype=torch.float32)
        assert not k[0, :, 64:80].any() and bool(k[0, :, 63].any())
        assert sp.spattn_device_error() == 4


def test_write_outside_the_table_leaves_the_cache():
    table = ints([[0, 1], [2, 3]]).cuda()
    cache = sp.Cache.empty(4, 1, 16, 32, table, dtype=torch.int8)
    x = torch.ones((2, 1, 3, 32), device="cuda")
    sp.spattn_cache_write(x, x, cache, ints([30, -1]).cuda())
    assert not raw(cache.k).any() and not cache.k_scale.any()
    assert sp.spattn_device_error() == 4
    sp.spattn_cache_write(x, x, cache, ints([29, 40]).cuda(), length=ints([3, 0]).cuda())
    assert raw(cache.k).any()
    assert sp.spattn_device_error() == 0


# ------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_prompt_then_tokens_then_full_pass(code):
    """A prompt in two chunks, then token by token; at the end the cache read back runs under the
    library's own causal window mask and gives the last token's rows."""
    g = torch.Generator().manual_seed(21)
    dtype = CODES[code]
    B, H, Hk, d, page, window = 2, 4, 2, 64, 16, 50
    lens, extra, m = [70, 41], 9, 48
    n = max(lens) + extra
    table = torch.randperm(16, generator=g).int().view(2, 8).cuda()
    cache = sp.Cache.empty(16, Hk, page, d, table, dtype=dtype)
    k, v = ((torch.randn((B, Hk, n, d), generator=g)).bfloat16() for _ in range(2))
    q = torch.randn((B, H, n, d), generator=g).bfloat16()
    codes = [torch.zeros((16, Hk, page, d), dtype=torch.int8) for _ in range(2)]
    scales = [torch.zeros((16, Hk)) for _ in range(2)]

    def step(start, count, width):
        rows = [torch.arange(s, s + width).clamp(max=n - 1) for s in start]
        kq = [torch.stack([t[b][:, rows[b]] for b in range(B)]) for t in (k, v, q)]
        st, ln = ints(start).cuda(), ints(count).cuda()
        sp.spattn_cache_write(kq[0].cuda(), kq[1].cuda(), cache, st, length=ln)
        for c, s, x in zip(codes, scales, kq):
            ref.write(c, s, table.cpu(), x, start, count, dtype)
        total = [s + c for s, c in zip(start, count)]
        out, lse = sp.spattn_fwd_cache(kq[2].cuda(), cache, ints(total).cuda(), qlen=ln, window=window, n_global=3)
        want = ref.attend(kq[2], codes, scales, table.cpu(), total, count, dtype, window, 3)
        assert_attend(out, lse, want)
        return out

    step([0, 0], [min(m, x) for x in lens], m)
    step([min(m, x) for x in lens], [x - min(m, x) for x in lens], m)
    for t in range(extra):
        out = step([x + t for x in lens], [1, 1], 1)
    total = [x + extra for x in lens]
    kr, vr = sp.spattn_cache_read(cache, n, length=ints(total).cuda())
    rep = [x.repeat_interleave(H // Hk, 1) for x in (kr, vr)]
    cols, rp = [], [0]
    for i in range(n):
        c = sorted(set(range(max(0, i - window), i + 1)) | set(range(min(3, i + 1))))
        cols += c
        rp.append(len(cols))
    with sp.spattn_create_csr_mask("csr", n, in_row_ptr=ints(rp).cuda(), in_col_idx=ints(cols).cuda()) as mask:
        full, _ = sp.spattn_fwd_mask_kpad(q.cuda(), rep[0], rep[1], mask, ints(total).cuda())
    for b in range(B):
        a, w = out[b, :, 0].double().cpu(), full[b, :, total[b] - 1].double().cpu()
        # K and V rounded to bf16 once (2^-8 each) and two bf16 outputs: scores move by 2^-8 sum |q k| scale
        # (at most about 2^-8 * 6 here), weights by that, the output by 2 * that * V + 3 * 2^-8 V with V < 4.5
        assert float((a - w).abs().max()) <= (2 * 6 + 3) * 2.0 ** -8 * 4.5


def test_streams_capture_and_replay():
    """Writes and attention captured into two graphs and replayed while other calls run on another stream;
    the captured calls see the buffers' contents at replay."""
    g = torch.Generator().manual_seed(31)
    table = torch.randperm(40, generator=g).int().view(2, 20).cuda()
    made, keep = [], []
    for real in ("bf16", "f32"):
        cache = sp.Cache.empty(40, 2, 32, 64, table, dtype=torch.int8)
        x = [torch.randn((2, h, 1, 64), generator=g).to(REAL[real]).cuda() for h in (2, 2, 8)]
        start, seqlen = ints([0, 0]).cuda(), ints([1, 1]).cuda()
        out = torch.empty_like(x[2])
        lse = torch.empty(16, device="cuda")

        def call():
            sp.spattn_cache_write(x[0], x[1], cache, start)
            sp.spattn_fwd_cache(x[2], cache, seqlen, out=out, lse=lse)
            start.add_(1)
            seqlen.add_(1)

        call()                                       # outside capture: the first call on the device
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        made.append((graph, cache, x, out, lse, real))
        keep.append((start, seqlen))                 # the graph reads and writes them
    steps = [[[torch.randn(t.shape, generator=g).to(t.dtype) for t in x] for _ in range(40)] for _, _, x, _, _, _ in made]
    side = torch.cuda.Stream()
    want = []
    for (graph, cache, x, out, lse, real), seq in zip(made, steps):
        codes = [torch.zeros((40, 2, 32, 64), dtype=torch.int8) for _ in range(2)]
        scales = [torch.zeros((40, 2)) for _ in range(2)]
        first = [t.cpu() for t in x]
        for t, new in enumerate([first] + seq):
            for c, s, y in zip(codes, scales, new):
                ref.write(c, s, table.cpu(), y, [t, t], [1, 1], torch.int8)
        want.append(ref.attend(seq[-1][2], codes, scales, table.cpu(), [41, 41], [1, 1], torch.int8))
    torch.cuda.synchronize()
    for t in range(40):
        for (graph, cache, x, out, lse, real), seq in zip(made, steps):
            s = side if real == "f32" else torch.cuda.current_stream()
            with torch.cuda.stream(s):
                for dst, new in zip(x, seq[t]):
                    dst.copy_(new)
                graph.replay()
    torch.cuda.synchronize()
    for (graph, cache, x, out, lse, real), w in zip(made, want):
        assert_attend(out, lse, w)


def test_runs_give_the_same_bits():
    a = run_attend(8, "e4m3", "bf16")
    b = run_attend(8, "e4m3", "bf16")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = run_attend(11, "i8", "f32"), run_attend(11, "i8", "f32")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
