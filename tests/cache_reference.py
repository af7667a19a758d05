"""The 8-bit cache in plain 64-bit arithmetic on the CPU, for the tests of the CUDA path, and the
inputs those tests share."""
from __future__ import annotations

import math

import torch

CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def quotient(x64, s32):
    """x / s held in 32 bits. Both are 32-bit numbers, and rounding their 64-bit quotient gives the
    correctly rounded 32-bit one (53 >= 2 * 24 + 2 bits)."""
    return (x64 / s32.double()).float()


def make_codes(x64, s32, dtype):
    """Codes (raw bytes, int8) of x under scale s (broadcast): NaN as 0, clipped, ties to even."""
    qmax = QMAX[dtype]
    q = quotient(x64, torch.where(s32 > 0, s32, torch.ones_like(s32))).clamp(-qmax, qmax)
    q = torch.where(torch.isnan(x64) | ~(s32 > 0), torch.zeros_like(q), q)
    return torch.round(q).to(torch.int8) if dtype == torch.int8 else q.to(dtype).view(torch.int8)


def write(codes, scale, table, new, start, length, dtype):
    """In place on CPU tensors. codes: raw bytes (int8) [pages, Hk, page, d]."""
    page = codes.shape[2]
    for b in range(table.shape[0]):
        s0, cnt = int(start[b]), int(length[b])
        for pi in range(s0 // page, -(-(s0 + cnt) // page) if cnt else s0 // page):
            pid = int(table[b, pi])
            lo, hi = max(s0, pi * page), min(s0 + cnt, (pi + 1) * page)
            x = new[b, :, lo - s0:hi - s0].double()
            a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax((1, 2))
            s = quotient(a, torch.full_like(a, QMAX[dtype]).float())
            older = lo - pi * page
            if older:
                before = scale[pid].clone()
                grown = s > before
                s = torch.where(grown, s, before)
                was = codes[pid, :, :older].view(dtype).float().double() * before.double()[:, None, None]
                redo = make_codes(was.float().double(), s[:, None, None], dtype)
                codes[pid, grown, :older] = redo[grown]
            codes[pid, :, older:older + hi - lo] = make_codes(x, s[:, None, None], dtype)
            scale[pid] = s


def tokens(codes, scale, table, b, n, dtype):
    """Values of the first n tokens of sequence b as fp32 products, [Hk, n, d] in 64 bits."""
    page = codes.shape[2]
    rows = table[b, :-(-n // page)].long()
    x = codes[rows].view(dtype).float() * scale[rows][..., None, None]
    return x.double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]


def attend(q, codes, scales, table, seqlen, qlen, dtype, window=-1, n_global=0, scale=None):
    """(out, lse, tolerance of out, tolerance of lse), all 64-bit [B, H, m, d] / [B, H, m].

    The tolerances, with S the largest sum |q_i k_i| * scale of a row and V the largest |v|: a score is
    a sum of d fp32 products and d additions, then two more products, each off by at most 2^-23
    relative (accumulation may truncate): ds = (d + 4) 2^-23 S; the exponent's argument adds 2^-22 (S + 8)
    for the subtraction of the maximum and the scale's logarithm, and the exponential and the sums
    2^-21. A weight is off by that relative amount, in numerator and denominator: 2 V times it. For
    bf16 queries weights are rounded to 11 bits (2^-11 V) and the result to bf16 (2^-8 |out|); for f32
    to two such parts (2^-22 V, and 2^-24 |out|)."""
    B, H, m, d = q.shape
    Hk = codes[0].shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros((B, H, m, d), dtype=torch.float64)
    lse = torch.full((B, H, m), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    half = q.dtype == torch.bfloat16
    for b in range(B):
        n, c = int(seqlen[b]), min(int(qlen[b]), m)
        if c <= 0:
            continue
        k = tokens(codes[0], scales[0], table, b, n, dtype).repeat_interleave(H // Hk, 0)
        v = tokens(codes[1], scales[1], table, b, n, dtype).repeat_interleave(H // Hk, 0)
        pos = torch.arange(n - c, n)[:, None]
        j = torch.arange(n)[None, :]
        sees = j <= pos
        if window >= 0:
            sees &= (j >= pos - window) | (j < n_global)
        x = q[b, :, :c].double()
        s = (x @ k.transpose(1, 2) * scale).masked_fill(~sees, -math.inf)
        S = (x.abs() @ k.abs().transpose(1, 2) * abs(scale)).masked_fill(~sees, 0).amax(-1) if n else torch.zeros(H, c)
        has = sees.any(-1)
        p = torch.softmax(s, -1).masked_fill(~sees, 0.0)
        p[:, ~has] = 0
        o = p @ v
        V = (v.abs().amax((1, 2)) if n else torch.zeros(H, dtype=torch.float64))[:, None]
        out[b, :, :c] = o
        if n:
            lse[b, :, :c] = torch.logsumexp(s, -1)
        ds = (d + 4) * 2.0 ** -23 * S + 2.0 ** -22 * (S + 8) + 2.0 ** -21
        round_p, round_o = (2.0 ** -11, 2.0 ** -8) if half else (2.0 ** -22, 2.0 ** -24)
        tol[b, :, :c] = ((2 * ds + round_p) * V)[..., None] + round_o * o.abs()
        tol_lse[b, :, :c] = ds + 2.0 ** -23 * lse[b, :, :c].abs().nan_to_num(posinf=0)
    return out, lse, tol, tol_lse


def make_cache(g, B, Hk, page, d, spans, dtype, layout="heads", spare=3):
    """A cache on the CPU whose sequences hold `spans` tokens: (codes of K and V as raw bytes
    [pages, Hk, page, d], scales, table). Pages of nobody, places behind a sequence and the scales of
    unused pages hold NaN codes (e4m3) or -128 (which is no code of a write), NaN scales and table
    entries -1. layout: the order in memory, "heads" [pages, Hk, page, d] or "tokens" [pages, page, Hk, d]."""
    need = [-(-s // page) for s in spans]
    total, width = sum(need) + spare, max(need + [1]) + 1
    order = torch.randperm(total, generator=g)[:sum(need)].int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    codes, scales = [], []
    for _ in range(2):
        shape = (total, Hk, page, d) if layout == "heads" else (total, page, Hk, d)
        raw = torch.full(shape, 127 if dtype != torch.int8 else -128, dtype=torch.int8)
        c = raw if layout == "heads" else raw.transpose(1, 2)
        sc = torch.full((total, Hk), math.nan)
        for b in range(B):
            for pi in range(need[b]):
                pid, cnt = int(table[b, pi]), min(page, spans[b] - pi * page)
                x = torch.randn((Hk, cnt, d), generator=g)
                if dtype == torch.int8:
                    c[pid, :, :cnt] = (x * 40).round().clamp(-127, 127).to(torch.int8)
                else:
                    c[pid, :, :cnt] = (x * 120).clamp(-448, 448).to(dtype).view(torch.int8)
                sc[pid] = (torch.rand((Hk,), generator=g) + 0.3) * 3.0 / QMAX[dtype]
        codes.append(c)
        scales.append(sc)
    return codes, scales, table
