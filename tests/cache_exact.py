"""Attention over the 8-bit cache in 64 bits with a tolerance for each element, from what that element
sums up rather than from the largest value of the sequence, and with page table entries left out."""
from __future__ import annotations

import math

import torch

import cache_reference as ref


def attend(q, codes, scales, table, seqlen, qlen, dtype, window=-1, n_global=0, scale=None, gone=()):
    """(out, lse, tolerance of out, tolerance of lse), 64-bit [B, H, m, d] / [B, H, m]. gone: (sequence,
    place in its row of the table) pairs whose tokens are not attended to.

    S is the largest sum |q_i k_i| * scale of a row, L the largest |log2| of its V scales, A = 1.45 S + L + 15
    a bound on a base-2 exponent and on the reference it is taken against. A score is d products and additions
    and two more products (2^-23 relative each, accumulation may truncate); an exponent is rounded three times
    at up to 2 A, and log2 of a V scale is off by 2^-22 L; times ln 2 that is 2^-22 (1.1 A + 0.7 L). The
    exponential and the reciprocals are off by 2^-21. n / 16 + 32 additions follow one another in a sum, 2^-23
    each. All that counts in the numerator and in the denominator, relative to sum_j p_j |v_j|.

    Weights are held in fp16 (bf16 queries), rounded once, and again where the reference moves: 2 * 2^-11; in two
    such parts, the second 2^11 times as large (fp32): 2^-22. The largest p_j * vs_j of a row (vs_j its V scale, at
    least 2^-64 here) is held as 2^8 or more, and fp16 is rounded by at most 2^-25 however small the weight is: a
    token is off by 2^-33 (twice for bf16, 2^-44 for fp32) times that and the largest code. The result is rounded
    at the end."""
    B, H, m, d = q.shape
    group = H // codes[0].shape[1]
    page, qmax = codes[0].shape[2], ref.QMAX[dtype]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros((B, H, m, d), dtype=torch.float64)
    lse = torch.full((B, H, m), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    half = q.dtype == torch.bfloat16
    for b in range(B):
        n, c = int(seqlen[b]), min(int(qlen[b]), m)
        if c <= 0 or n <= 0:
            continue
        k = ref.tokens(codes[0], scales[0], table, b, n, dtype).repeat_interleave(group, 0)
        v = ref.tokens(codes[1], scales[1], table, b, n, dtype).repeat_interleave(group, 0)
        pos = torch.arange(n - c, n)[:, None]
        j = torch.arange(n)[None, :]
        sees = j <= pos
        if window >= 0:
            sees = sees & ((j >= pos - window) | (j < n_global))
        for bb, slot in gone:
            if bb == b:
                sees = sees & ((j < slot * page) | (j >= (slot + 1) * page))
        has = sees.any(-1)
        x = q[b, :, :c].double()
        s = (x @ k.transpose(1, 2) * scale).masked_fill(~sees, -math.inf)
        S = (x.abs() @ k.abs().transpose(1, 2) * abs(scale)).masked_fill(~sees, 0).amax(-1)
        p = torch.softmax(s, -1).masked_fill(~sees, 0.0)
        p[:, ~has] = 0
        o = p @ v
        out[b, :, :c] = o
        lse[b, :, :c] = torch.logsumexp(s, -1)
        vs = scales[1][table[b, :-(-n // page)].long()].double().t().repeat_interleave(group, 0)  # [H, pages]
        vs = vs[:, ~torch.tensor([(b, i) in gone for i in range(vs.shape[1])])]
        L = torch.where(vs > 0, vs, torch.ones_like(vs)).log2().abs().amax(1)[:, None]
        A = 1.45 * S + L + 15
        off = (d + 4) * 2.0 ** -23 * S + 2.0 ** -22 * (1.1 * A + 0.7 * L) + 2.0 ** -21 + (n / 16 + 32) * 2.0 ** -23
        round_p, round_o, least = (2.0 ** -10, 2.0 ** -8, 2.0 ** -32) if half else (2.0 ** -22, 2.0 ** -24, 2.0 ** -44)
        of_token = scales[1][table[b, :-(-n // page)].long()].double().t().repeat_interleave(group, 0)
        of_token = of_token.repeat_interleave(page, 1)[:, None, :n].clamp(min=2.0 ** -64)
        floor = n * least * qmax * (p * of_token).amax(-1)
        tol[b, :, :c] = (2 * off + round_p)[..., None] * (p @ v.abs()) + floor[..., None] + round_o * o.abs()
        tol_lse[b, :, :c] = off + 2.0 ** -22 * A
    return out, lse, tol, tol_lse
