"""The key/value cache held in 8 bits: what is measured of it.

Three operators, over a paged cache. A page holds `page` tokens of every key/value head; its codes
are int8 or e4m3 numbers, with one fp32 scale for each page and head (K and V apart), and a code c
stands for c * scale. Row b of the page table lists the pages of sequence b in order; entries behind
the sequence's last page hold -1.

  write   new tokens of K and V are quantised at their places behind the sequence's older tokens.
          A page's scale is the largest magnitude of its new tokens / 127 (int8) or / 448 (e4m3);
          a page that already holds older tokens keeps its scale where that is larger, and where it
          grows the older codes are quantised again. The pass then reads back the pages it touched,
          which gives the stored values.
  read    a range of tokens as bf16 or fp32 values; places behind the range are zeros.
  attend  queries of the last tokens of each sequence attend to the cached tokens before them,
          all of them or a sliding window with global tokens; gives out and lse.

Lengths are made from the case alone, so that the work of a case is one number; values, page
numbers and scales are made from the seed.
"""
import math
import random

import torch

own = False

QMAX = {"i8": 127.0, "e4m3": 448.0}
CODE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
REAL = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's next token: a short call, where latency counts
        dict(name="decode-one", op="attend", B=1, H=12, Hk=12, m=1, n=4001, d=64, page=64, code="i8", real="bf16",
             window=-1, n_global=0, ragged=False),
        # a server's batch of conversations of many lengths, one token each, four query heads a K/V head
        dict(name="decode-batch", op="attend", B=48, H=16, Hk=4, m=1, n=8192, d=128, page=64, code="e4m3", real="bf16",
             window=-1, n_global=0, ragged=True),
        # two long documents, one token each
        dict(name="decode-long", op="attend", B=2, H=32, Hk=8, m=1, n=131071, d=128, page=128, code="i8", real="bf16",
             window=-1, n_global=0, ragged=False),
        # the sliding window with global tokens that the masks of this library have, token by token
        dict(name="decode-window", op="attend", B=32, H=16, Hk=16, m=1, n=16384, d=128, page=32, code="e4m3",
             real="bf16", window=1024, n_global=32, ragged=True),
        # five drafted tokens of each sequence checked at once, small pages
        dict(name="verify-five", op="attend", B=16, H=32, Hk=8, m=5, n=8192, d=128, page=16, code="i8", real="bf16",
             window=-1, n_global=0, ragged=True),
        # a chunk of a prompt behind what the cache holds already
        dict(name="prompt-chunk", op="attend", B=2, H=16, Hk=4, m=2048, n=8190, d=128, page=64, code="e4m3",
             real="bf16", window=-1, n_global=0, ragged=False),
        # fp32 queries
        dict(name="decode-f32", op="attend", B=8, H=16, Hk=16, m=1, n=8192, d=64, page=64, code="i8", real="f32",
             window=-1, n_global=0, ragged=True),
        # prompts written into an empty or partly filled cache
        dict(name="write-prompts", op="write", B=8, Hk=8, m=4096, at=500, d=128, page=64, code="e4m3", real="bf16",
             ragged=True),
        # the next token of each sequence of a large batch
        dict(name="write-tokens", op="write", B=256, Hk=8, m=1, at=4000, d=128, page=64, code="i8", real="bf16",
             ragged=True),
        # an odd chunk of fp32 tokens
        dict(name="write-odd-f32", op="write", B=3, Hk=12, m=517, at=77, d=64, page=32, code="i8", real="f32",
             ragged=True),
        # a cached prefix taken out for a pass that wants plain K and V
        dict(name="read-prefix", op="read", B=4, Hk=16, m=16384, at=0, d=128, page=128, code="e4m3", real="bf16",
             ragged=True),
        # a few tokens, odd sizes
        dict(name="read-few", op="read", B=3, Hk=4, m=77, at=130, d=32, page=16, code="i8", real="f32", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "write", "write", "read"])
    d, page = rng.choice([32, 64, 128, 128]), rng.choice([16, 32, 64, 128, 256])
    code, real = rng.choice(["i8", "e4m3"]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 4, 5, 8, 12, 16])
    B, ragged = _log(rng, 1, 64), rng.random() < 0.7
    if op != "attend":
        m = _log(rng, 1, max(1, min(16384, (1 << 22) // (B * Hk))))
        return dict(op=op, B=B, Hk=Hk, m=m, at=rng.choice([0, _log(rng, 1, 4000)]), d=d, page=page, code=code,
                    real=real, ragged=ragged)
    G = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    n = _log(rng, 1, max(64, min(131072, (1 << 21) // (B * Hk))))
    m = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1500)])
    m = max(1, min(m, n, (1 << 28) // (B * Hk * G * n)))
    window = rng.choice([-1, -1, _log(rng, 1, n)])
    return dict(op=op, B=B, H=Hk * G, Hk=Hk, m=m, n=n, d=d, page=page, code=code, real=real, window=window,
                n_global=rng.choice([0, 4, 33]) if window >= 0 else 0, ragged=ragged)


def _lengths(case):
    """Per sequence: attend: (tokens in the cache, queries); write, read: (place of the first token, tokens)."""
    r = random.Random("%(op)s %(B)d %(Hk)d %(m)d %(d)d %(page)d" % case)
    B, m, ragged = case["B"], case["m"], case["ragged"]
    if case["op"] == "attend":
        n = case["n"]
        tokens = [n] + [r.randint(max(1, n // 8), n) if ragged else n for _ in range(B - 1)]
        return tokens, [min(t, m) if b % 3 or not ragged else min(t, r.randint(1, m)) for b, t in enumerate(tokens)]
    start = [case["at"]] + [r.randint(0, case["at"]) if ragged else case["at"] for _ in range(B - 1)]
    return start, [m] + [r.randint(max(1, m // 4), m) if ragged else m for _ in range(B - 1)]


def _attended(case):
    """Per sequence: (query, token) pairs, and the tokens that any query attends to."""
    pairs, tokens = [], []
    for n, q in zip(*_lengths(case)):
        w, g = case["window"], case["n_global"]
        if w < 0:
            pairs.append(sum(range(n - q + 1, n + 1)))
            tokens.append(n)
        else:
            pairs.append(sum(min(p, w) + 1 + min(g, max(0, p - w)) for p in range(n - q, n)))
            first = max(0, n - q - w)
            tokens.append(n - first + min(g, first))
    return pairs, tokens


def work(case):
    d, Hk, B = case["d"], case["Hk"], case["B"]
    es = 2 if case["real"] == "bf16" else 4
    if case["op"] == "attend":
        pairs, tokens = _attended(case)
        rows = case["H"] * case["m"] * B
        pages = sum(-(-t // case["page"]) for t in tokens)
        return {"bytes": 2 * Hk * d * sum(tokens) + 8 * Hk * pages + 4 * pages + rows * (2 * d * es + 4),
                "flops": 4 * d * case["H"] * sum(pairs)}
    start, count = _lengths(case)
    values = 2 * Hk * d * sum(count)  # K and V
    scales = 8 * Hk * sum((s + c - 1) // case["page"] - s // case["page"] + 1 for s, c in zip(start, count))
    if case["op"] == "read":
        return {"bytes": values + scales + 2 * Hk * d * B * case["m"] * es, "flops": values}
    older = 2 * Hk * d * sum(s % case["page"] for s in start)
    back = 2 * Hk * d * B * (case["m"] + case["page"] - 1) * es
    # written: values in, codes out, the older codes of a first page in and out; read back: codes in, values out
    return {"bytes": values * (es + 1) + older * 2 + scales + (values + older) + back, "flops": 2 * values}


def _cache(case, g, spans):
    """A pool of pages with the tokens that each sequence holds, and pages of nobody between them."""
    page, d, Hk, code = case["page"], case["d"], case["Hk"], case["code"]
    need = [-(-t // page) for t in spans]
    used, width = sum(need), max(need) + 1
    pool = used + max(2, used // 16)
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)[:used]
    slots = torch.arange(width, device="cuda")[None, :]
    count = torch.tensor(need, device="cuda")[:, None]
    table = torch.full((len(spans), width), -1, dtype=torch.int32, device="cuda")
    table[slots < count] = order
    shape = (pool, Hk, page, d)

    def codes():
        x = torch.randn(shape, generator=g, device="cuda")
        if code == "i8":
            return (x * 36).round_().clamp_(-127, 127).to(torch.int8)
        return (x * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales():
        return (torch.rand((pool, Hk), generator=g, device="cuda") + 0.5) * (3.5 / QMAX[code])

    return dict(k=codes(), v=codes(), k_scale=scales(), v_scale=scales(), table=table)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    real, page = REAL[case["real"]], case["page"]
    a, b = _lengths(case)
    if case["op"] == "attend":
        state = _cache(case, g, a)
        q = torch.randn((case["B"], case["H"], case["m"], case["d"]), generator=g, device="cuda")
        state.update(q=q.to(real), seqlen=_ints(a), qlen=_ints(b))
    else:
        state = _cache(case, g, [s + c for s, c in zip(a, b)])
        state.update(start=_ints(a), length=_ints(b))
        if case["op"] == "write":
            shape = (case["B"], case["Hk"], case["m"], case["d"])
            state["new"] = [torch.randn(shape, generator=g, device="cuda").to(real) for _ in range(2)]
            # the touched pages from their first token on
            state["back_start"] = _ints([s // page * page for s in a])
            state["back_length"] = _ints([s % page + c for s, c in zip(a, b)])
    state["case"] = case
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import sparse_mask_scaled_b200 as sp
    case = state["case"]
    if "cache" not in state:  # the handle that a user's program keeps
        state["cache"] = sp.Cache(state["k"], state["v"], state["k_scale"], state["v_scale"], state["table"])
    cache, real = state["cache"], REAL[case["real"]]
    if case["op"] == "attend":
        out, lse = sp.spattn_fwd_cache(state["q"], cache, state["seqlen"], qlen=state["qlen"],
                                       window=case["window"], n_global=case["n_global"])
        return {"out": out, "lse": lse.view(out.shape[:3])}
    if case["op"] == "read":
        k, v = sp.spattn_cache_read(cache, case["m"], dtype=real, start=state["start"], length=state["length"])
        return {"k": k, "v": v}
    sp.spattn_cache_write(state["new"][0], state["new"][1], cache, state["start"], length=state["length"])
    k, v = sp.spattn_cache_read(cache, case["m"] + case["page"] - 1, dtype=real, start=state["back_start"],
                                length=state["back_length"])
    return {"k": k, "v": v, "k_scale": state["k_scale"], "v_scale": state["v_scale"]}


# ------------------------------------------------------------------ plain forms
def _run_plain(state):
    case = state["case"]
    if case["op"] == "attend":
        return _plain_attend(state, case)
    if case["op"] == "read":
        return {s: _plain_read(state, case, s, case["m"], state["start"], state["length"]) for s in ("k", "v")}
    _plain_write(state, case, "k", state["new"][0])
    _plain_write(state, case, "v", state["new"][1])
    m = case["m"] + case["page"] - 1
    back = {s: _plain_read(state, case, s, m, state["back_start"], state["back_length"]) for s in ("k", "v")}
    return {**back, "k_scale": state["k_scale"], "v_scale": state["v_scale"]}


def _plain_attend(state, case):
    B, H, Hk, m, d, page = (case[x] for x in ("B", "H", "Hk", "m", "d", "page"))
    table = state["table"].long().clamp(min=0)  # places behind a sequence are masked below
    N = table.shape[1] * page

    def values(s):
        x = state[s].view(torch.int8)[table].view(state[s].dtype).float() * state[s + "_scale"][table][..., None, None]  # [B, pages, Hk, page, d]
        return x.transpose(1, 2).reshape(B, Hk, N, d)

    seqlen, qlen = state["seqlen"].long(), state["qlen"].long()
    t, j = torch.arange(m, device="cuda"), torch.arange(N, device="cuda")
    pos = (seqlen - qlen)[:, None] + t  # [B, m]
    sees = (j <= pos[..., None]) & (t < qlen[:, None])[..., None]
    if case["window"] >= 0:
        sees &= (j >= pos[..., None] - case["window"]) | (j < case["n_global"])
    sees = sees[:, None, None]  # [B, 1, 1, m, N]
    q = state["q"].float().reshape(B, Hk, (H // Hk) * m, d)
    s = (q @ values("k").transpose(2, 3)).reshape(B, Hk, H // Hk, m, N) / math.sqrt(d)
    s = s.masked_fill(~sees, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    v = values("v").masked_fill((j >= seqlen[:, None])[:, None, :, None], 0.0)  # what lies behind a sequence is not read
    out = (p.reshape(B, Hk, (H // Hk) * m, N) @ v).reshape(B, Hk, H // Hk, m, d)
    out = out / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top)[..., 0]
    return {"out": out.reshape(B, H, m, d).to(state["q"].dtype), "lse": lse.reshape(B, H, m)}


def _plain_read(state, case, s, m, start, length):
    page = case["page"]
    t = torch.arange(m, device="cuda")
    at = start.long()[:, None] + t  # [B, m]
    there = t < length[:, None]
    at = torch.where(there, at, 0)
    pages = state["table"].long().gather(1, at // page).clamp(min=0)
    x = state[s].view(torch.int8)[pages, :, at % page].view(state[s].dtype).float()  # [B, m, Hk, d]
    x = x * state[s + "_scale"][pages][..., None]
    return x.masked_fill(~there[..., None, None], 0.0).transpose(1, 2).contiguous().to(REAL[case["real"]])


def _plain_write(state, case, s, new):
    page, m, qmax = case["page"], case["m"], QMAX[case["code"]]
    start, length = state["start"].long(), state["length"].long()
    slots = (m + page - 2) // page + 1
    slot = (start // page)[:, None] + torch.arange(slots, device="cuda")
    at = slot[..., None] * page + torch.arange(page, device="cuda")  # [B, slots, page]
    t = at - start[:, None, None]
    is_new = (t >= 0) & (t < length[:, None, None])
    is_old = t < 0
    touched = is_new.any(-1)
    pages = state["table"].long().gather(1, slot.clamp(max=state["table"].shape[1] - 1)).clamp(min=0)
    B, Hk, _, d = new.shape
    x = new.float().gather(2, t.clamp(0, m - 1).reshape(B, 1, -1, 1).expand(B, Hk, -1, d))
    x = x.reshape(B, Hk, slots, page, d).transpose(1, 2)  # [B, slots, Hk, page, d]
    x = x.masked_fill(~is_new[:, :, None, :, None], 0.0)
    scale = x.abs().amax((-1, -2))
    scale = scale / torch.full_like(scale, qmax)  # [B, slots, Hk]; a divisor that is a number would become a product
    before = torch.where(is_old.any(-1)[..., None], state[s + "_scale"][pages], 0.0)
    grown = scale > before
    scale = torch.maximum(scale, before)
    codes = state[s].view(torch.int8)[pages].view(state[s].dtype)
    x = torch.where(is_old[:, :, None, :, None], codes.float() * before[..., None, None], x)
    x = x / torch.where(scale > 0, scale, 1.0)[..., None, None]
    if case["code"] == "i8":
        made = x.round().clamp(-127, 127).to(torch.int8)
    else:
        made = x.clamp(-448, 448).to(torch.float8_e4m3fn)
    put = is_new[:, :, None, :] | (is_old[:, :, None, :] & grown[..., None])  # [B, slots, Hk, page]
    made = torch.where(put[..., None], made.view(torch.int8), codes.view(torch.int8))
    state[s].view(torch.int8)[pages[touched]] = made[touched]
    state[s + "_scale"][pages[touched]] = scale[touched]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(state, case)
    a, b = _lengths(case)
    if case["op"] == "write":
        if sum(y // case["page"] + 2 for y in b) > 12000:
            return None  # page by page this takes too long
        for s, new in zip(("k", "v"), state["new"]):
            _exact_write(state, case, s, new)
        m, a, b = case["m"] + case["page"] - 1, state["back_start"].tolist(), state["back_length"].tolist()
    else:
        m = case["m"]
    got = {}
    for s in ("k", "v"):
        got[s] = torch.zeros((case["B"], case["Hk"], m, case["d"]), dtype=torch.float64, device="cuda")
        for i in range(case["B"]):
            got[s][i, :, :b[i]] = _exact_tokens(state, case, s, i, a[i] + b[i])[:, a[i]:]
    if case["op"] == "write":
        got.update(k_scale=state["k_scale"].double(), v_scale=state["v_scale"].double())
    return got


def _exact_tokens(state, case, s, i, n):
    """The first n tokens of sequence i: [Hk, n, d]."""
    own_pages = state["table"][i, :-(-n // case["page"])].long()
    x = state[s].view(torch.int8)[own_pages].view(state[s].dtype).double()
    x = x * state[s + "_scale"][own_pages].double()[:, :, None, None]
    return x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n]


def _exact_attend(state, case):
    H, Hk, m, d = case["H"], case["Hk"], case["m"], case["d"]
    G = H // Hk
    out = torch.zeros((case["B"], H, m, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], H, m), -math.inf, dtype=torch.float64, device="cuda")
    for i, (n, c) in enumerate(zip(*_lengths(case))):
        k, v = (_exact_tokens(state, case, s, i, n) for s in ("k", "v"))
        place = torch.arange(n - c, n, device="cuda")[:, None]
        token = torch.arange(n, device="cuda")[None, :]
        hidden = token > place
        if case["window"] >= 0:
            hidden = hidden | ((place - token > case["window"]) & (token >= case["n_global"]))
        for h in range(H):
            s = state["q"][i, h, :c].double() @ k[h // G].T / math.sqrt(d)
            s[hidden] = -math.inf
            lse[i, h, :c] = torch.logsumexp(s, 1)
            out[i, h, :c] = torch.softmax(s, 1) @ v[h // G]
    return {"out": out, "lse": lse}


def _exact_write(state, case, s, new):
    """The scale is kept in 32 bits, and so are a code's quotient and an older code's value: each is worked out in 64 bits
    and rounded to 32 where the definition says so."""
    page, qmax = case["page"], QMAX[case["code"]]
    codes, scales = state[s].view(torch.int8), state[s + "_scale"]
    for i, (first, c) in enumerate(zip(*_lengths(case))):
        for p in range(first // page, (first + c - 1) // page + 1):
            at = int(state["table"][i, p])
            lo, hi = max(first, p * page), min(first + c, (p + 1) * page)
            x = new[i, :, lo - first:hi - first].double()
            scale = x.abs().amax((1, 2))
            scale = (scale / torch.full_like(scale, qmax)).float()
            older = lo - p * page
            if older:
                before = scales[at].clone()
                scale = torch.maximum(scale, before)
                was = (codes[at, :, :older].view(state[s].dtype).double() * before.double()[:, None, None]).float().double()
                redo = scale > before
                codes[at, redo, :older] = _exact_codes(was, scale, case)[redo]
            codes[at, :, older:older + hi - lo] = _exact_codes(x, scale, case)
            scales[at] = scale


def _exact_codes(x, scale, case):
    q = (x / torch.where(scale > 0, scale, 1.0).double()[:, None, None]).float()
    if case["code"] == "i8":
        return torch.round(q).clamp(-127, 127).to(torch.int8)
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.int8)
