"""The paged 8-bit KV cache: what is measured.

Four operators of one serving step, in the order a program calls them:
  plan     block tables, slot maps and positions from the requests' lengths (csa2_paged_plan)
  release  the pages of finished requests back on the free list (csa2_paged_release)
  append   new keys and values into E4M3 pages with one scale per page and head (csa2_kv8_append)
  attn     attention over those pages, ragged, causal (csa2_kv8_attn)
Lengths follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
LN2 = math.log(2.0)


def listed():
    return [
        # every request of a decode batch takes one token: the per-step bookkeeping
        dict(name="plan_decode", op="plan", R=256, page=64, lo=1, hi=8192, q=1, mix=0),
        # decode tokens and prefill chunks in one ragged batch, small pages, long contexts
        dict(name="plan_mixed", op="plan", R=48, page=16, lo=0, hi=131072, q=1024, mix=1),
        # a few requests of a batch ended
        dict(name="release_few", op="release", R=61, page=128, lo=1, hi=16384, every=8),
        # a large batch drained: a quarter of its requests ended, small pages
        dict(name="release_many", op="release", R=1024, page=16, lo=1, hi=32768, every=4),
        # one new token per sequence of a decode batch
        dict(name="append_decode", op="append", R=32, Hk=8, hd=128, page=64, dtype="bf16", lo=1, hi=2048, q=1, mix=0,
             fused=0),
        # drafted tokens of a verify step, starting anywhere in a page
        dict(name="append_verify", op="append", R=8, Hk=4, hd=128, page=128, dtype="fp16", lo=1, hi=1999, q=64, mix=0,
             fused=0),
        # prefill chunks, keys and values as views of one fused projection
        dict(name="append_prefill", op="append", R=9, Hk=8, hd=128, page=16, dtype="bf16", lo=0, hi=1024, q=2048, mix=1,
             fused=1),
        # one token of one short sequence: latency
        dict(name="attn_tiny", op="attn", R=1, Hq=16, Hk=2, hd=128, page=64, dtype="bf16", lo=4096, hi=4096, q=1, mix=0,
             window=0, cap=0.0),
        # a ragged decode batch, five query heads per key head, a window and capped scores
        dict(name="attn_ragged", op="attn", R=61, Hq=40, Hk=8, hd=64, page=16, dtype="fp16", lo=1, hi=8191, q=1, mix=0,
             window=1024, cap=30.0),
        # a long-context decode batch: 32 sequences of 64K to 128K tokens
        dict(name="attn_decode", op="attn", R=32, Hq=64, Hk=4, hd=128, page=64, dtype="bf16", lo=65536, hi=131072, q=1,
             mix=0, window=0, cap=0.0),
        # 64 drafted tokens per sequence checked at once
        dict(name="attn_verify", op="attn", R=8, Hq=64, Hk=8, hd=128, page=64, dtype="bf16", lo=8192, hi=32768, q=64,
             mix=0, window=0, cap=0.0),
        # prefill chunks of 1024 tokens next to single tokens
        dict(name="attn_chunk", op="attn", R=3, Hq=32, Hk=4, hd=128, page=128, dtype="bf16", lo=2000, hi=32768, q=1024,
             mix=1, window=0, cap=0.0),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["plan", "release", "append", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        R = _log(rng, 1, 1024)
        mix = rng.randrange(2)
        return dict(op=op, R=R, page=page, lo=0 if mix else 1, hi=_log(rng, 64, 65536 if R <= 128 else 8192),
                    q=_log(rng, 2, max(2, 24000 // R)) if mix else 1, mix=mix)
    if op == "release":
        R = _log(rng, 1, 1024)
        return dict(op=op, R=R, page=page, lo=1, hi=_log(rng, 64, 32768), every=rng.randrange(1, 9))
    hd = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    mix = rng.randrange(2)
    if op == "append":
        R = _log(rng, 1, 256)
        return dict(op=op, R=R, Hk=_log(rng, 1, 12), hd=hd, page=page, dtype=dtype, lo=0, hi=_log(rng, 64, 2048),
                    q=_log(rng, 2, max(2, min(2048, 12000 // R))) if mix else 1, mix=mix, fused=rng.randrange(2))
    Hk = _log(rng, 1, 8)
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if rng.random() < 0.5:  # single tokens
        R, q, mix = _log(rng, 1, 128), 1, 0
        hi = _log(rng, 16, min(131072, max(16, (1 << 29) // (R * Hk * hd))))
    else:  # drafts and chunks
        R = _log(rng, 1, 16)
        q = _log(rng, 2, max(2, min(1024, 4096 // R)))
        hi = _log(rng, 64, max(64, min(32768, (1 << 30) // (R * q * Hk * G))))
        q = min(q, hi)
    return dict(op=op, R=R, Hq=Hk * G, Hk=Hk, hd=hd, page=page, dtype=dtype, lo=min(hi, max(1, q)), hi=hi, q=q, mix=mix,
                window=rng.choice([0, 0, 0, 1, 100, 128, 1000]), cap=rng.choice([0.0, 0.0, 20.0, 50.0]))


def _lengths(case):
    """(length before the step, new tokens) of each request. For attn, lo..hi holds the length with
    the new tokens; with mix, one request in three brings a whole chunk, the others one token or a
    part of a chunk."""
    g = random.Random("lengths-%s-%d-%d-%d" % (case["op"], case["R"], case["lo"], case["hi"]))
    out = []
    for r in range(case["R"]):
        n = case["hi"] if r == 0 else g.randint(case["lo"], case["hi"])
        q = case.get("q", 0)
        if q > 1 and case.get("mix"):
            q = (q, 1, g.randint(1, q))[r % 3]
        if case["op"] == "attn":
            q = min(q, n)
            out.append((n - q, q))
        else:
            out.append((n, q))
    return out


def _pages(n, page):
    return -(-n // page)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _tables(case, lens, gen):
    """Block table over all pages that hold tokens before the step, and the pages left, shuffled."""
    page, R = case["page"], case["R"]
    have = [_pages(c, page) for c, _ in lens]
    want = [_pages(c + n, page) for c, n in lens]
    cols = max(1, max(want))
    total = max(1, sum(want)) + 7
    ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    h = _ints(have, torch.int64)
    first = torch.cumsum(h, 0) - h
    j = torch.arange(cols, device=DEV)
    at = (first[:, None] + j).clamp(max=total - 1)
    table = torch.where(j < h[:, None], ids[at], torch.full_like(ids[at], -1))
    left = ids[int(sum(have)):].contiguous()
    return table.contiguous(), left, total


def _slots(lens, table, page):
    """Slot map, query starts and lengths of a batch whose pages are all in the table."""
    c = _ints([a for a, _ in lens], torch.int64)
    n = _ints([b for _, b in lens], torch.int64)
    T = sum(b for _, b in lens)
    q_start = torch.zeros(len(lens) + 1, dtype=torch.int64, device=DEV)
    q_start[1:] = torch.cumsum(n, 0)
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(q_start, t, right=True) - 1
    pos = c[r] + t - q_start[r]
    slot = table[r, pos // page].to(torch.int64) * page + pos % page
    return slot.contiguous(), q_start.to(torch.int32), (c + n).to(torch.int32)


def _codes(shape, gen, spread):
    """E4M3 codes of normal values, their scale a power of two that differs by page and head."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=torch.uint8, device=DEV)
    step = 1 << 27
    for a in range(0, n, step):
        b = min(n, a + step)
        x = torch.randn(b - a, generator=gen, device=DEV, dtype=torch.float32).mul_(64.0).clamp_(-448.0, 448.0)
        out[a:b] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(-1, spread, shape[:2], generator=gen, device=DEV).float() - 6.0
    return out.view(shape), torch.exp2(e).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    lens = _lengths(case)
    page, R = case["page"], case["R"]
    s = dict(case)
    if case["op"] == "plan":
        table, left, total = _tables(case, lens, gen)
        T = sum(n for _, n in lens)
        s.update(ctx=_ints([c for c, _ in lens]), new=_ints([n for _, n in lens]), table=table, free=left,
                 n_free=_ints([left.numel()]), n_pages=total, T=T + 5,
                 seq_len=torch.zeros(R, dtype=torch.int32, device=DEV), n_free_out=_ints([0]),
                 q_start=torch.zeros(R + 1, dtype=torch.int32, device=DEV),
                 slot=torch.zeros(T + 5, dtype=torch.int64, device=DEV),
                 pos=torch.zeros(T + 5, dtype=torch.int64, device=DEV))
        return s
    if case["op"] == "release":
        table, left, total = _tables(case, [(c, 0) for c, _ in lens], gen)
        free = torch.zeros(total, dtype=torch.int32, device=DEV)
        free[:left.numel()] = left
        s.update(seq=_ints([c for c, _ in lens]), table=table, free=free, n_free=_ints([left.numel()]), n_pages=total,
                 release=_ints([int(r % case["every"] == 0) for r in range(R)], torch.uint8),
                 seq_len=torch.zeros(R, dtype=torch.int32, device=DEV), n_free_out=_ints([0]))
        return s
    Hk, hd = case["Hk"], case["hd"]
    full = [(c + n, 0) for c, n in lens]
    table, _, total = _tables(case, full, gen)
    slot, q_start, seq_len = _slots(lens, table, page)
    T = slot.numel()
    shape = (total, Hk, page, hd)
    kc, ks = _codes(shape, gen, 2)
    vc, vs = _codes(shape, gen, 2)
    s.update(table=table, slot=slot, q_start=q_start, seq_len=seq_len, kc=kc, ks=ks, vc=vc, vs=vs)
    if case["op"] == "append":
        if case["fused"]:  # [T][q heads | k heads | v heads][hd], as one projection writes them
            x = torch.randn(T, 4 * Hk, hd, generator=gen, device=DEV, dtype=torch.float32).to(_dtype(case))
            s.update(k=x[:, 2 * Hk:3 * Hk], v=x[:, 3 * Hk:])
        else:
            s.update(k=torch.randn(T, Hk, hd, generator=gen, device=DEV).to(_dtype(case)),
                     v=torch.randn(T, Hk, hd, generator=gen, device=DEV).to(_dtype(case)))
        return s
    # what lies behind a sequence's last token in its last page was never written: any bits
    last = table.gather(1, ((seq_len.to(torch.int64) - 1) // page)[:, None])[:, 0].to(torch.int64)
    behind = torch.arange(page, device=DEV) > ((seq_len.to(torch.int64) - 1) % page)[:, None]
    for cache in (kc, vc):
        rows = cache[last]
        cache[last] = torch.where(behind[:, None, :, None], torch.full_like(rows, 0x7F), rows)
    Hq = case["Hq"]
    s.update(q_in=torch.randn(T, Hq, hd, generator=gen, device=DEV).to(_dtype(case)),
             out=torch.zeros(T, Hq, hd, dtype=_dtype(case), device=DEV),
             lse=torch.zeros(T, Hq, dtype=torch.float32, device=DEV), scale=1.0 / math.sqrt(hd), T=T)
    return s


# ---- the plain forms ------------------------------------------------------------------------


def _plan(s):
    page, table, R = s["page"], s["table"], s["R"]
    c, n = s["ctx"].to(torch.int64), s["new"].to(torch.int64)
    have, want = (c + page - 1) // page, (c + n + page - 1) // page
    need = want - have
    off = torch.cumsum(need, 0) - need
    n_free = s["n_free"].to(torch.int64)
    j = torch.arange(table.shape[1], device=DEV)
    new = (j >= have[:, None]) & (j < want[:, None])
    at = (n_free - 1 - (off[:, None] + j - have[:, None])).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(new, s["free"][at], table))
    q_start = torch.zeros(R + 1, dtype=torch.int64, device=DEV)
    q_start[1:] = torch.cumsum(n, 0)
    t = torch.arange(s["T"], device=DEV)
    r = (torch.searchsorted(q_start, t, right=True) - 1).clamp(max=R - 1)
    used = t < q_start[R]
    pos = torch.where(used, c[r] + t - q_start[r], torch.zeros_like(t))
    slot = table[r, pos // page].to(torch.int64) * page + pos % page
    none = torch.full_like(t, -1)
    return dict(table=table, seq_len=(c + n).to(torch.int32), n_free=(n_free - need.sum()).to(torch.int32),
                q_start=q_start.to(torch.int32), slot=torch.where(used, slot, none), pos=torch.where(used, pos, none))


def _release(s):
    page, table = s["page"], s["table"]
    n, gone = s["seq"].to(torch.int64), s["release"] != 0
    j = torch.arange(table.shape[1], device=DEV)
    mine = ((j < ((n + page - 1) // page)[:, None]) & gone[:, None]).reshape(-1)
    n_free = s["n_free"].to(torch.int64)
    rank = torch.cumsum(mine.to(torch.int64), 0) - 1
    cap = s["free"].numel()
    wide = torch.cat([s["free"], s["free"][:1]])  # one more place, for what is not pushed
    at = torch.where(mine, n_free + rank, torch.full_like(rank, cap))
    wide[at] = table.reshape(-1)
    s["free"].copy_(wide[:cap])
    return dict(free=s["free"], n_free=(n_free + mine.sum()).to(torch.int32),
                seq_len=torch.where(gone, torch.zeros_like(s["seq"]), s["seq"]))


def _append_one(s, x, cache, scale):
    page, (P, Hk) = s["page"], scale.shape
    x = x.float()
    pid, row = s["slot"] // page, s["slot"] % page
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, and 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    want = torch.where(amax > 0, torch.exp2(e.clamp(-64, 127).float()), torch.full_like(amax, 2.0 ** -64))
    top = torch.zeros(P, Hk, device=DEV).scatter_reduce(0, pid[:, None].expand(-1, Hk), want, "amax")
    first = torch.full((P,), page, dtype=torch.int64, device=DEV).scatter_reduce(0, pid, row, "amin")
    new = torch.where((first > 0)[:, None], torch.maximum(scale, top), top)
    lead = s["q_start"][:-1].to(torch.int64)  # the token that may enter a page with earlier rows
    lp, lr = pid[lead], row[lead]
    old = cache[lp].view(torch.float8_e4m3fn).float() * (scale[lp] / new[lp])[:, :, None, None]
    keep = torch.arange(page, device=DEV) < lr[:, None]
    cache[lp] = torch.where(keep[:, None, :, None], old.to(torch.float8_e4m3fn).view(torch.uint8), cache[lp])
    cache[pid, :, row] = (x / new[pid][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(torch.where((first < page)[:, None], new, scale))


def _append(s):
    _append_one(s, s["k"], s["kc"], s["ks"])
    _append_one(s, s["v"], s["vc"], s["vs"])
    return _cache(s)


def _cache(s):
    return dict(kc=s["kc"].view(torch.float8_e4m3fn), ks=s["ks"], vc=s["vc"].view(torch.float8_e4m3fn), vs=s["vs"])


def _values(cache, scale, ids):
    """[R][Hk][L][hd] of the pages in `ids` [R][pages], times their scales."""
    x = cache[ids].view(torch.float8_e4m3fn).float() * scale[ids][..., None, None]
    R, n, Hk, page, hd = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(R, Hk, n * page, hd)


def _attn(s):
    R, Hq, Hk, hd, Q = s["R"], s["Hq"], s["Hk"], s["hd"], s["q"]
    G, T = Hq // Hk, s["T"]
    start, n_key = s["q_start"].to(torch.int64), s["seq_len"].to(torch.int64)
    n_q = start[1:] - start[:-1]
    ids = s["table"].clamp(min=0).to(torch.int64)
    i = torch.arange(Q, device=DEV)
    at = (start[:-1, None] + i).clamp(max=T - 1)
    q = s["q_in"][at].float().view(R, Q, Hk, G, hd).permute(0, 2, 1, 3, 4).reshape(R, Hk, Q * G, hd)
    k = _values(s["kc"], s["ks"], ids)
    L = k.shape[2]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(R, Hk, Q, G, L)
    del k
    if s["cap"]:
        x = torch.tanh(x / s["cap"]).mul_(s["cap"])
    j = torch.arange(L, device=DEV)
    p = (n_key - n_q)[:, None] + i  # position of each query
    sees = j <= p[..., None]
    if s["window"]:
        sees &= j > p[..., None] - s["window"]
    x.masked_fill_(~sees[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]
    v = _values(s["vc"], s["vs"], ids).masked_fill_((j >= n_key[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x.view(R, Hk, Q * G, L), v).view(R, Hk, Q, G, hd) / total
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(start, t, right=True) - 1
    i = t - start[r]
    o = o.permute(0, 2, 1, 3, 4)[r, i].reshape(T, Hq, hd)
    return dict(out=o.to(s["q_in"].dtype), lse=lse.permute(0, 2, 1, 3)[r, i].reshape(T, Hq))


def run(s):
    if not own:
        return {"plan": _plan, "release": _release, "append": _append, "attn": _attn}[s["op"]](s)
    from sparse_attention_fp4_pack_b200 import csa2
    if s["op"] == "plan":
        csa2.csa2_paged_plan(s["ctx"], s["new"], s["table"], s["free"], s["n_free"], s["page"], s["n_pages"], s["seq_len"],
                             s["n_free_out"], s["q_start"], s["slot"], s["pos"])
        return dict(table=s["table"], seq_len=s["seq_len"], n_free=s["n_free_out"], q_start=s["q_start"], slot=s["slot"],
                    pos=s["pos"])
    if s["op"] == "release":
        csa2.csa2_paged_release(s["seq"], s["table"], s["release"], s["free"], s["n_free"], s["page"], s["n_pages"],
                                s["seq_len"], s["n_free_out"])
        return dict(free=s["free"], n_free=s["n_free_out"], seq_len=s["seq_len"])
    if s["op"] == "append":
        csa2.csa2_kv8_append(s["k"], s["v"], s["slot"], s["kc"], s["vc"], s["ks"], s["vs"])
        return _cache(s)
    csa2.csa2_kv8_attn(s["q_in"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["q_start"], s["seq_len"], s["scale"],
                       s["out"], s["lse"], max_q=s["q"], window=s["window"], softcap=s["cap"])
    return dict(out=s["out"], lse=s["lse"])


# ---- what a pass cannot do without ----------------------------------------------------------


def _pairs(c, n, window):
    """Query-key pairs of n queries behind c keys."""
    if not window:
        return n * c + n * (n + 1) // 2
    short = max(0, min(n, window - c))  # queries that see fewer keys than the window
    return short * c + short * (short + 1) // 2 + (n - short) * window


def work(case):
    lens = _lengths(case)
    page, R = case["page"], case["R"]
    if case["op"] == "plan":
        T = sum(n for _, n in lens)
        new = sum(_pages(c + n, page) - _pages(c, page) for c, n in lens)
        return dict(bytes=8 * R + 4 * new + 4 * R + 4 + 4 * (2 * R + 1) + 4 + 16 * (T + 5) + 4 * new, flops=T + R)
    if case["op"] == "release":
        n = sum(_pages(c, page) for r, (c, _) in enumerate(lens) if r % case["every"] == 0)
        return dict(bytes=8 * n + 9 * R + 8, flops=n + R)
    Hk, hd = case["Hk"], case["hd"]
    T = sum(n for _, n in lens)
    if case["op"] == "append":
        touched = sum(_pages(c + n, page) - c // page for c, n in lens)
        return dict(bytes=2 * T * Hk * hd * 3 + 2 * 4 * touched * Hk * 2 + 8 * T, flops=4 * T * Hk * hd)
    Hq, w = case["Hq"], case["window"]
    keys = sum(c + n - (max(0, c + 1 - w) if w else 0) for c, n in lens)
    pages = sum(_pages(c + n, page) - ((max(0, c + 1 - w) if w else 0) // page) for c, n in lens)
    pairs = sum(_pairs(c, n, w) for c, n in lens)
    return dict(bytes=2 * keys * Hk * hd + pages * (4 + 8 * Hk) + 4 * T * Hq * hd + 4 * T * Hq + 8 * R,
                flops=4 * pairs * Hq * hd)


# ---- the definitions in 64 bits -------------------------------------------------------------


def _e4m3_nearest(y):
    """The E4M3 value nearest to y (ties to even), |y| <= 448, by its spacing in each binade."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(y / step) * step


def _decode(codes):
    b = codes.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
    return torch.where(b >= 128, -v, v)


def _exact_append(s, x, cache, scale):
    page = s["page"]
    values, scale = _decode(cache), scale.double()
    slots, starts = s["slot"].tolist(), s["q_start"].tolist()
    x = x.double()
    for a, b in zip(starts[:-1], starts[1:]):
        t = a
        while t < b:
            p, row = slots[t] // page, slots[t] % page
            n = min(page - row, b - t)
            chunk = x[t:t + n].permute(1, 0, 2)  # [Hk][n][hd]
            need = chunk.abs().amax((1, 2)) / E4M3_MAX
            new = torch.exp2(torch.ceil(torch.log2(need.clamp(min=2.0 ** -64))))
            new = torch.where(new < need, new * 2, torch.where(new / 2 >= need.clamp(min=2.0 ** -64), new / 2, new))
            if row:
                new = torch.maximum(new, scale[p])
                values[p, :, :row] = _e4m3_nearest(values[p, :, :row] * (scale[p] / new)[:, None, None])
            scale[p] = new
            values[p, :, row:row + n] = _e4m3_nearest(chunk / new[:, None, None])
            t += n
    return values, scale


def _exact_attn(s):
    Hq, Hk, hd, page, w = s["Hq"], s["Hk"], s["hd"], s["page"], s["window"]
    out = torch.zeros(s["T"], Hq, hd, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], Hq, dtype=torch.float64, device=DEV)
    starts, lens = s["q_start"].tolist(), s["seq_len"].tolist()
    for r, n in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        ids = s["table"][r, :_pages(n, page)].to(torch.int64)
        pos = torch.arange(n - (b - a), n, device=DEV)
        low = max(0, n - (b - a) + 1 - w) if w else 0
        for h in range(Hk):
            k = (_decode(s["kc"][ids, h]) * s["ks"][ids, h].double()[:, None, None]).reshape(-1, hd)[low:n]
            v = (_decode(s["vc"][ids, h]) * s["vs"][ids, h].double()[:, None, None]).reshape(-1, hd)[low:n]
            q = s["q_in"][a:b].double().view(b - a, Hk, Hq // Hk, hd)[:, h]
            x = (q @ k.T) * s["scale"]  # [queries][heads][keys]
            if s["cap"]:
                x = s["cap"] * torch.tanh(x / s["cap"])
            gap = pos[:, None] - torch.arange(low, n, device=DEV)
            hidden = (gap < 0) | (gap >= w) if w else gap < 0
            x = x.masked_fill(hidden[:, None], -math.inf)
            out.view(s["T"], Hk, Hq // Hk, hd)[a:b, h] = torch.softmax(x, -1) @ v
            lse.view(s["T"], Hk, Hq // Hk)[a:b, h] = torch.logsumexp(x, -1)
    return dict(out=out, lse=lse)


def exact(case, seed):
    if case["op"] in ("plan", "release"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    if sum(_pages(c + n, case["page"]) - c // case["page"] for c, n in _lengths(case)) > 4000:
        return None
    kc, ks = _exact_append(s, s["k"], s["kc"], s["ks"])
    vc, vs = _exact_append(s, s["v"], s["vc"], s["vs"])
    return dict(kc=kc, ks=ks, vc=vc, vs=vs)
