"""Plain implementations of the paged 8-bit KV cache calls (64 bits, one request or page at a
time), and the inputs their tests share.  They follow include/csa2.h, not the kernels."""
import math

import numpy as np
import torch

E4M3 = torch.tensor([i for i in range(256)], dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)


def plan(ctx, new, table, free, n_free, page, n_pages, t_cap):
    """Sequential definition of csa2_paged_plan on Python lists; returns its outputs and whether
    (bad index, bad count, out of pages) was met."""
    R, max_pages = table.shape
    table = table.copy()
    flags = [False, False, False]
    if n_free < 0 or n_free > len(free):
        flags[1] = True
        n_free = min(max(n_free, 0), len(free))
    seq, q_start, slot, pos = [], [0], [], []
    used = 0
    for r in range(R):
        c, n = int(ctx[r]), int(new[r])
        if c < 0 or n < 0:
            flags[1] = True
            c, n = max(c, 0), max(n, 0)
        if len(slot) + n > t_cap:
            flags[1] = True
            n = t_cap - len(slot)
        if math.ceil((c + n) / page) > max_pages:
            flags[1] = True
        for j in range(min(math.ceil(c / page), max_pages), min(math.ceil((c + n) / page), max_pages)):
            table[r, j] = -1
            if used < n_free:
                table[r, j] = free[n_free - 1 - used]
                if not 0 <= table[r, j] < n_pages:
                    flags[0] = True
                    table[r, j] = -1
            else:
                flags[2] = True
            used += 1
        for i in range(n):
            p = c + i
            id = table[r, p // page] if p // page < max_pages else -1
            if not 0 <= id < n_pages:
                if p // page < min(math.ceil(c / page), max_pages):
                    flags[0] = True
                id = -1
            slot.append(-1 if id < 0 else int(id) * page + p % page)
            pos.append(p)
        seq.append(c + n)
        q_start.append(len(slot))
    tail = [-1] * (t_cap - len(slot))
    return dict(table=table, seq_len=np.array(seq, np.int32), n_free=max(0, n_free - used),
                q_start=np.array(q_start, np.int32), slot=np.array(slot + tail, np.int64),
                pos=np.array(pos + tail, np.int64)), flags


def release(seq, table, gone, free, n_free, page, n_pages):
    free, out = free.copy(), seq.copy()
    flags = [False, False]
    if n_free < 0 or n_free > len(free):
        flags[1] = True
        n_free = min(max(n_free, 0), len(free))
    for r in range(len(seq)):
        if not gone[r]:
            continue
        out[r] = 0
        n = math.ceil(max(int(seq[r]), 0) / page)
        if seq[r] < 0 or n > table.shape[1]:
            flags[1] = True
            n = min(n, table.shape[1])
        for j in range(n):
            if not 0 <= table[r, j] < n_pages:
                flags[0] = True
                continue
            if n_free < len(free):
                free[n_free] = table[r, j]
                n_free += 1
            else:
                flags[1] = True
    return free, n_free, out, flags


def _encode(x):
    """float64 -> E4M3 codes; x holds at most 24 significant bits, so float32 holds it."""
    x32 = x.to(torch.float32)
    assert torch.equal(x32.to(torch.float64), x)
    return x32.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def append(x, slot, cache, scale):
    """csa2_kv8_append of one of K, V: x [T,Hk,hd], cache u8 [P,Hk,page,hd], scale f32 [P,Hk]
    (CPU; the cache and scale are updated in place)."""
    page = cache.shape[2]
    t, T = 0, len(slot)
    while t < T:
        if slot[t] < 0:
            t += 1
            continue
        p, row = divmod(int(slot[t]), page)
        n = 1
        while t + n < T and row + n < page and slot[t + n] == slot[t] + n:
            n += 1
        new = x[t:t + n].to(torch.float64)  # [n][Hk][hd]
        for h in range(cache.shape[1]):
            amax = float(new[:, h].abs().max())
            s = 2.0 ** -64
            while amax > 448.0 * s:
                s *= 2.0
            old = float(scale[p, h])
            if row > 0 and old > s:
                s = old
            if row > 0 and s != old:
                cache[p, h, :row] = _encode(E4M3[cache[p, h, :row].long()] * (old / s))
            cache[p, h, row:row + n] = _encode(new[:, h] / s)
            scale[p, h] = s
        t += n


def attn(q, kc, vc, ks, vs, table, q_start, seq_len, sm_scale, window, cap):
    """csa2_kv8_attn in float64 (CPU tensors).  Returns out, lse and, per output element, the sum
    of |p v| and per row the largest sm_scale * sum |q k| over its keys (for error bounds); rows
    outside every request are NaN."""
    T, Hq, hd = q.shape
    P, Hk, page, _ = kc.shape
    G = Hq // Hk
    out = torch.full((T, Hq, hd), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    absum = torch.zeros(T, Hq, hd, dtype=torch.float64)
    smax = torch.zeros(T, Hq, dtype=torch.float64)
    q = q.to(torch.float64)
    for r in range(len(seq_len)):
        a, b, L = int(q_start[r]), int(q_start[r + 1]), int(seq_len[r])
        if a == b:
            continue
        keys = torch.arange(min(L, table.shape[1] * page))
        ids = table[r].long()[keys // page]
        has = (ids >= 0) & (ids < P)
        ids = ids.clamp(0, P - 1)
        k = E4M3[kc[ids, :, keys % page].long()] * ks[ids].to(torch.float64)[..., None]  # [L][Hk][hd]
        v = E4M3[vc[ids, :, keys % page].long()] * vs[ids].to(torch.float64)[..., None]
        for i in range(b - a):
            p = L - (b - a) + i
            sees = has & (keys <= p)
            if window:
                sees &= keys > p - window
            kk, vv = k[sees], v[sees]
            for h in range(Hq):
                if kk.shape[0] == 0:
                    out[a + i, h] = 0.0
                    lse[a + i, h] = -math.inf
                    continue
                s = (kk[:, h // G] @ q[a + i, h]) * sm_scale
                smax[a + i, h] = ((kk[:, h // G].abs() @ q[a + i, h].abs()) * abs(sm_scale)).max()
                if cap:
                    s = cap * torch.tanh(s / cap)
                w = torch.softmax(s, 0)
                out[a + i, h] = w @ vv[:, h // G]
                absum[a + i, h] = w @ vv[:, h // G].abs()
                lse[a + i, h] = torch.logsumexp(s, 0)
    return out, lse, absum, smax


def assert_attn(got, got_lse, ref, cap, max_len, what):
    """Element bounds, from the arithmetic the header names:
      - the result is rounded once to its type: eps/2 of it;
      - probabilities are rounded to f16: 2^-11 of sum |p v|;
      - tensor-core sums truncate: at most 2^-21 of the sum of magnitudes per 32-key step (the
        accumulator's alignment), so steps * 2^-21 of sum |p v| for the output;
      - scores: digits to 2^-22 of the head's largest element (hd <= 128 products of it, at most
        16 times the mean magnitude: 2^-18), 4 truncating steps (2^-19), exp2 and the cap's tanh
        2^-20 of the score's size; a score error e moves every weight by a factor 1 +- 2 e.
    """
    out, lse, absum, smax = ref
    rows = ~torch.isnan(lse[:, 0])
    eps = torch.finfo(got.dtype).eps / 2
    e = (2.0 ** -17) * smax + (2.0 ** -20) * (cap + 1.0)
    steps = (max_len + 31) // 32 + 4
    tol = eps * out.abs() + absum * (2.0 ** -11 + steps * 2.0 ** -21 + 2 * e[..., None]) + 1e-30
    if got.dtype is torch.float16:
        tol = tol + 2.0 ** -25  # half a subnormal step
    err = (got.cpu().to(torch.float64) - out).abs()
    bad = (err > tol) & rows[:, None, None]
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol)[rows].max()):.2f} bounds"
    if got_lse is not None:
        fin = rows[:, None] & torch.isfinite(lse)
        gl = got_lse.cpu().to(torch.float64)
        assert torch.equal(torch.isneginf(gl[rows]), torch.isneginf(lse[rows])), f"{what}: lse -inf pattern"
        # the sum of weights: e, exp2's 2^-21 and the fp32 sums and log
        d = (gl - lse).abs()
        lt = e + 2.0 ** -19 * (1.0 + lse.abs())
        assert (d[fin] <= lt[fin]).all(), f"{what}: lse off by {float((d / lt)[fin].max()):.2f} bounds"


def make_cache(gen, lens, Hk, hd, page, extra=3, nan_behind=True):
    """Pages for requests of the given lengths in shuffled order: codes of normal values, scales
    that differ by page and head, and (nan_behind) NaN codes in every row no request holds."""
    n = [math.ceil(L / page) for L in lens]
    P = sum(n) + extra
    perm = torch.randperm(P, generator=gen)
    cols = max(1, max(n)) + 1
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    at = 0
    held = torch.zeros(P, page, dtype=torch.bool)
    for r, m in enumerate(n):
        table[r, :m] = perm[at:at + m].to(torch.int32)
        at += m
        for j in range(m):
            held[table[r, j].long(), :min(page, lens[r] - j * page)] = True
    def codes():
        x = torch.randn(P, Hk, page, hd, generator=gen) * 60.0
        c = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        if nan_behind:
            c = torch.where(held[:, None, :, None], c, torch.full_like(c, 0x7F))
        return c.contiguous()
    kc, vc = codes(), codes()
    ks = (2.0 ** torch.randint(-8, -5, (P, Hk), generator=gen)).float()
    vs = (2.0 ** torch.randint(-9, -3, (P, Hk), generator=gen)).float()
    return table, kc, vc, ks, vs
