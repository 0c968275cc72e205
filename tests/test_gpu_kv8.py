"""The paged 8-bit KV cache on the GPU: plan, release, append and attention against plain
64-bit implementations (tests/kv8_ref.py)."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as ref
from sparse_attention_fp4_pack_b200 import csa2

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda()


# ---- plan --------------------------------------------------------------------------------
def run_plan(ctx, new, table, free, n_free, page, n_pages, t_cap, in_place=False):
    c, t = dev(ctx, I32), dev(table, I32)
    nf = dev([n_free], I32)
    R = len(ctx)
    seq = c if in_place else torch.full((R,), 77, dtype=I32, device="cuda")
    nfo = nf if in_place else torch.full((1,), 77, dtype=I32, device="cuda")
    qs = torch.full((R + 1,), 77, dtype=I32, device="cuda")
    slot, pos = (torch.full((t_cap,), 77, dtype=I64, device="cuda") for _ in range(2))
    st = csa2.status_word()
    csa2.csa2_paged_plan(c, dev(new, I32), t, dev(free, I32), nf, page, n_pages, seq, nfo, qs, slot, pos, dev_status=st)
    torch.cuda.synchronize()
    return dict(table=t.cpu().numpy(), seq_len=seq.cpu().numpy(), n_free=int(nfo), q_start=qs.cpu().numpy(),
                slot=slot.cpu().numpy(), pos=pos.cpu().numpy()), int(st)


def check_plan(ctx, new, table, free, n_free, page, n_pages, t_cap, in_place=False):
    want, flags = ref.plan(ctx, new, table, free, n_free, page, n_pages, t_cap)
    got, word = run_plan(ctx, new, table, free, n_free, page, n_pages, t_cap, in_place)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    assert word == (csa2.DEV_BAD_INDEX * flags[0] | csa2.DEV_BAD_COUNT * flags[1] | csa2.DEV_NO_PAGES * flags[2])


def plan_inputs(rng, R, page, hi, q, spare):
    ctx = rng.integers(0, hi + 1, R)
    new = rng.integers(0, q + 1, R)
    have, want = -(-ctx // page), -(-(ctx + new) // page)
    P = int(want.sum()) + spare
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((R, max(1, int(want.max(initial=0)))), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    return ctx.astype(np.int32), new.astype(np.int32), table, ids[at:], P


@pytest.mark.parametrize("R,page,hi,q,in_place", [(1, 16, 0, 1, False), (1, 64, 100, 40, True), (7, 16, 50, 33, False),
                                                  (33, 128, 300, 1, True), (61, 32, 200, 90, False),
                                                  (1024, 16, 100, 3, True), (1025, 64, 400, 17, False),
                                                  (2100, 16, 60, 5, True)])
def test_plan(R, page, hi, q, in_place):
    rng = np.random.default_rng(R * 131 + page)
    ctx, new, table, free, P = plan_inputs(rng, R, page, hi, q, 5)
    check_plan(ctx, new, table, free, len(free), page, P, int(new.sum()) + 9, in_place)


def test_plan_edges():
    rng = np.random.default_rng(3)
    ctx, new, table, free, P = plan_inputs(rng, 40, 16, 60, 50, 0)
    T = int(new.sum())
    check_plan(ctx, new, table, free, 11, 16, P, T)                       # out of pages in the middle
    check_plan(ctx, new, table, free, 0, 16, P, T)                        # no page at all
    check_plan(ctx, new, table, free, len(free) + 3, 16, P, T)            # count beyond the list
    check_plan(ctx, new, table, free, -2, 16, P, T)                       # negative count
    check_plan(ctx, new, table, free, len(free), 16, P, T // 2)           # rows cut off
    check_plan(ctx, new, table, free, len(free), 16, P, 0)                # no rows at all
    check_plan(ctx, new, table[:, :4].copy(), free, len(free), 16, P, T)  # table too narrow
    check_plan(ctx, new, table, free, len(free), 16, P // 2, T)           # ids beyond the pool
    c2, n2 = ctx.copy(), new.copy()
    c2[5], n2[9] = -7, -1
    check_plan(c2, n2, table, free, len(free), 16, P, T)                  # negative lengths
    check_plan(ctx, np.zeros_like(new), table, free, len(free), 16, P, 6)  # nothing new
    check_plan(ctx[:0], new[:0], table[:0], free, len(free), 16, P, 6)    # no requests


# ---- release -----------------------------------------------------------------------------
def check_release(seq, table, gone, free, n_free, page, n_pages, in_place):
    want_free, want_n, want_seq, flags = ref.release(seq, table, gone, free, n_free, page, n_pages)
    s, f, nf = dev(seq, I32), dev(free, I32), dev([n_free], I32)
    so = s if in_place else torch.full_like(s, 77)
    nfo = nf if in_place else torch.full_like(nf, 77)
    st = csa2.status_word()
    csa2.csa2_paged_release(s, dev(table, I32), dev(gone, torch.uint8), f, nf, page, n_pages, so, nfo, dev_status=st)
    assert np.array_equal(f.cpu().numpy(), want_free)
    assert int(nfo) == want_n
    assert np.array_equal(so.cpu().numpy(), want_seq)
    assert int(st) == (csa2.DEV_BAD_INDEX * flags[0] | csa2.DEV_BAD_COUNT * flags[1])


@pytest.mark.parametrize("R,page,hi,in_place", [(1, 16, 40, True), (9, 64, 1000, False), (33, 16, 700, True),
                                                (500, 128, 3000, False), (1300, 32, 900, True)])
def test_release(R, page, hi, in_place):
    rng = np.random.default_rng(R)
    seq, _, table, left, P = plan_inputs(rng, R, page, hi, 0, 4)
    free = np.full(P, -5, np.int32)
    free[:len(left)] = left
    for gone in (rng.integers(0, 3, R) == 0, np.ones(R, bool), np.zeros(R, bool)):
        check_release(seq, table, gone.astype(np.uint8) * 3, free, len(left), page, P, in_place)


def test_release_edges():
    rng = np.random.default_rng(8)
    seq, _, table, left, P = plan_inputs(rng, 50, 16, 300, 0, 4)
    free = np.full(P, -5, np.int32)
    gone = np.ones(50, np.uint8)
    t2 = table.copy()
    t2[3, 0], t2[4, 1], t2[5, 0] = -1, P + 9, -44
    check_release(seq, t2, gone, free, 0, 16, P, False)           # bad entries are left out
    check_release(seq, table, gone, free[:20].copy(), 7, 16, P, False)  # the list is full
    check_release(seq, table, gone, free[:0].copy(), 0, 16, P, False)   # no list
    check_release(seq, table[:, :3].copy(), gone, free, 0, 16, P, False)  # lengths beyond the table
    s2 = seq.copy()
    s2[7] = -3
    check_release(s2, table, gone, free, 2, 16, P, False)
    check_release(seq, table, gone, free, -1, 16, P, False)
    check_release(seq[:0], table[:0], gone[:0], free, 3, 16, P, False)


# ---- append ------------------------------------------------------------------------------
def append_case(seed, lens, news, Hk, hd, page, dtype, fused=False, spread=0):
    gen = torch.Generator().manual_seed(seed)
    table, kc, vc, ks, vs = ref.make_cache(gen, [c + n for c, n in zip(lens, news)], Hk, hd, page, nan_behind=False)
    slot = [int(table[r, p // page]) * page + p % page for r, (c, n) in enumerate(zip(lens, news)) for p in range(c, c + n)]
    T = len(slot)
    heads = 3 * Hk if fused else Hk
    x = torch.randn(T, heads, hd, generator=gen) * 2.0 ** torch.randint(-spread, spread + 1, (T, heads, 1), generator=gen)
    x = x.to(dtype)
    y = torch.randn(T, heads, hd, generator=gen).to(dtype)
    return x, y, slot, kc, vc, ks, vs


def check_append(x, y, slot, kc, vc, ks, vs, fused=False, status=0):
    Hk = kc.shape[1]
    gk, gv, gks, gvs = kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda()
    xd, yd = x.cuda(), y.cuda()
    k, v = (xd[:, Hk:2 * Hk], yd[:, 2 * Hk:]) if fused else (xd, yd)
    st = csa2.status_word()
    csa2.csa2_kv8_append(k, v, dev(slot, I64), gk, gv, gks, gvs, dev_status=st)
    assert int(st) == status
    xc, yc = (x[:, Hk:2 * Hk], y[:, 2 * Hk:]) if fused else (x, y)
    ref.append(xc, slot, kc, ks)
    ref.append(yc, slot, vc, vs)
    for got, want, what in ((gks, ks, "k_scale"), (gvs, vs, "v_scale"), (gk, kc, "k"), (gv, vc, "v")):
        assert torch.equal(got.cpu(), want), what


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hk,hd,dtype", [(1, 64, torch.bfloat16), (3, 128, torch.float16), (2, 128, torch.bfloat16)])
def test_append(page, Hk, hd, dtype):
    fused = Hk == 3
    for seed, (lens, news) in enumerate((([0], [1]), ([5, 0, 37, 128, 255], [1, 1, 1, 1, 1]),
                                         ([3, 100, 64, 0], [150, 1, 64, 17]), ([127, 15, 31], [2, 2, 40]))):
        case = append_case(seed, lens, news, Hk, hd, page, dtype, fused, spread=seed * 3)
        check_append(*case, fused=fused)


def test_append_window_of_tokens():
    """Enough units that each walks several tokens, pages of one and of many rows mixed."""
    lens = [(7 * r) % 200 for r in range(700)]
    news = [1 + (r % 5) * (r % 3) for r in range(700)]
    check_append(*append_case(11, lens, news, 9, 64, 64, torch.bfloat16, spread=4))


def test_append_twice_and_extremes():
    x, y, slot, kc, vc, ks, vs = append_case(5, [4, 20], [20, 9], 2, 64, 16, torch.bfloat16)
    x[0] = 0.0           # a row of zeros
    x[5:9] = 3.0e38      # close to the type's largest
    y[:] = 0.0           # every new row zero: the smallest scale, or the page's own
    y[21] = -1.0e-30     # below the smallest scale's smallest code
    y[22] = -448.0       # exactly the largest code times one
    y[23] = 448.5 if y.dtype == torch.float32 else 450.0
    check_append(x, y, slot, kc, vc, ks, vs)
    a = [t.cuda() for t in (kc, vc, ks, vs)]
    for _ in range(2):   # the same rows again: nothing changes
        csa2.csa2_kv8_append(x.cuda(), y.cuda(), dev(slot, I64), *a)
    for got, want in zip(a, (kc, vc, ks, vs)):
        assert torch.equal(got.cpu(), want)


def test_append_one_token_at_a_time_equals_scale_growth():
    """A page filled row by row, each row larger than the last: every earlier row is re-encoded
    under each new scale exactly as the definition says."""
    gen = torch.Generator().manual_seed(1)
    kc, vc = (torch.zeros(2, 1, 16, 64, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.ones(2, 1) for _ in range(2))
    dk = [t.cuda() for t in (kc, vc, ks, vs)]
    for i in range(16):
        x = (torch.randn(1, 1, 64, generator=gen) * 1.7 ** i).to(torch.bfloat16)
        y = (torch.randn(1, 1, 64, generator=gen) * 0.6 ** i).to(torch.bfloat16)
        csa2.csa2_kv8_append(x.cuda(), y.cuda(), dev([16 + i], I64), *dk)
        ref.append(x, [16 + i], kc, ks)
        ref.append(y, [16 + i], vc, vs)
    for got, want in zip(dk, (kc, vc, ks, vs)):
        assert torch.equal(got.cpu(), want)


def test_append_bad_slots():
    x, y, slot, kc, vc, ks, vs = append_case(6, [0, 0], [20, 20], 1, 64, 16, torch.float16)
    P = kc.shape[0]
    slot[0] = -1                 # skipped in silence
    slot[39] = P * 16            # beyond the pool
    check = list(slot)
    check[39] = -1
    a = [t.cuda() for t in (kc, vc, ks, vs)]
    st = csa2.status_word()
    csa2.csa2_kv8_append(x.cuda(), y.cuda(), dev(slot, I64), *a, dev_status=st)
    assert int(st) == csa2.DEV_BAD_INDEX
    ref.append(x, check, kc, ks)
    ref.append(y, check, vc, vs)
    for got, want in zip(a, (kc, vc, ks, vs)):
        assert torch.equal(got.cpu(), want)
    # a row that repeats its neighbour's slot is refused
    st = csa2.status_word()
    csa2.csa2_kv8_append(x[:2].cuda(), y[:2].cuda(), dev([slot[5], slot[5]], I64), *a, dev_status=st)
    assert int(st) == csa2.DEV_BAD_INDEX


# ---- attention ---------------------------------------------------------------------------
def attn_inputs(seed, lens, news, Hq, Hk, hd, page, dtype, qscale=1.0):
    gen = torch.Generator().manual_seed(seed)
    table, kc, vc, ks, vs = ref.make_cache(gen, lens, Hk, hd, page)
    T = sum(news)
    q = (torch.randn(T + 2, Hq, hd, generator=gen) * qscale).to(dtype)
    q_start = torch.tensor([0] + list(np.cumsum(news)), dtype=I32)
    return q, kc, vc, ks, vs, table, q_start, torch.tensor(lens, dtype=I32)


def run_attn(args, sm_scale, window=0, cap=0.0, max_q=1, ws=None, want_status=0, stream=None):
    q, kc, vc, ks, vs, table, q_start, seq_len = [t.cuda() for t in args]
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    st = csa2.status_word()
    torch.cuda.synchronize()
    csa2.csa2_kv8_attn(q, kc, vc, ks, vs, table, q_start, seq_len, sm_scale, out, lse, max_q=max_q, window=window,
                       softcap=cap, ws=ws, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st) == want_status
    return out, lse


def check_attn(args, window=0, cap=0.0, max_q=1, sm_scale=None, want_status=0):
    q, hd = args[0], args[0].shape[-1]
    sm_scale = 1.0 / math.sqrt(hd) if sm_scale is None else sm_scale
    out, lse = run_attn(args, sm_scale, window, cap, max_q, want_status=want_status)
    want = ref.attn(*args, sm_scale, window, cap)
    ref.assert_attn(out, lse, want, cap, int(args[7].max()), f"Hq {q.shape[1]} hd {hd} window {window} cap {cap}")
    rest = torch.isnan(want[1][:, 0])
    assert rest.any() and (out.cpu()[rest] == 7.0).all() and (lse.cpu()[rest] == 7.0).all()  # left as they were


BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("Hq,Hk,hd,page,dtype", [(8, 1, 128, 64, BF), (16, 2, 128, 16, BF), (5, 1, 64, 32, HF),
                                                 (4, 4, 64, 128, BF), (12, 1, 128, 128, HF), (21, 3, 64, 16, BF),
                                                 (40, 2, 128, 32, BF), (40, 1, 128, 64, HF), (72, 1, 64, 64, BF),
                                                 (64, 1, 128, 16, BF)])
def test_attn_decode(Hq, Hk, hd, page, dtype):
    """One row per request: lengths around tile and page borders, every column count, groups
    larger than the largest tile."""
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 300, 640]
    check_attn(attn_inputs(Hq, lens, [1] * len(lens), Hq, Hk, hd, page, dtype))


@pytest.mark.parametrize("window,cap", [(1, 0.0), (100, 0.0), (128, 0.0), (1000, 0.0), (0, 20.0), (130, 5.0)])
@pytest.mark.parametrize("hd,dtype", [(128, BF), (64, HF)])
def test_attn_window_and_cap(window, cap, hd, dtype):
    lens, news = [1, 50, 129, 257, 700], [1, 9, 1, 30, 2]
    check_attn(attn_inputs(window + 7, lens, news, 6, 2, hd, 32, dtype), window, cap, max_q=9)


@pytest.mark.parametrize("Hq,Hk,hd,page,dtype,max_q", [(8, 2, 128, 64, BF, 64), (8, 2, 128, 64, BF, 1),
                                                       (5, 1, 64, 16, HF, 200), (16, 1, 128, 128, BF, 16),
                                                       (2, 2, 64, 32, BF, 30), (7, 1, 128, 16, HF, 3)])
def test_attn_ragged_rows(Hq, Hk, hd, page, dtype, max_q):
    """Requests of many, one and no rows; whole prompts and rows behind a long context; the tile
    hint too small, right and too large."""
    lens, news = [64, 300, 0, 1, 200, 513, 40], [64, 1, 0, 1, 130, 77, 0]
    check_attn(attn_inputs(max_q, lens, news, Hq, Hk, hd, page, dtype), max_q=max_q)


@pytest.mark.parametrize("length,Hq,Hk,hd", [(9000, 8, 1, 128), (5000, 4, 2, 64)])
def test_attn_split_over_ctas(length, Hq, Hk, hd):
    """One request whose key tiles are shared out over many CTAs and merged."""
    check_attn(attn_inputs(length, [length, 3], [1, 1], Hq, Hk, hd, 64, BF))


def test_attn_many_short_requests():
    lens = [1 + (r * 37) % 90 for r in range(900)]
    check_attn(attn_inputs(2, lens, [1] * 900, 2, 1, 64, 16, BF))


@pytest.mark.parametrize("qscale,dtype", [(40.0, BF), (1e-3, BF), (40.0, HF), (1e-3, HF)])
def test_attn_score_range(qscale, dtype):
    """Sharp and flat softmaxes: large scores move the running maximum, small ones never do."""
    check_attn(attn_inputs(3, [700, 30], [3, 1], 4, 2, 128, 64, dtype, qscale), max_q=3)


def test_attn_rising_scores():
    """Scores that grow from tile to tile: the accumulated output is rescaled every time."""
    args = list(attn_inputs(4, [900], [1], 8, 1, 128, 64, BF))
    q, kc, table = args[0], args[1], args[5]
    q[:] = q.abs()
    for j in range(15):
        kc[table[0, j].long()] &= 0x7F   # positive keys,
        args[3][table[0, j].long()] = 2.0 ** (j - 14)  # larger page by page
    kc[table[0, 14].long(), :, 4:] = 0x7F
    check_attn(args)


def test_attn_value_scales_apart():
    """Pages whose value scales differ by 2^60, zero included."""
    args = list(attn_inputs(5, [200, 64], [1, 1], 4, 1, 64, 16, HF))
    vs, table = args[4], args[5]
    for j in range(13):
        vs[table[0, j].long()] = [0.0, 2.0 ** -60, 2.0 ** -10, 1.0 / 3.0][j % 4]
    check_attn(args)


def test_attn_nothing_visible_and_bad_tables():
    """Rows before position 0, an empty request, and table entries that name no page."""
    args = list(attn_inputs(6, [40, 90, 300], [2, 1, 5], 4, 2, 64, 16, BF))
    args[7][0] = 1                         # two rows, one token: the first row sees nothing
    check_attn(args, max_q=5, want_status=csa2.DEV_BAD_COUNT)
    args = list(attn_inputs(6, [40, 90, 300], [2, 1, 5], 4, 2, 64, 16, BF))
    args[5][1, 2] = -1
    args[5][2, 0] = args[1].shape[0]
    check_attn(args, max_q=5, want_status=csa2.DEV_BAD_INDEX)
    args[5][1, :] = -1                     # nothing left to see
    check_attn(args, max_q=5, want_status=csa2.DEV_BAD_INDEX)
    args = list(attn_inputs(6, [40, 90], [1, 1], 4, 2, 64, 16, BF))
    args[5] = args[5][:, :4].contiguous()  # a length beyond the table
    check_attn(args, want_status=csa2.DEV_BAD_COUNT)


def test_attn_strided_queries_other_stream_and_no_lse():
    args = attn_inputs(9, [100, 300, 17], [4, 1, 2], 6, 3, 128, 64, BF)
    base_out, base_lse = run_attn(args, 0.1, max_q=4)
    q, kc, vc, ks, vs, table, q_start, seq_len = [t.cuda() for t in args]
    wide = torch.randn(q.shape[0], 12, 128, device="cuda").to(BF)
    wide[:, 3:9] = q
    side = torch.cuda.Stream()
    out = torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    csa2.csa2_kv8_attn(wide[:, 3:9], kc, vc, ks, vs, table, q_start, seq_len, 0.1, out, max_q=4, stream=side)
    side.synchronize()
    assert torch.equal(out, base_out)
    for _ in range(3):  # the same bits every time
        o, l = run_attn(args, 0.1, max_q=4)
        assert torch.equal(o, base_out) and torch.equal(l, base_lse)


# ---- plan and release on the cluster of eight CTAs: more rows and pages than one CTA takes ------
def test_release_edges_on_a_cluster():
    """test_release_edges with 2500 requests (three chunks) and a table beyond 16384 entries: bad
    entries in the first and in the last chunk alone, full lists, cut lengths and bad counts."""
    rng = np.random.default_rng(18)
    seq, _, table, left, P = plan_inputs(rng, 2500, 16, 200, 0, 4)
    assert table.size > 16384
    free = np.full(P, -5, np.int32)
    free[:len(left)] = left
    gone = (rng.integers(0, 3, 2500) > 0).astype(np.uint8)
    long = np.flatnonzero(seq > 32)  # three pages or more
    a, b, c, d = long[0], long[long < 1024][-1], long[long >= 2048][0], long[-1]
    gone[[a, b, c, d]] = 1
    t2, t3 = table.copy(), table.copy()
    t2[a, 0], t2[b, 1], t2[c, 0], t2[d, 1] = -1, P + 9, -44, P
    t3[d, 0] = -7
    for in_place in (False, True):
        check_release(seq, table, gone, free, len(left), 16, P, in_place)
        check_release(seq, t2, gone, free, len(left), 16, P, in_place)   # bad entries in two chunks
        check_release(seq, t3, gone, free, len(left), 16, P, in_place)   # in the last chunk alone
    check_release(seq, t2, gone, free[:900].copy(), 7, 16, P, False)     # the list is full in the middle of a chunk
    check_release(seq, table, gone, free[:900].copy(), 7, 16, P, True)
    check_release(seq, t2, gone, free[:0].copy(), 0, 16, P, False)       # no list
    narrow = np.ascontiguousarray(table[:, :7])
    assert narrow.size > 16384
    check_release(seq, narrow, gone, free, 0, 16, P, False)              # lengths beyond the table
    s2 = seq.copy()
    s2[[7, 1500]] = -3, -70000
    gone2 = gone.copy()
    gone2[[7, 1500]] = 1
    check_release(s2, t2, gone2, free, 2, 16, P, True)                   # negative lengths
    check_release(seq, table, gone, free, -1, 16, P, False)              # counts that cannot be
    check_release(seq, table, gone, free, P + 8, 16, P, False)
    check_release(seq, table, np.zeros(2500, np.uint8), free, 5, 16, P, True)


def test_plan_edges_on_a_cluster():
    """test_plan_edges with 2300 requests (three chunks) and more than 2048 rows."""
    rng = np.random.default_rng(13)
    ctx, new, table, free, P = plan_inputs(rng, 2300, 16, 60, 4, 0)
    T = int(new.sum())
    assert T > 2048
    for in_place in (False, True):
        check_plan(ctx, new, table, free, len(free) // 2, 16, P, T, in_place)      # out of pages in the middle
        check_plan(ctx, new, table, free, 0, 16, P, T + 3, in_place)               # no page at all
        check_plan(ctx, new, table, free, len(free) + 3, 16, P, T, in_place)       # count beyond the list
        check_plan(ctx, new, table, free, -2, 16, P, T, in_place)                  # negative count
        check_plan(ctx, new, table, free, len(free), 16, P, 2100, in_place)        # rows cut off
        check_plan(ctx, new, table[:, :3].copy(), free, len(free), 16, P, T, in_place)  # table too narrow
        check_plan(ctx, new, table, free, len(free), 16, P // 2, T, in_place)      # ids beyond the pool
        c2, n2 = ctx.copy(), new.copy()
        c2[[5, 2200]], n2[[9, 1100]] = -7, -1
        check_plan(c2, n2, table, free, len(free), 16, P, T, in_place)             # negative lengths
    check_plan(ctx, np.zeros_like(new), table, free, len(free), 16, P, 3000)       # nothing new
    check_plan(ctx[:0], new[:0], table[:0], free, len(free), 16, P, 3000)          # no requests
