"""csa2_kv8_attn with more than 16 rows per key head (the f16 kernel), and what both of its kernels
do with NaN, infinities, dirty workspaces, long offsets and other streams."""
import math

import pytest
import torch

import kv8_ref as ref
from sparse_attention_fp4_pack_b200 import csa2
from test_gpu_kv8 import BF, HF, I32, I64, attn_inputs, check_attn, dev, run_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,cap", [(0, 0.0), (1, 0.0), (100, 0.0), (128, 0.0), (300, 0.0), (0, 20.0), (130, 5.0)])
@pytest.mark.parametrize("hd,page,dtype", [(128, 64, BF), (64, 16, HF), (128, 16, HF), (64, 128, BF)])
def test_window_and_cap(window, cap, hd, page, dtype):
    lens, news = [1, 70, 129, 300, 513], [1, 33, 1, 140, 40]
    check_attn(attn_inputs(window + 3, lens, news, 4, 2, hd, page, dtype), window, cap, max_q=140)


@pytest.mark.parametrize("Hq,Hk", [(5, 1), (17, 1), (48, 1), (24, 8), (129, 1), (300, 1)])
def test_groups(Hq, Hk):
    """Rows that fill, overfill and leave parts of the 128-row slots; groups wider than a tile."""
    lens, news = [200, 31, 130, 64], [9, 31, 1, 3] if Hq < 100 else [2, 3, 1, 1]
    check_attn(attn_inputs(Hq, lens, news, Hq, Hk, 64, 32, BF), max_q=31)


@pytest.mark.parametrize("n", [1, 127, 128, 129, 255, 256, 257, 400])
def test_row_counts(n):
    """One request of n rows (two heads of one group): one slot, two, and several blocks."""
    check_attn(attn_inputs(n, [n + 5], [n], 2, 1, 64, 64, HF), max_q=n)


@pytest.mark.parametrize("length,n,hd", [(6000, 20, 128), (4000, 150, 64), (2600, 260, 128)])
def test_split_over_ctas(length, n, hd):
    """A few requests whose key tiles are shared out over all CTAs and merged, one slot and two."""
    check_attn(attn_inputs(length, [length, 7], [n, 1], 2, 1, hd, 64, BF), max_q=n)


@pytest.mark.parametrize("qscale,dtype", [(40.0, BF), (1e-3, BF), (40.0, HF), (1e-3, HF)])
def test_score_range(qscale, dtype):
    check_attn(attn_inputs(3, [700, 30], [40, 1], 4, 2, 128, 64, dtype, qscale), max_q=40)


def test_rising_scores():
    """Scores that grow from tile to tile: the accumulated output is rescaled again and again."""
    args = list(attn_inputs(4, [900], [40], 2, 1, 128, 64, BF))
    q, kc, table = args[0], args[1], args[5]
    q[:] = q.abs() * 8
    for j in range(15):
        kc[table[0, j].long()] &= 0x7F
        args[3][table[0, j].long()] = 2.0 ** (j - 14)
    kc[table[0, 14].long(), :, 4:] = 0x7F
    check_attn(args, max_q=40)


def test_value_scales_apart():
    args = list(attn_inputs(5, [200, 64], [30, 5], 4, 1, 64, 16, HF))
    for j in range(13):
        args[4][args[5][0, j].long()] = [0.0, 2.0 ** -60, 2.0 ** -10, 1.0 / 3.0][j % 4]
    check_attn(args, max_q=30)


def test_nothing_visible_and_bad_tables():
    make = lambda: list(attn_inputs(6, [40, 90, 300], [20, 1, 50], 4, 2, 64, 16, BF))
    args = make()
    args[7][0] = 10                        # twenty rows, ten tokens: ten rows see nothing
    check_attn(args, max_q=50, want_status=csa2.DEV_BAD_COUNT)
    args = make()
    args[5][1, 2] = -1
    args[5][2, 0] = args[1].shape[0]
    check_attn(args, max_q=50, want_status=csa2.DEV_BAD_INDEX)
    args[5][1, :] = -1
    check_attn(args, max_q=50, want_status=csa2.DEV_BAD_INDEX)
    args = make()
    args[5] = args[5][:, :4].contiguous()
    check_attn(args, max_q=50, want_status=csa2.DEV_BAD_COUNT)


@pytest.mark.parametrize("max_q", [1, 64])
def test_bad_query_ranges(max_q):
    """q_start beyond T or descending is cut: rows named by it that exist are still right."""
    args = list(attn_inputs(7, [40, 90, 30], [2, 3, 4], 4, 2, 64, 16, BF))
    good, good_lse = run_attn(args, 0.125, max_q=max_q)
    args[6] = torch.tensor([0, 2, 5, 50], dtype=I32)      # the last request runs past T = 11
    args[7][2] = 32                                       # six rows now
    out, lse = run_attn(args, 0.125, max_q=max_q, want_status=csa2.DEV_BAD_COUNT)
    assert torch.equal(out[:5], good[:5]) and torch.equal(lse[:5], good_lse[:5])
    args[6] = torch.tensor([0, 5, 2, 2], dtype=I32)       # descending
    out, _ = run_attn(args, 0.125, max_q=max_q, want_status=csa2.DEV_BAD_COUNT)
    assert (out[5:] == 7.0).all()
    args[6] = torch.tensor([-3, -1, 50, 60], dtype=I32)
    run_attn(args, 0.125, max_q=max_q, want_status=csa2.DEV_BAD_COUNT)


@pytest.mark.parametrize("max_q", [1, 64])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("length", [300, 9000])
def test_nan_and_infinity_stay_where_they_are(max_q, cap, length):
    """A NaN or an infinity in a query row gives NaN in that row and head alone; a NaN key code in
    the rows that see it."""
    args = list(attn_inputs(8, [length, 50], [5, 2], 4, 2, 64, 32, BF))
    clean, clean_lse = run_attn(args, 0.125, cap=cap, max_q=max_q)
    q = args[0].clone()
    q[1, 2, 7] = math.nan
    q[3, 0, 0] = math.inf
    out, lse = run_attn([q] + args[1:], 0.125, cap=cap, max_q=max_q)
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[3, 0] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])
    kc = args[1].clone()
    pos = length - 3                                      # seen by the last three rows of request 0
    kc[args[5][0, pos // 32].long(), 1, pos % 32, 3] = 0x7F
    out, lse = run_attn([args[0], kc] + args[2:], 0.125, cap=cap, max_q=max_q)
    bad[:] = False
    bad[2:5, 2:] = True                                   # key head 1: query heads 2 and 3
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


@pytest.mark.parametrize("max_q", [1, 64])
def test_dirty_workspace_and_repeats(max_q):
    """The workspace may hold anything, and the same call gives the same bits."""
    args = attn_inputs(9, [5000, 3, 900], [6, 1, 4], 4, 2, 128, 64, BF)
    want, want_lse = run_attn(args, 0.1, max_q=max_q)
    ref.assert_attn(want, want_lse, ref.attn(*args, 0.1, 0, 0.0), 0.0, 5000, "split")
    size = csa2.csa2_kv8_attn_workspace_size(4, 2, 128, max_q, BF)
    for fill in (0xFF, 0x7F, 0x01):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        out, lse = run_attn(args, 0.1, max_q=max_q, ws=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_strided_queries_other_stream_and_no_lse():
    args = attn_inputs(10, [100, 300, 17], [40, 30, 2], 6, 3, 128, 64, HF)
    want, _ = run_attn(args, 0.1, max_q=40)
    q, *rest = [t.cuda() for t in args]
    wide = torch.randn(q.shape[0], 12, 128, device="cuda").to(HF)
    wide[:, 3:9] = q
    side, out = torch.cuda.Stream(), torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    csa2.csa2_kv8_attn(wide[:, 3:9], *rest, 0.1, out, max_q=40, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_two_streams_at_once():
    """Two calls of both kernels in flight together, each with its own workspace."""
    a = attn_inputs(11, [3000, 90], [30, 1], 4, 2, 128, 64, BF)
    b = attn_inputs(12, [2500, 700], [1, 1], 4, 2, 128, 64, BF)
    want = [run_attn(a, 0.1, max_q=30), run_attn(b, 0.1)]
    args = [[t.cuda() for t in x] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.full_like(x[0], 7.0) for _ in range(10)] for x in args]
    torch.cuda.synchronize()
    for i in range(10):
        for k in range(2):
            csa2.csa2_kv8_attn(*args[k], 0.1, outs[k][i], max_q=30 if k == 0 else 1, stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            assert torch.equal(o, want[k][0])


@pytest.mark.parametrize("max_q", [1, 32])
def test_pages_far_into_a_large_pool(max_q):
    """A cache of 4.9 GB per tensor, its used pages at the end: offsets past 2^32 bytes."""
    P, Hk, page, hd = 38000, 8, 128, 128
    need = 2 * P * Hk * page * hd
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("not enough memory")
    small = attn_inputs(13, [300, 129], [3, 1], 8, 8, hd, page, BF)
    q, kc, vc, ks, vs, table, q_start, seq_len = small
    want, want_lse = run_attn(small, 0.1, max_q=max_q)
    n = kc.shape[0]
    bk, bv = (torch.empty(P, Hk, page, hd, dtype=torch.uint8, device="cuda") for _ in range(2))
    bks, bvs = (torch.ones(P, Hk, device="cuda") for _ in range(2))
    bk[P - n:], bv[P - n:], bks[P - n:], bvs[P - n:] = kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda()
    t2 = torch.where(table >= 0, table + (P - n), table).cuda()
    out, lse = torch.full_like(q, 7.0).cuda(), torch.full(q.shape[:2], 7.0, device="cuda")
    csa2.csa2_kv8_attn(q.cuda(), bk, bv, bks, bvs, t2, q_start.cuda(), seq_len.cuda(), 0.1, out, lse, max_q=max_q)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # and an append to the last page, against the same append to a small pool
    x, y = (torch.randn(20, Hk, hd, device="cuda").to(BF) for _ in range(2))
    slot = torch.arange(n * page - 20, n * page, device="cuda")
    sk, sv, sks, svs = [t.cuda().clone() for t in (kc, vc, ks, vs)]
    csa2.csa2_kv8_append(x, y, slot, sk, sv, sks, svs)
    csa2.csa2_kv8_append(x, y, slot + (P - n) * page, bk, bv, bks, bvs)
    for a, b in ((sk, bk), (sv, bv), (sks, bks), (svs, bvs)):
        assert torch.equal(a, b[P - n:])


def test_append_nan_and_infinity():
    """Stored as the header says, and not into other pages or heads."""
    x = torch.randn(20, 2, 64, dtype=torch.float32).to(BF)
    y = x.clone()
    y[3, 0, 5], y[18, 1, 0], y[18, 1, 1] = math.nan, math.inf, -math.inf
    slot = torch.arange(16, 36)
    caches = []
    for v in (x, y):
        kc, vc = (torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.ones(4, 2, device="cuda") for _ in range(2))
        csa2.csa2_kv8_append(v.cuda(), x.cuda(), dev(slot, I64), kc, vc, ks, vs)
        caches.append([t.cpu() for t in (kc, vc, ks, vs)])
    (kc, vc, ks, vs), (kc2, vc2, ks2, vs2) = caches
    assert torch.equal(vc, vc2) and torch.equal(vs, vs2)
    assert int(kc2[1, 0, 3, 5]) & 0x7F == 0x7F and float(ks2[2, 1]) == 2.0 ** 120
    assert kc2[2, 1, 2, 0] == 0x7E and kc2[2, 1, 2, 1] == 0xFE
    assert torch.equal(kc[1, 1], kc2[1, 1]) and torch.equal(kc[2, 0], kc2[2, 0]) and torch.equal(kc[0], kc2[0])
    keep = torch.ones(16, 64, dtype=torch.bool)
    keep[3, 5] = False
    if float(x[3, 0, 5].abs()) < float(x[:16, 0].abs().max()):
        assert torch.equal(kc[1, 0][keep], kc2[1, 0][keep])
