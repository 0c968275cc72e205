"""csa2_kv8_attn where scales and weights lie far apart: what the softmax sum, small weights beside a
dominating key and scores near the end of fp32 are held to.  max_q 1 takes the kernel of few rows per
key head, max_q 40 the f16 one."""
import math

import pytest
import torch

import kv8_ref as ref
from sparse_attention_fp4_pack_b200 import csa2
from test_gpu_kv8 import BF, HF, attn_inputs, run_attn

pytestmark = pytest.mark.gpu

ROWS = [(1, [1, 3]), (40, [40, 3])]


def check_lse(lse, want, what):
    """lse against the 64-bit one, with the bound of ref.assert_attn: the scores' error and 2^-19 of
    the value for exp2, the fp32 sums and the logarithm."""
    _, exact, _, smax = want
    rows = ~torch.isnan(exact[:, 0])
    tol = 2.0 ** -17 * smax + 2.0 ** -20 + 2.0 ** -19 * (1.0 + exact.abs())
    err = (lse.cpu().double() - exact).abs()
    assert (err <= tol)[rows].all(), f"{what}: lse off by {float(err[rows].max()):.3g}"


@pytest.mark.parametrize("max_q,news", ROWS)
@pytest.mark.parametrize("length", [200, 2000])
@pytest.mark.parametrize("scales", [(2.0 ** 60, 2.0 ** -60), (2.0 ** 120, 1.0), (2.0 ** -64, 2.0 ** 100, 3.0), (1.0, 2.0 ** -20, 2.0 ** 118)])
def test_softmax_sum_with_value_scales_far_apart(max_q, news, length, scales):
    """The sum of the weights does not depend on the value scales: keys on pages of small scale count
    in it whatever the other pages' scales are, and lower the share of the others."""
    args = list(attn_inputs(21, [length, 90], news, 4, 2, 64, 16, BF))
    vs, table = args[4], args[5]
    for r, n in enumerate((length, 90)):
        for j in range(-(-n // 16)):
            vs[table[r, j].long()] = scales[j % len(scales)]
    out, lse = run_attn(args, 0.125, max_q=max_q)
    want = ref.attn(*args, 0.125, 0, 0.0)
    check_lse(lse, want, f"scales {scales}")
    ref.assert_attn(out, None, want, 0.0, length, f"scales {scales}")


def dominated(seed, length, news, nats, hd, dtype):
    """Requests whose key 0 scores `nats` above the others (give or take one) in every row and has
    only zeros as its V: the output is carried by the small weights of the other keys."""
    args = list(attn_inputs(seed, [length, 90], news, 4, 2, hd, 16, dtype))
    q, kc, vc, ks, vs, table = args[:6]
    gen = torch.Generator().manual_seed(seed + 1)
    q[:] = (1.0 + torch.randn(q.shape, generator=gen) / 32).to(dtype)
    held = kc & 0x7F != 0x7F
    small = (torch.randn(kc.shape, generator=gen) * 12.0).to(torch.float8_e4m3fn).view(torch.uint8)
    kc[:] = torch.where(held, small, kc)
    ks[:], vs[:] = 1.0 / 64, 1.0 / 64
    code = int(torch.tensor([nats * 64.0 / 8.0]).to(torch.float8_e4m3fn).view(torch.uint8)[0])  # q . k is about hd, sm_scale 8 / hd
    for r in range(2):
        kc[table[r, 0].long(), :, 0] = code
        vc[table[r, 0].long(), :, 0] = 0
    return args, 8.0 / hd


@pytest.mark.parametrize("max_q,news", ROWS)
@pytest.mark.parametrize("length,hd,dtype", [(200, 64, BF), (2000, 128, BF), (2000, 64, HF)])
@pytest.mark.parametrize("nats", [8, 12, 16])
def test_small_weights_beside_a_dominating_key(max_q, news, length, hd, dtype, nats):
    """Weights down to e^-16 of the largest are held to f16's half step like any other by the kernel of
    few rows; the f16 kernel holds those below 2^-19 of the largest (13 nats) to 2^-30 of it."""
    args, sm_scale = dominated(31, length, news, nats, hd, dtype)
    out, lse = run_attn(args, sm_scale, max_q=max_q)
    want = ref.attn(*args, sm_scale, 0, 0.0)
    assert (want[0][:1].abs() < 0.1).all()
    check_lse(lse, want, f"{nats} nats")
    if max_q == 40 and nats > 12:  # in place of weights, their bound: as if each key's |p v| were 2^11 * 2^-30 |v| larger
        vc, vs, table = args[2], args[4], args[5]
        for r, (n, L) in enumerate(zip(news, (length, 90))):
            ids = table[r, :-(-L // 16)].long()
            v = (ref.E4M3[vc[ids].long()].abs() * vs[ids].double()[..., None, None]).permute(1, 0, 2, 3).reshape(2, -1, hd)[:, :L]
            a = sum(news[:r])
            want[2][a:a + n] += 2.0 ** (11 - 30) * v.sum(1).repeat_interleave(2, 0)[None]
    ref.assert_attn(out, None, want, 0.0, length, f"{nats} nats")


@pytest.mark.parametrize("max_q,news", ROWS)
@pytest.mark.parametrize("spread", [10, 16])
def test_small_value_scales_beside_a_large_one(max_q, news, spread):
    """One page holds an outlier in one channel, so its scale is 2^spread times the others'.  The other
    channels, where it holds zeros, come from the other pages alone and keep f16's half step."""
    args = list(attn_inputs(33, [600, 90], news, 4, 2, 64, 16, BF, qscale=0.25))
    vc, vs, table = args[2], args[4], args[5]
    vs[:] = 2.0 ** -8
    for r, j in ((0, 11), (1, 0)):
        page = table[r, j].long()
        vs[page] = 2.0 ** (spread - 8)
        vc[page] = 0
        vc[page, :, 3, 5] = 0x7E  # 448
    out, lse = run_attn(args, 0.125, max_q=max_q)
    want = ref.attn(*args, 0.125, 0, 0.0)
    check_lse(lse, want, f"spread {spread}")
    ref.assert_attn(out, None, want, 0.0, 600, f"spread {spread}")


@pytest.mark.parametrize("max_q,news", ROWS)
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("exponent", [100, 120])
def test_large_key_scales(max_q, news, cap, exponent):
    """Key scales up to the largest that csa2_kv8_append chooses: scores that fp32 holds are right
    whatever the scale and the query they come from."""
    args = list(attn_inputs(41, [700, 90], news, 4, 2, 64, 16, BF))
    args[0] = (args[0].float() * 2.0 ** (3 - exponent)).to(BF)
    args[3][:] = args[3] * 2.0 ** exponent
    out, lse = run_attn(args, 0.125, cap=cap, max_q=max_q)
    want = ref.attn(*args, 0.125, 0, cap)
    ref.assert_attn(out, lse, want, cap, 700, f"2^{exponent}")


@pytest.mark.parametrize("max_q,news", ROWS)
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_an_infinite_key_is_appended_and_read(max_q, news, cap):
    """csa2_kv8_append stores an infinity as 448 under a scale of 2^120.  Rows that see that key give it
    all their weight or none, or are NaN where its score leaves fp32; other rows and heads are as ever."""
    n, Hk, hd, page, at = news[0], 2, 64, 16, 333
    args = list(attn_inputs(43, [350, 90], news, 4, Hk, hd, page, BF))
    gen = torch.Generator().manual_seed(5)
    x, y = (torch.randn(350, Hk, hd, generator=gen).to(BF) for _ in range(2))
    x[at, 1, 7] = math.inf
    slot = [int(args[5][0, p // page]) * page + p % page for p in range(350)]
    cache = [t.cuda() for t in args[1:5]]
    csa2.csa2_kv8_append(x.cuda(), y.cuda(), torch.tensor(slot).cuda(), *cache)
    args[1:5] = [t.cpu() for t in cache]
    assert (args[3] == 2.0 ** 120).sum() == 1
    args[0][:, :, 7] = torch.where(torch.rand(args[0].shape[:2], generator=gen) < 0.5, 1.5, -1.5).to(BF)
    out, lse = run_attn(args, 0.125, cap=cap, max_q=max_q)
    exact, exact_lse, absum, smax = ref.attn(*args, 0.125, 0, cap)
    rows = ~torch.isnan(exact_lse[:, 0])
    small = torch.where(smax < 2.0 ** 60, smax, torch.full_like(smax, cap + 4.0))  # of the scores that share the weight
    ref.assert_attn(out, None, (exact, exact_lse, absum, small), cap, 350, "an infinite key")
    err = (lse.cpu().double() - exact_lse).abs()[rows]
    assert (err <= 2.0 ** -16 * (exact_lse.abs()[rows] + small[rows] + cap + 1.0)).all()
    big = list(args)
    big[0] = args[0].clone()
    big[0][:n] = args[0][:n] * 2.0 ** 7                   # the infinite key's scores leave fp32
    out, lse = run_attn(big, 0.125, cap=cap, max_q=max_q)
    exact, exact_lse, absum, smax = ref.attn(*big, 0.125, 0, cap)
    if not cap:
        sees = torch.zeros(out.shape[:2], dtype=torch.bool)
        sees[:n, 2:] = (350 - n + torch.arange(n) >= at)[:, None] & (big[0][:n, 2:, 7] > 0)
        assert sees.any() and torch.isnan(out.cpu()[sees]).all() and torch.isnan(lse.cpu()[sees]).all()
        exact_lse[sees] = math.nan
        finite = ~torch.isnan(exact_lse)
        assert not torch.isnan(out.cpu()[finite]).any() and not torch.isnan(lse.cpu()[finite]).any()
        exact, absum = (torch.where(finite[..., None], t, torch.zeros_like(t)) for t in (exact, absum))
        out = torch.where(finite[..., None], out.cpu(), torch.zeros_like(out.cpu()))
        exact_lse[~finite] = 0.0
        exact_lse[n + news[1]:] = math.nan
    small = torch.where(smax < 2.0 ** 60, smax, torch.full_like(smax, 2.0 ** 10))
    ref.assert_attn(out, None, (exact, exact_lse, absum, small), cap, 350, "scores past fp32")
