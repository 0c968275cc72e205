"""Plan, append, attention and release together, as a server runs them: steps of a growing and
shrinking batch, run directly and from one captured graph, against a plain cache in float64."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as ref
from sparse_attention_fp4_pack_b200 import csa2

pytestmark = pytest.mark.gpu
I32, I64, BF = torch.int32, torch.int64, torch.bfloat16


class Server:
    """One layer's cache and the buffers of a step; `rows` is the most a step may bring."""

    def __init__(self, R, Hq, Hk, hd, page, pages, cols, rows, window=0, cap=0.0):
        full = lambda *s, dtype=I32, v=0: torch.full(s, v, dtype=dtype, device="cuda")
        self.R, self.Hq, self.Hk, self.hd, self.page, self.pages, self.window, self.cap = R, Hq, Hk, hd, page, pages, window, cap
        self.ctx, self.new, self.gone = full(R), full(R), full(R, dtype=torch.uint8)
        self.table, self.free, self.n_free = full(R, cols, v=-1), torch.randperm(pages).to(I32).cuda(), full(1, v=pages)
        self.q_start, self.slot, self.pos = full(R + 1), full(rows, dtype=I64), full(rows, dtype=I64)
        self.seq = full(R)
        self.kc, self.vc = (full(pages, Hk, page, hd, dtype=torch.uint8, v=0x7F) for _ in range(2))
        self.ks, self.vs = (full(pages, Hk, dtype=torch.float32, v=1) for _ in range(2))
        self.q, self.k, self.v = (full(rows, h, hd, dtype=BF) for h in (Hq, Hk, Hk))
        self.out, self.lse = full(rows, Hq, hd, dtype=BF), full(rows, Hq, dtype=torch.float32)
        self.status = csa2.status_word()

    def step(self, max_q, ws):
        csa2.csa2_paged_release(self.ctx, self.table, self.gone, self.free, self.n_free, self.page, self.pages, self.ctx,
                                self.n_free, dev_status=self.status)
        csa2.csa2_paged_plan(self.ctx, self.new, self.table, self.free, self.n_free, self.page, self.pages, self.seq,
                             self.n_free, self.q_start, self.slot, self.pos, dev_status=self.status)
        csa2.csa2_kv8_append(self.k, self.v, self.slot, self.kc, self.vc, self.ks, self.vs, dev_status=self.status)
        csa2.csa2_kv8_attn(self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.q_start, self.seq,
                           1 / math.sqrt(self.hd), self.out, self.lse, max_q=max_q, window=self.window, softcap=self.cap,
                           ws=ws, dev_status=self.status)
        self.ctx.copy_(self.seq)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("Hq,Hk,hd,page,max_q,window,cap", [(4, 2, 64, 16, 1, 0, 0.0), (8, 1, 128, 32, 12, 70, 15.0)])
def test_steps(captured, Hq, Hk, hd, page, max_q, window, cap):
    R, rows, steps = 6, 60, 8
    rng = np.random.default_rng(page)
    torch.manual_seed(page)
    s = Server(R, Hq, Hk, hd, page, 40, 8, rows, window, cap)
    ws = csa2.workspace(csa2.csa2_kv8_attn_workspace_size(Hq, Hk, hd, max_q, BF))
    if captured:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):   # new = 0: a step that does nothing
            s.step(max_q, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step(max_q, ws)
    # the plain side: pages, codes and scales kept on the host
    kc, vc, ks, vs = s.kc.cpu(), s.vc.cpu(), s.ks.cpu(), s.vs.cpu()
    ctx, table, free, n_free = np.zeros(R, np.int32), s.table.cpu().numpy(), s.free.cpu().numpy(), 40
    for step in range(steps):
        gone = (rng.integers(0, 4, R) == 0).astype(np.uint8) if step else np.zeros(R, np.uint8)
        new = rng.integers(0, max_q + 1, R).astype(np.int32)
        if step < 2:
            new[step] = max_q
        s.gone.copy_(torch.from_numpy(gone))
        s.new.copy_(torch.from_numpy(new))
        for t in (s.q, s.k, s.v):
            t.copy_(torch.randn_like(t, dtype=torch.float32) * 2.0 ** (step % 3))
        s.out.fill_(7.0)
        s.lse.fill_(7.0)
        if captured:
            g.replay()
        else:
            s.step(max_q, ws)
        torch.cuda.synchronize()
        assert int(s.status) == 0
        free, n_free, ctx, flags = ref.release(ctx, table, gone, free, n_free, page, 40)
        assert not any(flags)
        plan, flags = ref.plan(ctx, new, table, free, n_free, page, 40, rows)
        assert not any(flags)
        table, n_free, ctx = plan["table"], plan["n_free"], plan["seq_len"]
        assert np.array_equal(s.free.cpu().numpy(), free) and int(s.n_free) == n_free
        assert np.array_equal(s.seq.cpu().numpy(), ctx) and np.array_equal(s.q_start.cpu().numpy(), plan["q_start"])
        assert np.array_equal(s.slot.cpu().numpy(), plan["slot"]) and np.array_equal(s.pos.cpu().numpy(), plan["pos"])
        for r in range(R):
            n = -(-int(ctx[r]) // page)
            assert np.array_equal(s.table.cpu().numpy()[r, :n], table[r, :n])
        ref.append(s.k.cpu(), plan["slot"], kc, ks)
        ref.append(s.v.cpu(), plan["slot"], vc, vs)
        for got, want in ((s.kc, kc), (s.vc, vc), (s.ks, ks), (s.vs, vs)):
            assert torch.equal(got.cpu(), want)
        want = ref.attn(s.q.cpu(), kc, vc, ks, vs, torch.from_numpy(table), plan["q_start"], ctx, 1 / math.sqrt(hd), window, cap)
        ref.assert_attn(s.out, s.lse, want, cap, int(ctx.max()), f"step {step}")
        T = int(plan["q_start"][-1])
        assert (s.out[T:] == 7.0).all() and (s.lse[T:] == 7.0).all()


def test_two_graphs_share_a_workspace():
    """Graphs of different shapes captured over one workspace, replayed in turn on one stream."""
    torch.manual_seed(0)
    servers, graphs, wants = [], [], []
    size = max(csa2.csa2_kv8_attn_workspace_size(8, 2, 64, q, BF) for q in (1, 10))
    ws = csa2.workspace(size)
    for max_q in (1, 10):
        s = Server(5, 8, 2, 64, 16, 2000, 300, 50)
        s.new.copy_(torch.tensor([4000 + 50 * i for i in range(5)]))
        s.k, s.v, s.slot, s.pos = (torch.randn(21000, 2, 64, device="cuda").to(BF), torch.randn(21000, 2, 64, device="cuda").to(BF),
                                   torch.zeros(21000, dtype=I64, device="cuda"), torch.zeros(21000, dtype=I64, device="cuda"))
        s.q, s.out, s.lse = (torch.randn(21000, 8, 64, device="cuda").to(BF), torch.zeros(21000, 8, 64, dtype=BF, device="cuda"),
                             torch.zeros(21000, 8, device="cuda"))
        s.step(10, csa2.workspace(size))              # a long prompt each
        s.new.fill_(max_q)
        n = 5 * max_q
        s.k, s.v, s.q, s.slot, s.pos, s.out, s.lse = (t[:n].contiguous() for t in (s.k, s.v, s.q, s.slot, s.pos, s.out, s.lse))
        s.ctx.copy_(s.seq)
        state = [t.clone() for t in (s.ctx, s.table, s.free, s.n_free, s.kc, s.vc, s.ks, s.vs)]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            s.step(max_q, ws)
        s.step(max_q, csa2.workspace(size))           # the same step outside the graph
        torch.cuda.synchronize()
        wants.append((s.out.clone(), s.lse.clone(), s.kc.clone()))
        servers.append((s, state))
        graphs.append(g)
    for _ in range(4):
        for (s, state), g, want in zip(servers, graphs, wants):
            for t, old in zip((s.ctx, s.table, s.free, s.n_free, s.kc, s.vc, s.ks, s.vs), state):
                t.copy_(old)
            s.out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for (s, _), want in zip(servers, wants):
            assert torch.equal(s.out, want[0]) and torch.equal(s.lse, want[1]) and torch.equal(s.kc, want[2])
            assert int(s.status) == 0


def test_empty_calls():
    s = Server(3, 4, 2, 64, 16, 5, 2, 4)
    ws = csa2.workspace(csa2.csa2_kv8_attn_workspace_size(4, 2, 64, 1, BF))
    s.out.fill_(7.0)
    s.step(1, ws)                                    # requests without tokens
    assert int(s.status) == 0 and (s.out == 7.0).all() and (s.slot == -1).all() and int(s.n_free) == 5
    e = Server(0, 4, 2, 64, 16, 5, 2, 4)             # no requests
    e.step(1, ws)
    assert int(e.status) == 0 and (e.slot == -1).all() and e.q_start.tolist() == [0]


def test_binding_refuses_on_the_device():
    s = Server(3, 4, 2, 64, 16, 5, 2, 4)
    with pytest.raises(ValueError, match="device"):
        csa2.csa2_kv8_append(s.k, s.v, s.slot.cpu(), s.kc, s.vc, s.ks, s.vs)
    with pytest.raises(ValueError, match="ws"):
        csa2.csa2_kv8_attn(s.q, s.kc, s.vc, s.ks, s.vs, s.table, s.q_start, s.seq, 0.1, s.out, ws=torch.zeros(9))
    with pytest.raises(csa2.CSA2Error):
        csa2.csa2_kv8_attn(s.q, s.kc, s.vc, s.ks, s.vs, s.table, s.q_start, s.seq, 0.1, s.out, ws=csa2.workspace(512))
    with pytest.raises(csa2.CSA2Error):
        csa2.csa2_kv8_attn(s.q, s.kc, s.vc, s.ks, s.vs, s.table, s.q_start, s.seq, 0.1, s.out, max_q=0)
    with pytest.raises(csa2.CSA2Error):
        csa2.csa2_paged_plan(s.ctx, s.new, s.table, s.free, s.n_free, 20, 5, s.seq, s.n_free, s.q_start, s.slot, s.pos)


def test_append_skipped_rows_inside_a_page():
    """A -1 row (or one beyond the pool) between two rows of a page: what follows is refused; -1 rows between pages, at the
    start and at the end are fine."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(40, 2, 64, generator=gen).to(BF)
    slot = [-1, -1] + list(range(16, 22)) + [-1, 999] + list(range(24, 28)) + [-1] * 20 + list(range(48, 52)) + [-1, -1]
    slot += [-1] * (40 - len(slot))
    want = list(slot)
    for i, s in enumerate(slot):
        if 24 <= s < 28 or s == 999:
            want[i] = -1
    kc, vc = (torch.randint(0, 126, (5, 2, 16, 64), generator=gen, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.ones(5, 2) for _ in range(2))
    got = [t.cuda() for t in (kc, vc, ks, vs)]
    st = csa2.status_word()
    csa2.csa2_kv8_append(x.cuda(), x.cuda(), torch.tensor(slot).cuda(), *got, dev_status=st)
    assert int(st) == csa2.DEV_BAD_INDEX
    ref.append(x, want, kc, ks)
    ref.append(x, want, vc, vs)
    for a, b in zip(got, (kc, vc, ks, vs)):
        assert torch.equal(a.cpu(), b)
    st = csa2.status_word()                      # the same without the second run: nothing to flag
    csa2.csa2_kv8_append(x.cuda(), x.cuda(), torch.tensor(want).cuda(), *got, dev_status=st)
    assert int(st) == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_long_gaps_inside_a_page(page):
    """The rows behind a gap inside their page are refused however long the gap is; behind the same
    gap the rows of another page are written."""
    gen = torch.Generator().manual_seed(page)
    for gap in (1, 2, page - 2, page - 1, page, page + 1, page + 2, 3 * page, 1000):
        run = [3 * page + i for i in range(4)]
        skipped = [-1] * gap
        skipped[gap // 2] = 7 * page if gap % 2 else -1          # beyond the pool in some
        slot = [-1] + run + skipped + [s + 6 for s in run] + [-1] * gap + [s + 10 for s in run] + [page, page + 1]
        slot += skipped + [5 * page, 5 * page + 1]
        keep = list(slot)
        for i, s in enumerate(slot):
            if s == 7 * page or 3 * page + 6 <= s < 4 * page:
                keep[i] = -1
        x, y = (torch.randn(len(slot), 1, 64, generator=gen).to(BF) for _ in range(2))
        kc, vc = (torch.randint(0, 126, (7, 1, page, 64), generator=gen, dtype=torch.uint8) for _ in range(2))
        ks, vs = (torch.full((7, 1), 2.0 ** -12) for _ in range(2))
        got = [t.cuda() for t in (kc, vc, ks, vs)]
        for again in range(3):
            st = csa2.status_word()
            csa2.csa2_kv8_append(x.cuda(), y.cuda(), torch.tensor(slot).cuda(), *got, dev_status=st)
            assert int(st) == csa2.DEV_BAD_INDEX
            ref.append(x, keep, kc, ks)
            ref.append(y, keep, vc, vs)
            for a, b in zip(got, (kc, vc, ks, vs)):
                assert torch.equal(a.cpu(), b), gap
