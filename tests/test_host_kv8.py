"""The paged 8-bit KV cache without a GPU: what the C entry points and the binding refuse, and the
plain implementations the GPU tests compare with, held against their own definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv8_ref as ref
from sparse_attention_fp4_pack_b200 import build as libbuild
from sparse_attention_fp4_pack_b200 import csa2

P = ctypes.c_void_p
FAKE, MIS4, MIS2 = P(0x10000), P(0x10004), P(0x10002)   # never dereferenced: refused before any launch
INVALID, UNSUPPORTED, OK = 1, 2, 0


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return csa2.lib()


def call(fn, base, **kw):
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    return fn(*args.values())


PLAN = dict(ctx=FAKE, new=FAKE, R=3, page=16, table=FAKE, max_pages=4, free=FAKE, cap=9, n_free=FAKE, n_pages=20,
            seq=FAKE, n_out=FAKE, q_start=FAKE, slot=FAKE, pos=FAKE, T=7, status=None, stream=None)


def test_plan_refuses(L):
    f = L.csa2_paged_plan
    for page in (0, 8, 17, 48, 256, -16):
        assert call(f, PLAN, page=page) == UNSUPPORTED
    for kw in (dict(R=-1), dict(max_pages=0), dict(n_pages=-1), dict(cap=-1), dict(T=-1)):
        assert call(f, PLAN, **kw) == INVALID
    for kw in (dict(max_pages=(1 << 30) // 16 + 1), dict(n_pages=1 << 31), dict(cap=1 << 31), dict(T=1 << 31)):
        assert call(f, PLAN, **kw) == UNSUPPORTED
    for name in ("ctx", "new", "table", "free", "n_free", "seq", "n_out", "q_start", "slot", "pos"):
        assert call(f, PLAN, **{name: None}) == INVALID, name
        assert call(f, PLAN, **{name: MIS2}) == INVALID, name
    for name in ("slot", "pos"):
        assert call(f, PLAN, **{name: MIS4}) == INVALID, name
    assert call(f, PLAN, status=MIS2) == INVALID


RELEASE = dict(seq=FAKE, table=FAKE, gone=FAKE, R=3, page=16, max_pages=4, free=FAKE, cap=9, n_free=FAKE, n_pages=20,
               seq_out=FAKE, n_out=FAKE, status=None, stream=None)


def test_release_refuses(L):
    f = L.csa2_paged_release
    assert call(f, RELEASE, page=24) == UNSUPPORTED
    for kw in (dict(R=-1), dict(max_pages=0), dict(n_pages=-1), dict(cap=-1)):
        assert call(f, RELEASE, **kw) == INVALID
    assert call(f, RELEASE, cap=1 << 31) == UNSUPPORTED
    for name in ("seq", "table", "free", "n_free", "seq_out", "n_out"):
        assert call(f, RELEASE, **{name: None}) == INVALID, name
        assert call(f, RELEASE, **{name: MIS2}) == INVALID, name
    assert call(f, RELEASE, gone=None) == INVALID


APPEND = dict(k=FAKE, v=FAKE, ks=0, vs=0, dtype=0, T=5, Hk=2, hd=128, slot=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE,
              n_pages=20, page=16, status=None, stream=None)


def test_append_refuses(L):
    f = L.csa2_kv8_append
    for kw in (dict(hd=96), dict(hd=0), dict(page=1), dict(dtype=2), dict(dtype=-1), dict(n_pages=1 << 31),
               dict(n_pages=1 << 26), dict(T=1 << 31)):
        assert call(f, APPEND, **kw) == UNSUPPORTED, kw
    for kw in (dict(Hk=0), dict(n_pages=0), dict(T=-1), dict(ks=255), dict(vs=260), dict(ks=-8)):
        assert call(f, APPEND, **kw) == INVALID, kw
    for name in ("k", "v", "slot", "kc", "vc", "ksc", "vsc"):
        assert call(f, APPEND, **{name: None}) == INVALID, name
        assert call(f, APPEND, **{name: MIS2}) == INVALID, name
    for name in ("k", "v", "slot", "kc", "vc"):
        assert call(f, APPEND, **{name: MIS4}) == INVALID, name
    assert call(f, APPEND, T=0, k=None, v=None, slot=None) == OK


ATTN = dict(q=FAKE, qs=0, dtype=0, T=5, Hq=8, Hk=2, hd=128, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, n_pages=20, page=16,
            table=FAKE, max_pages=4, q_start=FAKE, seq=FAKE, R=3, max_q=1, scale=0.1, window=0, cap=0.0, out=FAKE,
            lse=None, ws=FAKE, ws_bytes=1 << 40, status=None, stream=None)


def test_attn_refuses(L):
    f = L.csa2_kv8_attn
    for kw in (dict(hd=256), dict(page=129), dict(dtype=3), dict(T=1 << 31), dict(max_pages=1 << 27)):
        assert call(f, ATTN, **kw) == UNSUPPORTED, kw
    for kw in (dict(Hq=7), dict(Hq=1), dict(Hk=0), dict(T=-1), dict(R=-1), dict(max_q=0), dict(window=-1), dict(qs=4),
               dict(qs=1020), dict(scale=math.nan), dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.nan),
               dict(cap=1e-30), dict(cap=3e38), dict(cap=math.inf),
               dict(n_pages=0), dict(ws_bytes=1024), dict(ws=None), dict(ws=P(0x10080))):
        assert call(f, ATTN, **kw) == INVALID, kw
    for name in ("q", "kc", "vc", "ks", "vs", "table", "q_start", "seq", "out"):
        assert call(f, ATTN, **{name: None}) == INVALID, name
        assert call(f, ATTN, **{name: MIS2}) == INVALID, name
    assert call(f, ATTN, lse=MIS2) == INVALID
    assert call(f, ATTN, T=0, q=None, out=None) == OK
    assert call(f, ATTN, R=0, table=None, q_start=None, seq=None) == OK
    for hd in (64, 128):  # the workspace grows with the tile's columns, and is 0 for shapes that are refused
        a, b, c = (L.csa2_kv8_attn_workspace_size(16, 2, hd, n, 0) for n in (1, 2, 3))
        assert 0 < a < b < c and a % 256 == b % 256 == c % 256 == 0
    assert L.csa2_kv8_attn_workspace_size(15, 2, 128, 1, 0) == 0
    assert L.csa2_kv8_attn_workspace_size(16, 2, 96, 1, 0) == 0


def test_no_pages_maps_to_a_device_input_error(L):
    assert L.csa2_status_from_device_word(csa2.DEV_NO_PAGES) == 5
    assert L.csa2_status_from_device_word(csa2.DEV_NO_PAGES | csa2.DEV_TIMEOUT) == 4


def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def refused(fn, base, match, err=ValueError, **kw):
    with pytest.raises(err, match=match):
        fn(**{**base, **kw})


def test_binding_names_the_wrong_argument():
    """As the other calls: sizes and types are checked before the device, so host tensors of the
    right shapes fail only there."""
    i64, u8, f32, bf, hf = torch.int64, torch.uint8, torch.float32, torch.bfloat16, torch.float16
    plan = dict(ctx_len=z(3), new_len=z(3), block_table=z(3, 4), free_pages=z(9), n_free=z(1), page=16, n_pages=20,
                seq_len=z(3), n_free_out=z(1), q_start=z(4), slot_map=z(7, dtype=i64), pos=z(7, dtype=i64))
    rel = dict(seq_len=z(3), block_table=z(3, 4), release=z(3, dtype=u8), free_pages=z(9), n_free=z(1), page=16,
               n_pages=20, seq_len_out=z(3), n_free_out=z(1))
    cache = dict(k_cache=z(20, 2, 16, 64, dtype=u8), v_cache=z(20, 2, 16, 64, dtype=u8), k_scale=z(20, 2, dtype=f32),
                 v_scale=z(20, 2, dtype=f32))
    app = dict(k=z(5, 2, 64, dtype=bf), v=z(5, 2, 64, dtype=bf), slot_map=z(5, dtype=i64), **cache)
    att = dict(q=z(5, 8, 64, dtype=hf), **cache, block_table=z(3, 4), q_start=z(4), seq_len=z(3), sm_scale=0.1,
               out=z(5, 8, 64, dtype=hf), lse=z(5, 8, dtype=f32))
    for fn, base in ((csa2.csa2_paged_plan, plan), (csa2.csa2_paged_release, rel), (csa2.csa2_kv8_append, app),
                     (csa2.csa2_kv8_attn, att)):
        refused(fn, base, "CUDA")
        for name, t in base.items():
            if not torch.is_tensor(t) or name in ("ctx_len", "seq_len", "k_cache"):
                continue
            if name in ("free_pages", "slot_map") and fn is not csa2.csa2_kv8_append:
                wrong = t.unsqueeze(0)  # any length is one
            else:
                wrong = torch.zeros([n + 1 for n in t.shape], dtype=t.dtype)
            refused(fn, base, "must" if name in ("slot_map", "q") else rf"^{name}\b", **{name: wrong})
            refused(fn, base, f"^{name}", TypeError, **{name: t.to(torch.float64)})
    refused(csa2.csa2_kv8_append, app, "^k:", k=z(5, 2, 128, dtype=bf)[:, :, ::2])
    refused(csa2.csa2_kv8_append, app, "^v:", v=z(5, 132, dtype=bf)[:, :128].view(5, 2, 64))
    refused(csa2.csa2_kv8_append, app, "^v", TypeError, v=app["v"].to(hf))
    refused(csa2.csa2_kv8_append, app, "^k_cache", k_cache=z(20, 2, 16, 128, dtype=u8)[..., ::2])
    refused(csa2.csa2_kv8_attn, att, "^out", TypeError, out=att["out"].to(bf))
    refused(csa2.csa2_kv8_attn, att, "^q", q=z(5, 8, 128, dtype=hf))
    refused(csa2.csa2_paged_plan, plan, "^block_table", block_table=z(4, 3).T)
    # tensors without storage or strides end in an exception too
    for wrong in (z(3).to_sparse(), z(3, 4).to_sparse(), torch.zeros(3, dtype=torch.int32, device="meta")):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            csa2.csa2_paged_plan(**{**plan, "new_len": wrong})
    with pytest.raises((ValueError, TypeError, AttributeError)):
        csa2.csa2_paged_plan(**{**plan, "new_len": [1, 2, 3]})


def test_plain_plan_and_release_keep_every_page_once():
    """Plan, release, plan again: no page is held twice, none is lost."""
    rng = np.random.default_rng(0)
    R, page, P_, cols = 12, 16, 60, 9
    table = np.full((R, cols), -1, np.int32)
    free, n_free, ctx = rng.permutation(P_).astype(np.int32), P_, np.zeros(R, np.int32)
    for step in range(30):
        new = np.minimum(rng.integers(0, 20, R), cols * page - ctx).astype(np.int32)
        out, flags = ref.plan(ctx, new, table, free, n_free, page, P_, 400)
        if flags[2]:  # out of pages: release a third and go on without this step
            gone = (rng.integers(0, 3, R) == 0).astype(np.uint8)
            free, n_free, ctx, f2 = ref.release(ctx, table, gone, free, n_free, page, P_)
            assert not any(f2)
            continue
        assert not any(flags)
        table, n_free, ctx = out["table"], out["n_free"], out["seq_len"]
        held = [int(p) for r in range(R) for p in table[r, :-(-int(ctx[r]) // page)]]
        assert sorted(held + [int(p) for p in free[:n_free]]) == list(range(P_))
        assert len(set(out["slot"][:out["q_start"][-1]].tolist())) == out["q_start"][-1]


def test_plain_append_error_is_half_a_step():
    """What the cache holds is within half an E4M3 step (2^-4 of the value, half a subnormal step
    2^-10 of the scale) of what was appended; appends that re-scale a page move an earlier value
    by half a subnormal step of each new scale at most."""
    gen = torch.Generator().manual_seed(3)
    cache, scale = torch.zeros(2, 2, 16, 64, dtype=torch.uint8), torch.ones(2, 2)
    x = torch.randn(16, 2, 64, generator=gen).to(torch.float16) * torch.logspace(-2, 2, 16)[:, None, None].to(torch.float16)
    for a, b in ((0, 3), (3, 4), (4, 11), (11, 16)):
        ref.append(x[a:b], list(range(16 + a, 16 + b)), cache, scale)
    got = (ref.E4M3[cache[1].long()] * scale[1].to(torch.float64)[:, None, None]).permute(1, 0, 2)
    want = x.to(torch.float64)
    slack = 4 * 2.0 ** -10 * scale[1].to(torch.float64)[None, :, None]
    assert ((got - want).abs() <= want.abs() * 2.0 ** -4 + slack).all()


def test_binding_refuses_integers_that_do_not_fit():
    """A window, page or count past the C type's range is refused, not cut to its lower bits."""
    i64, u8, f32, bf = torch.int64, torch.uint8, torch.float32, torch.bfloat16
    plan = dict(ctx_len=z(3), new_len=z(3), block_table=z(3, 4), free_pages=z(9), n_free=z(1), page=16, n_pages=20,
                seq_len=z(3), n_free_out=z(1), q_start=z(4), slot_map=z(7, dtype=i64), pos=z(7, dtype=i64))
    rel = dict(seq_len=z(3), block_table=z(3, 4), release=z(3, dtype=u8), free_pages=z(9), n_free=z(1), page=16,
               n_pages=20, seq_len_out=z(3), n_free_out=z(1))
    cache = dict(k_cache=z(20, 2, 16, 64, dtype=u8), v_cache=z(20, 2, 16, 64, dtype=u8), k_scale=z(20, 2, dtype=f32),
                 v_scale=z(20, 2, dtype=f32))
    att = dict(q=z(5, 8, 64, dtype=bf), **cache, block_table=z(3, 4), q_start=z(4), seq_len=z(3), sm_scale=0.1,
               out=z(5, 8, 64, dtype=bf), lse=z(5, 8, dtype=f32))
    for fn, base in ((csa2.csa2_paged_plan, plan), (csa2.csa2_paged_release, rel)):
        refused(fn, base, "^page", page=(1 << 32) + 16)
        refused(fn, base, "^n_pages", n_pages=(1 << 64) + 20)
        refused(fn, base, "CUDA", page=np.int64(16))
        refused(fn, base, "", TypeError, page=16.0)
    for wide in ((1 << 32) + 5, 1 << 31, -(1 << 33)):
        refused(csa2.csa2_kv8_attn, att, "^window", window=wide)
        refused(csa2.csa2_kv8_attn, att, "^max_q", max_q=wide)
        with pytest.raises(ValueError, match="^max_q"):
            csa2.csa2_kv8_attn_workspace_size(8, 2, 64, wide)
    refused(csa2.csa2_kv8_attn, att, "", TypeError, window=1.5)


def test_binding_is_rebuilt_for_another_torch_or_python(L, monkeypatch, tmp_path):
    """_native.so goes by the torch and Python it was built for, not by file times alone."""
    libbuild.build_native()
    assert libbuild.native_up_to_date()
    monkeypatch.setattr(libbuild.importlib.metadata, "version", lambda name: "0.0.1")
    assert not libbuild.native_up_to_date()
    monkeypatch.undo()
    assert libbuild.native_up_to_date()
    monkeypatch.setattr(libbuild, "NATIVE_FOR", str(tmp_path / "none"))
    assert not libbuild.native_up_to_date()
