"""The two sets of argument checks of the paged 8-bit KV cache, in C++ (calls on the current stream) and
in Python (calls on a given stream, and the wording of every refusal): the same calls pass, the same
are refused, and by the same exception."""
import pytest
import torch

from sparse_attention_fp4_pack_b200 import csa2

pytestmark = pytest.mark.gpu
I32, I64, U8, F32, BF, HF = torch.int32, torch.int64, torch.uint8, torch.float32, torch.bfloat16, torch.float16


def z(*shape, dtype=I32, device="cuda"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def calls():
    cache = lambda: dict(k_cache=z(20, 2, 16, 64, dtype=U8), v_cache=z(20, 2, 16, 64, dtype=U8),
                         k_scale=z(20, 2, dtype=F32), v_scale=z(20, 2, dtype=F32))
    yield csa2.csa2_paged_plan, dict(ctx_len=z(3), new_len=z(3), block_table=z(3, 4), free_pages=z(9), n_free=z(1), page=16,
                                     n_pages=20, seq_len=z(3), n_free_out=z(1), q_start=z(4), slot_map=z(7, dtype=I64),
                                     pos=z(7, dtype=I64), dev_status=z(1))
    yield csa2.csa2_paged_release, dict(seq_len=z(3), block_table=z(3, 4), release=z(3, dtype=U8), free_pages=z(9), n_free=z(1),
                                        page=16, n_pages=20, seq_len_out=z(3), n_free_out=z(1), dev_status=z(1))
    yield csa2.csa2_kv8_append, dict(k=z(5, 2, 64, dtype=BF), v=z(5, 2, 64, dtype=BF), slot_map=z(5, dtype=I64) - 1, **cache(),
                                     dev_status=z(1))
    yield csa2.csa2_kv8_attn, dict(q=z(5, 8, 64, dtype=HF), **cache(), block_table=z(3, 4), q_start=z(4), seq_len=z(3),
                                   sm_scale=0.1, out=z(5, 8, 64, dtype=HF), lse=z(5, 8, dtype=F32), max_q=1, window=0,
                                   softcap=0.0, ws=csa2.workspace(csa2.csa2_kv8_attn_workspace_size(8, 2, 64, 1, HF)),
                                   dev_status=z(1))


def variants(name, x):
    """Other values of one argument: some are fine, most are not."""
    if not torch.is_tensor(x):
        yield from (None, "16", True, x, -1, 0, 1, 7, 1 << 20, 1 << 31, (1 << 32) + 16, 1 << 70, 1.5, float("nan"), float("inf"), -2.0)
        return
    yield None
    yield [1, 2, 3]
    yield x
    yield x.cpu()
    yield x.to(torch.float64)
    yield x.to(torch.int16)
    yield x.unsqueeze(0)
    yield x.reshape(-1)
    yield x[:0]
    yield x[1:]
    yield x.clone().requires_grad_() if x.is_floating_point() else x.clone()
    yield torch.empty(x.shape, dtype=x.dtype, device="meta")
    yield x.flatten()[:1].expand(x.shape)
    yield torch.cat([x, x[:1]])
    wide = torch.zeros(*x.shape, 2, dtype=x.dtype, device="cuda")
    yield wide[..., 0]                                                  # every dimension strided
    if x.dim() == 3:
        yield torch.zeros(x.shape[0], x.shape[1] + 3, x.shape[2], dtype=x.dtype, device="cuda")[:, 1:1 + x.shape[1]]   # tokens strided
        yield torch.zeros(x.shape[0], x.shape[1] * x.shape[2] + 4, dtype=x.dtype, device="cuda")[:, :-4].view(x.shape)  # by 4 more
        yield x.transpose(0, 1).contiguous().transpose(0, 1)            # heads first
        yield x.flip(0).contiguous().expand_as(x)
    raw = torch.zeros(x.numel() * x.element_size() + 64, dtype=U8, device="cuda")
    for by in (2, 4, 8):                                                # aligned to less than the call wants
        if by % x.element_size() == 0:
            yield raw[by:by + x.numel() * x.element_size()].view(x.dtype).view(x.shape)


def outcome(fn, args, stream):
    try:
        fn(**args, stream=stream)
    except Exception as e:
        return type(e)
    torch.cuda.synchronize()
    return None


def test_both_sets_of_checks_agree():
    fine = refused = 0
    for fn, base in calls():
        assert outcome(fn, base, None) is None and outcome(fn, base, torch.cuda.current_stream()) is None
        for name, x in base.items():
            for i, other in enumerate(variants(name, x)):
                args = {**base, name: other}
                fast, slow = outcome(fn, args, None), outcome(fn, args, torch.cuda.current_stream())
                assert fast == slow, f"{fn.__name__}({name}= variant {i}): {fast} on the current stream, {slow} on a given one"
                fine, refused = fine + (fast is None), refused + (fast is not None)
    assert fine > 40 and refused > 300
    assert torch.ones(3, device="cuda").sum() == 3                      # nothing was refused by a fault


def test_all_the_same_arguments_pass_through_both():
    """One that is left out, and several at once in place: the calls' documented aliases."""
    for stream in (None, torch.cuda.current_stream()):
        for fn, base in calls():
            for name in ("dev_status", "lse", "ws"):
                if name in base:
                    assert outcome(fn, {**base, name: None}, stream) is None
            if "ctx_len" in base:
                assert outcome(fn, {**base, "seq_len": base["ctx_len"], "n_free_out": base["n_free"]}, stream) is None
                assert outcome(fn, {**base, "seq_len": base["new_len"]}, stream) is csa2.CSA2Error
            if "release" in base:
                assert outcome(fn, {**base, "seq_len_out": base["seq_len"], "n_free_out": base["n_free"]}, stream) is None
