"""Thin ctypes binding of libcsa2 (C ABI in include/csa2.h).

Argument marshalling only: every function checks that its tensors' shapes agree with the
sizes it passes (the C entry points take sizes and cannot see a buffer's extent, so a
smaller buffer would be accessed out of bounds), then their devices, dtypes and layout,
passes raw device pointers and the current CUDA stream to the C entry point of the same
name, and raises CSA2Error on a non-OK status (the paged 8-bit cache's calls do the same in
_native, csrc/binding.cpp).  All compute runs in libcsa2's kernels; there
is no other code path.  Workspaces are plain uint8 device tensors from torch's
allocator (``workspace``).
"""
import ctypes
import functools
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2.so")

CSA2_OK = 0
STATUS_NAMES = {0: "CSA2_OK", 1: "CSA2_ERR_INVALID_ARG", 2: "CSA2_ERR_UNSUPPORTED", 3: "CSA2_ERR_CUDA",
                4: "CSA2_ERR_TIMEOUT", 5: "CSA2_ERR_DEVICE_INPUT"}
DEV_BAD_INDEX, DEV_BAD_COUNT, DEV_TIMEOUT, DEV_NO_PAGES = 0x1, 0x2, 0x4, 0x8

D, DI, KV_BYTES, IK_BYTES = 512, 128, 288, 68

_lib = None


class CSA2Error(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")


def lib():
    """Load libcsa2.so (raises if it was not built: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        L.csa2_status_string.restype = ctypes.c_char_p
        L.csa2_status_string.argtypes = [I32]
        L.csa2_status_from_device_word.restype = I32
        L.csa2_status_from_device_word.argtypes = [ctypes.c_uint32]
        L.csa2_version.restype = I32
        L.csa2_pack_kv.restype = I32
        L.csa2_pack_kv.argtypes = [P, P, I64, I32, P, I64, P, P, P, P]
        L.csa2_pack_kv_normed.restype = I32
        L.csa2_pack_kv_normed.argtypes = [P, P, I64, I32, P, P, P, I64, P, F32, P, I64, P, P, P, P]
        L.csa2_index_full_workspace_size.restype = SZ
        L.csa2_index_full_workspace_size.argtypes = [I32, I32, I32, I32, I64]
        L.csa2_index_full.restype = I32
        L.csa2_index_full.argtypes = [P, P, P, I64, P, P, I32, I32, I32, I32, I64, P, P, P, SZ, P, P]
        L.csa2_test_index_full_withheld_copy.restype = I32
        L.csa2_test_index_full_withheld_copy.argtypes = [P, P, P, I64, P, P, I32, I32, I32, I32, I64, P, P, P, SZ,
                                                         P, P, I32]
        L.csa2_index_hier_workspace_size.restype = SZ
        L.csa2_index_hier_workspace_size.argtypes = [I32, I32, I32, I32, I32, I64]
        L.csa2_index_hier.restype = I32
        L.csa2_index_hier.argtypes = [P, P, P, I64, P, P, I32, I32, I32, I32, I32, I64, P, P, P, SZ, P, P]
        L.csa2_reindex_workspace_size.restype = SZ
        L.csa2_reindex_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32]
        L.csa2_reindex.restype = I32
        L.csa2_reindex.argtypes = [P, P, P, I64, P, P, P, I32, I32, I32, I32, I32, I32, P, P, P, SZ, P, P]
        L.csa2_static_scratch_bytes.restype = SZ
        L.csa2_static_scratch_bytes.argtypes = []
        L.csa2_reindex_static.restype = I32
        L.csa2_reindex_static.argtypes = [P, P, P, I64, P, P, P, I32, I32, I32, I32, I32, I32, P, P, P, P]
        L.csa2_sparse_attn_workspace_size.restype = SZ
        L.csa2_sparse_attn_workspace_size.argtypes = [I32, I32, I32, I32, I32]
        L.csa2_sparse_attn.restype = I32
        L.csa2_sparse_attn.argtypes = [P, P, I64, P, P, I32, P, I32, P, P, I32, I32, I32, I32, F32, P, P, P,
                                       SZ, P, P]
        L.csa2_cp_shard_vis.restype = I32
        L.csa2_cp_shard_vis.argtypes = [P, P, P, I32, I32, P, P, P]
        L.csa2_topk_merge_workspace_size.restype = SZ
        L.csa2_topk_merge_workspace_size.argtypes = [I32, I32, I32, I32]
        L.csa2_topk_merge.restype = I32
        L.csa2_topk_merge.argtypes = [P, P, I64, P, I32, I32, I32, I32, I32, P, P, P, SZ, P, P]
        L.csa2_topk_localize.restype = I32
        L.csa2_topk_localize.argtypes = [P, I32, I32, I32, P, P, P, P, P]
        L.csa2_attn_combine.restype = I32
        L.csa2_attn_combine.argtypes = [P, I64, P, I64, I32, I32, I32, I32, P, P, P]
        L.csa2_paged_plan.restype = I32
        L.csa2_paged_plan.argtypes = [P, P, I32, I32, P, I32, P, I64, P, I64, P, P, P, P, P, I64, P, P]
        L.csa2_paged_release.restype = I32
        L.csa2_paged_release.argtypes = [P, P, P, I32, I32, I32, P, I64, P, I64, P, P, P, P]
        L.csa2_kv8_append.restype = I32
        L.csa2_kv8_append.argtypes = [P, P, I64, I64, I32, I64, I32, I32, P, P, P, P, P, I64, I32, P, P]
        L.csa2_kv8_attn_workspace_size.restype = SZ
        L.csa2_kv8_attn_workspace_size.argtypes = [I32, I32, I32, I32, I32]
        L.csa2_kv8_attn.restype = I32
        L.csa2_kv8_attn.argtypes = [P, I64, I32, I64, I32, I32, I32, P, P, P, P, I64, I32, P, I32, P, P, I32, I32, F32,
                                    I32, F32, P, P, P, SZ, P, P]
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, what):
    if status != CSA2_OK:
        raise CSA2Error(status, what)


def _need(t, dtype, name, ndim=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _shape(t, shape, name):
    """Raise unless `t` (when given) has exactly `shape`; None in `shape` matches any size.
    The C entry points take sizes, not buffers, and cannot check a buffer's extent: a
    tensor smaller than the sizes say would be read or written out of bounds."""
    if t is None:
        return
    if t.dim() != len(shape) or any(e is not None and d != e for d, e in zip(t.shape, shape)):
        want = ", ".join("*" if e is None else str(e) for e in shape)
        raise ValueError(f"{name} must have shape ({want}), got {tuple(t.shape)}")


def _rows(t, n, name):
    """Raise unless the 1-D `t` (when given) has at least n entries (per-sequence arrays)."""
    if t is not None and (t.dim() != 1 or t.shape[0] < n):
        raise ValueError(f"{name} must be 1-D with at least {n} entries, got {tuple(t.shape)}")


def _status(t):
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1 or not t.is_cuda):
        raise ValueError("dev_status must be a CUDA int32 tensor with at least one element")


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A uint8 device buffer usable as csa2 workspace (torch's allocator aligns to 512 B)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device or "cuda")


def status_word(device=None) -> torch.Tensor:
    """A zeroed device status word for the dev_status argument."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def status_from_device_word(word: int) -> int:
    return lib().csa2_status_from_device_word(word & 0xFFFFFFFF)


def version() -> int:
    return lib().csa2_version()


# ---- a1 ---------------------------------------------------------------------------------
def csa2_pack_kv(kv, ik, ratio, kv_pool, ik_pool, dst_entry=None, dev_status=None, stream=None):
    """kv bf16 [T,512], ik bf16 [T,128] -> entries written into kv_pool u8 [P,288] and
    ik_pool u8 [P,68] (slots dst_entry int64 [T/ratio], or 0..T/ratio-1)."""
    _shape(kv, (None, D), "kv")
    T = kv.shape[0]
    _shape(ik, (T, DI), "ik")
    _shape(kv_pool, (None, KV_BYTES), "kv_pool")
    _shape(ik_pool, (kv_pool.shape[0], IK_BYTES), "ik_pool")
    if dst_entry is not None and (dst_entry.dim() != 1 or dst_entry.numel() != T // max(int(ratio), 1)):
        raise ValueError("dst_entry must hold one slot per new entry (T // ratio)")
    _need(kv, torch.bfloat16, "kv", 2)
    _need(ik, torch.bfloat16, "ik", 2)
    _need(kv_pool, torch.uint8, "kv_pool", 2)
    _need(ik_pool, torch.uint8, "ik_pool", 2)
    _need(dst_entry, torch.int64, "dst_entry", 1)
    _status(dev_status)
    _check(lib().csa2_pack_kv(_ptr(kv), _ptr(ik), T, int(ratio), _ptr(dst_entry), kv_pool.shape[0],
                              _ptr(kv_pool), _ptr(ik_pool), _ptr(dev_status), _stream(stream)),
           "csa2_pack_kv")


def csa2_pack_kv_normed(kv, ik, ratio, pos, rope_cos, rope_sin, kv_pool, ik_pool, gamma=None, eps=1e-6,
                        dst_entry=None, dev_status=None, stream=None):
    """Raw kv bf16 [T,512] normalised and rotated (pos int64 [T] into rope_cos / rope_sin
    f32 [n_pos,256]; gamma f32 [512] or None), then packed like csa2_pack_kv."""
    _shape(kv, (None, D), "kv")
    T = kv.shape[0]
    _shape(ik, (T, DI), "ik")
    _shape(pos, (T,), "pos")
    _shape(rope_cos, (None, D // 2), "rope_cos")
    _shape(rope_sin, (rope_cos.shape[0], D // 2), "rope_sin")
    _shape(gamma, (D,), "gamma")
    _shape(kv_pool, (None, KV_BYTES), "kv_pool")
    _shape(ik_pool, (kv_pool.shape[0], IK_BYTES), "ik_pool")
    if dst_entry is not None and (dst_entry.dim() != 1 or dst_entry.numel() != T // max(int(ratio), 1)):
        raise ValueError("dst_entry must hold one slot per new entry (T // ratio)")
    _need(kv, torch.bfloat16, "kv", 2)
    _need(ik, torch.bfloat16, "ik", 2)
    _need(pos, torch.int64, "pos", 1)
    _need(rope_cos, torch.float32, "rope_cos", 2)
    _need(rope_sin, torch.float32, "rope_sin", 2)
    _need(gamma, torch.float32, "gamma", 1)
    _need(kv_pool, torch.uint8, "kv_pool", 2)
    _need(ik_pool, torch.uint8, "ik_pool", 2)
    _need(dst_entry, torch.int64, "dst_entry", 1)
    _status(dev_status)
    _check(lib().csa2_pack_kv_normed(_ptr(kv), _ptr(ik), T, int(ratio), _ptr(pos), _ptr(rope_cos), _ptr(rope_sin),
                                     rope_cos.shape[0], _ptr(gamma), float(eps), _ptr(dst_entry), kv_pool.shape[0],
                                     _ptr(kv_pool), _ptr(ik_pool), _ptr(dev_status), _stream(stream)),
           "csa2_pack_kv_normed")


def _query_dims(q, w, ik_pool, seq_base, n_vis):
    """(B, Q, HI) of an indexer call, after checking the shapes its inputs must share."""
    _shape(q, (None, None, None, DI), "q")
    B, Q, HI, _ = q.shape
    _shape(w, (B, Q, HI), "w")
    _shape(ik_pool, (None, IK_BYTES), "ik_pool")
    _rows(seq_base, B, "seq_base")
    _shape(n_vis, (B, Q), "n_vis")
    return B, Q, HI


# ---- a2/a3 ------------------------------------------------------------------------------
def csa2_index_full_workspace_size(B, Q, HI, K, max_n_vis):
    return lib().csa2_index_full_workspace_size(B, Q, HI, K, max_n_vis)


def csa2_index_full(q, w, ik_pool, seq_base, n_vis, K, max_n_vis, topk, topk_score=None, ws=None,
                    dev_status=None, stream=None):
    """q f32 [B,Q,HI,128], w f32 [B,Q,HI], ik_pool u8 [P,68], seq_base i64 [B],
    n_vis i32 [B,Q] -> topk i32 [B,Q,K] (+ topk_score f32 [B,Q,K])."""
    B, Q, HI = _query_dims(q, w, ik_pool, seq_base, n_vis)
    _shape(topk, (B, Q, K), "topk")
    _shape(topk_score, (B, Q, K), "topk_score")
    _need(q, torch.float32, "q", 4)
    _need(w, torch.float32, "w", 3)
    _need(ik_pool, torch.uint8, "ik_pool", 2)
    _need(seq_base, torch.int64, "seq_base", 1)
    _need(n_vis, torch.int32, "n_vis", 2)
    _need(topk, torch.int32, "topk", 3)
    _need(topk_score, torch.float32, "topk_score", 3)
    _status(dev_status)
    if ws is None:
        ws = workspace(csa2_index_full_workspace_size(B, Q, HI, K, max_n_vis), q.device)
    _check(lib().csa2_index_full(_ptr(q), _ptr(w), _ptr(ik_pool), ik_pool.shape[0], _ptr(seq_base),
                                 _ptr(n_vis), B, Q, HI, K, int(max_n_vis), _ptr(topk), _ptr(topk_score),
                                 _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream)),
           "csa2_index_full")


def csa2_test_index_full_withheld_copy(q, w, ik_pool, seq_base, n_vis, K, max_n_vis, topk, withheld_tile,
                                       topk_score=None, ws=None, dev_status=None, stream=None):
    """Test hook: csa2_index_full whose streaming scan withholds one tile copy, so a bounded
    device wait expires and CSA2_DEV_TIMEOUT is set in dev_status (results unspecified)."""
    B, Q, HI = _query_dims(q, w, ik_pool, seq_base, n_vis)
    _shape(topk, (B, Q, K), "topk")
    _shape(topk_score, (B, Q, K), "topk_score")
    _need(q, torch.float32, "q", 4)
    _need(w, torch.float32, "w", 3)
    _need(ik_pool, torch.uint8, "ik_pool", 2)
    _need(seq_base, torch.int64, "seq_base", 1)
    _need(n_vis, torch.int32, "n_vis", 2)
    _need(topk, torch.int32, "topk", 3)
    _need(topk_score, torch.float32, "topk_score", 3)
    _status(dev_status)
    if ws is None:
        ws = workspace(csa2_index_full_workspace_size(B, Q, HI, K, max_n_vis), q.device)
    _check(lib().csa2_test_index_full_withheld_copy(
        _ptr(q), _ptr(w), _ptr(ik_pool), ik_pool.shape[0], _ptr(seq_base), _ptr(n_vis), B, Q, HI, K,
        int(max_n_vis), _ptr(topk), _ptr(topk_score), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream),
        int(withheld_tile)), "csa2_test_index_full_withheld_copy")


# ---- a4 ---------------------------------------------------------------------------------
def csa2_index_hier_workspace_size(B, Q, HI, n_blocks, block, max_n_vis):
    return lib().csa2_index_hier_workspace_size(B, Q, HI, n_blocks, block, max_n_vis)


def csa2_index_hier(q, w, ik_pool, seq_base, n_vis, n_blocks, block, max_n_vis, blocks, block_score=None,
                    ws=None, dev_status=None, stream=None):
    B, Q, HI = _query_dims(q, w, ik_pool, seq_base, n_vis)
    _shape(blocks, (B, Q, n_blocks), "blocks")
    _shape(block_score, (B, Q, n_blocks), "block_score")
    _need(q, torch.float32, "q", 4)
    _need(w, torch.float32, "w", 3)
    _need(ik_pool, torch.uint8, "ik_pool", 2)
    _need(seq_base, torch.int64, "seq_base", 1)
    _need(n_vis, torch.int32, "n_vis", 2)
    _need(blocks, torch.int32, "blocks", 3)
    _need(block_score, torch.float32, "block_score", 3)
    _status(dev_status)
    if ws is None:
        ws = workspace(csa2_index_hier_workspace_size(B, Q, HI, n_blocks, block, max_n_vis), q.device)
    _check(lib().csa2_index_hier(_ptr(q), _ptr(w), _ptr(ik_pool), ik_pool.shape[0], _ptr(seq_base),
                                 _ptr(n_vis), B, Q, HI, n_blocks, block, int(max_n_vis), _ptr(blocks),
                                 _ptr(block_score), _ptr(ws), ws.numel(), _ptr(dev_status),
                                 _stream(stream)),
           "csa2_index_hier")


# ---- a5 ---------------------------------------------------------------------------------
def csa2_reindex_workspace_size(B, Q, HI, n_blocks, block, K):
    return lib().csa2_reindex_workspace_size(B, Q, HI, n_blocks, block, K)


def csa2_reindex(q, w, ik_pool, seq_base, n_vis, blocks, block, K, topk, topk_score=None, ws=None,
                 dev_status=None, stream=None):
    B, Q, HI = _query_dims(q, w, ik_pool, seq_base, n_vis)
    _shape(blocks, (B, Q, None), "blocks")
    _shape(topk, (B, Q, K), "topk")
    _shape(topk_score, (B, Q, K), "topk_score")
    _need(q, torch.float32, "q", 4)
    _need(w, torch.float32, "w", 3)
    _need(ik_pool, torch.uint8, "ik_pool", 2)
    _need(seq_base, torch.int64, "seq_base", 1)
    _need(n_vis, torch.int32, "n_vis", 2)
    _need(blocks, torch.int32, "blocks", 3)
    _need(topk, torch.int32, "topk", 3)
    _need(topk_score, torch.float32, "topk_score", 3)
    _status(dev_status)
    n_blocks = blocks.shape[-1]
    if ws is None:
        ws = workspace(csa2_reindex_workspace_size(B, Q, HI, n_blocks, block, K), q.device)
    _check(lib().csa2_reindex(_ptr(q), _ptr(w), _ptr(ik_pool), ik_pool.shape[0], _ptr(seq_base),
                              _ptr(n_vis), _ptr(blocks), n_blocks, block, B, Q, HI, K, _ptr(topk),
                              _ptr(topk_score), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream)),
           "csa2_reindex")


def csa2_static_scratch_bytes():
    return lib().csa2_static_scratch_bytes()


def csa2_reindex_static(q, w, ik_pool, seq_base, n_vis, blocks, block, K, topk, topk_score=None,
                        dev_status=None, stream=None):
    """csa2_reindex with the library's own static device scratch instead of a workspace:
    for callers that cannot allocate device memory for the call (see include/csa2.h)."""
    B, Q, HI = _query_dims(q, w, ik_pool, seq_base, n_vis)
    _shape(blocks, (B, Q, None), "blocks")
    _shape(topk, (B, Q, K), "topk")
    _shape(topk_score, (B, Q, K), "topk_score")
    _need(q, torch.float32, "q", 4)
    _need(w, torch.float32, "w", 3)
    _need(ik_pool, torch.uint8, "ik_pool", 2)
    _need(seq_base, torch.int64, "seq_base", 1)
    _need(n_vis, torch.int32, "n_vis", 2)
    _need(blocks, torch.int32, "blocks", 3)
    _need(topk, torch.int32, "topk", 3)
    _need(topk_score, torch.float32, "topk_score", 3)
    _status(dev_status)
    n_blocks = blocks.shape[-1]
    _check(lib().csa2_reindex_static(_ptr(q), _ptr(w), _ptr(ik_pool), ik_pool.shape[0], _ptr(seq_base),
                                     _ptr(n_vis), _ptr(blocks), n_blocks, block, B, Q, HI, K, _ptr(topk),
                                     _ptr(topk_score), _ptr(dev_status), _stream(stream)),
           "csa2_reindex_static")


# ---- a6/a7 ------------------------------------------------------------------------------
def csa2_sparse_attn_workspace_size(B, Q, H, K, window):
    return lib().csa2_sparse_attn_workspace_size(B, Q, H, K, window)


def csa2_sparse_attn(q, kv_pool, seq_base, topk, swa, swa_start, q_pos, sm_scale, out, lse, window=128,
                     ws=None, dev_status=None, stream=None):
    """q f32 [B,Q,H,512]; kv_pool u8 [P,288]; topk i32 [B,Q,K]; swa u8 [B,S_w,512] or None;
    swa_start i64 [B]; q_pos i64 [B,Q] -> out f32 [B,Q,H,512], lse f32 [B,Q,H]."""
    _shape(q, (None, None, None, D), "q")
    B, Q, H, _ = q.shape
    _shape(kv_pool, (None, KV_BYTES), "kv_pool")
    _rows(seq_base, B, "seq_base")
    _shape(topk, (B, Q, None), "topk")
    _shape(swa, (None, None, D), "swa")
    if swa is not None and swa.shape[0] < B:
        raise ValueError(f"swa must hold at least {B} sequences, got {tuple(swa.shape)}")
    if swa is not None and swa.shape[1] > 0 and swa_start is None:
        raise ValueError("swa_start is required with a window buffer")
    _rows(swa_start, B, "swa_start")
    _shape(q_pos, (B, Q), "q_pos")
    _shape(out, (B, Q, H, D), "out")
    _shape(lse, (B, Q, H), "lse")
    _need(q, torch.float32, "q", 4)
    _need(kv_pool, torch.uint8, "kv_pool", 2)
    _need(seq_base, torch.int64, "seq_base", 1)
    _need(topk, torch.int32, "topk", 3)
    _need(swa, torch.uint8, "swa", 3)
    _need(swa_start, torch.int64, "swa_start", 1)
    _need(q_pos, torch.int64, "q_pos", 2)
    _need(out, torch.float32, "out", 4)
    _need(lse, torch.float32, "lse", 3)
    _status(dev_status)
    K = topk.shape[-1] if topk is not None else 0
    S_w = swa.shape[1] if swa is not None else 0
    if ws is None:
        ws = workspace(csa2_sparse_attn_workspace_size(B, Q, H, K, window), q.device)
    _check(lib().csa2_sparse_attn(_ptr(q), _ptr(kv_pool), kv_pool.shape[0], _ptr(seq_base), _ptr(topk), K,
                                  _ptr(swa), S_w, _ptr(swa_start), _ptr(q_pos), int(window), B, Q, H,
                                  float(sm_scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                  _ptr(dev_status), _stream(stream)),
           "csa2_sparse_attn")


# ---- context-parallel decode ------------------------------------------------------------
def csa2_cp_shard_vis(n_vis, shard_lo, shard_len, n_vis_local, dev_status=None, stream=None):
    """n_vis i32 [B,Q]; shard_lo, shard_len i64 [B] -> n_vis_local i32 [B,Q] (the visible
    count inside this rank's shard)."""
    _shape(n_vis, (None, None), "n_vis")
    B, Q = n_vis.shape
    _rows(shard_lo, B, "shard_lo")
    _rows(shard_len, B, "shard_len")
    _shape(n_vis_local, (B, Q), "n_vis_local")
    _need(n_vis, torch.int32, "n_vis", 2)
    _need(shard_lo, torch.int64, "shard_lo", 1)
    _need(shard_len, torch.int64, "shard_len", 1)
    _need(n_vis_local, torch.int32, "n_vis_local", 2)
    _status(dev_status)
    _check(lib().csa2_cp_shard_vis(_ptr(n_vis), _ptr(shard_lo), _ptr(shard_len), B, Q, _ptr(n_vis_local),
                                   _ptr(dev_status), _stream(stream)), "csa2_cp_shard_vis")


def csa2_topk_merge_workspace_size(C, B, Q, Kc):
    return lib().csa2_topk_merge_workspace_size(C, B, Q, Kc)


def _part_stride(t, name):
    """Elements from one part to the next of a [C, ...] tensor whose parts are each
    contiguous (0 for a single part: the library then takes the dense stride)."""
    if t.dim() < 1 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor with a leading part dimension")
    if not t[0].is_contiguous():
        raise ValueError(f"{name}: each part must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else 0


def csa2_topk_merge(cand, cand_score, shard_off, K, topk, topk_score=None, ws=None, dev_status=None,
                    stream=None):
    """cand i32 [C,B,Q,Kc] (labels local to each shard, -1 empty), cand_score f32 [C,B,Q,Kc],
    shard_off i64 [C,B] -> topk i32 [B,Q,K] global labels (+ topk_score f32 [B,Q,K]).
    cand and cand_score may be strided views (parts each contiguous, same part stride),
    e.g. the two halves of one gathered buffer per shard."""
    _shape(cand, (None, None, None, None), "cand")
    C, B, Q, Kc = cand.shape
    _shape(cand_score, (C, B, Q, Kc), "cand_score")
    _shape(shard_off, (C, B), "shard_off")
    _shape(topk, (B, Q, K), "topk")
    _shape(topk_score, (B, Q, K), "topk_score")
    if cand.dtype != torch.int32 or cand_score.dtype != torch.float32:
        raise TypeError("cand must be int32 and cand_score float32")
    ps = _part_stride(cand, "cand")
    if _part_stride(cand_score, "cand_score") != ps:
        raise ValueError("cand and cand_score must have the same part stride")
    _need(shard_off, torch.int64, "shard_off", 2)
    _need(topk, torch.int32, "topk", 3)
    _need(topk_score, torch.float32, "topk_score", 3)
    _status(dev_status)
    if ws is None:
        ws = workspace(csa2_topk_merge_workspace_size(C, B, Q, Kc), cand.device)
    _check(lib().csa2_topk_merge(_ptr(cand), _ptr(cand_score), int(ps), _ptr(shard_off), C, B, Q, Kc, int(K),
                                 _ptr(topk), _ptr(topk_score), _ptr(ws), ws.numel(), _ptr(dev_status),
                                 _stream(stream)), "csa2_topk_merge")


def csa2_topk_localize(topk, shard_off, shard_len, topk_local, dev_status=None, stream=None):
    """topk i32 [B,Q,K] global labels; shard_off, shard_len i64 [B] -> topk_local i32
    [B,Q,K]: this shard's labels minus its offset, compacted, -1 after them."""
    _shape(topk, (None, None, None), "topk")
    B, Q, K = topk.shape
    _rows(shard_off, B, "shard_off")
    _rows(shard_len, B, "shard_len")
    _shape(topk_local, (B, Q, K), "topk_local")
    _need(topk, torch.int32, "topk", 3)
    _need(shard_off, torch.int64, "shard_off", 1)
    _need(shard_len, torch.int64, "shard_len", 1)
    _need(topk_local, torch.int32, "topk_local", 3)
    _status(dev_status)
    _check(lib().csa2_topk_localize(_ptr(topk), B, Q, K, _ptr(shard_off), _ptr(shard_len), _ptr(topk_local),
                                    _ptr(dev_status), _stream(stream)), "csa2_topk_localize")


def csa2_attn_combine(out_parts, lse_parts, out, lse, stream=None):
    """out_parts f32 [C,B,Q,H,512], lse_parts f32 [C,B,Q,H] (parts each contiguous; dense,
    or views of one gathered [out | lse] buffer per part) -> out f32 [B,Q,H,512], lse f32
    [B,Q,H]: attention over the union."""
    _shape(out_parts, (None, None, None, None, D), "out_parts")
    C, B, Q, H, _ = out_parts.shape
    _shape(lse_parts, (C, B, Q, H), "lse_parts")
    _shape(out, (B, Q, H, D), "out")
    _shape(lse, (B, Q, H), "lse")
    if out_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise TypeError("out_parts and lse_parts must be float32")
    pso = _part_stride(out_parts, "out_parts")
    psl = _part_stride(lse_parts, "lse_parts")
    _need(out, torch.float32, "out", 4)
    _need(lse, torch.float32, "lse", 3)
    _check(lib().csa2_attn_combine(_ptr(out_parts), int(pso), _ptr(lse_parts), int(psl), C, B, Q, H, _ptr(out),
                                   _ptr(lse), _stream(stream)), "csa2_attn_combine")


# ---- paged 8-bit KV cache ----------------------------------------------------------------
# These calls are made per layer of a decode step, where the host's time shows: on the current
# stream they go through _native (csrc/binding.cpp), which makes the same checks in C++.  What it
# does not take (another stream, an argument that is not as it should be) comes here, where the
# checks read each tensor's properties once and name what they refuse.
_BF16, _F16, _I32, _I64, _F32, _U8 = (torch.bfloat16, torch.float16, torch.int32, torch.int64, torch.float32, torch.uint8)
_KV_DTYPES = {_BF16: 0, _F16: 1}


_fast = None


def _load_fast():
    global _fast
    lib()
    try:
        from . import _native
    except ImportError as e:
        raise RuntimeError("_native.so is missing; build it with __graft_entry__.build()") from e
    _fast = _native
    return _native


def _refuse(t, dtype, shape, name, dev):
    """The shape first: it is what the C entry points cannot check."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the first argument, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, dtype, shape, name, dev):
    """Raise unless t is a contiguous `dtype` tensor of exactly `shape` on device `dev` (-1: the
    host, refused when everything else is right); its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, dtype, shape, name, dev)
    return t.data_ptr()


def _tokens(t, dtype, shape, name, dev):
    """The same for a [T, heads, hd] view whose tokens are each contiguous: (address, token stride)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, dtype, shape, name, dev)
    T, heads, hd = shape
    s0, s1, s2 = t.stride()
    if T > 0 and (s2 != 1 or (s1 != hd and heads > 1)):
        raise ValueError(f"{name}: each token's [heads, hd] must be contiguous")
    if T <= 1:
        return t.data_ptr(), heads * hd
    if s0 < heads * hd or s0 % 8:
        raise ValueError(f"{name}: the token stride must be a multiple of 8 elements and at least heads * hd")
    return t.data_ptr(), s0


def _flag_arg(dev_status, dev):
    if dev_status is None:
        return None
    if dev_status.dtype is not _I32 or dev_status.numel() < 1 or dev_status.get_device() != dev:
        raise ValueError(f"dev_status must be an int32 tensor with at least one element on cuda:{dev}")
    return dev_status.data_ptr()


def _whole(x, name, bits=32):
    """x as an int that `bits` bits hold: ctypes would cut a larger one without a word."""
    v = operator.index(x)
    if not -(1 << (bits - 1)) <= v < 1 << (bits - 1):
        raise ValueError(f"{name} must fit a signed {bits}-bit integer, got {v}")
    return v


def _need_cuda(dev, name):
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")


def _length(t, name):
    sh = t.shape
    if len(sh) != 1:
        raise ValueError(f"{name} must be 1-D, got {tuple(sh)}")
    return sh[0]


def _table(t, R, dev):
    """(address, columns) of the block table of R requests."""
    sh = t.shape
    if len(sh) != 2:
        raise ValueError(f"block_table must be 2-D, got {tuple(sh)}")
    return _arg(t, _I32, (R, sh[1]), "block_table", dev), sh[1]


def _call_on(dev, stream, fn, *args):
    """fn(*args, stream) with cuda:`dev` current (the library launches on the current device)."""
    _need_cuda(dev, "every tensor")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        return fn(*args, raw)
    with torch.cuda.device(dev):
        return fn(*args, raw)


def csa2_paged_plan(ctx_len, new_len, block_table, free_pages, n_free, page, n_pages, seq_len, n_free_out, q_start,
                    slot_map, pos, dev_status=None, stream=None):
    """ctx_len, new_len i32 [R], block_table i32 [R,max_pages] (new pages are added),
    free_pages i32 [F] with n_free i32 [1] valid -> seq_len i32 [R], n_free_out i32 [1],
    q_start i32 [R+1], slot_map and pos i64 [T_cap] (see include/csa2.h).  seq_len may be
    ctx_len and n_free_out may be n_free."""
    if stream is None:
        st = (_fast or _load_fast()).paged_plan(ctx_len, new_len, block_table, free_pages, n_free, page, n_pages, seq_len,
                                               n_free_out, q_start, slot_map, pos, dev_status)
        if st >= 0:
            return _check(st, "csa2_paged_plan")
    page, n_pages = _whole(page, "page"), _whole(n_pages, "n_pages", 64)
    dev = ctx_len.get_device()
    R, F, T = _length(ctx_len, "ctx_len"), _length(free_pages, "free_pages"), _length(slot_map, "slot_map")
    ta, cols = _table(block_table, R, dev)
    _check(_call_on(
        dev, stream, lib().csa2_paged_plan, _arg(ctx_len, _I32, (R,), "ctx_len", dev),
        _arg(new_len, _I32, (R,), "new_len", dev), R, page, ta, cols, _arg(free_pages, _I32, (F,), "free_pages", dev), F,
        _arg(n_free, _I32, (1,), "n_free", dev), n_pages, _arg(seq_len, _I32, (R,), "seq_len", dev),
        _arg(n_free_out, _I32, (1,), "n_free_out", dev), _arg(q_start, _I32, (R + 1,), "q_start", dev),
        _arg(slot_map, _I64, (T,), "slot_map", dev), _arg(pos, _I64, (T,), "pos", dev), T, _flag_arg(dev_status, dev)),
        "csa2_paged_plan")


def csa2_paged_release(seq_len, block_table, release, free_pages, n_free, page, n_pages, seq_len_out, n_free_out,
                       dev_status=None, stream=None):
    """The pages of requests whose release u8 [R] is nonzero, pushed onto free_pages i32 [F]
    after its n_free i32 [1] entries; seq_len_out i32 [R] (0 for those) and n_free_out i32 [1]
    may be seq_len and n_free."""
    if stream is None:
        st = (_fast or _load_fast()).paged_release(seq_len, block_table, release, free_pages, n_free, page, n_pages,
                                                  seq_len_out, n_free_out, dev_status)
        if st >= 0:
            return _check(st, "csa2_paged_release")
    page, n_pages = _whole(page, "page"), _whole(n_pages, "n_pages", 64)
    dev = seq_len.get_device()
    R, F = _length(seq_len, "seq_len"), _length(free_pages, "free_pages")
    ta, cols = _table(block_table, R, dev)
    _check(_call_on(
        dev, stream, lib().csa2_paged_release, _arg(seq_len, _I32, (R,), "seq_len", dev), ta,
        _arg(release, _U8, (R,), "release", dev), R, page, cols, _arg(free_pages, _I32, (F,), "free_pages", dev), F,
        _arg(n_free, _I32, (1,), "n_free", dev), n_pages, _arg(seq_len_out, _I32, (R,), "seq_len_out", dev),
        _arg(n_free_out, _I32, (1,), "n_free_out", dev), _flag_arg(dev_status, dev)), "csa2_paged_release")


def _cache_args(k_cache, v_cache, k_scale, v_scale, dev):
    """(n_pages, Hk, page, hd) and the four addresses of one layer's cache."""
    sh = k_cache.shape
    if len(sh) != 4:
        raise ValueError(f"k_cache must be [n_pages, Hk, page, hd], got {tuple(sh)}")
    per = (sh[0], sh[1])
    return sh, (_arg(k_cache, _U8, sh, "k_cache", dev), _arg(v_cache, _U8, sh, "v_cache", dev),
                _arg(k_scale, _F32, per, "k_scale", dev), _arg(v_scale, _F32, per, "v_scale", dev))


def csa2_kv8_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, dev_status=None, stream=None):
    """k, v bf16 or fp16 [T,Hk,hd] (token-strided views allowed) written as E4M3 codes into
    k_cache, v_cache u8 [n_pages,Hk,page,hd] at slot_map i64 [T], with one power-of-two scale
    per page and head in k_scale, v_scale f32 [n_pages,Hk] (see include/csa2.h)."""
    if stream is None:
        st = (_fast or _load_fast()).kv8_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, dev_status)
        if st >= 0:
            return _check(st, "csa2_kv8_append")
    dev = k.get_device()
    (P, Hk, page, hd), cache = _cache_args(k_cache, v_cache, k_scale, v_scale, dev)
    dtype = k.dtype
    if dtype not in _KV_DTYPES:
        raise TypeError(f"k must be bfloat16 or float16, got {dtype}")
    T = _length(slot_map, "slot_map")
    rows = (T, Hk, hd)
    ka, ks = _tokens(k, dtype, rows, "k", dev)
    va, vs = _tokens(v, dtype, rows, "v", dev)
    _check(_call_on(dev, stream, lib().csa2_kv8_append, ka, va, ks, vs, _KV_DTYPES[dtype], T, Hk, hd,
                    _arg(slot_map, _I64, (T,), "slot_map", dev), *cache, P, page, _flag_arg(dev_status, dev)),
           "csa2_kv8_append")


@functools.lru_cache(maxsize=256)
def _kv8_ws(dev, Hq, Hk, hd, max_q, kind):
    """Workspace bytes on cuda:`dev` (by its number of SMs); at least 1, refusals come from the call."""
    with torch.cuda.device(dev):
        return max(lib().csa2_kv8_attn_workspace_size(Hq, Hk, hd, max_q, kind), 1)


def csa2_kv8_attn_workspace_size(Hq, Hk, hd, max_q, dtype=torch.bfloat16):
    Hq, Hk, hd, max_q = _whole(Hq, "Hq"), _whole(Hk, "Hk"), _whole(hd, "hd"), _whole(max_q, "max_q")
    return lib().csa2_kv8_attn_workspace_size(Hq, Hk, hd, max_q, _KV_DTYPES[dtype])


def csa2_kv8_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, q_start, seq_len, sm_scale, out, lse=None,
                  max_q=1, window=0, softcap=0.0, ws=None, dev_status=None, stream=None):
    """q bf16 or fp16 [T,Hq,hd] (token-strided views allowed), the cache of csa2_kv8_append,
    block_table i32 [R,max_pages], q_start i32 [R+1], seq_len i32 [R] -> out like q
    (contiguous) and lse f32 [T,Hq] or None (see include/csa2.h)."""
    if stream is None:
        st = (_fast or _load_fast()).kv8_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, q_start, seq_len,
                                             sm_scale, out, lse, max_q, window, softcap, ws, dev_status)
        if st >= 0:
            return _check(st, "csa2_kv8_attn")
    max_q, window = _whole(max_q, "max_q"), _whole(window, "window")
    dev = q.get_device()
    (P, Hk, page, hd), cache = _cache_args(k_cache, v_cache, k_scale, v_scale, dev)
    dtype, sh = q.dtype, q.shape
    if dtype not in _KV_DTYPES:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    if len(sh) != 3 or sh[2] != hd:
        raise ValueError(f"q must be [T, Hq, {hd}], got {tuple(sh)}")
    T, Hq = sh[0], sh[1]
    R, kind = _length(seq_len, "seq_len"), _KV_DTYPES[dtype]
    qa, qs = _tokens(q, dtype, sh, "q", dev)
    ta, cols = _table(block_table, R, dev)
    qsa, sla = _arg(q_start, _I32, (R + 1,), "q_start", dev), _arg(seq_len, _I32, (R,), "seq_len", dev)
    oa = _arg(out, dtype, (T, Hq, hd), "out", dev)
    la = None if lse is None else _arg(lse, _F32, (T, Hq), "lse", dev)
    L = lib()
    _need_cuda(dev, "q")
    if ws is None:
        # taken on the stream that uses it, so the allocator keeps it until the kernels are done
        need = _kv8_ws(dev, Hq, Hk, hd, max_q, kind)
        if stream is None:
            ws = q.new_empty(need, dtype=_U8)
        else:
            with torch.cuda.stream(stream):
                ws = q.new_empty(need, dtype=_U8)
    elif ws.dtype is not _U8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{dev}")
    _check(_call_on(
        dev, stream, L.csa2_kv8_attn, qa, qs, kind, T, Hq, Hk, hd, *cache, P, page, ta, cols,
        qsa, sla, R, max_q, sm_scale, window, softcap, oa, la, ws.data_ptr(), ws.numel(), _flag_arg(dev_status, dev)),
        "csa2_kv8_attn")
