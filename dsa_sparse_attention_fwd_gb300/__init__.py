"""GB300 (sm_103a) DSA lightning-indexer forward.

A thin ctypes binding over the C ABI in `include/dsa_indexer.h`.  This module
only marshals arguments: it allocates outputs and workspace with PyTorch,
passes raw device pointers and the current CUDA stream, and raises on error
codes.  Every step of the computation runs in the library's CUDA kernels; if
the library is missing, every call raises instead of falling back.

Interface after the DeepSeek-V4 SBHD indexer of NeMo AutoModel
("tilelang_indexer" page: `v4_lighting_indexer(index_q, index_k, weights,
compress_ratio, topk, topk_indices=None)`):
    index_q  [S, B, H, D] bf16, index_k [S_kv, B, D] bf16,
    weights  [S, B, H] fp32, topk_indices [B, S, topk] int32 (optional)
returns (scores [B, S, topk] fp32, indices [B, S, topk] int32).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

from ._build import LIB_PATH, build

__all__ = [
    "DsaError", "load_library", "build", "dsa_indexer_workspace_size",
    "dsa_set_prefill_policy", "dsa_indexer_fwd_launches", "PREFILL_AUTO",
    "PREFILL_ONE_KERNEL", "PREFILL_TWO_KERNELS",
    "dsa_indexer_fwd", "dsa_indexer_logits", "dsa_indexer_check",
    "dsa_status_string", "dsa_selftest_wait_limit", "v4_lighting_indexer",
    "indexer_logits", "dsa_indexer_host_buffer_size", "dsa_indexer_fwd_host",
    "dsa_indexer_varlen_workspace_size", "dsa_indexer_fwd_varlen",
    "dsa_indexer_bwd", "dsa_indexer_bwd_workspace_size",
    "dsa_kpool_compress", "dsa_expand_selection",
    "dsa_indexer_pooled_workspace_size", "dsa_indexer_fwd_pooled",
    "dsa_sparse_mla_fwd", "dsa_sparse_mla_workspace_size", "STATUS",
    "rope_inv_freq", "dsa_norm_rope_fwd", "dsa_norm_rope_bwd",
    "dsa_norm_rope_bwd_workspace_size", "dsa_paged_append",
    "dsa_block_attn_fwd", "dsa_block_attn_paged_fwd", "dsa_block_attn_bwd",
    "dsa_block_attn_workspace_size", "dsa_block_attn_bwd_workspace_size",
    "dsa_paged_append_q8", "dsa_paged_read_q8", "dsa_block_attn_paged_q8_fwd",
    "dsa_block_attn_q8_workspace_size",
]

STATUS = {
    0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED",
    3: "DSA_ERR_WORKSPACE", 4: "DSA_ERR_CUDA", 5: "DSA_ERR_DEVICE_TIMEOUT",
    6: "DSA_ERR_INDEX_RANGE",
}

_lib = None
_lock = threading.Lock()


class DsaError(RuntimeError):
    """A non-zero dsa_status from the library."""

    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} "
                         f"({dsa_status_string(code)})")


def load_library(path: str | None = None):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library not built ({p}); run "
                "dsa_sparse_attention_fwd_gb300.build() first")
        lib = ctypes.CDLL(p)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.dsa_indexer_workspace_size.restype = Z
        lib.dsa_indexer_workspace_size.argtypes = [I] * 8
        lib.dsa_set_prefill_policy.restype = I
        lib.dsa_set_prefill_policy.argtypes = [I]
        lib.dsa_indexer_fwd_launches.restype = I
        lib.dsa_indexer_fwd_launches.argtypes = [I] * 8
        lib.dsa_indexer_fwd.restype = I
        lib.dsa_indexer_fwd.argtypes = [P, P, P, I, I, I, I, I, I, I, P, P, P,
                                        P, P, Z, P]
        lib.dsa_indexer_fwd_profiled.restype = I
        lib.dsa_indexer_fwd_profiled.argtypes = [P, P, P, I, I, I, I, I, I, I,
                                                 P, P, P, P, P, Z, P, P, I]
        lib.dsa_indexer_logits_workspace_size.restype = Z
        lib.dsa_indexer_logits_workspace_size.argtypes = []
        lib.dsa_indexer_logits.restype = I
        lib.dsa_indexer_logits.argtypes = [P, P, P, I, I, I, I, I, I, P, P, P,
                                           Z, P]
        lib.dsa_indexer_check.restype = I
        lib.dsa_indexer_check.argtypes = [P, P]
        lib.dsa_status_string.restype = ctypes.c_char_p
        lib.dsa_status_string.argtypes = [I]
        lib.dsa_selftest_wait_limit.restype = I
        lib.dsa_selftest_wait_limit.argtypes = [I, P, Z, P]
        lib.dsa_indexer_host_buffer_size.restype = Z
        lib.dsa_indexer_host_buffer_size.argtypes = [I] * 8
        lib.dsa_indexer_host_plan.restype = I
        lib.dsa_indexer_host_plan.argtypes = [I, I, I, I, I, I, I, P, I, I,
                                              P, P]
        lib.dsa_indexer_varlen_workspace_size.restype = Z
        lib.dsa_indexer_varlen_workspace_size.argtypes = [I, P, P, I, I, I, I,
                                                          I]
        lib.dsa_indexer_fwd_varlen.restype = I
        lib.dsa_indexer_fwd_varlen.argtypes = [P, P, P, I, P, P, I, I, I, I,
                                               P, P, P, P, P, Z, P]
        lib.dsa_indexer_fwd_host.restype = I
        lib.dsa_indexer_fwd_host.argtypes = [P, P, P, I, I, I, I, I, I, I, P,
                                             P, P, P, P, Z, P]
        lib.dsa_indexer_bwd_workspace_size.restype = Z
        lib.dsa_indexer_bwd_workspace_size.argtypes = []
        lib.dsa_indexer_bwd.restype = I
        lib.dsa_indexer_bwd.argtypes = [P, P, P, I, I, I, I, I, I, I, P, P, P,
                                        P, P, P, P, Z, P]
        L = ctypes.c_longlong
        lib.dsa_kpool_compress.restype = I
        lib.dsa_kpool_compress.argtypes = [P, P, P, P, I, I, I, I, I, P, P, P]
        lib.dsa_expand_selection.restype = I
        lib.dsa_expand_selection.argtypes = [P, L, I, I, I, P, P]
        lib.dsa_indexer_pooled_workspace_size.restype = Z
        lib.dsa_indexer_pooled_workspace_size.argtypes = [I] * 8
        lib.dsa_indexer_fwd_pooled.restype = I
        lib.dsa_indexer_fwd_pooled.argtypes = [P, P, P, P, P, P, I, I, I, I,
                                               I, I, I, I, P, P, P, P, P, Z,
                                               P]
        lib.dsa_sparse_mla_workspace_size.restype = Z
        lib.dsa_sparse_mla_workspace_size.argtypes = []
        lib.dsa_sparse_mla_fwd.restype = I
        lib.dsa_sparse_mla_fwd.argtypes = [P, P, P, I, I, I, I, I, I,
                                           ctypes.c_float, P, P, P, Z, P]
        F = ctypes.c_float
        lib.dsa_norm_rope_fwd.restype = I
        lib.dsa_norm_rope_fwd.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P,
                                          F, P, P, I, I, I, F, P, P, P]
        lib.dsa_norm_rope_bwd_workspace_size.restype = Z
        lib.dsa_norm_rope_bwd_workspace_size.argtypes = [I]
        lib.dsa_norm_rope_bwd.restype = I
        lib.dsa_norm_rope_bwd.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I,
                                          P, P, F, P, P, I, I, I, F, P, P, P,
                                          P, P, Z, P]
        lib.dsa_paged_append.restype = I
        lib.dsa_paged_append.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P,
                                         P, P, I, I, P, I, P, P, P, F, P, I,
                                         I, I, F, P, P, Z, P]
        for name in ("dsa_block_attn_workspace_size",
                     "dsa_block_attn_bwd_workspace_size",
                     "dsa_block_attn_q8_workspace_size"):
            getattr(lib, name).restype = Z
            getattr(lib, name).argtypes = [I] * 9
        lib.dsa_block_attn_fwd.restype = I
        lib.dsa_block_attn_fwd.argtypes = [P, P, P, P, I, I, I, I, I, I, P, I,
                                           I, I, I, P, F, P, P, P, Z, P]
        lib.dsa_block_attn_paged_fwd.restype = I
        lib.dsa_block_attn_paged_fwd.argtypes = [
            P, P, P, P, I, I, P, I, I, I, I, I, I, P, I, I, I, I, P, F, P, P,
            P, Z, P]
        lib.dsa_block_attn_bwd.restype = I
        lib.dsa_block_attn_bwd.argtypes = [
            P, P, P, P, P, P, P, I, I, I, I, I, I, P, I, I, I, I, P, F, P, P,
            P, P, Z, P]
        lib.dsa_paged_append_q8.restype = I
        lib.dsa_paged_append_q8.argtypes = [
            P, P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, I, I, I, P, I, P,
            P, P, P, F, P, I, I, I, F, P, P, Z, P]
        lib.dsa_paged_read_q8.restype = I
        lib.dsa_paged_read_q8.argtypes = [
            P, P, P, P, P, I, I, I, P, I, I, I, I, I, P, P, P, P, P, Z, P]
        lib.dsa_block_attn_paged_q8_fwd.restype = I
        lib.dsa_block_attn_paged_q8_fwd.argtypes = [
            P, P, P, P, P, P, I, I, I, P, I, I, I, I, I, I, P, I, I, I, I, P,
            F, P, P, P, Z, P]
        _lib = lib
        return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(stream, shape, dt, device):
    """torch.empty() in the memory of the stream that a call runs on (the
    current one where none is given): memory that was freed by work on the
    current stream may still be in use by what is queued there.  A result used
    on another stream afterwards follows torch's rules for that
    (record_stream)."""
    if stream is None:
        return torch.empty(shape, dtype=dt, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dt, device=device)


def _zeroed_workspace(stream, size, device):
    """A workspace whose first 256 bytes are cleared in the stream's order."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _zeroed_workspace(None, size, device)
    if size <= 256:
        return torch.zeros(size, dtype=torch.uint8, device=device)
    workspace = torch.empty(size, dtype=torch.uint8, device=device)
    workspace[:256].zero_()
    return workspace


def dsa_status_string(code: int) -> str:
    return load_library().dsa_status_string(int(code)).decode()


# prefill top-k path policies (dsa_set_prefill_policy)
PREFILL_AUTO, PREFILL_ONE_KERNEL, PREFILL_TWO_KERNELS = 0, 1, 2


def dsa_set_prefill_policy(policy: int) -> None:
    """Process-wide choice between the one-kernel and the two-kernel prefill
    forward (PREFILL_AUTO picks by row length)."""
    rc = load_library().dsa_set_prefill_policy(int(policy))
    if rc != 0:
        raise DsaError(rc, "dsa_set_prefill_policy")


def dsa_indexer_fwd_launches(S, B, H, D, S_kv, compress_ratio, topk,
                             has_in_idx=False) -> int:
    """Kernels one forward of this shape launches under the current policy."""
    return int(load_library().dsa_indexer_fwd_launches(
        S, B, H, D, S_kv, compress_ratio, topk, 1 if has_in_idx else 0))


def dsa_indexer_workspace_size(S, B, H, D, S_kv, compress_ratio, topk,
                               has_in_idx=False) -> int:
    return int(load_library().dsa_indexer_workspace_size(
        S, B, H, D, S_kv, compress_ratio, topk, int(bool(has_in_idx))))


def _require_cuda(where: str, **tensors):
    """Device entry points read every tensor's pointer as device memory:
    each given tensor must be a CUDA tensor, all on one device (host
    tensors go through dsa_indexer_fwd_host / v4_lighting_indexer)."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{where}: {name} must be a CUDA tensor, got "
                             f"{t.device}")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{where}: {name} is on {t.device}, the other "
                             f"tensors on {dev}")
    if dev is not None:
        _require_current(where, dev.index)


def _require_current(where: str, index: int):
    """Kernels run on the current device: tensors of another one are refused
    before it reads their pointers."""
    if index is not None and index != torch.cuda.current_device():
        raise ValueError(f"{where}: the tensors are on cuda:{index}, the "
                         f"current device is cuda:"
                         f"{torch.cuda.current_device()} (call within "
                         f"torch.cuda.device({index}))")


def _check_inputs(q, k, w, q_pos, in_idx):
    for name, t, dt in (("index_q", q, torch.bfloat16),
                        ("index_k", k, torch.bfloat16),
                        ("weights", w, torch.float32)):
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    S, B, H, D = q.shape
    S_kv = k.shape[0]
    if tuple(k.shape) != (S_kv, B, D):
        raise ValueError(f"index_k shape {tuple(k.shape)} != "
                         f"({S_kv}, {B}, {D})")
    if tuple(w.shape) != (S, B, H):
        raise ValueError(f"weights shape {tuple(w.shape)} != ({S}, {B}, {H})")
    if q_pos is not None and (q_pos.dtype != torch.int32
                              or q_pos.numel() != B):
        raise ValueError("q_pos must be int32 [B]")
    if in_idx is not None and (in_idx.dtype != torch.int32
                               or not in_idx.is_contiguous()):
        raise ValueError("topk_indices must be contiguous int32")
    return S, B, H, D, S_kv


def dsa_indexer_fwd(q, k, w, compress_ratio, topk, q_pos=None, in_idx=None,
                    out_idx=None, out_scores=None, workspace=None,
                    stream=None, stage_events=None):
    """Enqueue the forward on device tensors; returns (out_scores, out_idx,
    workspace).  Raises DsaError on a synchronous error.  `stage_events`
    (torch.cuda.Event created with enable_timing, at most 1024) are recorded
    before the first kernel and after each kernel launch, in launch order
    (dsa_indexer_fwd_launches gives the count); events left over after the
    last launch are recorded at the end."""
    lib = load_library()
    _require_cuda("dsa_indexer_fwd", q=q, k=k, w=w, q_pos=q_pos,
                  in_idx=in_idx, out_idx=out_idx, out_scores=out_scores,
                  workspace=workspace)
    S, B, H, D, S_kv = _check_inputs(q, k, w, q_pos, in_idx)
    dev = q.device
    if in_idx is not None and tuple(in_idx.shape) != (B, S, topk):
        raise ValueError("topk_indices must be [B, S, topk]")
    if out_idx is None:
        out_idx = _empty(stream, (B, S, topk), torch.int32, dev)
    if out_scores is None:
        out_scores = _empty(stream, (B, S, topk), torch.float32, dev)
    ws = dsa_indexer_workspace_size(S, B, H, D, S_kv, compress_ratio, topk,
                                    in_idx is not None)
    if workspace is None:
        workspace = _empty(stream, max(ws, 256), torch.uint8, dev)
    if stage_events:
        evs = (ctypes.c_void_p * len(stage_events))(
            *[ctypes.c_void_p(e.cuda_event) for e in stage_events])
        rc = lib.dsa_indexer_fwd_profiled(
            _ptr(q), _ptr(k), _ptr(w), S, B, H, D, S_kv, int(compress_ratio),
            int(topk), _ptr(q_pos), _ptr(in_idx), _ptr(out_idx),
            _ptr(out_scores), _ptr(workspace), workspace.numel(),
            _stream(stream), evs, len(stage_events))
    else:
        rc = lib.dsa_indexer_fwd(
            _ptr(q), _ptr(k), _ptr(w), S, B, H, D, S_kv, int(compress_ratio),
            int(topk), _ptr(q_pos), _ptr(in_idx), _ptr(out_idx),
            _ptr(out_scores), _ptr(workspace), workspace.numel(),
            _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_indexer_fwd")
    return out_scores, out_idx, workspace


def dsa_indexer_bwd_workspace_size() -> int:
    return int(load_library().dsa_indexer_bwd_workspace_size())


def dsa_indexer_bwd(q, k, w, compress_ratio, idx, grad_scores, q_pos=None,
                    grad_q=None, grad_k=None, grad_w=None, workspace=None,
                    stream=None):
    """Enqueue the backward of the given-slots scores on device tensors:
    idx [B, S, topk] int32 and grad_scores [B, S, topk] fp32 give grad_q
    [S, B, H, D], grad_k [S_kv, B, D] and grad_w [S, B, H] (fp32).  Returns
    (grad_q, grad_k, grad_w, workspace)."""
    lib = load_library()
    _require_cuda("dsa_indexer_bwd", q=q, k=k, w=w, idx=idx,
                  grad_scores=grad_scores, q_pos=q_pos, grad_q=grad_q,
                  grad_k=grad_k, grad_w=grad_w, workspace=workspace)
    S, B, H, D, S_kv = _check_inputs(q, k, w, q_pos, idx)
    topk = idx.shape[-1]
    if tuple(idx.shape) != (B, S, topk):
        raise ValueError("idx must be [B, S, topk]")
    if (grad_scores.dtype != torch.float32 or not grad_scores.is_contiguous()
            or tuple(grad_scores.shape) != (B, S, topk)):
        raise ValueError("grad_scores must be contiguous fp32 [B, S, topk]")
    dev = q.device
    if grad_q is None:
        grad_q = _empty(stream, (S, B, H, D), torch.float32, dev)
    if grad_k is None:
        grad_k = _empty(stream, (S_kv, B, D), torch.float32, dev)
    if grad_w is None:
        grad_w = _empty(stream, (S, B, H), torch.float32, dev)
    if workspace is None:
        workspace = _empty(stream, dsa_indexer_bwd_workspace_size(),
                           torch.uint8, dev)
    rc = lib.dsa_indexer_bwd(
        _ptr(q), _ptr(k), _ptr(w), S, B, H, D, S_kv, int(compress_ratio),
        int(topk), _ptr(q_pos), _ptr(idx), _ptr(grad_scores), _ptr(grad_q),
        _ptr(grad_k), _ptr(grad_w), _ptr(workspace), workspace.numel(),
        _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_indexer_bwd")
    return grad_q, grad_k, grad_w, workspace


def _pool_inputs(k, gate, ape, valid, kpool):
    if k.dtype != torch.bfloat16 or k.dim() != 3 or not k.is_contiguous():
        raise ValueError("k must be contiguous bf16 [T, B, D]")
    T, B, D = k.shape
    if (gate.dtype != torch.float32 or tuple(gate.shape) != (T, B, D)
            or not gate.is_contiguous()):
        raise ValueError("gate must be contiguous fp32 [T, B, D]")
    if (ape.dtype != torch.float32 or tuple(ape.shape) != (kpool, D)
            or not ape.is_contiguous()):
        raise ValueError("ape must be contiguous fp32 [kpool, D]")
    if valid is not None and (valid.dtype != torch.uint8
                              or tuple(valid.shape) != (T, B)
                              or not valid.is_contiguous()):
        raise ValueError("valid must be contiguous uint8 [T, B]")
    return T, B, D


def dsa_kpool_compress(k, gate, ape, kpool, first_key=0, valid=None,
                       stream=None):
    """Pool compression on device tensors: returns (keys [P, B, D] bf16,
    pool_valid [P, B] uint8)."""
    lib = load_library()
    _require_cuda("dsa_kpool_compress", k=k, gate=gate, ape=ape,
                  valid=valid)
    T, B, D = _pool_inputs(k, gate, ape, valid, kpool)
    P = max(0, (T - first_key) // kpool)
    keys = _empty(stream, (max(P, 1), B, D), torch.bfloat16, k.device)
    pv = _empty(stream, (max(P, 1), B), torch.uint8, k.device)
    rc = lib.dsa_kpool_compress(_ptr(k), _ptr(gate), _ptr(ape), _ptr(valid),
                                T, B, D, int(kpool), int(first_key),
                                _ptr(keys), _ptr(pv), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_kpool_compress")
    return keys[:P], pv[:P]


def dsa_expand_selection(pools, kpool, first_key=0, out=None, stream=None):
    """Pool ids [..., select_k] int32 -> token ids [..., select_k*kpool]."""
    lib = load_library()
    _require_cuda("dsa_expand_selection", pools=pools, out=out)
    if pools.dtype != torch.int32 or not pools.is_contiguous():
        raise ValueError("pools must be contiguous int32")
    select_k = pools.shape[-1]
    if out is None:
        out = _empty(stream, tuple(pools.shape[:-1]) + (select_k * kpool,),
                     torch.int32, pools.device)
    rows = pools.numel() // select_k
    rc = lib.dsa_expand_selection(_ptr(pools), rows, select_k, int(kpool),
                                  int(first_key), _ptr(out), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_expand_selection")
    return out


def dsa_indexer_pooled_workspace_size(S, B, H, D, T, kpool, first_key,
                                      index_topk) -> int:
    return int(load_library().dsa_indexer_pooled_workspace_size(
        S, B, H, D, T, kpool, first_key, index_topk))


def dsa_indexer_fwd_pooled(q, k, gate, ape, w, kpool, first_key, index_topk,
                           valid=None, q_pos=None, out_tokens=None,
                           out_pools=None, out_scores=None, workspace=None,
                           stream=None):
    """The pool variant on device tensors: q [S,B,H,D] bf16, per-token k
    [T,B,D] bf16, gate [T,B,D] fp32, ape [kpool,D] fp32, w [S,B,H] fp32,
    valid [T,B] uint8 or None.  Returns (tokens [B,S,index_topk] int32,
    pools [B,S,index_topk/kpool] int32, scores [B,S,index_topk/kpool] fp32,
    workspace)."""
    lib = load_library()
    _require_cuda("dsa_indexer_fwd_pooled", q=q, k=k, gate=gate, ape=ape,
                  w=w, valid=valid, q_pos=q_pos, out_tokens=out_tokens,
                  out_pools=out_pools, out_scores=out_scores,
                  workspace=workspace)
    T, B, D = _pool_inputs(k, gate, ape, valid, kpool)
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16")
    S, Bq, H, Dq = q.shape
    if (Bq, Dq) != (B, D) or tuple(w.shape) != (S, B, H):
        raise ValueError("q / w shapes do not match k")
    if index_topk % kpool:
        raise ValueError("index_topk must be a multiple of kpool")
    sk = index_topk // kpool
    dev = q.device
    if out_tokens is None:
        out_tokens = _empty(stream, (B, S, index_topk), torch.int32, dev)
    if out_pools is None:
        out_pools = _empty(stream, (B, S, sk), torch.int32, dev)
    if out_scores is None:
        out_scores = _empty(stream, (B, S, sk), torch.float32, dev)
    if workspace is None:
        n = dsa_indexer_pooled_workspace_size(S, B, H, D, T, kpool,
                                              first_key, index_topk)
        if n == 0:
            raise DsaError(2, "dsa_indexer_pooled_workspace_size")
        workspace = _empty(stream, n, torch.uint8, dev)
    rc = lib.dsa_indexer_fwd_pooled(
        _ptr(q), _ptr(k), _ptr(gate), _ptr(ape), _ptr(valid), _ptr(w), S, B,
        H, D, T, int(kpool), int(first_key), int(index_topk), _ptr(q_pos),
        _ptr(out_tokens), _ptr(out_pools), _ptr(out_scores), _ptr(workspace),
        workspace.numel(), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_indexer_fwd_pooled")
    return out_tokens, out_pools, out_scores, workspace


def dsa_sparse_mla_workspace_size() -> int:
    return int(load_library().dsa_sparse_mla_workspace_size())


def dsa_sparse_mla_fwd(q, c, idx, scale, out_o=None, out_lse=None,
                       workspace=None, stream=None):
    """Sparse MLA forward on device tensors: q [S,B,H,Dc] bf16, latent
    cache c [T,B,Dc] bf16, idx [B,S,topk] int32 token ids.  Returns (o
    [S,B,H,Dc] fp32, lse [S,B,H] fp32, workspace)."""
    lib = load_library()
    _require_cuda("dsa_sparse_mla_fwd", q=q, c=c, idx=idx, out_o=out_o,
                  out_lse=out_lse, workspace=workspace)
    for name, t, dt in (("q", q, torch.bfloat16), ("c", c, torch.bfloat16),
                        ("idx", idx, torch.int32)):
        if t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dt}")
    S, B, H, Dc = q.shape
    T = c.shape[0]
    if tuple(c.shape) != (T, B, Dc) or idx.shape[:2] != (B, S):
        raise ValueError("c must be [T, B, Dc] and idx [B, S, topk]")
    topk = idx.shape[-1]
    dev = q.device
    if out_o is None:
        out_o = _empty(stream, (S, B, H, Dc), torch.float32, dev)
    if out_lse is None:
        out_lse = _empty(stream, (S, B, H), torch.float32, dev)
    if workspace is None:
        workspace = _empty(stream, dsa_sparse_mla_workspace_size(),
                           torch.uint8, dev)
    rc = lib.dsa_sparse_mla_fwd(_ptr(q), _ptr(c), _ptr(idx), S, B, H, Dc, T,
                                topk, float(scale), _ptr(out_o),
                                _ptr(out_lse), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_sparse_mla_fwd")
    return out_o, out_lse, workspace


_ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def rope_inv_freq(rot_dim, base=10000.0, scaling=None, device=None):
    """Rotation frequencies [rot_dim / 2] fp64 (radians a position) of
    base^(-2i / rot_dim), and the factor on cos and sin (rot_scale).

    scaling: None, or a dict with "type" and "factor" (> 1) that stretches
    the positions for contexts longer than those trained on:
      "linear"  every frequency divided by factor (position interpolation);
      "ntk"     the base raised so that the lowest frequency is divided by
                factor and the highest stays;
      "yarn"    frequencies that turn more than "beta_fast" (32) times within
                "original_max_position" stay, those that turn less than
                "beta_slow" (1) times are divided by factor, a linear ramp
                over the index between; cos and sin are multiplied by
                0.1 ln(factor) + 1 (or "attention_factor").
    Returns (inv_freq, rot_scale)."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be positive and even")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    rot_scale = 1.0
    if scaling is None:
        inv = base ** (-2.0 * i / rot_dim)
    else:
        kind, factor = scaling["type"], float(scaling["factor"])
        if not factor >= 1.0:
            raise ValueError("the scaling factor must be at least 1")
        if kind == "linear":
            inv = base ** (-2.0 * i / rot_dim) / factor
        elif kind == "ntk":
            if rot_dim > 2:
                base = base * factor ** (rot_dim / (rot_dim - 2))
            inv = base ** (-2.0 * i / rot_dim)
        elif kind == "yarn":
            inv = base ** (-2.0 * i / rot_dim)
            length = float(scaling["original_max_position"])
            fast = float(scaling.get("beta_fast", 32))
            slow = float(scaling.get("beta_slow", 1))

            def index_of(turns):  # the index that turns this often
                return (rot_dim * math.log(length / (turns * 2 * math.pi))
                        / (2 * math.log(base)))
            lo = max(math.floor(index_of(fast)), 0)
            hi = min(math.ceil(index_of(slow)), rot_dim - 1)
            ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
            inv = inv * (1 - ramp) + inv / factor * ramp
            rot_scale = float(scaling.get("attention_factor",
                                          0.1 * math.log(factor) + 1.0))
        else:
            raise ValueError(f"unknown scaling type {kind!r}")
    return inv.to(device) if device is not None else inv, rot_scale


# The calls below run once a layer for a single token, where the host's time
# is the call's: their checks touch each tensor a few times only.
_I3, _I6 = ctypes.c_int64 * 3, ctypes.c_int64 * 6


def _on_gpu(where, names, *tensors):
    """_require_cuda() of the tensors by these names, without building device
    objects or a dict while all is well: the device's index."""
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()  # -1: not on a GPU
            if d < 0 or d != dev >= 0:
                break
            dev = d
    else:
        if dev != torch._C._cuda_getDevice():
            _require_current(where, dev)
        return dev
    _require_cuda(where, **dict(zip(names.split(), tensors)))


def _raw_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _strides(t):
    """Host array of the three leading element strides (None: dense)."""
    return None if t.is_contiguous() else _I3(*t.stride()[:3])


def _strides2(a, b):
    return (None if a.is_contiguous() and b.is_contiguous()
            else _I6(*a.stride()[:3], *b.stride()[:3]))


def _last_contiguous(name, t, dt, shape):
    if t.dtype != dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _dense(name, t, dt, shape):
    if t.dtype != dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rope_inputs(q, k, inv_freq, positions, wq, wk, dt, q_name="q",
                 k_name="k"):
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q [S, B, H, D] and k [S, B, Hk, D] expected")
    S, B, H, D = q.shape
    Hk = 0 if k is None else k.shape[2]
    _last_contiguous(q_name, q, dt, (S, B, H, D))
    if k is not None:
        _last_contiguous(k_name, k, dt, (S, B, Hk, D))
    if inv_freq is not None and (inv_freq.dtype != torch.float64
                                 or inv_freq.dim() != 1
                                 or not inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be contiguous fp64 [rot_dim / 2]")
    if positions is not None:
        _dense("positions", positions, torch.int32, (S, B))
    if wq is not None:
        _dense("w" + q_name, wq, torch.float32, (D,))
    if wk is not None:
        _dense("w" + k_name, wk, torch.float32, (D,))
    return S, B, H, Hk, D, 0 if inv_freq is None else 2 * inv_freq.numel()


def dsa_norm_rope_fwd(q, k, inv_freq, positions=None, wq=None, wk=None,
                      eps=1e-6, rot_start=0, interleaved=False,
                      rot_scale=1.0, out_q=None, out_k=None, stream=None):
    """Per-head RMS norm (where a weight is given) and rotation of q
    [S, B, H, D] and k [S, B, Hk, D] (or None) on device tensors, bf16, fp16
    or fp32 with any strides over a contiguous last dimension.  inv_freq
    [rot_dim / 2] fp64 (rope_inv_freq; None: no rotation), positions [S, B]
    int32 (None: row s at s).  Returns (out_q, out_k), dense."""
    lib = load_library()
    dev = _on_gpu("dsa_norm_rope_fwd",
                  "q k inv_freq positions wq wk out_q out_k",
                  q, k, inv_freq, positions, wq, wk, out_q, out_k)
    dt = q.dtype
    if dt not in _ROPE_DTYPES:
        raise TypeError(f"q must be bf16, fp16 or fp32, got {dt}")
    S, B, H, Hk, D, R = _rope_inputs(q, k, inv_freq, positions, wq, wk, dt)
    if out_q is None:
        out_q = _empty(stream, (S, B, H, D), dt, q.device)
    else:
        _dense("out_q", out_q, dt, (S, B, H, D))
    if k is not None:
        if out_k is None:
            out_k = _empty(stream, (S, B, Hk, D), dt, q.device)
        else:
            _dense("out_k", out_k, dt, (S, B, Hk, D))
    rc = lib.dsa_norm_rope_fwd(
        _addr(q), _strides(q), _addr(k), None if k is None else _strides(k),
        _ROPE_DTYPES[dt], S, B, H, Hk, D, _addr(wq), _addr(wk), float(eps),
        _addr(positions), _addr(inv_freq), int(rot_start), R,
        int(bool(interleaved)), float(rot_scale), _addr(out_q), _addr(out_k),
        _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_norm_rope_fwd")
    return out_q, out_k


def dsa_norm_rope_bwd_workspace_size(D) -> int:
    return int(load_library().dsa_norm_rope_bwd_workspace_size(int(D)))


def dsa_norm_rope_bwd(q, k, grad_out_q, grad_out_k, inv_freq, positions=None,
                      wq=None, wk=None, eps=1e-6, rot_start=0,
                      interleaved=False, rot_scale=1.0, workspace=None,
                      stream=None):
    """Backward of dsa_norm_rope_fwd from its inputs and the gradients of its
    outputs (dense).  Returns (grad_q, grad_k, grad_wq, grad_wk, workspace);
    the weights' gradients are fp32 [D], None without the weight."""
    lib = load_library()
    dev = _on_gpu("dsa_norm_rope_bwd",
                  "q k grad_out_q grad_out_k inv_freq positions wq wk "
                  "workspace",
                  q, k, grad_out_q, grad_out_k, inv_freq, positions, wq, wk,
                  workspace)
    dt = q.dtype
    if dt not in _ROPE_DTYPES:
        raise TypeError(f"q must be bf16, fp16 or fp32, got {dt}")
    S, B, H, Hk, D, R = _rope_inputs(q, k, inv_freq, positions, wq, wk, dt)
    _dense("grad_out_q", grad_out_q, dt, (S, B, H, D))
    gk = gwq = gwk = None
    gq = _empty(stream, (S, B, H, D), dt, q.device)
    if k is not None:
        if grad_out_k is None:
            raise ValueError("grad_out_k is needed with k")
        _dense("grad_out_k", grad_out_k, dt, (S, B, Hk, D))
        gk = _empty(stream, (S, B, Hk, D), dt, q.device)
    if wq is not None:
        gwq = _empty(stream, D, torch.float32, q.device)
    if wk is not None and k is not None:
        gwk = _empty(stream, D, torch.float32, q.device)
    if workspace is None:
        workspace = _empty(stream,
                           max(dsa_norm_rope_bwd_workspace_size(D), 256),
                           torch.uint8, q.device)
    rc = lib.dsa_norm_rope_bwd(
        _addr(q), _strides(q), _addr(k), None if k is None else _strides(k),
        _addr(grad_out_q), None if k is None else _addr(grad_out_k),
        _ROPE_DTYPES[dt], S, B, H, Hk, D, _addr(wq), _addr(wk), float(eps),
        _addr(positions), _addr(inv_freq), int(rot_start), R,
        int(bool(interleaved)), float(rot_scale), _addr(gq), _addr(gk),
        _addr(gwq), _addr(gwk), _addr(workspace), workspace.numel(),
        _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_norm_rope_bwd")
    return gq, gk, gwq, gwk, workspace


def _paged_cache(k_cache, v_cache, page_table, B):
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, Hk, D]")
    shape = tuple(k_cache.shape)
    _last_contiguous("k_cache", k_cache, torch.bfloat16, shape)
    _last_contiguous("v_cache", v_cache, torch.bfloat16, shape)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    _dense("page_table", page_table, torch.int32, (B, page_table.shape[1]))
    return shape


def dsa_paged_append(k, v, k_cache, v_cache, page_table, positions,
                     inv_freq=None, wk=None, eps=1e-6, rot_start=0,
                     interleaved=False, rot_scale=1.0, q=None, wq=None,
                     out_q=None, workspace=None, stream=None):
    """Append k and v [S, B, Hk, D] bf16 (any strides over a contiguous last
    dimension) at positions [S, B] int32 (< 0: skipped) to the paged caches
    [pages, page_size, Hk, D] through page_table [B, max_pages] int32, the
    keys normed and rotated as by dsa_norm_rope_fwd; q [S, B, H, D] given
    with them is normed and rotated into out_q in the same launch.  Returns
    (out_q, workspace).  The call only sets bits in the workspace's status
    word (256 zeroed bytes to begin with; dsa_indexer_check reads it); an
    indexer call in the same workspace clears it, so an error that has not been
    read by then is lost: give the append, or it and the block attention, a
    workspace of their own."""
    lib = load_library()
    dev = _on_gpu("dsa_paged_append",
                  "k v k_cache v_cache page_table positions inv_freq wk q "
                  "wq out_q workspace",
                  k, v, k_cache, v_cache, page_table, positions, inv_freq, wk,
                  q, wq, out_q, workspace)
    bf = torch.bfloat16
    S, B, Hk, H, D, R = _rope_inputs(k, q, inv_freq, positions, wk,
                                     None if q is None else wq, bf, "k", "q")
    _last_contiguous("v", v, bf, (S, B, Hk, D))
    pages, page_size, cache_heads, cache_dim = _paged_cache(
        k_cache, v_cache, page_table, B)
    if cache_heads != Hk or cache_dim != D:
        raise ValueError("the cache's heads or head size differ from k's")
    if q is not None:
        if out_q is None:
            out_q = _empty(stream, (S, B, H, D), bf, q.device)
        else:
            _dense("out_q", out_q, bf, (S, B, H, D))
    if workspace is None:
        workspace = _zeroed_workspace(stream, 256, k.device)
    rc = lib.dsa_paged_append(
        _addr(k), _strides(k), _addr(v), _strides(v), _addr(q),
        None if q is None else _strides(q), S, B, H, Hk, D, _addr(k_cache),
        _addr(v_cache), _strides2(k_cache, v_cache), pages, page_size,
        _addr(page_table), page_table.shape[1], _addr(positions), _addr(wq),
        _addr(wk), float(eps), _addr(inv_freq), int(rot_start), R,
        int(bool(interleaved)), float(rot_scale),
        None if q is None else _addr(out_q), _addr(workspace),
        workspace.numel(), _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_paged_append")
    return out_q, workspace


def dsa_block_attn_workspace_size(S, B, H, Hk, D, T, block_size, topk,
                                  local_blocks=0) -> int:
    """Workspace bytes of dsa_block_attn_fwd and, with T = max_pages *
    page_size, of dsa_block_attn_paged_fwd (0: invalid sizes)."""
    return int(load_library().dsa_block_attn_workspace_size(
        S, B, H, Hk, D, T, block_size, topk, local_blocks))


def dsa_block_attn_bwd_workspace_size(S, B, H, Hk, D, T, block_size, topk,
                                      local_blocks=0) -> int:
    return int(load_library().dsa_block_attn_bwd_workspace_size(
        S, B, H, Hk, D, T, block_size, topk, local_blocks))


def _selection(blocks, B, S, Hk, q_pos):
    """(sel_heads, topk) of blocks [B, S, topk] or [B, S, Hk, topk]."""
    if q_pos is not None:
        _dense("q_pos", q_pos, torch.int32, (B,))
    if blocks is None:
        return 1, 0
    if blocks.dim() == 3:
        shape = (B, S, blocks.shape[-1])
    else:
        shape = (B, S, Hk, blocks.shape[-1])
    _dense("blocks", blocks, torch.int32, shape)
    return (1 if blocks.dim() == 3 else Hk), blocks.shape[-1]


def _block_attn_out(q, shape, out_o, out_lse, workspace, stream,
                    workspace_size=dsa_block_attn_workspace_size):
    """The outputs and the workspace of a forward, made where not given."""
    S, B, H, D = q.shape
    if out_o is None:
        out_o = (torch.empty_like(q) if stream is None  # (q is dense)
                 else _empty(stream, (S, B, H, D), q.dtype, q.device))
    else:
        _dense("out_o", out_o, torch.bfloat16, (S, B, H, D))
    if out_lse is None:
        out_lse = _empty(stream, (S, B, H), torch.float32, q.device)
    else:
        _dense("out_lse", out_lse, torch.float32, (S, B, H))
    if workspace is None:
        size = workspace_size(*shape)
        if size == 0:
            raise DsaError(1, workspace_size.__name__)
        workspace = _zeroed_workspace(stream, size, q.device)
    return out_o, out_lse, workspace


def dsa_block_attn_fwd(q, k, v, blocks, block_size, scale, q_pos=None,
                       local_blocks=0, out_o=None, out_lse=None,
                       workspace=None, stream=None):
    """Attention over selected blocks on device tensors: q [S, B, H, D] bf16,
    k and v [T, B, Hk, D] bf16 (any strides over a contiguous last
    dimension), blocks [B, S, topk] or [B, S, Hk, topk] int32 block ids (-1:
    empty; None: local blocks only), q_pos [B] int32 (row s at q_pos[b] + s;
    None: at s), local_blocks trailing blocks always attended to.  Returns
    (o [S, B, H, D] bf16, lse [S, B, H] fp32, workspace); a workspace of the
    caller's has its first 256 bytes zeroed once, before its first use."""
    lib = load_library()
    dev = _on_gpu("dsa_block_attn_fwd",
                  "q k v blocks q_pos out_o out_lse workspace",
                  q, k, v, blocks, q_pos, out_o, out_lse, workspace)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q [S, B, H, D] and k [T, B, Hk, D] expected")
    S, B, H, D = q.shape
    T, _, Hk, _ = k.shape
    _dense("q", q, torch.bfloat16, (S, B, H, D))
    _last_contiguous("k", k, torch.bfloat16, (T, B, Hk, D))
    _last_contiguous("v", v, torch.bfloat16, (T, B, Hk, D))
    sel_heads, topk = _selection(blocks, B, S, Hk, q_pos)
    out_o, out_lse, workspace = _block_attn_out(
        q, (S, B, H, Hk, D, T, block_size, topk, local_blocks), out_o,
        out_lse, workspace, stream)
    rc = lib.dsa_block_attn_fwd(
        _addr(q), _addr(k), _addr(v), _strides2(k, v), S, B, H, Hk, D, T,
        _addr(blocks), sel_heads, topk, int(block_size), int(local_blocks),
        _addr(q_pos), float(scale), _addr(out_o), _addr(out_lse),
        _addr(workspace), workspace.numel(), _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_block_attn_fwd")
    return out_o, out_lse, workspace


def dsa_block_attn_paged_fwd(q, k_cache, v_cache, page_table, blocks,
                             block_size, scale, q_pos=None, local_blocks=0,
                             out_o=None, out_lse=None, workspace=None,
                             stream=None):
    """dsa_block_attn_fwd over paged caches [pages, page_size, Hk, D] bf16
    through page_table [B, max_pages] int32 (S = 1: one token of each
    sequence at q_pos[b])."""
    lib = load_library()
    dev = _on_gpu("dsa_block_attn_paged_fwd",
                  "q k_cache v_cache page_table blocks q_pos out_o out_lse "
                  "workspace",
                  q, k_cache, v_cache, page_table, blocks, q_pos, out_o,
                  out_lse, workspace)
    if q.dim() != 4:
        raise ValueError("q [S, B, H, D] expected")
    S, B, H, D = q.shape
    _dense("q", q, torch.bfloat16, (S, B, H, D))
    pages, page_size, Hk, Dk = _paged_cache(k_cache, v_cache, page_table, B)
    if Dk != D:
        raise ValueError(f"the cache's head size {Dk} differs from q's {D}")
    max_pages = page_table.shape[1]
    sel_heads, topk = _selection(blocks, B, S, Hk, q_pos)
    out_o, out_lse, workspace = _block_attn_out(
        q, (S, B, H, Hk, D, max_pages * page_size, block_size, topk,
            local_blocks), out_o, out_lse, workspace, stream)
    rc = lib.dsa_block_attn_paged_fwd(
        _addr(q), _addr(k_cache), _addr(v_cache), _strides2(k_cache, v_cache),
        pages, page_size, _addr(page_table), max_pages, S, B, H, Hk, D,
        _addr(blocks), sel_heads, topk, int(block_size), int(local_blocks),
        _addr(q_pos), float(scale), _addr(out_o), _addr(out_lse),
        _addr(workspace), workspace.numel(), _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_block_attn_paged_fwd")
    return out_o, out_lse, workspace


def dsa_block_attn_bwd(q, k, v, o, lse, grad_o, blocks, block_size, scale,
                       q_pos=None, local_blocks=0, grad_q=None, grad_k=None,
                       grad_v=None, workspace=None, stream=None):
    """Backward of dsa_block_attn_fwd from its inputs, its outputs o and lse,
    and grad_o [S, B, H, D] bf16.  Returns (grad_q [S, B, H, D], grad_k and
    grad_v [T, B, Hk, D], dense bf16, workspace)."""
    lib = load_library()
    dev = _on_gpu("dsa_block_attn_bwd",
                  "q k v o lse grad_o blocks q_pos grad_q grad_k grad_v "
                  "workspace",
                  q, k, v, o, lse, grad_o, blocks, q_pos, grad_q, grad_k,
                  grad_v, workspace)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q [S, B, H, D] and k [T, B, Hk, D] expected")
    S, B, H, D = q.shape
    T, _, Hk, _ = k.shape
    bf = torch.bfloat16
    for name, t in (("q", q), ("o", o), ("grad_o", grad_o)):
        _dense(name, t, bf, (S, B, H, D))
    _dense("lse", lse, torch.float32, (S, B, H))
    _last_contiguous("k", k, bf, (T, B, Hk, D))
    _last_contiguous("v", v, bf, (T, B, Hk, D))
    sel_heads, topk = _selection(blocks, B, S, Hk, q_pos)
    if grad_q is None:
        grad_q = _empty(stream, (S, B, H, D), bf, q.device)
    else:
        _dense("grad_q", grad_q, bf, (S, B, H, D))
    if grad_k is None:
        grad_k = _empty(stream, (T, B, Hk, D), bf, q.device)
    else:
        _dense("grad_k", grad_k, bf, (T, B, Hk, D))
    if grad_v is None:
        grad_v = _empty(stream, (T, B, Hk, D), bf, q.device)
    else:
        _dense("grad_v", grad_v, bf, (T, B, Hk, D))
    if workspace is None:
        n = dsa_block_attn_bwd_workspace_size(S, B, H, Hk, D, T, block_size,
                                              topk, local_blocks)
        # (0: invalid or not supported, and the call below says which)
        workspace = _zeroed_workspace(stream, max(n, 256), q.device)
    rc = lib.dsa_block_attn_bwd(
        _addr(q), _addr(k), _addr(v), _strides2(k, v), _addr(o), _addr(lse),
        _addr(grad_o), S, B, H, Hk, D, T, _addr(blocks), sel_heads, topk,
        int(block_size), int(local_blocks), _addr(q_pos), float(scale),
        _addr(grad_q), _addr(grad_k), _addr(grad_v), _addr(workspace),
        workspace.numel(), _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_block_attn_bwd")
    return grad_q, grad_k, grad_v, workspace


# The three calls below look at each tensor once, all in one expression; where
# that does not hold, the named checks say what is wrong (or that a layout is
# fine after all: strided caches).
_BF, _E4M3 = torch.bfloat16, torch.float8_e4m3fn
_F32, _I32 = torch.float32, torch.int32
_I9 = ctypes.c_int64 * 9


def _cache_q8_ok(dev, k_cache, v_cache, k_scale, v_scale, page_table):
    """Whether these are the dense tensors of an 8-bit cache on device dev."""
    shape = k_cache.shape
    return (k_cache.dtype is _E4M3 and v_cache.dtype is _E4M3
            and k_scale.dtype is _F32 and v_scale.dtype is _F32
            and page_table.dtype is _I32 and v_cache.shape == shape
            and v_scale.shape == k_scale.shape
            and k_cache.get_device() == dev and v_cache.get_device() == dev
            and k_scale.get_device() == dev and v_scale.get_device() == dev
            and page_table.get_device() == dev and k_cache.is_contiguous()
            and v_cache.is_contiguous() and k_scale.is_contiguous()
            and v_scale.is_contiguous() and page_table.is_contiguous())


def _cache_q8_sizes(k_cache, k_scale, page_table):
    """(pages, page_size, Hk, D, group, B, max_pages)."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, Hk, D]")
    if k_scale.dim() != 3:
        raise ValueError("k_scale must be [pages, page_size / group, Hk]")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    pages, page_size, Hk, D = k_cache.shape
    pages_s, n, heads_s = k_scale.shape
    if n <= 0 or page_size % n:
        raise ValueError(f"k_scale: {n} scales do not divide a page of "
                         f"{page_size} tokens")
    if pages_s != pages or heads_s != Hk:
        raise ValueError(f"k_scale shape {tuple(k_scale.shape)} != "
                         f"{(pages, n, Hk)}")
    B, max_pages = page_table.shape
    return pages, page_size, Hk, D, page_size // n, B, max_pages


def _check_cache_q8(k_cache, v_cache, k_scale, v_scale, page_table):
    _last_contiguous("k_cache", k_cache, _E4M3, k_cache.shape)
    _last_contiguous("v_cache", v_cache, _E4M3, k_cache.shape)
    _dense("k_scale", k_scale, _F32, k_scale.shape)
    _dense("v_scale", v_scale, _F32, k_scale.shape)
    _dense("page_table", page_table, _I32, page_table.shape)


def _three_strides(k, v, q):
    """Host arrays of k's, v's and q's leading strides: addresses in one
    array, which the caller keeps."""
    a = _I9(*k.stride()[:3], *v.stride()[:3],
            *((0, 0, 0) if q is None else q.stride()[:3]))
    at = ctypes.addressof(a)
    return a, at, at + 24, None if q is None else at + 48


def dsa_paged_append_q8(k, v, k_cache, v_cache, k_scale, v_scale, page_table,
                        start, count=None, inv_freq=None, wk=None, eps=1e-6,
                        rot_start=0, interleaved=False, rot_scale=1.0, q=None,
                        wq=None, out_q=None, workspace=None, stream=None):
    """Append rows s < count[b] of k and v [S, B, Hk, D] bf16 (any strides
    over a contiguous last dimension; count [B] int32, None: all rows) at
    positions start[b] + s (start [B] int32; < 0: nothing is appended) to
    paged caches held in 8 bits: k_cache, v_cache [pages, page_size, Hk, D]
    float8_e4m3fn, k_scale, v_scale [pages, page_size / group, Hk] fp32, a
    power of two for each group of tokens and head.  The keys are normed and
    rotated as by dsa_norm_rope_fwd; q [S, B, H, D] given with them is normed
    and rotated into out_q in the same launch.  An append ends its sequence: a
    group's scale may grow with it, which rounds the group's earlier tokens
    again.  Returns (out_q, workspace); the status word is that of
    dsa_paged_append."""
    lib = _lib or load_library()
    dev = k.get_device()
    pages, page_size, Hk, D, group, B, max_pages = _cache_q8_sizes(
        k_cache, k_scale, page_table)
    if k.dim() != 4 or (q is not None and q.dim() != 4):
        raise ValueError("q [S, B, H, D] and k [S, B, Hk, D] expected")
    S = k.shape[0]
    shape = (S, B, Hk, D)
    H, R = 0, 0
    if q is not None:
        H = q.shape[2]
    if inv_freq is not None:
        R = 2 * inv_freq.numel()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice()
            and _cache_q8_ok(dev, k_cache, v_cache, k_scale, v_scale,
                             page_table)
            and k.dtype is _BF and v.dtype is _BF and k.shape == shape
            and v.shape == shape and k.stride(3) == 1 and v.stride(3) == 1
            and v.get_device() == dev
            and start.dtype is _I32 and start.shape == (B,)
            and start.is_contiguous() and start.get_device() == dev
            and (count is None or (
                count.dtype is _I32 and count.shape == (B,)
                and count.is_contiguous() and count.get_device() == dev))
            and (q is None or (
                q.dtype is _BF and q.shape == (S, B, H, D)
                and q.stride(3) == 1 and q.get_device() == dev))
            and (inv_freq is None or (
                inv_freq.dtype is torch.float64 and inv_freq.dim() == 1
                and inv_freq.is_contiguous() and inv_freq.get_device() == dev))
            and (wk is None or (
                wk.dtype is _F32 and wk.shape == (D,) and wk.is_contiguous()
                and wk.get_device() == dev))
            and (wq is None or (
                wq.dtype is _F32 and wq.shape == (D,) and wq.is_contiguous()
                and wq.get_device() == dev))
            and (workspace is None or workspace.get_device() == dev)
            and (out_q is None or out_q.get_device() == dev)):
        dev = _on_gpu("dsa_paged_append_q8",
                      "k v k_cache v_cache k_scale v_scale page_table start "
                      "count inv_freq wk q wq out_q workspace",
                      k, v, k_cache, v_cache, k_scale, v_scale, page_table,
                      start, count, inv_freq, wk, q, wq, out_q, workspace)
        _rope_inputs(k, q, inv_freq, None, wk, wq, _BF, "k", "q")
        _last_contiguous("k", k, _BF, shape)
        _last_contiguous("v", v, _BF, shape)
        _check_cache_q8(k_cache, v_cache, k_scale, v_scale, page_table)
        _dense("start", start, _I32, (B,))
        if count is not None:
            _dense("count", count, _I32, (B,))
    if q is not None:
        if out_q is None:
            out_q = _empty(stream, (S, B, H, D), _BF, q.device)
        else:
            _dense("out_q", out_q, _BF, (S, B, H, D))
    if workspace is None:
        workspace = _zeroed_workspace(stream, 256, k.device)
    keep, k_st, v_st, q_st = _three_strides(k, v, q)
    rc = lib.dsa_paged_append_q8(
        k.data_ptr(), k_st, v.data_ptr(), v_st, _addr(q), q_st, S, B, H, Hk,
        D, k_cache.data_ptr(), v_cache.data_ptr(), _strides2(k_cache, v_cache),
        k_scale.data_ptr(), v_scale.data_ptr(), group, pages, page_size,
        page_table.data_ptr(), max_pages, start.data_ptr(), _addr(count),
        None if q is None else _addr(wq), _addr(wk), float(eps),
        _addr(inv_freq), int(rot_start), R, 1 if interleaved else 0,
        float(rot_scale),
        None if q is None else out_q.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _raw_stream(stream, dev))
    del keep
    if rc != 0:
        raise DsaError(rc, "dsa_paged_append_q8")
    return out_q, workspace


def dsa_paged_read_q8(k_cache, v_cache, k_scale, v_scale, page_table, T,
                      first=None, length=None, out_k=None, out_v=None,
                      workspace=None, stream=None):
    """Read a cache held in 8 bits back: (k, v, workspace), k and v [T, B, Hk,
    D] bf16 with row t of sequence b token first[b] + t (first [B] int32,
    None: t) where t < length[b] (None: T), zeros behind.  For caches as
    dsa_paged_append_q8 writes them."""
    lib = _lib or load_library()
    dev = k_cache.get_device()
    pages, page_size, Hk, D, group, B, max_pages = _cache_q8_sizes(
        k_cache, k_scale, page_table)
    T = int(T)
    shape = (T, B, Hk, D)
    if not (dev >= 0 and dev == torch._C._cuda_getDevice()
            and _cache_q8_ok(dev, k_cache, v_cache, k_scale, v_scale,
                             page_table)
            and (first is None or (
                first.dtype is _I32 and first.shape == (B,)
                and first.is_contiguous() and first.get_device() == dev))
            and (length is None or (
                length.dtype is _I32 and length.shape == (B,)
                and length.is_contiguous() and length.get_device() == dev))
            and (workspace is None or workspace.get_device() == dev)
            and out_k is None and out_v is None):
        dev = _on_gpu("dsa_paged_read_q8",
                      "k_cache v_cache k_scale v_scale page_table first "
                      "length out_k out_v workspace",
                      k_cache, v_cache, k_scale, v_scale, page_table, first,
                      length, out_k, out_v, workspace)
        _check_cache_q8(k_cache, v_cache, k_scale, v_scale, page_table)
        for name, t in (("first", first), ("length", length)):
            if t is not None:
                _dense(name, t, _I32, (B,))
        for name, t in (("out_k", out_k), ("out_v", out_v)):
            if t is not None:
                _dense(name, t, _BF, shape)
    if out_k is None:
        out_k = _empty(stream, shape, _BF, k_cache.device)
    if out_v is None:
        out_v = _empty(stream, shape, _BF, k_cache.device)
    if workspace is None:
        workspace = _zeroed_workspace(stream, 256, k_cache.device)
    rc = lib.dsa_paged_read_q8(
        k_cache.data_ptr(), v_cache.data_ptr(), _strides2(k_cache, v_cache),
        k_scale.data_ptr(), v_scale.data_ptr(), group, pages, page_size,
        page_table.data_ptr(), max_pages, T, B, Hk, D, _addr(first),
        _addr(length), out_k.data_ptr(), out_v.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_paged_read_q8")
    return out_k, out_v, workspace


def dsa_block_attn_q8_workspace_size(S, B, H, Hk, D, T, block_size, topk,
                                     local_blocks=0) -> int:
    """Workspace bytes of dsa_block_attn_paged_q8_fwd, T = max_pages *
    page_size (0: invalid sizes)."""
    return int(load_library().dsa_block_attn_q8_workspace_size(
        S, B, H, Hk, D, T, block_size, topk, local_blocks))


def dsa_block_attn_paged_q8_fwd(q, k_cache, v_cache, k_scale, v_scale,
                                page_table, blocks, block_size, scale,
                                q_pos=None, local_blocks=0, out_o=None,
                                out_lse=None, workspace=None, stream=None):
    """dsa_block_attn_paged_fwd over caches held in 8 bits, as
    dsa_paged_append_q8 writes them.  blocks None with local_blocks =
    max_pages * page_size / block_size: all keys up to each row's position."""
    lib = _lib or load_library()
    dev = q.get_device()
    if q.dim() != 4:
        raise ValueError("q [S, B, H, D] expected")
    pages, page_size, Hk, Dk, group, Bt, max_pages = _cache_q8_sizes(
        k_cache, k_scale, page_table)
    S, B, H, D = q.shape
    sel_heads, topk = 1, 0
    ids = None
    if blocks is not None:
        topk = blocks.shape[-1]
        if blocks.dim() == 3:
            ids = (B, S, topk)
        else:
            ids, sel_heads = (B, S, Hk, topk), Hk
    if not (dev >= 0 and dev == torch._C._cuda_getDevice()
            and _cache_q8_ok(dev, k_cache, v_cache, k_scale, v_scale,
                             page_table)
            and q.dtype is _BF and q.is_contiguous() and Dk == D and Bt == B
            and (blocks is None or (
                blocks.dtype is _I32 and blocks.shape == ids
                and blocks.is_contiguous() and blocks.get_device() == dev))
            and (q_pos is None or (
                q_pos.dtype is _I32 and q_pos.shape == (B,)
                and q_pos.is_contiguous() and q_pos.get_device() == dev))
            and (workspace is None or workspace.get_device() == dev)
            and (out_o is None or out_o.get_device() == dev)
            and (out_lse is None or out_lse.get_device() == dev)):
        dev = _on_gpu("dsa_block_attn_paged_q8_fwd",
                      "q k_cache v_cache k_scale v_scale page_table blocks "
                      "q_pos out_o out_lse workspace",
                      q, k_cache, v_cache, k_scale, v_scale, page_table,
                      blocks, q_pos, out_o, out_lse, workspace)
        _dense("q", q, _BF, q.shape)
        _check_cache_q8(k_cache, v_cache, k_scale, v_scale, page_table)
        if Bt != B:
            raise ValueError(f"page_table is for {Bt} sequences, q for {B}")
        if Dk != D:
            raise ValueError(f"the cache's head size {Dk} differs from q's "
                             f"{D}")
        _selection(blocks, B, S, Hk, q_pos)
    out_o, out_lse, workspace = _block_attn_out(
        q, (S, B, H, Hk, D, max_pages * page_size, block_size, topk,
            local_blocks), out_o, out_lse, workspace, stream,
        dsa_block_attn_q8_workspace_size)
    rc = lib.dsa_block_attn_paged_q8_fwd(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _strides2(k_cache, v_cache), k_scale.data_ptr(), v_scale.data_ptr(),
        group, pages, page_size, page_table.data_ptr(), max_pages, S, B, H, Hk,
        D, _addr(blocks), sel_heads, topk, int(block_size), int(local_blocks),
        _addr(q_pos), float(scale), out_o.data_ptr(), out_lse.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if rc != 0:
        raise DsaError(rc, "dsa_block_attn_paged_q8_fwd")
    return out_o, out_lse, workspace


def dsa_indexer_logits(q, k, w, compress_ratio, q_pos=None, logits=None,
                       workspace=None, stream=None):
    """Enqueue the scoring step alone: logits [B, S, S_kv] fp32 (-inf where
    a key is not visible).  Returns (logits, workspace)."""
    lib = load_library()
    _require_cuda("dsa_indexer_logits", q=q, k=k, w=w, q_pos=q_pos,
                  logits=logits, workspace=workspace)
    S, B, H, D, S_kv = _check_inputs(q, k, w, q_pos, None)
    dev = q.device
    if logits is None:
        logits = _empty(stream, (B, S, S_kv), torch.float32, dev)
    if workspace is None:
        workspace = _empty(stream,
                           int(lib.dsa_indexer_logits_workspace_size()),
                           torch.uint8, dev)
    rc = lib.dsa_indexer_logits(
        _ptr(q), _ptr(k), _ptr(w), S, B, H, D, S_kv, int(compress_ratio),
        _ptr(q_pos), _ptr(logits), _ptr(workspace), workspace.numel(),
        _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_indexer_logits")
    return logits, workspace


def dsa_indexer_check(workspace, stream=None) -> int:
    """Synchronise the stream and return the device status code (0 = ok)."""
    _require_cuda("dsa_indexer_check", workspace=workspace)
    return int(load_library().dsa_indexer_check(_ptr(workspace),
                                                 _stream(stream)))


def dsa_selftest_wait_limit(limit_us: int, workspace, stream=None) -> int:
    _require_cuda("dsa_selftest_wait_limit", workspace=workspace)
    return int(load_library().dsa_selftest_wait_limit(
        int(limit_us), _ptr(workspace), workspace.numel(), _stream(stream)))


def _host_i32(a):
    """A contiguous host int32 tensor (kept alive by the caller)."""
    t = torch.as_tensor(a, dtype=torch.int32, device="cpu").contiguous()
    return t


def dsa_indexer_varlen_workspace_size(cu_seqlens_q, cu_seqlens_k, H, D,
                                      compress_ratio, topk,
                                      has_in_idx=False) -> int:
    cq, ck = _host_i32(cu_seqlens_q), _host_i32(cu_seqlens_k)
    if cq.numel() != ck.numel() or cq.numel() < 2:
        raise ValueError("cu_seqlens_q / cu_seqlens_k must both be [N + 1]")
    return int(load_library().dsa_indexer_varlen_workspace_size(
        cq.numel() - 1, _ptr(cq), _ptr(ck), H, D, compress_ratio, topk,
        int(bool(has_in_idx))))


def dsa_indexer_fwd_varlen(q, k, w, cu_seqlens_q, cu_seqlens_k,
                           compress_ratio, topk, q_pos=None, in_idx=None,
                           out_idx=None, out_scores=None, workspace=None,
                           stream=None):
    """The forward over packed variable-length sequences: q [T, H, D] bf16,
    k [T_kv, D] bf16, w [T, H] fp32 and the optional q_pos [N] / in_idx
    [T, topk] on the device; cu_seqlens_q / cu_seqlens_k are host int32
    offsets [N + 1].  Returns (out_scores [T, topk], out_idx [T, topk],
    workspace); indices are local to each row's sequence."""
    lib = load_library()
    _require_cuda("dsa_indexer_fwd_varlen", q=q, k=k, w=w, q_pos=q_pos,
                  in_idx=in_idx, out_idx=out_idx, out_scores=out_scores,
                  workspace=workspace)
    cq, ck = _host_i32(cu_seqlens_q), _host_i32(cu_seqlens_k)
    N = cq.numel() - 1
    if ck.numel() != N + 1 or N < 1:
        raise ValueError("cu_seqlens_q / cu_seqlens_k must both be [N + 1]")
    if q.dim() != 3 or k.dim() != 2 or w.dim() != 2:
        raise ValueError("q [T, H, D], k [T_kv, D], w [T, H] expected")
    T, H, D = q.shape
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16),
                        ("w", w, torch.float32)):
        if t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dt}")
    if int(cq[-1]) != T or int(ck[-1]) != k.shape[0] or k.shape[1] != D or \
            tuple(w.shape) != (T, H):
        raise ValueError("shapes do not match the offsets")
    if q_pos is not None and (q_pos.dtype != torch.int32 or
                              q_pos.numel() != N):
        raise ValueError("q_pos must be int32 [N]")
    if in_idx is not None and (in_idx.dtype != torch.int32 or
                               tuple(in_idx.shape) != (T, topk) or
                               not in_idx.is_contiguous()):
        raise ValueError("in_idx must be contiguous int32 [T, topk]")
    dev = q.device
    if out_idx is None:
        out_idx = _empty(stream, (T, topk), torch.int32, dev)
    if out_scores is None:
        out_scores = _empty(stream, (T, topk), torch.float32, dev)
    if workspace is None:
        need = dsa_indexer_varlen_workspace_size(cq, ck, H, D,
                                                 compress_ratio, topk,
                                                 in_idx is not None)
        if need == 0:
            raise DsaError(2, "dsa_indexer_varlen_workspace_size")
        workspace = _empty(stream, need, torch.uint8, dev)
    rc = lib.dsa_indexer_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(w), N, _ptr(cq), _ptr(ck), H, D,
        int(compress_ratio), int(topk), _ptr(q_pos), _ptr(in_idx),
        _ptr(out_idx), _ptr(out_scores), _ptr(workspace), workspace.numel(),
        _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_indexer_fwd_varlen")
    return out_scores, out_idx, workspace


def dsa_indexer_host_buffer_size(S, B, H, D, S_kv, compress_ratio, topk,
                                 has_in_idx=False) -> int:
    return int(load_library().dsa_indexer_host_buffer_size(
        S, B, H, D, S_kv, compress_ratio, topk, int(bool(has_in_idx))))


def dsa_indexer_host_plan(S, B, H, D, S_kv, compress_ratio, topk,
                          q_pos=None, has_in_idx=False, sms=0):
    """How dsa_indexer_fwd_host splits and orders the query rows: returns
    (chunk starts, the last one S; processing order).  q_pos: host int32
    [B] or None.  sms: the SM count the chunk starts assume (0: the current
    device's).  Raises DsaError for an invalid shape."""
    lib = load_library()
    starts = (ctypes.c_int * 17)()
    order = (ctypes.c_int * 16)()
    pos = None
    if q_pos is not None:
        pos = _host_i32(q_pos)
    n = lib.dsa_indexer_host_plan(
        S, B, H, D, S_kv, int(compress_ratio), int(topk),
        None if pos is None else pos.data_ptr(), int(bool(has_in_idx)),
        int(sms), starts, order)
    if n <= 0:
        raise DsaError(1, "dsa_indexer_host_plan")
    return list(starts[:n + 1]), list(order[:n])


def dsa_indexer_fwd_host(q, k, w, compress_ratio, topk, q_pos=None,
                         in_idx=None, out_idx=None, out_scores=None,
                         device_buf=None, stream=None):
    """The forward on host (CPU) tensors through the C entry point that
    pipelines the copies against the kernels; returns (out_scores, out_idx,
    status).  Outputs are page-locked when q is.  `device_buf` (uint8 on the
    current CUDA device) is allocated when not given.  The call returns with
    the results in the host outputs; `status` is the library's return code
    (0, or the device status of the run)."""
    lib = load_library()
    S, B, H, D, S_kv = _check_inputs(q, k, w, q_pos, in_idx)
    for name, t in (("index_q", q), ("index_k", k), ("weights", w),
                    ("q_pos", q_pos), ("topk_indices", in_idx),
                    ("out_idx", out_idx), ("out_scores", out_scores)):
        if t is not None and t.device.type != "cpu":
            raise ValueError(f"{name} must be a host tensor")
    _require_cuda("dsa_indexer_fwd_host", device_buf=device_buf)
    if in_idx is not None and tuple(in_idx.shape) != (B, S, topk):
        raise ValueError("topk_indices must be [B, S, topk]")
    pinned = q.is_pinned()
    if out_idx is None:
        out_idx = torch.empty((B, S, topk), dtype=torch.int32,
                              pin_memory=pinned)
    if out_scores is None:
        out_scores = torch.empty((B, S, topk), dtype=torch.float32,
                                 pin_memory=pinned)
    need = dsa_indexer_host_buffer_size(S, B, H, D, S_kv, compress_ratio,
                                        topk, in_idx is not None)
    if need == 0:
        raise DsaError(2, "dsa_indexer_host_buffer_size")
    if device_buf is None:
        device_buf = _empty(stream, need, torch.uint8,
                            torch.device("cuda", torch.cuda.current_device()))
    rc = lib.dsa_indexer_fwd_host(
        _ptr(q), _ptr(k), _ptr(w), S, B, H, D, S_kv, int(compress_ratio),
        int(topk), _ptr(q_pos), _ptr(in_idx), _ptr(out_idx),
        _ptr(out_scores), _ptr(device_buf), device_buf.numel(),
        _stream(stream))
    if rc not in (0, 5, 6):  # device status codes are returned, not raised
        raise DsaError(rc, "dsa_indexer_fwd_host")
    return out_scores, out_idx, rc


def v4_lighting_indexer(index_q, index_k, weights, compress_ratio, topk,
                        topk_indices=None, q_pos=None, check=True):
    """The indexer forward with the V4 argument order.

    Device tensors run on the current stream.  Host (CPU) tensors are copied
    to the current CUDA device, run there, and the results copied back into
    host tensors (pinned when the inputs are pinned); the whole host round
    trip happens inside this call.  Returns (scores [B,S,topk] fp32,
    indices [B,S,topk] int32).  With check=True the call synchronises and
    raises on a device-side status (bad given index, expired wait).
    """
    if index_q.device.type == "cpu":
        # host buffers: the C entry point copies in, runs and copies out,
        # overlapping the copies with the kernels
        scores, idx, rc = dsa_indexer_fwd_host(
            index_q, index_k, weights, compress_ratio, topk, q_pos=q_pos,
            in_idx=topk_indices)
        if check and rc != 0:
            raise DsaError(rc, "device status")
        return scores, idx
    scores, idx, ws = dsa_indexer_fwd(index_q, index_k, weights,
                                      compress_ratio, topk, q_pos=q_pos,
                                      in_idx=topk_indices)
    if check:
        rc = dsa_indexer_check(ws)
        if rc != 0:
            raise DsaError(rc, "device status")
    return scores, idx


def indexer_logits(index_q, index_k, weights, compress_ratio, q_pos=None):
    """Logits [B, S, S_kv] fp32 on the device (-inf where masked)."""
    logits, _ = dsa_indexer_logits(index_q, index_k, weights, compress_ratio,
                                   q_pos=q_pos)
    return logits
