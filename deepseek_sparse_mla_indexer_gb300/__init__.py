"""Python binding of the sparse-attention C ABI (include/nsa.h).

Argument marshalling only: every computation runs in libnsa.so's CUDA
kernels (the local virtual-batch builder runs in its host C++).  Device
buffers are torch CUDA tensors; work is enqueued on the current torch stream
unless `stream` is given.  There is no CPU fallback: if the library cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Dict, Optional

import numpy as np
import torch

from . import _build

__all__ = [
    "NsaError", "load", "MODE_DECODE", "MODE_EXTEND", "MODE_TARGET_VERIFY", "DT_F32", "DT_BF16",
    "DT_E4M3", "nsa_metadata", "alloc_metadata", "alloc_score_hist", "nsa_local_virtual_batches", "nsa_effective_chunk_size",
    "nsa_indexer_logits", "nsa_topk_transform", "nsa_topk_launches", "nsa_sparse_mla",
    "nsa_sparse_mla_workspace_bytes", "nsa_sparse_mla_plan", "nsa_set_mla_kv", "nsa_quantize_kv_cache", "nsa_dequantize_kv_paged",
    "nsa_set_index_k", "nsa_topk_transform_ragged", "nsa_flatten_page_table", "nsa_copy_buffers",
    "nsa_check_bounded_wait", "nsa_local_attention", "nsa_paged_mla", "nsa_paged_mla_workspace_bytes",
    "alloc_paged_mla_workspace", "nsa_mla_key_weights", "nsa_evict_select", "nsa_evict_compact",
    "nsa_evict_compact_workspace_bytes", "alloc_evict_workspace", "nsa_mla_expand_kv",
    "nsa_mla_expand_kv_workspace_bytes", "alloc_mla_expand_workspace", "nsa_mla_prefill",
    "nsa_mla_prefill_workspace_bytes", "alloc_mla_prefill_workspace", "nsa_merge_attention", "nsa_mla_absorb_q",
    "nsa_mla_project_v", "nsa_status_read", "nsa_status_string", "nsa_abi_version",
    "EXPORTED_SYMBOLS",
]

MODE_DECODE, MODE_EXTEND, MODE_TARGET_VERIFY = 0, 1, 2
DT_F32, DT_BF16, DT_E4M3 = 0, 1, 2
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_BOUNDS, ERR_TIMEOUT = range(6)

EXPORTED_SYMBOLS = [
    "nsa_status_string", "nsa_abi_version", "nsa_status_read", "nsa_metadata",
    "nsa_effective_chunk_size", "nsa_local_virtual_batches", "nsa_indexer_logits",
    "nsa_topk_transform", "nsa_topk_workspace_bytes", "nsa_topk_launches", "nsa_sparse_mla",
    "nsa_sparse_mla_workspace_bytes",
    "nsa_sparse_mla_plan", "nsa_set_mla_kv", "nsa_quantize_kv_cache", "nsa_dequantize_kv_paged", "nsa_set_index_k",
    "nsa_topk_transform_ragged", "nsa_flatten_page_table", "nsa_copy_buffers",
    "nsa_check_bounded_wait", "nsa_local_attention", "nsa_paged_mla", "nsa_paged_mla_workspace_bytes",
    "nsa_mla_key_weights", "nsa_evict_select", "nsa_evict_compact", "nsa_evict_compact_workspace_bytes",
    "nsa_mla_expand_kv", "nsa_mla_expand_kv_workspace_bytes", "nsa_mla_prefill", "nsa_mla_prefill_workspace_bytes",
    "nsa_merge_attention", "nsa_mla_absorb_q", "nsa_mla_project_v",
]

_lib = None


class NsaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {nsa_status_string(code)} ({code})")


def load(build_if_missing: bool = True):
    """Load libnsa.so (building it with nvcc when missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if build_if_missing:
        path = _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"libnsa.so is missing ({path}); run __graft_entry__.build()")
    lib = C.CDLL(path)
    P, I, L, F, S = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t
    sig = {
        "nsa_status_string": ([I], C.c_char_p),
        "nsa_abi_version": ([], I),
        "nsa_status_read": ([P, P, P], I),
        "nsa_metadata": ([I, I, I, I, I, I, I, P, P, P, L, L, P, P, P, P], I),
        "nsa_effective_chunk_size": ([I, I, I], I),
        "nsa_local_virtual_batches": ([I, I, I, P, P, P, L, L, I, P, P, P, P, P, P], I),
        "nsa_indexer_logits": ([I, P, P, P, P, L, I, I, I, P, L, P, P, I, I, I, P, L, P, P, P], I),
        "nsa_topk_transform": ([P, L, P, P, P, L, P, L, I, I, I, P, L, P, P, S, P, P], I),
        "nsa_topk_workspace_bytes": ([I, I, I], S),
        "nsa_topk_launches": ([I, I, I], I),
        "nsa_sparse_mla": ([I, I, P, L, L, P, L, L, P, L, P, L, I, I, I, I, I, F, P, P, P, S, P, P], I),
        "nsa_sparse_mla_workspace_bytes": ([I, I, I, I, I, I, I], S),
        "nsa_sparse_mla_plan": ([I, I, I, I, I, I, I, P, P], I),
        "nsa_set_mla_kv": ([I, P, L, P, L, P, I, I, I, P, L, P, P], I),
        "nsa_quantize_kv_cache": ([P, L, I, I, P, P], I),
        "nsa_dequantize_kv_paged": ([P, L, I, I, P, L, P, P, P], I),
        "nsa_set_index_k": ([P, L, P, I, I, P, P, L, P, P], I),
        "nsa_topk_transform_ragged": ([P, L, P, P, P, I, I, I, P, L, P, P, S, P, P], I),
        "nsa_flatten_page_table": ([I, P, L, P, P, P, L, P, P], I),
        "nsa_copy_buffers": ([I, P, P, P, P], I),
        "nsa_check_bounded_wait": ([P, C.c_longlong, P], I),
        "nsa_local_attention": ([P, L, P, P, L, I, P, L, P, P, I, I, I, I, I, F, P, P, P, P], I),
        "nsa_paged_mla": ([I, I, P, L, L, P, L, L, P, L, I, P, L, P, I, I, I, I, I, I, F, P, P, P, S, P, P], I),
        "nsa_paged_mla_workspace_bytes": ([I, I, I, I, I, I, I, I], S),
        "nsa_mla_key_weights": ([I, I, P, L, L, P, L, L, P, L, I, P, L, P, I, I, I, I, I, I, F, P, P, L, P, P], I),
        "nsa_evict_select": ([P, L, P, I, I, I, I, I, P, L, P, P, P], I),
        "nsa_evict_compact": ([I, P, L, I, P, P, I, P, L, I, L, I, P, P, P, L, P, S, P, P], I),
        "nsa_evict_compact_workspace_bytes": ([I, I], S),
        "nsa_mla_expand_kv": ([I, P, L, P, I, P, I, I, I, I, I, P, P, P, S, P, P], I),
        "nsa_mla_expand_kv_workspace_bytes": ([I], S),
        "nsa_mla_prefill": ([P, L, L, P, L, L, P, L, L, P, L, P, L, L, P, P, I, I, I, I, I, I, I, I, F, P, P, P, S, P, P], I),
        "nsa_mla_prefill_workspace_bytes": ([], S),
        "nsa_merge_attention": ([I, I, I, P, P, L, I, P, P, P], I),
        "nsa_mla_absorb_q": ([P, L, L, P, I, I, I, I, I, P, P, P], I),
        "nsa_mla_project_v": ([P, L, L, P, I, I, I, I, I, P, P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    _lib = lib
    return lib


class _MetadataOut(C.Structure):
    _fields_ = [("cache_seqlens", C.c_void_p), ("cu_seqlens_k", C.c_void_p), ("cu_seqlens_q", C.c_void_p),
                ("seqlens_expanded", C.c_void_p), ("nsa_cache_seqlens", C.c_void_p),
                ("nsa_cu_seqlens_k", C.c_void_p), ("nsa_cu_seqlens_q", C.c_void_p),
                ("row_to_req", C.c_void_p), ("page_table_1", C.c_void_p), ("page_table_1_ld", C.c_int64),
                ("real_page_table", C.c_void_p), ("real_page_table_ld", C.c_int64),
                ("indexer_ks", C.c_void_p), ("indexer_ke", C.c_void_p), ("req_rows", C.c_void_p)]


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return C.c_void_p(t.data_ptr())


def _ld(t: torch.Tensor) -> int:
    """Leading dimension of a row-major 2D tensor: its row stride, or for a single
    row (whose stride is arbitrary, 0 for a broadcast view) its row length.  The
    library reads every row as packed, so elements of a row must be adjacent."""
    if t.dim() != 2:
        raise ValueError(f"expected a 2D tensor, got shape {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("the elements of each row must be adjacent (stride 1 in the last dimension)")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def alloc_score_hist(R: int, device="cuda") -> torch.Tensor:
    """A zeroed [R, 2048] uint32 (stored as int32) digit-count buffer shared by
    nsa_indexer_logits and nsa_topk_transform (the top-k leaves it zeroed)."""
    return torch.zeros((max(R, 1), 2048), dtype=torch.int32, device=device)


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn: str, code: int):
    if code != OK:
        raise NsaError(fn, code)


def nsa_status_string(code: int) -> str:
    return load().nsa_status_string(code).decode()


def nsa_abi_version() -> int:
    return load().nsa_abi_version()


def nsa_status_read(status: torch.Tensor, stream=None) -> int:
    """Synchronize `stream` and return the device status word."""
    v = C.c_int32(0)
    _check("nsa_status_read", load().nsa_status_read(_ptr(status), C.byref(v), _stream(stream)))
    return int(v.value)


# ------------------------------------------------------------------ metadata

def alloc_metadata(mode: int, B: int, R: int, W: int, page_size: int, device="cuda",
                   with_ks_ke: bool = False, with_page_table_1: bool = True,
                   with_req_rows: bool = False) -> Dict[str, torch.Tensor]:
    """Device buffers for nsa_metadata's outputs (page_table_1 left out, and so not
    written, when with_page_table_1 is False; req_rows added with with_req_rows)."""
    i32 = dict(dtype=torch.int32, device=device)
    nq = R + 1 if mode == MODE_TARGET_VERIFY else B + 1
    npg = (W + page_size - 1) // page_size
    out = dict(cache_seqlens=torch.empty(B, **i32), cu_seqlens_k=torch.empty(B + 1, **i32),
               cu_seqlens_q=torch.empty(nq, **i32), seqlens_expanded=torch.empty(R, **i32),
               nsa_cache_seqlens=torch.empty(R, **i32), nsa_cu_seqlens_k=torch.empty(R + 1, **i32),
               nsa_cu_seqlens_q=torch.empty(R + 1, **i32), row_to_req=torch.empty(R, **i32),
               real_page_table=torch.empty((B, max(npg, 1)), **i32))
    if with_page_table_1:
        out["page_table_1"] = torch.empty((B, max(W, 1)), **i32)
    if with_req_rows:
        out["req_rows"] = torch.empty(B, **i32)
    if with_ks_ke:
        out["indexer_ks"] = torch.empty(R, **i32)
        out["indexer_ke"] = torch.empty(R, **i32)
    return out


def nsa_metadata(mode: int, B: int, R: int, W: int, n_draft: int, topk: int, page_size: int,
                 seq_lens: torch.Tensor, extend_lens: Optional[torch.Tensor], req_to_token: torch.Tensor,
                 req_pool_indices: torch.Tensor, out: Dict[str, torch.Tensor],
                 status: Optional[torch.Tensor] = None, stream=None) -> None:
    pt1 = out.get("page_table_1")
    o = _MetadataOut(*(_ptr(out[k]) for k in ["cache_seqlens", "cu_seqlens_k", "cu_seqlens_q",
                                              "seqlens_expanded", "nsa_cache_seqlens", "nsa_cu_seqlens_k",
                                              "nsa_cu_seqlens_q", "row_to_req"]),
                     _ptr(pt1), _ld(pt1) if pt1 is not None else 0, _ptr(out["real_page_table"]),
                     _ld(out["real_page_table"]), _ptr(out.get("indexer_ks")), _ptr(out.get("indexer_ke")),
                     _ptr(out.get("req_rows")))
    rc = load().nsa_metadata(mode, B, R, W, n_draft, topk, page_size, _ptr(seq_lens), _ptr(extend_lens),
                             _ptr(req_to_token), _ld(req_to_token), req_to_token.shape[0],
                             _ptr(req_pool_indices), C.byref(o), _ptr(status), _stream(stream))
    _check("nsa_metadata", rc)


# ------------------------------------------------------------------ local attention (host)

def nsa_effective_chunk_size(attn_chunk_size: int, max_seq_len: int, page_size: int) -> int:
    v = load().nsa_effective_chunk_size(attn_chunk_size, max_seq_len, page_size)
    if v < 0:
        raise NsaError("nsa_effective_chunk_size", ERR_INVALID_ARG)
    return v


def nsa_local_virtual_batches(attn_chunk_size: int, page_size: int, cu_seqlens_q, seq_lens, block_table):
    """Host call.  Returns numpy arrays (seqlens_q_local, cu_seqlens_q_local,
    seqlens_k_local, k_seqstarts_absolute, block_table_local)."""
    lib = load()
    cq = np.ascontiguousarray(cu_seqlens_q, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    B = len(sl)
    n = C.c_int(0)
    P = lambda a: a.ctypes.data_as(C.c_void_p)
    _check("nsa_local_virtual_batches",
           lib.nsa_local_virtual_batches(attn_chunk_size, page_size, B, P(cq), P(sl), P(bt), bt.shape[1],
                                         bt.shape[1], 0, C.byref(n), None, None, None, None, None))
    V, ppl = n.value, attn_chunk_size // page_size
    sq, cu, sk = np.zeros(V, np.int32), np.zeros(V + 1, np.int32), np.zeros(V, np.int32)
    st, btl = np.zeros(V, np.int32), np.zeros((V, ppl), np.int32)
    _check("nsa_local_virtual_batches",
           lib.nsa_local_virtual_batches(attn_chunk_size, page_size, B, P(cq), P(sl), P(bt), bt.shape[1],
                                         bt.shape[1], V, C.byref(n), P(sq), P(cu), P(sk), P(st), P(btl)))
    return sq, cu, sk, st, btl


# ------------------------------------------------------------------ indexer / top-k / attention

def nsa_indexer_logits(dtype: int, q_idx: torch.Tensor, weights: torch.Tensor, k_cache: torch.Tensor,
                       k_scale: torch.Tensor, real_page_table: torch.Tensor, row_to_req: torch.Tensor,
                       row_len: torch.Tensor, max_row_len: int, logits: torch.Tensor,
                       status: Optional[torch.Tensor] = None, stream=None, rows_per_group: int = 1,
                       score_hist: Optional[torch.Tensor] = None) -> None:
    R, Hi, Di = q_idx.shape
    num_pages, ps = k_cache.shape[0], k_cache.shape[1]
    assert q_idx.is_contiguous() and k_cache.is_contiguous() and weights.is_contiguous() and k_scale.is_contiguous()
    rc = load().nsa_indexer_logits(dtype, _ptr(q_idx), _ptr(weights), _ptr(k_cache), _ptr(k_scale), num_pages,
                                   ps, Hi, Di, _ptr(real_page_table), _ld(real_page_table),
                                   _ptr(row_to_req), _ptr(row_len), R, rows_per_group, max_row_len, _ptr(logits),
                                   _ld(logits), _ptr(_hist(score_hist, R)), _ptr(status), _stream(stream))
    _check("nsa_indexer_logits", rc)


def _hist(h: Optional[torch.Tensor], R: int) -> Optional[torch.Tensor]:
    if h is not None:
        assert h.is_contiguous() and h.element_size() == 4 and h.shape[-1] == 2048 and h.numel() >= R * 2048
    return h


def nsa_topk_workspace_bytes(R: int, max_row_len: int, with_score_hist: bool) -> int:
    return int(load().nsa_topk_workspace_bytes(R, max_row_len, 1 if with_score_hist else 0))


def nsa_topk_launches(R: int, max_row_len: int, with_score_hist: bool) -> int:
    return int(load().nsa_topk_launches(R, max_row_len, 1 if with_score_hist else 0))


def alloc_topk_workspace(R: int, max_row_len: int, with_score_hist: bool, device="cuda") -> torch.Tensor:
    """A zeroed top-k workspace (the calls leave it zeroed for the next one)."""
    n = max(256, nsa_topk_workspace_bytes(R, max_row_len, with_score_hist))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _topk_ws(ws: Optional[torch.Tensor], R: int, max_row_len: int, score_hist, device):
    if ws is None:  # a fresh zeroed one (a caller running many steps keeps its own)
        ws = alloc_topk_workspace(R, max_row_len, score_hist is not None, device)
    return ws, ws.numel() * ws.element_size()


def nsa_topk_transform(logits: torch.Tensor, row_len: torch.Tensor, row_to_req: torch.Tensor,
                       page_table_1: torch.Tensor, topk: int, max_row_len: int, indices: torch.Tensor,
                       status: Optional[torch.Tensor] = None, stream=None,
                       score_hist: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       pt_rows: Optional[torch.Tensor] = None) -> None:
    """pt_rows: request b's slots are row pt_rows[b] of page_table_1 (e.g. req_to_token
    with nsa_metadata's req_rows); None: row b."""
    R = row_len.shape[0]
    ws, ws_bytes = _topk_ws(workspace, R, max_row_len, score_hist, logits.device)
    rc = load().nsa_topk_transform(_ptr(logits), _ld(logits), _ptr(row_len), _ptr(row_to_req),
                                   _ptr(page_table_1), _ld(page_table_1), _ptr(pt_rows),
                                   int(page_table_1.shape[0]) if pt_rows is not None else 0, R, topk, max_row_len,
                                   _ptr(indices), _ld(indices), _ptr(_hist(score_hist, R)), _ptr(ws), ws_bytes,
                                   _ptr(status), _stream(stream))
    _check("nsa_topk_transform", rc)


def nsa_sparse_mla_workspace_bytes(q_dtype: int, kv_dtype: int, R: int, H: int, d_latent: int, d_rope: int,
                                   topk: int) -> int:
    return int(load().nsa_sparse_mla_workspace_bytes(q_dtype, kv_dtype, R, H, d_latent, d_rope, topk))


def nsa_sparse_mla_plan(q_dtype: int, kv_dtype: int, R: int, H: int, d_latent: int, d_rope: int,
                        topk: int):
    """(splits per top-k list, kernel launches per call) of nsa_sparse_mla for this shape."""
    ns, nl = C.c_int(0), C.c_int(0)
    _check("nsa_sparse_mla_plan", load().nsa_sparse_mla_plan(q_dtype, kv_dtype, R, H, d_latent, d_rope, topk,
                                                             C.byref(ns), C.byref(nl)))
    return int(ns.value), int(nl.value)


def nsa_sparse_mla(q_dtype: int, kv_dtype: int, q_nope: torch.Tensor, q_rope: torch.Tensor, kv: torch.Tensor,
                   indices: torch.Tensor, sm_scale: float, out: torch.Tensor, lse: torch.Tensor,
                   workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                   stream=None, num_slots: Optional[int] = None) -> None:
    """q_nope [R,H,d_latent] and q_rope [R,H,d_rope] (any row / head strides,
    unit stride in the last dim); kv [slots, row]; indices [R, topk]."""
    R, H, d_latent = q_nope.shape
    d_rope = q_rope.shape[2]
    topk = indices.shape[1]
    assert q_nope.stride(2) == 1 and q_rope.stride(2) == 1 and out.is_contiguous() and lse.is_contiguous()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().nsa_sparse_mla(q_dtype, kv_dtype, _ptr(q_nope), q_nope.stride(0), q_nope.stride(1), _ptr(q_rope),
                               q_rope.stride(0), q_rope.stride(1), _ptr(kv),
                               kv.shape[0] if num_slots is None else num_slots, _ptr(indices),
                               _ld(indices), R, H, d_latent, d_rope, topk, float(sm_scale), _ptr(out),
                               _ptr(lse), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream))
    _check("nsa_sparse_mla", rc)


# ---------------------------------------------------------------- KV-cache write side

def nsa_set_mla_kv(kv_dtype: int, k_nope: torch.Tensor, k_rope: torch.Tensor, loc: torch.Tensor,
                   kv: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """New tokens' latent [n, 512] and rope [n, 64] (bf16) into the KV cache at slots `loc` (int32)."""
    n = loc.shape[0]
    num_slots = kv.shape[0]
    rc = load().nsa_set_mla_kv(kv_dtype, _ptr(k_nope), k_nope.stride(0), _ptr(k_rope), k_rope.stride(0), _ptr(loc),
                               n, k_nope.shape[1], k_rope.shape[1], _ptr(kv), num_slots, _ptr(status),
                               _stream(stream))
    _check("nsa_set_mla_kv", rc)


def nsa_quantize_kv_cache(kv_bf16: torch.Tensor, kv_fp8: torch.Tensor, d_latent: int = 512, d_rope: int = 64,
                          stream=None) -> None:
    rc = load().nsa_quantize_kv_cache(_ptr(kv_bf16), kv_bf16.shape[0], d_latent, d_rope, _ptr(kv_fp8),
                                      _stream(stream))
    _check("nsa_quantize_kv_cache", rc)


def nsa_dequantize_kv_paged(kv_fp8: torch.Tensor, slots: torch.Tensor, out_bf16: torch.Tensor,
                            d_latent: int = 512, d_rope: int = 64, status: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    rc = load().nsa_dequantize_kv_paged(_ptr(kv_fp8), kv_fp8.shape[0], d_latent, d_rope, _ptr(slots),
                                        slots.shape[0], _ptr(out_bf16), _ptr(status), _stream(stream))
    _check("nsa_dequantize_kv_paged", rc)


def nsa_set_index_k(k: torch.Tensor, loc: torch.Tensor, k_cache: torch.Tensor, k_scale: torch.Tensor,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Indexer keys [n, 128] (bf16) -> e4m3 codes and fp32 scales at slots `loc` of the paged key cache."""
    num_slots = k_scale.numel()
    rc = load().nsa_set_index_k(_ptr(k), k.stride(0), _ptr(loc), loc.shape[0], k.shape[1], _ptr(k_cache),
                                _ptr(k_scale), num_slots, _ptr(status), _stream(stream))
    _check("nsa_set_index_k", rc)


# ---------------------------------------------------------------- RAGGED extend

def nsa_topk_transform_ragged(logits: torch.Tensor, row_len: torch.Tensor, row_to_req: torch.Tensor,
                              req_offset: torch.Tensor, topk: int, max_row_len: int, indices: torch.Tensor,
                              status: Optional[torch.Tensor] = None, stream=None,
                              score_hist: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None) -> None:
    R = row_len.shape[0]
    ws, ws_bytes = _topk_ws(workspace, R, max_row_len, score_hist, logits.device)
    rc = load().nsa_topk_transform_ragged(_ptr(logits), _ld(logits), _ptr(row_len), _ptr(row_to_req),
                                          _ptr(req_offset), R, topk, max_row_len, _ptr(indices), _ld(indices),
                                          _ptr(_hist(score_hist, R)), _ptr(ws), ws_bytes, _ptr(status),
                                          _stream(stream))
    _check("nsa_topk_transform_ragged", rc)


def nsa_flatten_page_table(page_table_1: torch.Tensor, kv_len: torch.Tensor, kv_start: torch.Tensor,
                           out: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    B = kv_len.shape[0]
    rc = load().nsa_flatten_page_table(B, _ptr(page_table_1), _ld(page_table_1), _ptr(kv_len), _ptr(kv_start),
                                       _ptr(out), out.numel(), _ptr(status), _stream(stream))
    _check("nsa_flatten_page_table", rc)


# ---------------------------------------------------------------- copies

def nsa_copy_buffers(pairs, stream=None) -> None:
    """[(dst, src), ...] tensors of equal byte size (device or pinned host), copied in one launch."""
    n = len(pairs)
    src = (C.c_void_p * max(1, n))(*[p[1].data_ptr() for p in pairs])
    dst = (C.c_void_p * max(1, n))(*[p[0].data_ptr() for p in pairs])
    nb = (C.c_int64 * max(1, n))(*[p[1].numel() * p[1].element_size() for p in pairs])
    for d, s in pairs:
        assert d.numel() * d.element_size() == s.numel() * s.element_size()
    _check("nsa_copy_buffers", load().nsa_copy_buffers(n, src, dst, nb, _stream(stream)))


def nsa_check_bounded_wait(status: torch.Tensor, budget_cycles: int, stream=None) -> None:
    _check("nsa_check_bounded_wait", load().nsa_check_bounded_wait(_ptr(status), int(budget_cycles), _stream(stream)))


# ---------------------------------------------------------------- chunk-local attention

def nsa_local_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        cu_seqlens_q: torch.Tensor, seqused_k: torch.Tensor, sm_scale: float, out: torch.Tensor,
                        lse: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q bf16 [total_q, Hq, D] (rows may be strided); k_cache / v_cache bf16 [pages, page_size, Hkv, D];
    block_table int32 [nvb, bt_ld]; cu_seqlens_q int32 [nvb + 1]; seqused_k int32 [nvb];
    out bf16 [total_q, Hq, D]; lse float32 [total_q, Hq]."""
    total_q, Hq, D = q.shape
    assert q.stride(2) == 1 and q.stride(1) == D
    num_pages, ps, Hkv, Dk = k_cache.shape
    assert Dk == D and tuple(v_cache.shape) == tuple(k_cache.shape)
    assert k_cache.is_contiguous() and v_cache.is_contiguous() and block_table.stride(1) == 1
    assert out.is_contiguous() and lse.is_contiguous()
    nvb = seqused_k.shape[0]
    # the library reads bt_ld as the row stride and as the row's capacity: a column
    # slice of a wider table (stride beyond the row length) would overstate it
    if block_table.shape[0] > 1 and block_table.stride(0) != block_table.shape[1]:
        raise ValueError("block_table rows must be packed (row stride == row length)")
    bt_ld = _ld(block_table)
    rc = load().nsa_local_attention(_ptr(q), q.stride(0), _ptr(k_cache), _ptr(v_cache), num_pages, ps,
                                    _ptr(block_table), bt_ld, _ptr(cu_seqlens_q), _ptr(seqused_k),
                                    nvb, total_q, Hq, Hkv, D, float(sm_scale), _ptr(out), _ptr(lse), _ptr(status),
                                    _stream(stream))
    _check("nsa_local_attention", rc)


# ---------------------------------------------------------------- dense paged MLA attention

_Q_TYPES = {DT_F32: torch.float32, DT_BF16: torch.bfloat16}
_CACHE_TYPES = {**_Q_TYPES, DT_E4M3: torch.float8_e4m3fn}


def _paged_q(q_dtype: int, q_nope: torch.Tensor, q_rope: torch.Tensor):
    """The query arguments of the C calls; a single row's or head's stride, which is
    arbitrary, is replaced by what a packed tensor would have."""
    R, H, dl = q_nope.shape
    Rr, Hr, dr = q_rope.shape
    if Rr != R or Hr != H:
        raise ValueError(f"q_rope {tuple(q_rope.shape)} does not match q_nope {tuple(q_nope.shape)}")
    sn, sr = q_nope.stride(), q_rope.stride()
    if (dl > 1 and sn[2] != 1) or (dr > 1 and sr[2] != 1):
        raise ValueError("the elements of each query head must be adjacent (stride 1 in the last dimension)")
    want = _Q_TYPES.get(q_dtype)
    if q_nope.dtype != want or q_rope.dtype != want:
        raise ValueError(f"q must be {want} for this q_dtype, got {q_nope.dtype} and {q_rope.dtype}")
    hn, hr = (sn[1], sr[1]) if H > 1 else (dl, dr)
    rn, rr = (sn[0], sr[0]) if R > 1 else (H * hn, H * hr)
    return q_nope.data_ptr(), rn, hn, q_rope.data_ptr(), rr, hr


def _paged_cache(kv_dtype: int, kv: torch.Tensor, page_size: int, d_latent: int, d_rope: int) -> int:
    """Checks a cache of [slots, row] (or [pages, page_size, row]; of its own type, or raw bytes in an
    integer type) and returns its page count."""
    dtype = kv.dtype
    if dtype is not _CACHE_TYPES.get(kv_dtype) and dtype.is_floating_point:
        raise ValueError(f"the cache must be {_CACHE_TYPES.get(kv_dtype)} (or bytes) for this kv_dtype, got {dtype}")
    if kv_dtype == DT_E4M3:
        want = d_latent + 4 * (d_latent // 128) + 2 * d_rope
    else:
        want = (4 if kv_dtype == DT_F32 else 2) * (d_latent + d_rope)
    row = kv.shape[-1]
    if not kv.is_contiguous() or kv.dim() not in (2, 3) or row * kv.element_size() != want:
        raise ValueError(f"the cache must be contiguous rows of {want} bytes, got shape {tuple(kv.shape)} of {kv.dtype}")
    slots = kv.numel() // row
    if page_size < 1 or slots % page_size:
        raise ValueError(f"{slots} slots are no whole pages of {page_size}")
    return slots // page_size


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# without the check for an initialised CUDA that a CUDA tensor makes superfluous
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch_on(stream, *tensors: Optional[torch.Tensor]):
    """The stream handle of a call on these tensors, which must live on the current device (the
    library launches there)."""
    dev = _current_device() if tensors[0].is_cuda else -1
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0):
            raise ValueError(f"expected CUDA tensors on the current device, got one on {t.device}")
    if stream is None and _raw_stream is not None:  # the current stream without building its object
        return _raw_stream(dev)
    return _stream(stream)


def _scratch(t: Optional[torch.Tensor]) -> int:
    """The bytes of a workspace."""
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return t.numel() * t.element_size()


def _status_word(t: Optional[torch.Tensor]) -> None:
    if t is not None and (t.dtype is not torch.int32 or t.numel() < 1):
        raise ValueError(f"status must be an int32 word, got shape {tuple(t.shape)} of {t.dtype}")


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _i32(name: str, t: torch.Tensor, n: int) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous int32 values, got shape {tuple(t.shape)} of {t.dtype}")
    return t


def _table(t: torch.Tensor, B: int) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != B:
        raise ValueError(f"page_table must be int32 [{B}, pages], got shape {tuple(t.shape)} of {t.dtype}")
    return t


def _table_ld(t: torch.Tensor, max_len: int, page_size: int) -> int:
    if t.shape[1] * page_size < max_len:
        raise ValueError(f"a page-table row of {t.shape[1]} pages of {page_size} does not hold {max_len} positions")
    return _ld(t)


def nsa_paged_mla_workspace_bytes(q_dtype: int, kv_dtype: int, R: int, rows_per_req: int, H: int, max_row_len: int,
                                  d_latent: int = 512, d_rope: int = 64) -> int:
    return int(load().nsa_paged_mla_workspace_bytes(q_dtype, kv_dtype, R, rows_per_req, H, d_latent, d_rope, max_row_len))


def alloc_paged_mla_workspace(q_dtype: int, kv_dtype: int, R: int, rows_per_req: int, H: int, max_row_len: int,
                              d_latent: int = 512, d_rope: int = 64, device="cuda") -> Optional[torch.Tensor]:
    """Scratch for nsa_paged_mla calls of these types and at most this shape (no more rows, rows a request,
    heads or positions; None if they need none)."""
    n = nsa_paged_mla_workspace_bytes(q_dtype, kv_dtype, R, rows_per_req, H, max_row_len, d_latent, d_rope)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def nsa_paged_mla(q_dtype: int, kv_dtype: int, q_nope: torch.Tensor, q_rope: torch.Tensor, kv: torch.Tensor,
                  page_size: int, page_table: torch.Tensor, row_len: torch.Tensor, rows_per_req: int, max_row_len: int,
                  sm_scale: float, out: torch.Tensor, lse: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q_nope [R, H, d_latent] and q_rope [R, H, d_rope] (any row / head strides); kv [slots, row];
    page_table int32 [R / rows_per_req, pages]; row_len int32 [R]; out [R, H, d_latent] (q's type) and
    lse float32 [R, H].  workspace: alloc_paged_mla_workspace's, for this shape or a larger one (see there)."""
    R, H, dl = q_nope.shape
    dr = q_rope.shape[2]
    if rows_per_req < 1 or R % rows_per_req:
        raise ValueError(f"{R} rows are no whole requests of {rows_per_req}")
    pages = _paged_cache(kv_dtype, kv, page_size, dl, dr)
    pt = _table(page_table, R // rows_per_req)
    if tuple(out.shape) != (R, H, dl) or tuple(lse.shape) != (R, H) or lse.dtype != torch.float32 or \
            out.dtype != q_nope.dtype or not out.is_contiguous() or not lse.is_contiguous():
        raise ValueError("out must be [R, H, d_latent] in q's type and lse float32 [R, H], both contiguous")
    q_args, pt_ld, ws_bytes = _paged_q(q_dtype, q_nope, q_rope), _table_ld(pt, max_row_len, page_size), _scratch(workspace)
    _i32("row_len", row_len, R)
    _status_word(status)
    handle = _launch_on(stream, q_nope, q_rope, kv, page_table, row_len, out, lse, workspace, status)
    rc = load().nsa_paged_mla(q_dtype, kv_dtype, *q_args, _at(kv), pages, page_size, _at(pt), pt_ld, _at(row_len), R,
                              rows_per_req, H, dl, dr, max_row_len, float(sm_scale), _at(out), _at(lse), _at(workspace),
                              ws_bytes, _at(status), handle)
    _check("nsa_paged_mla", rc)


# ---------------------------------------------------------------- eviction

def nsa_mla_key_weights(q_dtype: int, kv_dtype: int, q_nope: torch.Tensor, q_rope: torch.Tensor, kv: torch.Tensor,
                        page_size: int, page_table: torch.Tensor, row_len: torch.Tensor, rows_per_req: int,
                        max_row_len: int, sm_scale: float, lse: torch.Tensor, total: torch.Tensor,
                        status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Adds to total (float32 [requests, positions]) the attention weight each cached position got
    from its request's rows; the other arguments as nsa_paged_mla's, lse as that call wrote it."""
    R, H, dl = q_nope.shape
    dr = q_rope.shape[2]
    if rows_per_req < 1 or R % rows_per_req:
        raise ValueError(f"{R} rows are no whole requests of {rows_per_req}")
    B = R // rows_per_req
    pages = _paged_cache(kv_dtype, kv, page_size, dl, dr)
    pt = _table(page_table, B)
    if tuple(lse.shape) != (R, H) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [R, H]")
    q_args, pt_ld = _paged_q(q_dtype, q_nope, q_rope), _table_ld(pt, max_row_len, page_size)
    total_ld = _total_ld(total, B, max_row_len)
    _i32("row_len", row_len, R)
    _status_word(status)
    handle = _launch_on(stream, q_nope, q_rope, kv, page_table, row_len, lse, total, status)
    rc = load().nsa_mla_key_weights(q_dtype, kv_dtype, *q_args, _at(kv), pages, page_size, _at(pt), pt_ld, _at(row_len), R,
                                    rows_per_req, H, dl, dr, max_row_len, float(sm_scale), _at(lse), _at(total),
                                    total_ld, _at(status), handle)
    _check("nsa_mla_key_weights", rc)


def _total_ld(total: torch.Tensor, B: int, max_len: int) -> int:
    if total.dtype != torch.float32 or total.dim() != 2 or total.shape[0] != B or total.shape[1] < max_len:
        raise ValueError(f"total must be float32 [{B}, >= {max_len}], got shape {tuple(total.shape)} of {total.dtype}")
    return _ld(total)


def nsa_evict_select(total: torch.Tensor, lens: torch.Tensor, max_len: int, sinks: int, recent: int, budget: int,
                     keep: torch.Tensor, new_len: torch.Tensor, status: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """keep int32 [B, >= budget]: the kept positions of each request, ascending, then -1; new_len int32 [B]."""
    B = lens.shape[0]
    if keep.dtype != torch.int32 or keep.dim() != 2 or keep.shape[0] != B or keep.shape[1] < budget:
        raise ValueError(f"keep must be int32 [{B}, >= {budget}], got shape {tuple(keep.shape)} of {keep.dtype}")
    total_ld, keep_ld = _total_ld(total, B, max_len), _ld(keep)
    _i32("lens", lens, B)
    _i32("new_len", new_len, B)
    _status_word(status)
    handle = _launch_on(stream, total, lens, keep, new_len, status)
    rc = load().nsa_evict_select(_at(total), total_ld, _at(lens), B, max_len, sinks, recent, budget, _at(keep), keep_ld,
                                 _at(new_len), _at(status), handle)
    _check("nsa_evict_select", rc)


def nsa_evict_compact_workspace_bytes(B: int, max_len: int) -> int:
    return int(load().nsa_evict_compact_workspace_bytes(B, max_len))


def alloc_evict_workspace(B: int, max_len: int, device="cuda") -> torch.Tensor:
    """Scratch for nsa_evict_compact calls of at most B requests and max_len positions."""
    return torch.empty(max(16, nsa_evict_compact_workspace_bytes(B, max_len)), dtype=torch.uint8, device=device)


def nsa_evict_compact(keep: torch.Tensor, new_len: torch.Tensor, old_len: torch.Tensor, max_len: int,
                      page_table: torch.Tensor, page_size: int, arrays, total: Optional[torch.Tensor],
                      workspace: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Moves, in place, position keep[b, i] of every paged array to position i, and total likewise.
    arrays: contiguous tensors whose first dimension is the slot (a cache kept as [pages, page_size, ...]
    is passed as a view(-1, ...) of it); workspace: alloc_evict_workspace's."""
    B = old_len.shape[0]
    if keep.dtype != torch.int32 or keep.dim() != 2 or keep.shape[0] != B:
        raise ValueError(f"keep must be int32 [{B}, budget], got shape {tuple(keep.shape)} of {keep.dtype}")
    pt = _table(page_table, B)
    if page_size < 1:
        raise ValueError(f"page_size must be positive, got {page_size}")
    slots = arrays[0].shape[0] if len(arrays) else pt.shape[1] * page_size
    for a in arrays:
        if not a.is_contiguous() or a.shape[0] != slots or slots < 1 or slots % page_size:
            raise ValueError(f"the arrays must be contiguous with one first dimension of whole pages of {page_size}, "
                             f"got shape {tuple(a.shape)}")
    total_ld = 0 if total is None else _total_ld(total, B, max_len)
    keep_ld, pt_ld, ws_bytes = _ld(keep), _table_ld(pt, max_len, page_size), _scratch(workspace)
    _i32("new_len", new_len, B)
    _i32("old_len", old_len, B)
    _status_word(status)
    handle = _launch_on(stream, keep, new_len, old_len, page_table, total, workspace, status, *arrays)
    n = len(arrays)
    ptrs = (C.c_void_p * max(1, n))(*[a.data_ptr() for a in arrays])
    nb = (C.c_int64 * max(1, n))(*[a.numel() * a.element_size() // slots for a in arrays])
    rc = load().nsa_evict_compact(B, _at(keep), keep_ld, keep.shape[1], _at(new_len), _at(old_len), max_len, _at(pt),
                                  pt_ld, page_size, slots // page_size, n, ptrs, nb, _at(total), total_ld, _at(workspace),
                                  ws_bytes, _at(status), handle)
    _check("nsa_evict_compact", rc)


# ---------------------------------------------------------------- latent attention's two forms

_D_LATENT, _D_ROPE, _D_NOPE, _D_V = 512, 64, 128, 128


def _bf16(name: str, t: torch.Tensor, shape, contiguous: bool = True) -> torch.Tensor:
    """A bf16 tensor of this shape (None: any size there), contiguous or with an adjacent last dimension."""
    if t.dtype is torch.bfloat16 and (t.shape == shape or (
            None in shape and t.dim() == len(shape) and all(n is None or n == m for n, m in zip(shape, t.shape)))):
        if t.is_contiguous() or (not contiguous and (t.stride(-1) == 1 or t.shape[-1] <= 1)):
            return t
    want = ", ".join("any" if n is None else str(n) for n in shape)
    raise ValueError(f"{name} must be bf16 [{want}], {'contiguous' if contiguous else 'its last dimension adjacent'}, "
                     f"got shape {tuple(t.shape)}, strides {t.stride()} of {t.dtype}")


def _rows(name: str, t: torch.Tensor, d: int, heads: Optional[int] = None):
    """(rows, heads) of a bf16 tensor [rows, heads, d] (None: any number) whose last dimension is adjacent."""
    shape = t.shape
    if len(shape) == 3 and shape[2] == d and (heads is None or shape[1] == heads) and t.dtype is torch.bfloat16 and \
            t.stride(2) == 1:
        return shape[0], shape[1]
    return _bf16(name, t, (None, heads, d), False).shape[:2]


def _heads_of(w: torch.Tensor) -> int:
    """The heads of an up-projection."""
    n = w.shape[0] if w.dim() == 2 else 0
    if n < 1 or n % (_D_NOPE + _D_V):
        raise ValueError(f"w must be bf16 [heads * {_D_NOPE + _D_V}, {_D_LATENT}], got shape {tuple(w.shape)}")
    if w.shape[1] != _D_LATENT or w.dtype is not torch.bfloat16 or not w.is_contiguous():
        _bf16("w", w, (None, _D_LATENT))
    return n // (_D_NOPE + _D_V)


def nsa_mla_expand_kv_workspace_bytes(m: int) -> int:
    return int(load().nsa_mla_expand_kv_workspace_bytes(m))


def alloc_mla_expand_workspace(m: int, device="cuda") -> torch.Tensor:
    """Scratch for nsa_mla_expand_kv calls of at most m rows."""
    return torch.empty(max(16, nsa_mla_expand_kv_workspace_bytes(m)), dtype=torch.uint8, device=device)


def nsa_mla_expand_kv(kv_dtype: int, kv: torch.Tensor, slots: torch.Tensor, w: torch.Tensor, kv_out: torch.Tensor,
                      k_rope_out: torch.Tensor, workspace: torch.Tensor, status: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """Rows `slots` (int32 [m]) of the cache [slots, row] through w [H * 256, 512]: kv_out [m, H, 256] (a head's
    128 key values, then its 128 values) and k_rope_out [m, 64].  workspace: alloc_mla_expand_workspace's."""
    H, m = _heads_of(w), slots.numel()
    num_slots = _paged_cache(kv_dtype, kv, 1, _D_LATENT, _D_ROPE)
    _i32("slots", slots, m)
    _bf16("kv_out", kv_out, (m, H, _D_NOPE + _D_V))
    _bf16("k_rope_out", k_rope_out, (m, _D_ROPE))
    ws_bytes = _scratch(workspace)
    _status_word(status)
    handle = _launch_on(stream, kv, slots, w, kv_out, k_rope_out, workspace, status)
    rc = load().nsa_mla_expand_kv(kv_dtype, _at(kv), num_slots, _at(slots), m, _at(w), H, _D_LATENT, _D_ROPE, _D_NOPE, _D_V,
                                  _at(kv_out), _at(k_rope_out), _at(workspace), ws_bytes, _at(status), handle)
    _check("nsa_mla_expand_kv", rc)


def nsa_mla_prefill_workspace_bytes() -> int:
    return int(load().nsa_mla_prefill_workspace_bytes())


def alloc_mla_prefill_workspace(device="cuda") -> torch.Tensor:
    """Scratch for nsa_mla_prefill calls of any shape on this device."""
    with torch.cuda.device(device):
        n = nsa_mla_prefill_workspace_bytes()
    return torch.empty(n, dtype=torch.uint8, device=device)


def nsa_mla_prefill(q_nope: torch.Tensor, q_rope: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor,
                    v: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, causal: bool,
                    sm_scale: float, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q_nope [total_q, H, 128], q_rope [total_q, H, 64], k_nope and v [total_k, H, 128] (any row / head strides),
    k_rope [total_k, 64]; cu_seqlens_q / cu_seqlens_k int32 [B + 1]; out bf16 [total_q, H, 128], lse float32
    [total_q, H].  workspace: alloc_mla_prefill_workspace's."""
    total_q, H = _rows("q_nope", q_nope, _D_NOPE)
    bf16, kr = torch.bfloat16, k_rope.shape
    if len(kr) != 2 or kr[1] != _D_ROPE or k_rope.dtype is not bf16 or k_rope.stride(1) != 1:
        _bf16("k_rope", k_rope, (None, _D_ROPE), False)
    total_k, B = kr[0], cu_seqlens_q.numel() - 1
    heads_k = (total_k, H, _D_NOPE)
    qn, qr, kn, vv = q_nope.stride(), q_rope.stride(), k_nope.stride(), v.stride()
    if not (q_rope.shape == (total_q, H, _D_ROPE) and k_nope.shape == heads_k and v.shape == heads_k and
            out.shape == q_nope.shape and q_rope.dtype is bf16 and k_nope.dtype is bf16 and v.dtype is bf16 and
            out.dtype is bf16 and qr[2] == 1 and kn[2] == 1 and vv[2] == 1 and out.is_contiguous()):
        # (something is not as it should be: which)
        _bf16("q_rope", q_rope, (total_q, H, _D_ROPE), False)
        _bf16("k_nope", k_nope, (total_k, H, _D_NOPE), False)
        _bf16("v", v, (total_k, H, _D_V), False)
        _bf16("out", out, (total_q, H, _D_V))
    if lse.shape != (total_q, H) or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous float32 [{total_q}, {H}], got shape {tuple(lse.shape)} of {lse.dtype}")
    _i32("cu_seqlens_q", cu_seqlens_q, max(B, 0) + 1)
    _i32("cu_seqlens_k", cu_seqlens_k, B + 1)
    ws_bytes = _scratch(workspace)
    _status_word(status)
    handle = _launch_on(stream, q_nope, q_rope, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, out, lse, workspace, status)
    rc = load().nsa_mla_prefill(q_nope.data_ptr(), qn[0], qn[1], q_rope.data_ptr(), qr[0], qr[1], k_nope.data_ptr(), kn[0],
                                kn[1], k_rope.data_ptr(), k_rope.stride(0), v.data_ptr(), vv[0], vv[1],
                                cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, total_q, total_k, H, _D_NOPE, _D_ROPE,
                                _D_V, 1 if causal else 0, sm_scale, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                ws_bytes, _at(status), handle)
    _check("nsa_mla_prefill", rc)


_DTYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}


def nsa_merge_attention(parts, lses, out: torch.Tensor, lse: torch.Tensor, stream=None) -> None:
    """parts: tensors [..., D] (all bf16 or all float32), lses: float32 tensors [...], one each; out (parts' type, or
    bf16) and lse get the attention over all parts' keys, and may be a part's own tensors."""
    n = len(parts)
    if n < 1 or len(lses) != n:
        raise ValueError(f"expected as many lse as parts, at least one: got {len(lses)} and {n}")
    shape, dtype = out.shape, parts[0].dtype
    rows = shape[:-1]
    if dtype not in _DTYPES or out.dtype not in _DTYPES:
        raise ValueError(f"parts and out must be float32 or bf16, got {dtype} and {out.dtype}")
    ptrs, lptrs = [], []  # (addresses; this call is as short as its checks)
    for p, l in zip(parts, lses):
        if p.shape != shape or l.shape != rows or p.dtype is not dtype or l.dtype is not torch.float32 or \
                not p.is_contiguous() or not l.is_contiguous():
            _refuse_part(p, l, dtype, shape)
        ptrs.append(p.data_ptr())
        lptrs.append(l.data_ptr())
    if not shape or lse.shape != rows or lse.dtype is not torch.float32 or not out.is_contiguous() or not lse.is_contiguous():
        _refuse_part(out, lse, out.dtype, shape)
    handle = _launch_on(stream, out, lse, *parts, *lses)
    _check("nsa_merge_attention", load().nsa_merge_attention(
        _DTYPES[dtype], _DTYPES[out.dtype], n, struct.pack(f"{n}P", *ptrs), struct.pack(f"{n}P", *lptrs), lse.numel(), shape[-1],
        _at(out), _at(lse), handle))


def _refuse_part(p: torch.Tensor, l: torch.Tensor, dtype, shape):
    raise ValueError(f"parts must be contiguous {dtype} {list(shape)} and lses contiguous float32 {list(shape[:-1])}, "
                     f"got {p.dtype} {list(p.shape)} and {l.dtype} {list(l.shape)}")


def nsa_mla_absorb_q(q_nope: torch.Tensor, w: torch.Tensor, out: torch.Tensor, status: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """q_nope [R, H, 128] (any row / head strides) through each head's W_k: out [R, H, 512]."""
    H = _heads_of(w)
    R, _ = _rows("q_nope", q_nope, _D_NOPE, H)
    _bf16("out", out, (R, H, _D_LATENT))
    _status_word(status)
    handle = _launch_on(stream, q_nope, w, out, status)
    _check("nsa_mla_absorb_q", load().nsa_mla_absorb_q(_at(q_nope), q_nope.stride(0), q_nope.stride(1), _at(w), R, H, _D_NOPE,
                                                       _D_V, _D_LATENT, _at(out), _at(status), handle))


def nsa_mla_project_v(latent: torch.Tensor, w: torch.Tensor, out: torch.Tensor, status: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """latent [R, H, 512] (any row / head strides) through each head's W_v: out [R, H, 128]."""
    H = _heads_of(w)
    R, _ = _rows("latent", latent, _D_LATENT, H)
    _bf16("out", out, (R, H, _D_V))
    _status_word(status)
    handle = _launch_on(stream, latent, w, out, status)
    _check("nsa_mla_project_v", load().nsa_mla_project_v(_at(latent), latent.stride(0), latent.stride(1), _at(w), R, H,
                                                         _D_NOPE, _D_V, _D_LATENT, _at(out), _at(status), handle))
