"""Python binding of libmtpsd: the C-ABI calls under the same names, taking
torch CUDA tensors.  Argument marshalling only: every step runs in the
library's CUDA kernels on the current torch stream (or the stream given: a
torch stream or a raw handle).  Outputs not passed in are allocated with torch
before the call, in the memory of the stream that the call runs on."""
from __future__ import annotations

import ctypes as C
from typing import Optional

import numpy as np
import torch

from . import _native as N
from ._native import check, lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype, ndim: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _torch_stream(stream, device):
    """A torch stream, or a raw handle as one (None, the current stream, stays None)."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream(stream).value or 0
    # 0 and 1 are the handles of the default stream
    return torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)


def _empty(stream, *shape, dtype, device) -> torch.Tensor:
    """A new output.  torch's allocator hands a freed block out again in the order of the stream it was allocated on, so
    with a stream given the block has to be that stream's: one of the current stream may still be in use there, and after
    the caller has dropped it the current stream could take it while the call still writes.  The current stream, where the
    caller is, is recorded as a user of the block, so that it is not handed out while work queued there still reads it."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    stream = _torch_stream(stream, device)
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if current != stream:
        t.record_stream(current)
    return t


class Workspace:
    """A reusable device scratch buffer, grown outside the timed path."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = torch.empty(0, dtype=torch.uint8, device=device)

    def get(self, nbytes: int) -> torch.Tensor:
        if self.buf.numel() < nbytes:
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        return self.buf


_default_ws = {}


def _ws(workspace: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    if workspace is not None:
        return workspace
    key = str(device)
    if key not in _default_ws:
        _default_ws[key] = Workspace(device)
    return _default_ws[key].get(nbytes)


def _paged(paged):
    """(block_table [B, n] int32 CUDA tensor, page_size) -> a PagedKV (None stays None)."""
    if paged is None:
        return None
    bt, page_size = paged
    _need(bt, "block_table", torch.int32, 2)
    return N.PagedKV(block_table=bt.data_ptr(), bt_stride=bt.shape[1], page_size=int(page_size))


def _byref(x):
    return None if x is None else C.byref(x)


# --------------------------------------------------------------------------- merge

def merge_tokens(prompt_tokens, prompt_offsets, draft_tokens, merged_tokens=None, merged_offsets=None,
                 stream=None):
    _need(prompt_tokens, "prompt_tokens", torch.int64, 1)
    _need(prompt_offsets, "prompt_offsets", torch.uint32, 1)
    _need(draft_tokens, "draft_tokens", torch.int64, 2)
    B, K = draft_tokens.shape
    S = prompt_tokens.numel()
    if prompt_offsets.numel() != B + 1:
        raise ValueError("prompt_offsets must have B+1 entries")
    if merged_tokens is None:
        merged_tokens = _empty(stream, S + B * K, dtype=torch.int64, device=prompt_tokens.device)
    if merged_offsets is None:
        merged_offsets = _empty(stream, B + 1, dtype=torch.uint32, device=prompt_tokens.device)
    check("mtpsd_merge_tokens", lib().mtpsd_merge_tokens(
        _ptr(prompt_tokens), S, _ptr(prompt_offsets), _ptr(draft_tokens), B, K,
        _ptr(merged_tokens), _ptr(merged_offsets), _stream(stream)))
    return merged_tokens, merged_offsets


def host_merged_offsets(prompt_offsets: np.ndarray, K: int) -> np.ndarray:
    po = np.ascontiguousarray(prompt_offsets, dtype=np.uint32)
    out = np.empty_like(po)
    lib().mtpsd_host_merged_offsets(po.ctypes.data_as(C.c_void_p), len(po) - 1, K,
                                    out.ctypes.data_as(C.c_void_p))
    return out


def pack_latent_fp8(latent, packed=None, stream=None):
    """latent [T, 576] bf16 or float32 -> the FP8 latent cache rows [T, 656] uint8."""
    f32 = latent.dtype == torch.float32
    _need(latent, "latent", torch.float32 if f32 else torch.bfloat16, 2)
    if latent.shape[1] != 576:
        raise ValueError("latent rows must have 576 values")
    T = latent.shape[0]
    if packed is None:
        packed = _empty(stream, T, 656, dtype=torch.uint8, device=latent.device)
    check("mtpsd_pack_latent_fp8", lib().mtpsd_pack_latent_fp8(
        _ptr(latent), N.MTPSD_F32 if f32 else N.MTPSD_BF16, T, _ptr(packed), _stream(stream)))
    return packed


def resolve_indexer_types(n_layers: int, explicit=None, pattern=None, freq=None, offset=None):
    """Per-layer indexer schedule as a list of "full" / "shared" (an explicit list is checked and
    returned; otherwise the library resolves the pattern or the frequency and offset)."""
    if explicit is not None and len(explicit) > 0:
        types = [str(t) for t in explicit]
        if len(types) != n_layers or any(t not in ("full", "shared") for t in types) or types[0] != "full":
            raise ValueError("an explicit schedule needs one full/shared entry per layer, the first full")
        return types
    out = np.zeros(max(n_layers, 1), dtype=np.int32)
    check("mtpsd_resolve_indexer_types", lib().mtpsd_resolve_indexer_types(
        n_layers, pattern.encode() if pattern else None, 0 if freq is None else int(freq),
        -1 if offset is None else int(offset), out.ctypes.data_as(C.c_void_p)))
    return ["full" if x else "shared" for x in out[:n_layers]]


# --------------------------------------------------------------------------- FP8

def quantize_fp8_block128(x, codes=None, scales=None, stream=None):
    _need(x, "x", torch.float32)
    if x.numel() % 128:
        raise ValueError("x must hold a multiple of 128 values")
    nb = x.numel() // 128
    if codes is None:
        codes = _empty(stream, x.shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = _empty(stream, x.shape[:-1] + (x.shape[-1] // 128,), dtype=torch.float32, device=x.device)
    check("mtpsd_quantize_fp8_block128", lib().mtpsd_quantize_fp8_block128(
        _ptr(x), nb, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


# --------------------------------------------------------------------------- indexer + top-k

def scores_ld(max_visible: int) -> int:
    return int(lib().mtpsd_scores_ld(max_visible))


def indexer_topk_workspace_size(B, R, max_visible, topk) -> int:
    return int(lib().mtpsd_indexer_topk_workspace_size(B, R, max_visible, topk))


def indexer_plan_bytes(B, R) -> int:
    return int(lib().mtpsd_indexer_topk_plan_bytes(B, R))


def indexer_topk_aux_bytes(B, R, max_visible, topk) -> int:
    return int(lib().mtpsd_indexer_topk_aux_bytes(B, R, max_visible, topk))


def topk_workspace_size(R, max_len, k) -> int:
    return int(lib().mtpsd_topk_workspace_size(R, max_len, k))


def _indexer_args(q, q_scale, weights, k_cache, k_scale, cache_start, row_offsets, row_pos, topk, max_visible,
                  topk_idx, topk_score, scores, ws, dev_status):
    fp8 = q.dtype == torch.uint8
    _need(q, "q", torch.uint8 if fp8 else torch.float32, 3)
    _need(k_cache, "k_cache", q.dtype, 2)
    _need(weights, "weights", torch.float32, 2)
    if cache_start is not None:
        _need(cache_start, "cache_start", torch.int64, 1)
    _need(row_offsets, "row_offsets", torch.uint32, 1)
    _need(row_pos, "row_pos", torch.int64, 1)
    if fp8:
        _need(q_scale, "q_scale", torch.float32)
        _need(k_scale, "k_scale", torch.float32)
    if scores is not None:
        _need(scores, "scores", torch.float32, 2)
        if scores.shape[0] != q.shape[0] or scores.shape[1] != scores_ld(max_visible):
            raise ValueError("scores must be [R, scores_ld(max_visible)]")
    R, H, D = q.shape
    return N.IndexerArgs(B=row_offsets.numel() - 1, R=R, n_heads=H, head_dim=D, topk=topk,
                         dtype=N.MTPSD_FP8_E4M3 if fp8 else N.MTPSD_F32,
                         q=q.data_ptr(), q_scale=q_scale.data_ptr() if fp8 else None,
                         weights=weights.data_ptr(), k_cache=k_cache.data_ptr(),
                         k_scale=k_scale.data_ptr() if fp8 else None, pool_tokens=k_cache.shape[0],
                         cache_start=None if cache_start is None else cache_start.data_ptr(),
                         row_offsets=row_offsets.data_ptr(),
                         row_pos=row_pos.data_ptr(), max_visible=max_visible,
                         topk_idx=None if topk_idx is None else topk_idx.data_ptr(),
                         topk_score=None if topk_score is None else topk_score.data_ptr(),
                         scores=None if scores is None else scores.data_ptr(),
                         workspace=ws.data_ptr(), workspace_bytes=ws.numel(),
                         dev_status=None if dev_status is None else dev_status.data_ptr())


def indexer_topk(q, q_scale, weights, k_cache, k_scale, cache_start, row_offsets, row_pos, topk: int,
                 max_visible: int, topk_idx=None, topk_score=None, scores=None, workspace=None,
                 dev_status=None, stream=None, paged=None):
    """paged = (block_table [B, n] int32, page_size) reads the caches through the block table
    (cache_start is then ignored and may be None)."""
    R = q.shape[0]
    B = row_offsets.numel() - 1
    if topk_idx is None:
        topk_idx = _empty(stream, R, topk, dtype=torch.int32, device=q.device)
    nbytes = indexer_topk_aux_bytes(B, R, max_visible, topk) if scores is not None else \
        indexer_topk_workspace_size(B, R, max_visible, topk)
    ws = _ws(workspace, nbytes, q.device)
    a = _indexer_args(q, q_scale, weights, k_cache, k_scale, cache_start, row_offsets, row_pos, topk, max_visible,
                      topk_idx, topk_score, scores, ws, dev_status)
    if paged is None:
        check("mtpsd_indexer_topk", lib().mtpsd_indexer_topk(C.byref(a), _stream(stream)))
    else:
        check("mtpsd_indexer_topk_paged", lib().mtpsd_indexer_topk_paged(C.byref(a), _byref(_paged(paged)),
                                                                           _stream(stream)))
    return topk_idx


def indexer_scores(q, q_scale, weights, k_cache, k_scale, cache_start, row_offsets, row_pos, max_visible: int,
                   scores=None, workspace=None, dev_status=None, stream=None, paged=None):
    """The score matrix [R, scores_ld(max_visible)] alone (row r valid up to row_pos[r])."""
    R = q.shape[0]
    B = row_offsets.numel() - 1
    if scores is None:
        scores = _empty(stream, R, scores_ld(max_visible), dtype=torch.float32, device=q.device)
    ws = _ws(workspace, indexer_plan_bytes(B, R), q.device)
    a = _indexer_args(q, q_scale, weights, k_cache, k_scale, cache_start, row_offsets, row_pos, 1, max_visible,
                      None, None, scores, ws, dev_status)
    if paged is None:
        check("mtpsd_indexer_scores", lib().mtpsd_indexer_scores(C.byref(a), _stream(stream)))
    else:
        check("mtpsd_indexer_scores_paged", lib().mtpsd_indexer_scores_paged(C.byref(a), _byref(_paged(paged)),
                                                                             _stream(stream)))
    return scores


def topk(scores, row_len, max_len: int, k: int, out_idx=None, out_score=None, dev_status=None, stream=None,
         row_len_add: int = 0, workspace=None):
    """Top-k per row; row r's valid prefix has row_len[r] + row_len_add scores."""
    _need(scores, "scores", torch.float32, 2)
    _need(row_len, "row_len", torch.int64, 1)
    R, ld = scores.shape
    if out_idx is None:
        out_idx = _empty(stream, R, k, dtype=torch.int32, device=scores.device)
    nbytes = topk_workspace_size(R, max_len, k)
    ws = _ws(workspace, nbytes, scores.device) if nbytes else None
    check("mtpsd_topk", lib().mtpsd_topk(
        _ptr(scores), ld, R, _ptr(row_len), row_len_add, max_len, k, _ptr(out_idx), _ptr(out_score), _ptr(ws),
        0 if ws is None else ws.numel(), _ptr(dev_status), _stream(stream)))
    return out_idx


# --------------------------------------------------------------------------- sparse MLA

def sparse_mla_workspace_size(R, H, n_idx, n_append, dtype) -> int:
    return int(lib().mtpsd_sparse_mla_workspace_size(R, H, n_idx, n_append, dtype))


def indexer_topk_launch_count(H, D, dtype, max_visible, topk) -> int:
    """Kernel launches of one indexer_topk call (aligned q and k_cache)."""
    return int(lib().mtpsd_indexer_topk_launch_count(H, D, dtype, max_visible, topk))


def topk_launch_count(max_len, k) -> int:
    """Kernel launches of one topk call (aligned score rows)."""
    return int(lib().mtpsd_topk_launch_count(max_len, k))


def indexer_scores_launch_count(H, D, dtype) -> int:
    """Kernel launches of one indexer_scores call (aligned q and k_cache)."""
    return int(lib().mtpsd_indexer_scores_launch_count(H, D, dtype))


def sparse_mla_launch_count(R, H, n_idx, n_append, dtype) -> int:
    """Kernel launches of one sparse_mla_decode call (16-byte aligned output)."""
    return int(lib().mtpsd_sparse_mla_launch_count(R, H, n_idx, n_append, dtype))


def sparse_mla_decode(q, latent, cache_start, row_offsets, row_pos, idx, softmax_scale: float,
                      n_append: int = 0, append_base=None, row_pos_add: int = 0, out=None, lse=None,
                      workspace=None, dev_status=None, stream=None, paged=None):
    """paged = (block_table [B, n] int32, page_size) gathers through the block table (cache_start is
    then ignored and may be None)."""
    bf16 = q.dtype == torch.bfloat16
    _need(q, "q", torch.bfloat16 if bf16 else torch.float32, 3)
    packed = latent.dtype == torch.uint8     # a packed latent cache (656-byte FP8 or 416-byte 4-bit rows)
    if packed:
        _need(latent, "latent", torch.uint8, 2)
        if not bf16 or latent.shape[1] not in (656, 416):
            raise ValueError("a packed latent cache needs bf16 queries and 656-byte (FP8) or 416-byte (4-bit) rows")
    else:
        _need(latent, "latent", q.dtype, 2)
    if cache_start is not None:
        _need(cache_start, "cache_start", torch.int64, 1)
    _need(row_offsets, "row_offsets", torch.uint32, 1)
    _need(row_pos, "row_pos", torch.int64, 1)
    _need(idx, "idx", torch.int32, 2)
    if append_base is not None:
        _need(append_base, "append_base", torch.int64, 1)
    R, H, DL = q.shape
    dt = _latent_dtype(latent)
    if out is None:
        out = _empty(stream, R, H, 512, dtype=q.dtype, device=q.device)
    nbytes = sparse_mla_workspace_size(R, H, idx.shape[1], n_append, dt)
    if nbytes and workspace is None and dt == N.MTPSD_FP4_MLA:
        ws = _empty(stream, nbytes, dtype=torch.uint8, device=q.device)     # the call's own: calls on two streams do not share it
    else:
        ws = _ws(workspace, nbytes, q.device) if nbytes else workspace
    a = N.MlaArgs(B=row_offsets.numel() - 1, R=R, n_heads=H, d_latent=DL, d_v=512, n_idx=idx.shape[1],
                  n_append=n_append, dtype=dt, softmax_scale=softmax_scale, row_pos_add=row_pos_add,
                  q=q.data_ptr(), latent=latent.data_ptr(), pool_tokens=latent.shape[0],
                  cache_start=None if cache_start is None else cache_start.data_ptr(),
                  row_offsets=row_offsets.data_ptr(), row_pos=row_pos.data_ptr(), idx=idx.data_ptr(),
                  append_base=None if append_base is None else append_base.data_ptr(),
                  out=out.data_ptr(), lse=None if lse is None else lse.data_ptr(),
                  workspace=None if ws is None else ws.data_ptr(),
                  workspace_bytes=0 if ws is None else ws.numel(),
                  dev_status=None if dev_status is None else dev_status.data_ptr())
    if paged is None:
        check("mtpsd_sparse_mla_decode", lib().mtpsd_sparse_mla_decode(C.byref(a), _stream(stream)))
    else:
        check("mtpsd_sparse_mla_decode_paged", lib().mtpsd_sparse_mla_decode_paged(
            C.byref(a), _byref(_paged(paged)), _stream(stream)))
    return out


# --------------------------------------------------------------------------- accept / write-back / share

def accept_greedy(draft, target_argmax, magic_draft_id: int = -1, num_accepted=None, next_tokens=None,
                  stream=None):
    _need(draft, "draft", torch.int64, 2)
    _need(target_argmax, "target_argmax", torch.int64, 2)
    B, K = draft.shape
    if target_argmax.shape != (B, K + 1):
        raise ValueError("target_argmax must be [B, K+1]")
    if num_accepted is None:
        num_accepted = _empty(stream, B, dtype=torch.int32, device=draft.device)
    if next_tokens is None:
        next_tokens = _empty(stream, B, dtype=torch.int64, device=draft.device)
    check("mtpsd_accept_greedy", lib().mtpsd_accept_greedy(
        _ptr(draft), _ptr(target_argmax), B, K, magic_draft_id, _ptr(num_accepted), _ptr(next_tokens),
        _stream(stream)))
    return num_accepted, next_tokens


def accept_stochastic(draft, draft_probs, target_probs, u_accept, u_sample, num_accepted=None, next_tokens=None,
                      dev_status=None, stream=None):
    """Rejection-sampling acceptance: draft [B, K] int64, draft_probs [B, K, V] and target_probs [B, K+1, V]
    float32, u_accept [B, K] and u_sample [B] float32 uniforms."""
    _need(draft, "draft", torch.int64, 2)
    _need(draft_probs, "draft_probs", torch.float32, 3)
    _need(target_probs, "target_probs", torch.float32, 3)
    _need(u_accept, "u_accept", torch.float32, 2)
    _need(u_sample, "u_sample", torch.float32, 1)
    B, K = draft.shape
    V = target_probs.shape[2]
    if target_probs.shape != (B, K + 1, V) or draft_probs.shape != (B, K, V) or u_accept.shape != (B, K) \
            or u_sample.shape != (B,):
        raise ValueError("shapes must be draft [B,K], draft_probs [B,K,V], target_probs [B,K+1,V], "
                         "u_accept [B,K], u_sample [B]")
    if num_accepted is None:
        num_accepted = _empty(stream, B, dtype=torch.int32, device=draft.device)
    if next_tokens is None:
        next_tokens = _empty(stream, B, dtype=torch.int64, device=draft.device)
    check("mtpsd_accept_stochastic", lib().mtpsd_accept_stochastic(
        _ptr(draft), _ptr(draft_probs), _ptr(target_probs), _ptr(u_accept), _ptr(u_sample), B, K, V,
        _ptr(num_accepted), _ptr(next_tokens), _ptr(dev_status), _stream(stream)))
    return num_accepted, next_tokens


def kv_writeback(src_latent, src_idxk, src_idxs, num_accepted, dst_latent, dst_idxk, dst_idxs, cache_start, dst_pos,
                 next_pos=None, dev_status=None, stream=None):
    bf16 = src_latent.dtype == torch.bfloat16
    packed = src_latent.dtype == torch.uint8   # packed latent rows (656 or 416 bytes)
    _need(src_latent, "src_latent", src_latent.dtype if packed else (torch.bfloat16 if bf16 else torch.float32), 3)
    _need(dst_latent, "dst_latent", src_latent.dtype, 2)
    _need(num_accepted, "num_accepted", torch.int32, 1)
    _need(cache_start, "cache_start", torch.int64, 1)
    _need(dst_pos, "dst_pos", torch.int64, 1)
    B, W, _ = src_latent.shape
    idx_dim = 0
    if src_idxk is not None:
        _need(src_idxk, "src_idxk", torch.uint8, 3)
        _need(dst_idxk, "dst_idxk", torch.uint8, 2)
        idx_dim = src_idxk.shape[2]
    if src_idxs is not None:
        _need(src_idxs, "src_idxs", torch.float32)
        _need(dst_idxs, "dst_idxs", torch.float32)
    check("mtpsd_kv_writeback", lib().mtpsd_kv_writeback(
        _ptr(src_latent), _ptr(src_idxk), _ptr(src_idxs), B, W,
        _latent_dtype(src_latent, dst_latent), idx_dim,
        _ptr(num_accepted), _ptr(dst_latent), _ptr(dst_idxk), _ptr(dst_idxs), _ptr(cache_start), _ptr(dst_pos),
        dst_latent.shape[0], _ptr(next_pos), _ptr(dev_status), _stream(stream)))
    return next_pos


def topk_share_gather(step0_topk, row_offsets, num_accepted=None, shared_idx=None, dev_status=None, stream=None,
                      row_pos=None, shared_pos=None):
    """shared_idx[b] = step0_topk[row_offsets[b] + num_accepted[b]] (row 0 without num_accepted); with
    row_pos, shared_pos[b] receives the position of that row."""
    _need(step0_topk, "step0_topk", torch.int32, 2)
    _need(row_offsets, "row_offsets", torch.uint32, 1)
    if num_accepted is not None:
        _need(num_accepted, "num_accepted", torch.int32, 1)
    B = row_offsets.numel() - 1
    k = step0_topk.shape[1]
    if shared_idx is None:
        shared_idx = _empty(stream, B, k, dtype=torch.int32, device=step0_topk.device)
    if row_pos is not None:
        _need(row_pos, "row_pos", torch.int64, 1)
        if shared_pos is None:
            shared_pos = _empty(stream, B, dtype=torch.int64, device=step0_topk.device)
    check("mtpsd_topk_share_gather", lib().mtpsd_topk_share_gather(
        _ptr(step0_topk), _ptr(row_offsets), _ptr(num_accepted), B, k, _ptr(shared_idx), _ptr(row_pos),
        _ptr(shared_pos if row_pos is not None else None), _ptr(dev_status), _stream(stream)))
    return shared_idx


# --------------------------------------------------------------------------- paged caches

_LATENT_TYPES = {(torch.bfloat16, 576): N.MTPSD_BF16, (torch.float32, 576): N.MTPSD_F32, (torch.uint8, 656): N.MTPSD_FP8_DS_MLA,
                 (torch.uint8, 416): N.MTPSD_FP4_MLA}


def _latent_dtype(t, dst=None):
    """The type of latent rows (the last dim); dst: the cache that such rows are written to."""
    dt = _LATENT_TYPES.get((t.dtype, t.shape[-1]))
    if dt is None:
        raise ValueError("latent rows must be 576 bfloat16 or float32 values, or 656 (FP8) or 416 (4-bit) bytes, got "
                         f"{t.shape[-1]} of {t.dtype}")
    if dst is not None and dst.shape[-1] != t.shape[-1]:
        raise ValueError(f"rows of {t.shape[-1]} cannot be written to a cache whose rows have {dst.shape[-1]}")
    return dt


def assign_cache_locs(block_table, page_size: int, start_pos, W: int, out_cache_loc=None, dev_status=None,
                      stream=None):
    """out_cache_loc [B, W] int64: the slots of positions start_pos[b] + j (j < W), -1 where none."""
    _need(start_pos, "start_pos", torch.int64, 1)
    B = start_pos.numel()
    if out_cache_loc is None:
        out_cache_loc = _empty(stream, B, W, dtype=torch.int64, device=start_pos.device)
    pk = _paged((block_table, page_size))
    check("mtpsd_assign_cache_locs", lib().mtpsd_assign_cache_locs(
        C.byref(pk), B, _ptr(start_pos), W, _ptr(out_cache_loc), _ptr(dev_status), _stream(stream)))
    return out_cache_loc


def kv_move_accepted(latent, idxk, idxs, out_cache_loc, accept_index, num_accepted, dev_status=None, stream=None):
    """Moves the accepted rows' KV (window slots out_cache_loc[b, accept_index[b, i]]) to the front slots
    out_cache_loc[b, i], i < num_accepted[b] + 1, in every cache of the layer (in place)."""
    _need(latent, "latent", latent.dtype, 2)
    _need(out_cache_loc, "out_cache_loc", torch.int64, 2)
    _need(accept_index, "accept_index", torch.int32, 2)
    _need(num_accepted, "num_accepted", torch.int32, 1)
    B, W = out_cache_loc.shape
    idx_dim = 0
    if idxk is not None:
        _need(idxk, "idxk", torch.uint8, 2)
        idx_dim = idxk.shape[1]
    if idxs is not None:
        _need(idxs, "idxs", torch.float32, 1)
    check("mtpsd_kv_move_accepted", lib().mtpsd_kv_move_accepted(
        _ptr(latent), _latent_dtype(latent), _ptr(idxk), idx_dim, _ptr(idxs), latent.shape[0],
        _ptr(out_cache_loc), _ptr(accept_index), _ptr(num_accepted), B, W, _ptr(dev_status), _stream(stream)))


def kv_writeback_slots(src_latent, src_idxk, src_idxs, num_accepted, dst_latent, dst_idxk, dst_idxs, dst_slots,
                       dst_pos=None, next_pos=None, dev_status=None, stream=None):
    """The accepted rows (num_accepted + 1, clamped to [1, W]) of each window to pool slots dst_slots [B, W];
    with dst_pos, next_pos[b] = dst_pos[b] + the rows written."""
    _need(src_latent, "src_latent", src_latent.dtype, 3)
    _need(dst_latent, "dst_latent", src_latent.dtype, 2)
    _need(num_accepted, "num_accepted", torch.int32, 1)
    _need(dst_slots, "dst_slots", torch.int64, 2)
    B, W, _ = src_latent.shape
    idx_dim = 0
    if src_idxk is not None:
        _need(src_idxk, "src_idxk", torch.uint8, 3)
        _need(dst_idxk, "dst_idxk", torch.uint8, 2)
        idx_dim = src_idxk.shape[2]
    if src_idxs is not None:
        _need(src_idxs, "src_idxs", torch.float32)
        _need(dst_idxs, "dst_idxs", torch.float32)
    check("mtpsd_kv_writeback_slots", lib().mtpsd_kv_writeback_slots(
        _ptr(src_latent), _ptr(src_idxk), _ptr(src_idxs), B, W, _latent_dtype(src_latent, dst_latent), idx_dim,
        _ptr(num_accepted), _ptr(dst_latent), _ptr(dst_idxk), _ptr(dst_idxs), _ptr(dst_slots), dst_latent.shape[0],
        _ptr(dst_pos), _ptr(next_pos), _ptr(dev_status), _stream(stream)))
    return next_pos


# --------------------------------------------------------------------------- head and logits

def _current(t, name: str) -> int:
    """The current device, on whose stream the launch goes: every tensor has to be there, t the first of them."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch.cuda.current_device()


def _tensor(t, name: str, dev: int, dtype, ndim: int):
    """Checks a contiguous tensor on device dev; returns its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device cuda:{dev}, is on {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name: str, dev: int, dtypes, R: int, V: int):
    """Checks a tensor [R, V] on device dev whose rows are contiguous; returns its address and its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device cuda:{dev}, is on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != R or t.shape[1] != V:
        raise ValueError(f"{name} must be [{R}, {V}], got {list(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), max(V, 1)
    ld, step = t.stride()
    if R and V > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if R > 1 and ld < V:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t.data_ptr(), ld if R > 1 else max(V, 1)


def _status_ptr(t, dev: int):
    if t is None:
        return None
    if t.numel() < 1:
        raise ValueError("dev_status must hold one int32")
    return _tensor(t, "dev_status", dev, torch.int32, t.dim())


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_OUT_TYPES = (torch.bfloat16, torch.float32)
_F32_ONLY = (torch.float32,)


def gemm_fp8_block128(a, a_scale, w, w_scale, out=None, out_dtype=None, dev_status=None, stream=None):
    """out [M, N] = the product of E4M3 codes a [M, K] and w [N, K] (uint8) with a float32 scale per block of 128:
    a_scale [M, K/128]; w_scale [N, K/128] (quantize_fp8_block128 of the weight) or [ceil(N/128), K/128] (128 x 128
    blocks).  out is bf16 (or out_dtype float32); an out given may have any row stride."""
    dev = _current(a, "a")
    pa, pw = _tensor(a, "a", dev, torch.uint8, 2), _tensor(w, "w", dev, torch.uint8, 2)
    M, K = a.shape
    n_out, k_w = w.shape
    if k_w != K:
        raise ValueError("a and w must have the same K")
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    kbs = K // 128
    psa, psw = _tensor(a_scale, "a_scale", dev, torch.float32, a_scale.dim()), _tensor(w_scale, "w_scale", dev, torch.float32, 2)
    if a_scale.shape not in ((M, kbs), (M * kbs,)):
        raise ValueError("a_scale must be [M, K/128]")
    if w_scale.shape == (n_out, kbs):
        rows = 1
    elif w_scale.shape == (-(-n_out // 128), kbs):
        rows = 128
    else:
        raise ValueError("w_scale must be [N, K/128] or [ceil(N/128), K/128]")
    if out is None:
        out = _empty(stream, M, n_out, dtype=out_dtype or torch.bfloat16, device=a.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    po, ld = _rows(out, "out", dev, _OUT_TYPES, M, n_out)
    check("mtpsd_gemm_fp8_block128", lib().mtpsd_gemm_fp8_block128(
        pa, psa, pw, psw, rows, M, n_out, K, N.MTPSD_F32 if out.dtype == torch.float32 else N.MTPSD_BF16, po, ld,
        _status_ptr(dev_status, dev), _raw_stream(stream, dev)))
    return out


def token_counts_ld(V: int) -> int:
    """Row stride (int16 words) of a token table of V tokens."""
    return int(lib().mtpsd_token_counts_ld(V))


def _counts(counts, V, B, count_rows, dev):
    """Checks a token table and the requests' rows in it; returns their addresses."""
    p = _tensor(counts, "counts", dev, torch.int16, 2)
    n_rows, ld = counts.shape
    if ld < V or ld % 8:
        raise ValueError("counts rows must have at least V words, a multiple of 8 (token_counts_ld)")
    if count_rows is None:
        if n_rows < B:
            raise ValueError("counts has fewer rows than requests")
        return p, None
    if count_rows.numel() != B:
        raise ValueError("count_rows must have one entry per request")
    return p, _tensor(count_rows, "count_rows", dev, torch.int32, 1)


def token_counts_build(tokens, offsets, V: int, n_prompt=None, counts=None, count_rows=None, dev_status=None,
                       stream=None):
    """The token table rows of B requests from their tokens [S] int64 (ragged, offsets [B+1] uint32): the first
    n_prompt[b] (int64; all without it) set the prompt bit, the others count as output.  Request b fills row b, or
    count_rows[b] of a larger table."""
    dev = _current(tokens, "tokens")
    pt, po = _tensor(tokens, "tokens", dev, torch.int64, 1), _tensor(offsets, "offsets", dev, torch.uint32, 1)
    B = offsets.numel() - 1
    if B < 0:
        raise ValueError("offsets must have B+1 entries")
    pn = None
    if n_prompt is not None:
        pn = _tensor(n_prompt, "n_prompt", dev, torch.int64, 1)
        if n_prompt.numel() != B:
            raise ValueError("n_prompt must have one entry per request")
    if counts is None:
        if count_rows is not None:
            raise ValueError("count_rows needs a table")
        counts = _empty(stream, B, token_counts_ld(V), dtype=torch.int16, device=tokens.device)
    pc, pr = _counts(counts, V, B, count_rows, dev)
    check("mtpsd_token_counts_build", lib().mtpsd_token_counts_build(
        pt, tokens.numel(), po, pn, B, V, pc, counts.shape[1], counts.shape[0], pr, _status_ptr(dev_status, dev),
        _raw_stream(stream, dev)))
    return counts


def token_counts_accept(counts, V: int, draft, num_accepted, next_tokens, count_rows=None, dev_status=None, stream=None):
    """Adds draft[b, :num_accepted[b]] and next_tokens[b] to the token table (in place); draft and num_accepted may be
    None (one token per request)."""
    dev = _current(next_tokens, "next_tokens")
    px = _tensor(next_tokens, "next_tokens", dev, torch.int64, 1)
    B = next_tokens.numel()
    K, pd, pn = 0, None, None
    if (draft is None) != (num_accepted is None):
        raise ValueError("give draft and num_accepted together or neither")
    if draft is not None:
        pd, pn = _tensor(draft, "draft", dev, torch.int64, 2), _tensor(num_accepted, "num_accepted", dev, torch.int32, 1)
        K = draft.shape[1]
        if draft.shape[0] != B or num_accepted.numel() != B:
            raise ValueError("draft [B, K], num_accepted [B] and next_tokens [B] must have the same B")
    pc, pr = _counts(counts, V, B, count_rows, dev)
    check("mtpsd_token_counts_accept", lib().mtpsd_token_counts_accept(
        pd, pn, px, B, K, V, pc, counts.shape[1], counts.shape[0], pr, _status_ptr(dev_status, dev),
        _raw_stream(stream, dev)))
    return counts


def process_logits(logits, row_offsets, draft=None, counts=None, count_rows=None, repetition=None, frequency=None,
                   presence=None, bias_offsets=None, bias_tokens=None, bias_values=None, bitmask=None, mask_rows=None,
                   temperature=None, argmax=None, probs=None, out_logits=None, dev_status=None, stream=None):
    """Penalties, biases and grammar masks on logits [R, V] (bf16 or float32, any row stride), then the outputs given:
    argmax [R] int64, probs [R, V] float32, out_logits [R, V] float32 (may be logits itself).  With none given, argmax
    is allocated.  Returns argmax.

    draft [B, K] int64 (row i of a request counts its first i drafts as output); counts: the token table (rows by
    request, or count_rows [B] int32); repetition, frequency, presence, temperature [B] float32; biases as ragged lists
    (bias_offsets [B+1] uint32, bias_tokens int32, bias_values float32); bitmask [n, ceil(V/32)] int32, one row per
    logits row, or mask_rows [R] int32 (-1: none)."""
    dev = _current(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [R, V]")
    R, V = logits.shape
    px, ld = _rows(logits, "logits", dev, _OUT_TYPES, R, V)
    po = _tensor(row_offsets, "row_offsets", dev, torch.uint32, 1)
    B = row_offsets.numel() - 1
    K, pd = 0, None
    if draft is not None:
        pd = _tensor(draft, "draft", dev, torch.int64, 2)
        if draft.shape[0] != B:
            raise ValueError("draft must be [B, K]")
        K = draft.shape[1]
    pc = pr = None
    c_ld = c_rows = 0
    if counts is not None:
        pc, pr = _counts(counts, V, B, count_rows, dev)
        c_rows, c_ld = counts.shape
    elif count_rows is not None:
        raise ValueError("count_rows without counts")

    def per_request(t, name):
        if t is None:
            return None
        p = _tensor(t, name, dev, torch.float32, 1)
        if t.numel() != B:
            raise ValueError(f"{name} must have one entry per request")
        return p

    p_rep, p_freq = per_request(repetition, "repetition"), per_request(frequency, "frequency")
    p_pres, p_temp = per_request(presence, "presence"), per_request(temperature, "temperature")
    p_bo = p_bt = p_bv = None
    n_bias = 0
    if bias_offsets is not None or bias_tokens is not None or bias_values is not None:
        if bias_offsets is None or bias_tokens is None or bias_values is None:
            raise ValueError("give bias_offsets, bias_tokens and bias_values together or none")
        p_bo = _tensor(bias_offsets, "bias_offsets", dev, torch.uint32, 1)
        p_bt = _tensor(bias_tokens, "bias_tokens", dev, torch.int32, 1)
        p_bv = _tensor(bias_values, "bias_values", dev, torch.float32, 1)
        n_bias = bias_tokens.numel()
        if bias_offsets.numel() != B + 1 or bias_values.numel() != n_bias:
            raise ValueError("bias_offsets must be [B+1], bias_tokens and bias_values of one length")
    p_mask = p_mrows = None
    n_masks = 0
    if bitmask is not None:
        p_mask = _tensor(bitmask, "bitmask", dev, torch.int32, 2)
        n_masks, words = bitmask.shape
        if words != -(-V // 32):
            raise ValueError("bitmask rows must have ceil(V/32) words")
    if mask_rows is not None:
        p_mrows = _tensor(mask_rows, "mask_rows", dev, torch.int32, 1)
        if mask_rows.numel() != R:
            raise ValueError("mask_rows must have one entry per row")
    if argmax is None and probs is None and out_logits is None:
        argmax = _empty(stream, R, dtype=torch.int64, device=logits.device)
    p_arg = None
    if argmax is not None:
        if argmax.numel() != R:
            raise ValueError("argmax must have one entry per row")
        p_arg = _tensor(argmax, "argmax", dev, torch.int64, argmax.dim())
    p_probs, ld_probs = (None, 0) if probs is None else _rows(probs, "probs", dev, _F32_ONLY, R, V)
    p_out, ld_out = (None, 0) if out_logits is None else _rows(out_logits, "out_logits", dev, _F32_ONLY, R, V)
    # in the order of the structure's fields
    a = N.LogitsArgs(B, R, V, N.MTPSD_F32 if logits.dtype == torch.float32 else N.MTPSD_BF16, K, px, ld, po, pc, c_ld, c_rows,
                     n_bias, pr, pd, p_rep, p_freq, p_pres, p_bo, p_bt, p_bv, p_mask, p_mrows, n_masks, p_temp, p_arg,
                     p_probs, ld_probs, p_out, ld_out, _status_ptr(dev_status, dev))
    check("mtpsd_process_logits", lib().mtpsd_process_logits(C.byref(a), _raw_stream(stream, dev)))
    return argmax


# --------------------------------------------------------------------------- filling the caches

def _opt(t, name: str, dev: int, dtype, ndim: int, numel: Optional[int] = None):
    """The address of an optional tensor (None stays None), checked like _tensor."""
    if t is None:
        return None
    if type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.ndim == ndim and (
            numel is None or t.numel() == numel):
        return t.data_ptr()
    p = _tensor(t, name, dev, dtype, ndim)      # says what is wrong
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} entries, got {t.numel()}")
    return p


def block_table_grow(block_table, page_size: int, new_len, free_pages, n_free, old_len=None, lengths=None, n_free_out=None,
                     token_offsets=None, slots=None, positions=None, dev_status=None, stream=None):
    """Block tables from the requests' lengths: request b of block_table [B, n] int32 gets the pages between old_len[b] and
    new_len[b] tokens (int64 [B]; without old_len the tables are built anew) off the end of free_pages [cap] int32, of which
    n_free [1] int32 are free; n_free_out (in place without it) receives what is left.  Requests that the list has too few
    pages for get -1 (STATUS_NO_PAGES).  lengths [B] int64 (may be old_len) receives the tokens that each request has pages for, the
    next call's old_len.

    With token_offsets [B+1] uint32 (request b's tokens of this step, the last of its new length), slots [T] int64 and
    positions [T] int64 (optional) receive each token's pool slot (-1: none) and position.  Returns lengths."""
    dev = _current(block_table, "block_table")
    pt = _tensor(block_table, "block_table", dev, torch.int32, 2)
    B, width = block_table.shape
    pn = _opt(new_len, "new_len", dev, torch.int64, 1, B)
    if pn is None:
        raise TypeError("new_len must be a torch tensor")
    po = _opt(old_len, "old_len", dev, torch.int64, 1, B)
    pf = _tensor(free_pages, "free_pages", dev, torch.int32, 1)
    pc = _opt(n_free, "n_free", dev, torch.int32, 1, 1)
    if pc is None:
        raise TypeError("n_free must be a torch tensor")
    pco = pc if n_free_out is None else _opt(n_free_out, "n_free_out", dev, torch.int32, 1, 1)
    if lengths is None:
        lengths = _empty(stream, B, dtype=torch.int64, device=block_table.device)
    pl = _opt(lengths, "lengths", dev, torch.int64, 1, B)
    pto = ps = pp = None
    T = 0
    if token_offsets is not None:
        if slots is None:
            raise ValueError("token_offsets needs slots")
        pto = _opt(token_offsets, "token_offsets", dev, torch.uint32, 1, B + 1)
        ps = _tensor(slots, "slots", dev, torch.int64, 1)
        T = slots.numel()
        pp = _opt(positions, "positions", dev, torch.int64, 1, T)
    elif slots is not None or positions is not None:
        raise ValueError("slots and positions need token_offsets")
    # in the order of the structure's fields
    a = N.BlockTableArgs(pt, width, int(page_size), B, free_pages.numel(), po, pn, pf, pc, pco, pl, pto, ps, pp, T,
                         _status_ptr(dev_status, dev))
    check("mtpsd_block_table_grow", lib().mtpsd_block_table_grow(C.byref(a), _raw_stream(stream, dev)))
    return lengths


def block_table_release(block_table, page_size: int, old_len, free_pages, n_free, keep_len=None, dev_status=None, stream=None):
    """Returns the pages behind keep_len[b] tokens (none are kept without it) of each request to the free list: behind its
    n_free entries, which grow in place; their table entries become -1."""
    dev = _current(block_table, "block_table")
    pt = _tensor(block_table, "block_table", dev, torch.int32, 2)
    B, width = block_table.shape
    po = _opt(old_len, "old_len", dev, torch.int64, 1, B)
    if po is None:
        raise TypeError("old_len must be a torch tensor")
    pk = _opt(keep_len, "keep_len", dev, torch.int64, 1, B)
    pf = _tensor(free_pages, "free_pages", dev, torch.int32, 1)
    pc = _opt(n_free, "n_free", dev, torch.int32, 1, 1)
    if pc is None:
        raise TypeError("n_free must be a torch tensor")
    check("mtpsd_block_table_release", lib().mtpsd_block_table_release(
        pt, width, int(page_size), B, po, pk, pf, free_pages.numel(), pc, _status_ptr(dev_status, dev),
        _raw_stream(stream, dev)))


def slot_map(block_table, page_size: int, token_offsets, lengths, slots, positions=None, dev_status=None, stream=None):
    """slots [T] int64 (and positions [T] int64) of ragged tokens: request b's are tokens token_offsets[b] ..
    token_offsets[b+1]-1 (uint32 [B+1]), the last ones of its lengths[b] (int64) tokens.  Returns slots."""
    dev = _current(block_table, "block_table")
    pt = _tensor(block_table, "block_table", dev, torch.int32, 2)
    B, width = block_table.shape
    pto = _opt(token_offsets, "token_offsets", dev, torch.uint32, 1, B + 1)
    pl = _opt(lengths, "lengths", dev, torch.int64, 1, B)
    if pto is None or pl is None:
        raise TypeError("token_offsets and lengths must be torch tensors")
    ps = _tensor(slots, "slots", dev, torch.int64, 1)
    T = slots.numel()
    pp = _opt(positions, "positions", dev, torch.int64, 1, T)
    pk = N.PagedKV(pt, width, int(page_size))
    check("mtpsd_slot_map", lib().mtpsd_slot_map(C.byref(pk), B, pto, pl, T, ps, pp, _status_ptr(dev_status, dev),
                                                 _raw_stream(stream, dev)))
    return slots


_NORMS = {None: N.MTPSD_NORM_NONE, "rms": N.MTPSD_NORM_RMS, "layer": N.MTPSD_NORM_LAYER}
_TYPES = {torch.bfloat16: N.MTPSD_BF16, torch.float32: N.MTPSD_F32}


def _head_side(t, name, dev, norm, weight, bias, norm_dim, rot_start, out, scale, pool, stream):
    """One side of norm_rope: (HeadSide, out).  out: [T (pool), heads, D] (or without the head dimension for one head), codes or
    cache rows as uint8."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device cuda:{dev}, is on {t.device}")
    in_type = _TYPES.get(t.dtype)
    if in_type is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) == 3:
        T, heads, D = shape
        x_hs = st[1]
    elif len(shape) == 2:
        (T, D), heads = shape, 1
        x_hs = D
    else:
        raise ValueError(f"{name} must be [T, heads, D] or [T, D]")
    if D > 1 and st[-1] != 1 and T and heads:
        raise ValueError(f"{name} must have contiguous heads")
    kind = _NORMS.get(norm, -1)
    if kind < 0:
        raise ValueError(f"{name}_norm must be None, 'rms' or 'layer'")
    nd = D if norm_dim is None else int(norm_dim)
    pw = None if weight is None else _opt(weight, f"{name}_weight", dev, torch.float32, 1, nd)
    pb = None if bias is None else _opt(bias, f"{name}_bias", dev, torch.float32, 1, nd)
    rows = T if pool is None else pool
    if out is None:
        if pool is not None:
            raise ValueError(f"slots need {name}_out, the cache")
        out = _empty(stream, *shape, dtype=t.dtype, device=t.device)
    if not isinstance(out, torch.Tensor):
        raise TypeError(f"{name}_out must be a torch tensor")
    if out.get_device() != dev:
        raise ValueError(f"{name}_out must be a CUDA tensor on the current device cuda:{dev}, is on {out.device}")
    o_shape, so = out.shape, out.stride()
    psc = None
    dtype = _TYPES.get(out.dtype)
    width = D
    if dtype is None:
        if out.dtype is not torch.uint8:
            raise TypeError(f"{name}_out must be bfloat16, float32 or uint8, got {out.dtype}")
        dtype = N.MTPSD_FP8_E4M3
        if D == 576 and len(o_shape) == 2 and heads == 1 and o_shape[1] in (656, 416):     # cache rows
            width = o_shape[1]
            dtype = N.MTPSD_FP4_MLA if width == 416 else N.MTPSD_FP8_DS_MLA
        else:
            if scale is None:
                raise ValueError(f"{name}_out of codes needs {name}_scale")
            psc = _opt(scale, f"{name}_scale", dev, torch.float32, scale.dim(), rows * heads)
    if o_shape != (rows, heads, width) and not (heads == 1 and o_shape == (rows, width)):
        raise ValueError(f"{name}_out must be [{rows}, {heads}, {width}], got {list(o_shape)}")
    o_ts, o_hs = so[0], so[1] if len(so) == 3 else width
    if rows and heads:
        if width > 1 and so[-1] != 1:
            raise ValueError(f"{name}_out must have contiguous rows")
        # heads side by side within a token, or tokens within a head
        if heads > 1 and o_hs < width or rows > 1 and o_ts < width or \
                heads > 1 and rows > 1 and o_ts < (heads - 1) * o_hs + width and o_hs < (rows - 1) * o_ts + width:
            raise ValueError(f"{name}_out must have heads that do not overlap")
    # in the order of the structure's fields
    return N.HeadSide(t.data_ptr(), st[0], x_hs, heads, D, in_type, kind, nd, rot_start, pw, pb, out.data_ptr(), o_ts, o_hs, dtype,
                      psc), out


def norm_rope(positions, cos_sin, q=None, k=None, q_norm=None, q_weight=None, q_bias=None, q_norm_dim=None, q_rot_start=0,
              q_out=None, q_scale=None, k_norm=None, k_weight=None, k_bias=None, k_norm_dim=None, k_rot_start=0, k_out=None,
              k_scale=None, slots=None, interleaved=False, eps=1e-6, dev_status=None, stream=None):
    """The norms of queries q [T, heads, D] and keys k [T, heads, D] (or [T, D]; bf16 or float32, any token and head strides)
    for each head, and their rotation by the angles of positions [T] int64, in one pass.

    q_norm, k_norm: None, "rms" or "layer", over dims 0 .. norm_dim - 1 (all without it), with float32 weight and bias.
    cos_sin [n_pos, rot_dim] float32: the cosines and then the sines of each position's rot_dim / 2 angles, which turn dims rot_start ..
    rot_start + rot_dim - 1: dim i with dim i + rot_dim / 2, or neighbours (interleaved).  positions and cos_sin None: no rotation.

    Outputs: like the input without one given; bf16 or float32 [T, heads, D]; uint8 codes [T, heads, 128] with a float32 scale
    [T, heads] (what indexer_topk reads).  k_out may be a cache of `pool` rows with slots [T] int64: those types, or uint8 latent rows
    [pool, 656] (FP8) or [pool, 416] (4 bits).  Returns (q_out, k_out)."""
    if q is None and k is None:
        raise ValueError("give q, k or both")
    first, name = (q, "q") if q is not None else (k, "k")
    dev = _current(first, name)
    T = first.shape[0]
    if q is not None and k is not None and k.shape[0] != T:
        raise ValueError("q and k must have the same tokens")
    if (positions is None) != (cos_sin is None):
        raise ValueError("give positions and cos_sin together or neither")
    pp = _opt(positions, "positions", dev, torch.int64, 1, T)
    pcs = _opt(cos_sin, "cos_sin", dev, torch.float32, 2)
    n_pos, rot = (0, 0) if cos_sin is None else cos_sin.shape
    psl = _opt(slots, "slots", dev, torch.int64, 1, T)
    pool = None
    if slots is not None:
        if k is None or not isinstance(k_out, torch.Tensor):
            raise ValueError("slots need k and k_out, the cache")
        pool = k_out.shape[0]
    sq = sk = None
    if q is not None:
        sq, q_out = _head_side(q, "q", dev, q_norm, q_weight, q_bias, q_norm_dim, q_rot_start, q_out, q_scale, None, stream)
    if k is not None:
        sk, k_out = _head_side(k, "k", dev, k_norm, k_weight, k_bias, k_norm_dim, k_rot_start, k_out, k_scale, pool, stream)
    check("mtpsd_norm_rope", lib().mtpsd_norm_rope(
        _byref(sq), _byref(sk), T, pp, pcs, n_pos, rot, 1 if interleaved else 0, float(eps), psl, 0 if pool is None else pool,
        _status_ptr(dev_status, dev), _raw_stream(stream, dev)))
    return q_out, k_out


def pack_latent_fp4(latent, packed=None, slots=None, dev_status=None, stream=None):
    """latent [T, 576] bf16 or float32 -> 4-bit latent cache rows of 416 bytes: packed [T, 416] uint8, or rows slots [T] int64 of
    the cache packed [pool, 416].  Returns packed."""
    dev = _current(latent, "latent")
    if latent.dtype not in _TYPES:
        raise TypeError(f"latent must be bfloat16 or float32, got {latent.dtype}")
    pl = _tensor(latent, "latent", dev, latent.dtype, 2)
    T = latent.shape[0]
    if latent.shape[1] != 576:
        raise ValueError("latent rows must have 576 values")
    psl = _opt(slots, "slots", dev, torch.int64, 1, T)
    if packed is None:
        if slots is not None:
            raise ValueError("slots need packed, the cache")
        packed = _empty(stream, T, 416, dtype=torch.uint8, device=latent.device)
    pk = _tensor(packed, "packed", dev, torch.uint8, 2)
    if packed.shape[1] != 416 or (slots is None and packed.shape[0] != T):
        raise ValueError("packed must be [T, 416], or [pool, 416] with slots")
    check("mtpsd_pack_latent_fp4", lib().mtpsd_pack_latent_fp4(
        pl, _TYPES[latent.dtype], T, pk, psl, packed.shape[0], _status_ptr(dev_status, dev), _raw_stream(stream, dev)))
    return packed
