"""ctypes binding of libmars' packed-sequence entry points (include/mars.h): attention of whole
prompts and its gradient, attention of new tokens over the paged cache, and the append of
their K/V. Like mars.py, argument marshalling only; the rows of q, k and v may be slices of a
wider tensor (a fused projection's output).
"""
from __future__ import annotations

import torch

from .mars import PAGE_SIZE, _check, _ptr, _rc, _stream, lib

OP_ATTN_PACKED, OP_ATTN_CHUNK, OP_ATTN_PACKED_GRAD = 6, 7, 8


def _check_rows(t, name, shape):
    """A bf16 [total, heads, d] tensor whose rows may be slices of a wider tensor (the heads of
    a row contiguous); returns its row pitch in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (libmars has no CPU path)")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    total, heads, d = shape
    if t.numel() == 0:
        return heads * d
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"the heads of each row of {name} must be contiguous")
    if total == 1:
        return heads * d
    if t.stride(0) < heads * d or t.stride(0) % 8 or t.stride(0) > 0x7fffffff:
        raise ValueError(f"{name} has row pitch {t.stride(0)}: it must be a multiple of 8, at "
                         f"least {heads * d} and below 2^31")
    return t.stride(0)


def _check_one_device(stream, **tensors):
    """Every tensor on the device whose stream the call goes to."""
    want = torch.cuda.current_device() if stream is None else stream.device.index
    for name, t in tensors.items():
        if t is not None and t.device.index != want:
            raise ValueError(f"{name} is on cuda:{t.device.index}, the stream's device is "
                             f"cuda:{want}")
    if want != torch.cuda.current_device():
        raise ValueError(f"the stream is on cuda:{want}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def mars_packed_workspace_bytes(op, batch, total, hq=1, hkv=1, d=64, max_len=0):
    return int(lib().mars_packed_workspace_bytes(op, batch, total, hq, hkv, d, max_len))


def _packed_args(q, k, v, cu_seqlens, o, workspace, status):
    total, hq, d = q.shape
    hkv = k.shape[1]
    strides = (_check_rows(q, "q", (total, hq, d)), _check_rows(k, "k", (total, hkv, d)),
               _check_rows(v, "v", (total, hkv, d)))
    _check(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must hold batch + 1 boundaries")
    _check(o, "o", torch.bfloat16, (total, hq, d))
    _check(workspace, "workspace", torch.uint8)
    if status is not None:
        _check(status, "status", torch.int32, (1,))
    return cu_seqlens.shape[0] - 1, total, hq, hkv, d, strides


def mars_attn_packed(q, k, v, cu_seqlens, o, workspace, lse=None, scale: float = 0.0,
                     status=None, stream=None):
    """o[total, hq, d] (bf16) = causal attention inside each sequence of a packed batch; lse
    [hq, total] (float32, optional) its log2 row statistics (see include/mars.h)."""
    batch, total, hq, hkv, d, (qs, ks, vs) = _packed_args(q, k, v, cu_seqlens, o, workspace, status)
    if lse is not None:
        _check(lse, "lse", torch.float32, (hq, total))
    _check_one_device(stream, q=q, k=k, v=v, cu_seqlens=cu_seqlens, o=o, lse=lse,
                      workspace=workspace, status=status)
    _rc(lib().mars_attn_packed(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(o), _ptr(lse),
                               batch, total, hq, hkv, d, qs, ks, vs, float(scale),
                               _ptr(workspace), workspace.numel(), _ptr(status),
                               _stream(stream)), "mars_attn_packed")


def mars_attn_packed_grad(q, k, v, o, d_o, lse, cu_seqlens, dq, dk, dv, workspace,
                          scale: float = 0.0, status=None, stream=None):
    """dq, dk, dv (bf16) of mars_attn_packed for the upstream gradient d_o, from its o and lse
    (see include/mars.h); dq, dk, dv may be slices of a wider tensor, like q, k, v."""
    batch, total, hq, hkv, d, (qs, ks, vs) = _packed_args(q, k, v, cu_seqlens, o, workspace, status)
    _check(d_o, "d_o", torch.bfloat16, (total, hq, d))
    _check(lse, "lse", torch.float32, (hq, total))
    dqs = _check_rows(dq, "dq", (total, hq, d))
    dks, dvs = _check_rows(dk, "dk", (total, hkv, d)), _check_rows(dv, "dv", (total, hkv, d))
    _check_one_device(stream, q=q, k=k, v=v, o=o, d_o=d_o, lse=lse, cu_seqlens=cu_seqlens, dq=dq,
                      dk=dk, dv=dv, workspace=workspace, status=status)
    _rc(lib().mars_attn_packed_grad(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(d_o), _ptr(lse), _ptr(cu_seqlens), _ptr(dq),
        _ptr(dk), _ptr(dv), batch, total, hq, hkv, d, qs, ks, vs, dqs, dks, dvs, float(scale),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)), "mars_attn_packed_grad")


def mars_attn_chunk(q, k, v, cu_seqlens, k_pool, v_pool, block_table, seq_lens,
                    max_len_hint: int, o, workspace, status=None, scale: float = 0.0,
                    stream=None):
    """o[total, hq, d] (bf16) = attention of each sequence's new rows over its seq_lens[s]
    cached tokens and, causally, its own new keys (see include/mars.h)."""
    batch, total, hq, hkv, d, (qs, ks, vs) = _packed_args(q, k, v, cu_seqlens, o, workspace, status)
    num_pages = k_pool.shape[0]
    _check(k_pool, "k_pool", torch.bfloat16, (num_pages, hkv, PAGE_SIZE, d))
    _check(v_pool, "v_pool", torch.bfloat16, (num_pages, hkv, PAGE_SIZE, d))
    _check(seq_lens, "seq_lens", torch.int32, (batch,))
    _check(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}, expected [{batch}, "
                         "max_pages]")
    _check_one_device(stream, q=q, k=k, v=v, cu_seqlens=cu_seqlens, k_pool=k_pool, v_pool=v_pool,
                      block_table=block_table, seq_lens=seq_lens, o=o, workspace=workspace,
                      status=status)
    _rc(lib().mars_attn_chunk(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(k_pool),
                              _ptr(v_pool), num_pages, _ptr(block_table), block_table.shape[1],
                              _ptr(seq_lens), int(max_len_hint), _ptr(o), batch, total, hq, hkv,
                              d, PAGE_SIZE, qs, ks, vs, float(scale), _ptr(workspace),
                              workspace.numel(), _ptr(status), _stream(stream)),
        "mars_attn_chunk")


def mars_kv_append(k, v, cu_seqlens, seq_lens, block_table, k_pool, v_pool, new_lens=None,
                   slots=None, status=None, stream=None):
    """Copy each sequence's new K/V rows to its pages, after its seq_lens[s] cached tokens;
    new_lens [batch] and slots [total] (int32) are optional outputs (see include/mars.h)."""
    total, hkv, d = k.shape
    num_pages = k_pool.shape[0]
    ks, vs = _check_rows(k, "k", (total, hkv, d)), _check_rows(v, "v", (total, hkv, d))
    _check(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must hold batch + 1 boundaries")
    batch = cu_seqlens.shape[0] - 1
    _check(seq_lens, "seq_lens", torch.int32, (batch,))
    _check(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}, expected [{batch}, "
                         "max_pages]")
    _check(k_pool, "k_pool", torch.bfloat16, (num_pages, hkv, PAGE_SIZE, d))
    _check(v_pool, "v_pool", torch.bfloat16, (num_pages, hkv, PAGE_SIZE, d))
    if new_lens is not None:
        _check(new_lens, "new_lens", torch.int32, (batch,))
    if slots is not None:
        _check(slots, "slots", torch.int32, (total,))
    if status is not None:
        _check(status, "status", torch.int32, (1,))
    _check_one_device(stream, k=k, v=v, cu_seqlens=cu_seqlens, seq_lens=seq_lens,
                      block_table=block_table, k_pool=k_pool, v_pool=v_pool, new_lens=new_lens,
                      slots=slots, status=status)
    _rc(lib().mars_kv_append(_ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(seq_lens), _ptr(new_lens),
                             _ptr(block_table), block_table.shape[1], _ptr(k_pool), _ptr(v_pool),
                             num_pages, _ptr(slots), batch, total, hkv, d, PAGE_SIZE, ks, vs,
                             _ptr(status), _stream(stream)), "mars_kv_append")
