"""ctypes binding of libmars' packed-sequence entry points (include/mars.h): attention of whole
prompts and its gradient, attention of new tokens over the paged cache, and the append of
their K/V; rotary positions; and the append to, and attention over, the 8-bit paged cache. Like
mars.py, argument marshalling only (but for rotary_frequencies, which makes a table); the rows of
q, k and v may be slices of a wider tensor (a fused projection's output).

A call for the current stream goes through csrc/packed_calls.c, which checks its arguments in C
and declines what is not right (or not of the plainest kind: an integer scale, a workspace of
2 GiB or more); the checks here then raise the error, or make the call.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .mars import MarsError, PAGE_SIZE, lib

OP_ATTN_PACKED, OP_ATTN_CHUNK, OP_ATTN_PACKED_GRAD, OP_ATTN_CHUNK_Q8 = 6, 7, 8, 9

_INT_MAX = 0x7fffffff
_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_E4M3 = torch.float8_e4m3fn

_calls = None


def _ready(first):
    """Load the C form of the calls, once there is a CUDA tensor to call it for."""
    global _calls
    if not (isinstance(first, torch.Tensor) and first.is_cuda):
        return False
    entry = lib()
    try:
        from . import _packed_calls
    except ImportError as e:
        raise RuntimeError("the C form of the packed calls is not built; run "
                           "`python -m block_masked_token_gb300.build`") from e
    _packed_calls.setup(torch.Tensor, _BF16, _I32, _F32, _U8, torch._C._cuda_getDevice,
                        torch._C._cuda_getCurrentRawStream,
                        *(ctypes.cast(f, ctypes.c_void_p).value for f in (
                            entry.mars_attn_packed, entry.mars_attn_packed_grad,
                            entry.mars_attn_chunk, entry.mars_kv_append)))
    _packed_calls.setup_q8(_E4M3, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
        entry.mars_rotary, entry.mars_kv_append_q8, entry.mars_attn_chunk_q8)))
    _calls = _packed_calls
    return True


# Pointers are passed as plain integers (0 for none).


def _refuse(t, name, dtype, shape, dev):
    """Raise for the first thing that is wrong with t (something is)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libmars has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call goes to cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _counts(name, shape):
    """The library counts in 31 bits, and ctypes would pass on the low ones of more."""
    if max(shape) > _INT_MAX:
        raise ValueError(f"{name} has a size that 31 bits do not count")


def _ptr(t, name, dtype, shape, dev):
    """Address of a contiguous tensor."""
    try:
        if (t.get_device() == dev and t.dtype is dtype and t.shape == shape and
                t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:                       # not a tensor
        pass
    _refuse(t, name, dtype, shape, dev)


def _opt(t, name, dtype, shape, dev):
    return 0 if t is None else _ptr(t, name, dtype, shape, dev)


def _rows(t, name, shape, dev):
    """Address and row pitch, in elements, of a bf16 [total, heads, d] tensor whose rows may be
    slices of a wider tensor (the heads of a row contiguous)."""
    try:
        good = t.get_device() == dev and t.dtype is _BF16 and t.shape == shape
    except AttributeError:
        good = False
    total, heads, d = shape
    _counts(name, shape)
    if not good:
        _refuse(t, name, _BF16, shape, dev)
    pitch, head, one = t.stride()
    if total == 0 or heads == 0 or d == 0:
        return t.data_ptr(), heads * d
    if (one != 1 and d > 1) or (head != d and heads > 1):
        raise ValueError(f"the heads of each row of {name} must be contiguous")
    if total == 1:
        return t.data_ptr(), heads * d
    if pitch < heads * d or pitch % 8 or pitch > _INT_MAX:
        raise ValueError(f"{name} has row pitch {pitch}: it must be a multiple of 8, at least "
                         f"{heads * d} and below 2^31")
    return t.data_ptr(), pitch


def _target(first, name, stream):
    """Device and raw handle of the stream that a call goes to; the device has to be current
    (the library launches there). first: a tensor argument, since a host tensor is refused
    before the CUDA runtime is asked for anything."""
    if not isinstance(first, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not first.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libmars has no CPU path)")
    dev = torch._C._cuda_getDevice()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device.index}, the current device is "
                         f"cuda:{dev}")
    return dev, stream.cuda_stream


def _batch(cu_seqlens, dev):
    """Address of the boundaries and the number of sequences."""
    if not isinstance(cu_seqlens, torch.Tensor):
        raise ValueError("cu_seqlens must hold batch + 1 boundaries")
    shape = cu_seqlens.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError("cu_seqlens must hold batch + 1 boundaries")
    _counts("cu_seqlens", shape)
    return _ptr(cu_seqlens, "cu_seqlens", _I32, shape, dev), shape[0] - 1


def _table(block_table, batch, dev):
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages]")
    width = block_table.shape[1]
    _counts("block_table", block_table.shape)
    return _ptr(block_table, "block_table", _I32, (batch, width), dev), width


def _workspace(ws, dev):
    if not isinstance(ws, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    size = ws.numel()
    return _ptr(ws, "workspace", _U8, (size,), dev), size


def _rc(code, where):
    if code:
        raise MarsError(code, where)


def mars_packed_workspace_bytes(op, batch, total, hq=1, hkv=1, d=64, max_len=0):
    sizes = (batch, total, hq, hkv, d, max_len)
    if not all(-1 <= n <= _INT_MAX for n in sizes):
        return 0
    return int(lib().mars_packed_workspace_bytes(op, *sizes))


def mars_attn_packed(q, k, v, cu_seqlens, o, workspace, lse=None, scale: float = 0.0,
                     status=None, stream=None):
    """o[total, hq, d] (bf16) = causal attention inside each sequence of a packed batch; lse
    [hq, total] (float32, optional) its log2 row statistics (see include/mars.h)."""
    if stream is None and (_calls is not None or _ready(q)):
        rc = _calls.attn_packed(q, k, v, cu_seqlens, o, workspace, lse, scale, status)
        if rc is not None:
            return _rc(rc, "mars_attn_packed")
    dev, raw = _target(q, "q", stream)
    total, hq, d = q.shape
    hkv = k.shape[1]
    cu, batch = _batch(cu_seqlens, dev)
    qp, qs = _rows(q, "q", (total, hq, d), dev)
    kp, ks = _rows(k, "k", (total, hkv, d), dev)
    vp, vs = _rows(v, "v", (total, hkv, d), dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _rc(lib().mars_attn_packed(
        qp, kp, vp, cu,
        _ptr(o, "o", _BF16, (total, hq, d), dev), _opt(lse, "lse", _F32, (hq, total), dev), batch,
        total, hq, hkv, d, qs, ks, vs, scale, ws, ws_bytes,
        _opt(status, "status", _I32, (1,), dev), raw), "mars_attn_packed")


def mars_attn_packed_grad(q, k, v, o, d_o, lse, cu_seqlens, dq, dk, dv, workspace,
                          scale: float = 0.0, status=None, stream=None):
    """dq, dk, dv (bf16) of mars_attn_packed for the upstream gradient d_o, from its o and lse
    (see include/mars.h); dq, dk, dv may be slices of a wider tensor, like q, k, v."""
    if stream is None and (_calls is not None or _ready(q)):
        rc = _calls.attn_packed_grad(q, k, v, o, d_o, lse, cu_seqlens, dq, dk, dv, workspace,
                                     scale, status)
        if rc is not None:
            return _rc(rc, "mars_attn_packed_grad")
    dev, raw = _target(q, "q", stream)
    total, hq, d = q.shape
    hkv = k.shape[1]
    cu, batch = _batch(cu_seqlens, dev)
    qp, qs = _rows(q, "q", (total, hq, d), dev)
    kp, ks = _rows(k, "k", (total, hkv, d), dev)
    vp, vs = _rows(v, "v", (total, hkv, d), dev)
    dqp, dqs = _rows(dq, "dq", (total, hq, d), dev)
    dkp, dks = _rows(dk, "dk", (total, hkv, d), dev)
    dvp, dvs = _rows(dv, "dv", (total, hkv, d), dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _rc(lib().mars_attn_packed_grad(
        qp, kp, vp, _ptr(o, "o", _BF16, (total, hq, d), dev),
        _ptr(d_o, "d_o", _BF16, (total, hq, d), dev), _ptr(lse, "lse", _F32, (hq, total), dev),
        cu, dqp, dkp, dvp, batch, total, hq,
        hkv, d, qs, ks, vs, dqs, dks, dvs, scale, ws, ws_bytes,
        _opt(status, "status", _I32, (1,), dev), raw), "mars_attn_packed_grad")


def mars_attn_chunk(q, k, v, cu_seqlens, k_pool, v_pool, block_table, seq_lens,
                    max_len_hint: int, o, workspace, status=None, scale: float = 0.0,
                    stream=None):
    """o[total, hq, d] (bf16) = attention of each sequence's new rows over its seq_lens[s]
    cached tokens and, causally, its own new keys (see include/mars.h)."""
    if stream is None and (_calls is not None or _ready(q)):
        rc = _calls.attn_chunk(q, k, v, cu_seqlens, k_pool, v_pool, block_table, seq_lens,
                               max_len_hint, o, workspace, status, scale, PAGE_SIZE)
        if rc is not None:
            return _rc(rc, "mars_attn_chunk")
    dev, raw = _target(q, "q", stream)
    if max_len_hint > _INT_MAX:
        raise ValueError("max_len_hint is beyond 31 bits")
    total, hq, d = q.shape
    hkv = k.shape[1]
    cu, batch = _batch(cu_seqlens, dev)
    pages = k_pool.shape[0]
    pool = (pages, hkv, PAGE_SIZE, d)
    qp, qs = _rows(q, "q", (total, hq, d), dev)
    kp, ks = _rows(k, "k", (total, hkv, d), dev)
    vp, vs = _rows(v, "v", (total, hkv, d), dev)
    table, width = _table(block_table, batch, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _rc(lib().mars_attn_chunk(
        qp, kp, vp, cu,
        _ptr(k_pool, "k_pool", _BF16, pool, dev), _ptr(v_pool, "v_pool", _BF16, pool, dev), pages,
        table, width, _ptr(seq_lens, "seq_lens", _I32, (batch,), dev), max_len_hint,
        _ptr(o, "o", _BF16, (total, hq, d), dev), batch, total, hq, hkv, d, PAGE_SIZE, qs, ks, vs,
        scale, ws, ws_bytes, _opt(status, "status", _I32, (1,), dev), raw), "mars_attn_chunk")


def mars_kv_append(k, v, cu_seqlens, seq_lens, block_table, k_pool, v_pool, new_lens=None,
                   slots=None, status=None, stream=None):
    """Copy each sequence's new K/V rows to its pages, after its seq_lens[s] cached tokens;
    new_lens [batch] and slots [total] (int32) are optional outputs (see include/mars.h)."""
    if stream is None and (_calls is not None or _ready(k)):
        rc = _calls.kv_append(k, v, cu_seqlens, k_pool, v_pool, block_table, seq_lens, new_lens,
                              slots, status, PAGE_SIZE)
        if rc is not None:
            return _rc(rc, "mars_kv_append")
    dev, raw = _target(k, "k", stream)
    total, hkv, d = k.shape
    cu, batch = _batch(cu_seqlens, dev)
    pages = k_pool.shape[0]
    pool = (pages, hkv, PAGE_SIZE, d)
    kp, ks = _rows(k, "k", (total, hkv, d), dev)
    vp, vs = _rows(v, "v", (total, hkv, d), dev)
    table, width = _table(block_table, batch, dev)
    _rc(lib().mars_kv_append(
        kp, vp, cu,
        _ptr(seq_lens, "seq_lens", _I32, (batch,), dev),
        _opt(new_lens, "new_lens", _I32, (batch,), dev), table, width,
        _ptr(k_pool, "k_pool", _BF16, pool, dev), _ptr(v_pool, "v_pool", _BF16, pool, dev), pages,
        _opt(slots, "slots", _I32, (total,), dev), batch, total, hkv, d, PAGE_SIZE, ks, vs,
        _opt(status, "status", _I32, (1,), dev), raw), "mars_kv_append")


def rotary_frequencies(rot, base: float = 10000.0, scaling=None, stretch: float = 1.0,
                       trained: int = 0, low: float = 1.0, high: float = 32.0):
    """(inv_freq [rot / 2] float32 on the host, factor) for mars_rotary: pair j turns by
    base^(-2j / rot) radians per position, for contexts of up to `stretch` times those trained on
    changed by `scaling`:
      None       not at all
      "linear"   every frequency divided by stretch (positions squeezed into the trained range)
      "base"     base times stretch^(rot / (rot - 2)): the slowest pair is divided by stretch, the
                 fastest not at all
      "parts"    a pair that turns fewer than `low` times over the `trained` positions is divided
                 by stretch, one that turns more than `high` times is not, and between the two the
                 share falls linearly in the number of turns; factor = 1 + 0.1 ln(stretch) keeps the
                 softmax as sharp.
    A model that was trained with another scaling, one whose share falls linearly in j among them, needs
    its own table: mars_rotary takes any."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot is {rot}: it must be even and at least 2")
    if not base > 0 or not stretch >= 1:
        raise ValueError("base must be positive and stretch at least 1")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base" and rot == 2:
        raise ValueError("one pair has no base to scale")
    if scaling == "base":
        base = base * stretch ** (rot / (rot - 2))
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    factor = 1.0
    if scaling == "linear":
        freq = freq / stretch
    elif scaling == "parts":
        if trained < 1 or not 0 < low < high:
            raise ValueError("parts needs the number of trained positions, and 0 < low < high")
        turns = trained * freq / (2 * math.pi)
        kept = ((turns - low) / (high - low)).clamp(0, 1)
        freq = freq * kept + freq / stretch * (1 - kept)
        factor = 1.0 + 0.1 * math.log(stretch)
    return freq.float(), factor


def mars_rotary(q, k, cu_seqlens, inv_freq, q_out, k_out, seq_lens=None, interleaved: bool = False,
                factor: float = 1.0, inverse: bool = False, status=None, stream=None):
    """q_out, k_out = q and k with their pairs turned by their positions, seq_lens[s] + row;
    inverse gives the gradient. q_out may be q and k_out k (see include/mars.h)."""
    if stream is None and (_calls is not None or _ready(q)):
        rc = _calls.rotary(q, k, cu_seqlens, inv_freq, q_out, k_out, seq_lens, interleaved, factor,
                           inverse, status)
        if rc is not None:
            return _rc(rc, "mars_rotary")
    dev, raw = _target(q, "q", stream)
    total, hq, d = q.shape
    hkv = k.shape[1]
    cu, batch = _batch(cu_seqlens, dev)
    qp, qs = _rows(q, "q", (total, hq, d), dev)
    kp, ks = _rows(k, "k", (total, hkv, d), dev)
    qop, qos = _rows(q_out, "q_out", (total, hq, d), dev)
    kop, kos = _rows(k_out, "k_out", (total, hkv, d), dev)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1 or inv_freq.shape[0] > d // 2:
        raise ValueError("inv_freq must hold a frequency for each pair, d / 2 at most")
    half = inv_freq.shape[0]
    _rc(lib().mars_rotary(
        qp, kp, cu, _opt(seq_lens, "seq_lens", _I32, (batch,), dev),
        _ptr(inv_freq, "inv_freq", _F32, (half,), dev), qop, kop, batch, total, hq, hkv, d,
        2 * half, bool(interleaved), bool(inverse), factor, qs, ks, qos, kos,
        _opt(status, "status", _I32, (1,), dev), raw), "mars_rotary")


def _cache_q8(k_pool, v_pool, k_scale, v_scale, hkv, d, dev):
    """Addresses of an 8-bit cache's four tensors, and its pages."""
    for t, name, dim in ((k_pool, "k_pool", 4), (v_pool, "v_pool", 4)):
        if not isinstance(t, torch.Tensor) or t.dim() != dim:
            raise ValueError(f"{name} must be [pages, hkv, {PAGE_SIZE}, d]")
    pages = k_pool.shape[0]
    _counts("k_pool", k_pool.shape)
    pool = (pages, hkv, PAGE_SIZE, d)
    return (_ptr(k_pool, "k_pool", _E4M3, pool, dev), _ptr(v_pool, "v_pool", _E4M3, pool, dev),
            _ptr(k_scale, "k_scale", _U8, (pages, hkv), dev),
            _ptr(v_scale, "v_scale", _U8, (pages, hkv), dev)), pages


def mars_kv_append_q8(k, v, cu_seqlens, seq_lens, block_table, k_pool, v_pool, k_scale, v_scale,
                      counts=None, new_lens=None, slots=None, status=None, stream=None):
    """mars_kv_append into the 8-bit cache: float8_e4m3fn pools and uint8 scales [pages, hkv];
    counts [batch] (int32, optional): how many of a sequence's rows (see include/mars.h)."""
    if stream is None and (_calls is not None or _ready(k)):
        rc = _calls.kv_append_q8(k, v, cu_seqlens, k_pool, v_pool, k_scale, v_scale, block_table,
                                 seq_lens, counts, new_lens, slots, status, PAGE_SIZE)
        if rc is not None:
            return _rc(rc, "mars_kv_append_q8")
    dev, raw = _target(k, "k", stream)
    total, hkv, d = k.shape
    cu, batch = _batch(cu_seqlens, dev)
    kp, ks = _rows(k, "k", (total, hkv, d), dev)
    vp, vs = _rows(v, "v", (total, hkv, d), dev)
    table, width = _table(block_table, batch, dev)
    cache, pages = _cache_q8(k_pool, v_pool, k_scale, v_scale, hkv, d, dev)
    _rc(lib().mars_kv_append_q8(
        kp, vp, cu, _ptr(seq_lens, "seq_lens", _I32, (batch,), dev),
        _opt(counts, "counts", _I32, (batch,), dev),
        _opt(new_lens, "new_lens", _I32, (batch,), dev), table, width, *cache, pages,
        _opt(slots, "slots", _I32, (total,), dev), batch, total, hkv, d, PAGE_SIZE, ks, vs,
        _opt(status, "status", _I32, (1,), dev), raw), "mars_kv_append_q8")


def mars_attn_chunk_q8(q, k, v, cu_seqlens, k_pool, v_pool, k_scale, v_scale, block_table,
                       seq_lens, max_len_hint: int, o, workspace, status=None, scale: float = 0.0,
                       stream=None):
    """mars_attn_chunk over the 8-bit cache (see include/mars.h); its workspace is that of
    OP_ATTN_CHUNK_Q8."""
    if stream is None and (_calls is not None or _ready(q)):
        rc = _calls.attn_chunk_q8(q, k, v, cu_seqlens, k_pool, v_pool, k_scale, v_scale,
                                  block_table, seq_lens, max_len_hint, o, workspace, status, scale,
                                  PAGE_SIZE)
        if rc is not None:
            return _rc(rc, "mars_attn_chunk_q8")
    dev, raw = _target(q, "q", stream)
    if max_len_hint > _INT_MAX:
        raise ValueError("max_len_hint is beyond 31 bits")
    total, hq, d = q.shape
    hkv = k.shape[1]
    cu, batch = _batch(cu_seqlens, dev)
    qp, qs = _rows(q, "q", (total, hq, d), dev)
    kp, ks = _rows(k, "k", (total, hkv, d), dev)
    vp, vs = _rows(v, "v", (total, hkv, d), dev)
    table, width = _table(block_table, batch, dev)
    cache, pages = _cache_q8(k_pool, v_pool, k_scale, v_scale, hkv, d, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _rc(lib().mars_attn_chunk_q8(
        qp, kp, vp, cu, *cache, pages, table, width,
        _ptr(seq_lens, "seq_lens", _I32, (batch,), dev), max_len_hint,
        _ptr(o, "o", _BF16, (total, hq, d), dev), batch, total, hq, hkv, d, PAGE_SIZE, qs, ks, vs,
        scale, ws, ws_bytes, _opt(status, "status", _I32, (1,), dev), raw), "mars_attn_chunk_q8")
