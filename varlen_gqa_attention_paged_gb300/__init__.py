"""Unified paged varlen GQA attention for GB300 (sm_103a).

Python binding of the C ABI in ``include/ua.h``: it only turns torch tensors into
device pointers, the current CUDA stream and host-side sizes, and calls
``ua_append_kv`` (new keys and values into the paged cache, rotated by position) and
``ua_unified_attention`` (attention over it) in ``libua.so``.  Every step of the computation
runs in the library's CUDA kernels; without the built library this module raises.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import (UA_BACKEND_2D, UA_BACKEND_AUTO, UA_BACKEND_SPLIT, UA_DT_BF16, UA_DT_F8E4M3,
                   UA_DT_F16, UA_DT_F32, UA_DT_I8, UA_PATH_2D, UA_PATH_SPLIT)

__all__ = ["unified_attention", "prepare", "PreparedAttention", "append_kv", "prepare_append",
           "PreparedAppend", "rope_table", "plan", "device_status", "device_status_reset",
           "UaError", "BACKENDS", "library_path"]

BACKENDS = {"auto": UA_BACKEND_AUTO, "2d": UA_BACKEND_2D, "split": UA_BACKEND_SPLIT}
_DTYPES = {torch.float16: UA_DT_F16, torch.bfloat16: UA_DT_BF16,
           torch.float8_e4m3fn: UA_DT_F8E4M3, torch.float32: UA_DT_F32,
           torch.int8: UA_DT_I8}


class UaError(RuntimeError):
    def __init__(self, code: int, what: str):
        lib = _lib.load()
        super().__init__(f"{what}: {lib.ua_status_string(code).decode()} (status {code})")
        self.code = code


def library_path() -> str:
    return _lib.LIB_PATH


def _dtype_code(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _new(shape, dtype, device, stream):
    """A result for a call on `stream` to write: the current stream's, as any new tensor, and (if
    `stream` is another) not handed out again before that is done with it."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None and stream.cuda_stream != torch.cuda.current_stream(device).cuda_stream:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
        t.record_stream(stream)
    return t


def _shape(q, k_cache, block_table, cu_seqlens_q, max_seqlen_q, max_seqlen_k, qq_bias,
           out_dtype_code, num_splits, workspace, events, k_scale_tok=None, v_scale_tok=None,
           k_scale_blk=None, v_scale_blk=None):
    sh = _lib.UaShape()
    sh.num_seqs = cu_seqlens_q.numel() - 1
    sh.total_q = q.shape[0]
    sh.max_seqlen_q = int(max_seqlen_q)
    sh.max_seqlen_k = int(max_seqlen_k)
    sh.max_blocks_per_seq = block_table.shape[-1]
    sh.num_blocks = k_cache.shape[0]
    sh.qq_bias_stride = qq_bias.shape[-1] if qq_bias is not None else 0
    sh.q_dtype = _dtype_code(q)
    sh.out_dtype = out_dtype_code
    sh.num_splits = int(num_splits)
    if workspace is not None:
        sh.workspace = workspace.data_ptr()
        sh.workspace_bytes = workspace.numel() * workspace.element_size()
    if events is not None:
        for e in events:
            if not e.cuda_event:  # torch creates the CUDA event lazily, on its first record
                e.record()
        arr = (ctypes.c_void_p * 3)(*[e.cuda_event for e in events])
        sh.events = ctypes.cast(arr, ctypes.c_void_p)
        sh._events_keepalive = arr  # noqa: SLF001 -- keep the array alive for the call
    if (k_scale_tok is None) != (v_scale_tok is None):
        raise ValueError("per-token scales: give both k_scale_tok and v_scale_tok, or neither")
    if k_scale_tok is not None:
        for t, ptr, strides in ((k_scale_tok, "k_scale_tok", "k_scale_stride"),
                                (v_scale_tok, "v_scale_tok", "v_scale_stride")):
            if t.dtype != torch.float32 or t.device != k_cache.device or t.dim() != 3:
                raise ValueError("per-token scales are float32 tensors [blocks, slots, H_kv] on "
                                 "the caches' device")
            if tuple(t.shape) != tuple(k_cache.shape[:3]):
                raise ValueError("per-token scales must be [num_blocks, block_size, H_kv]")
            setattr(sh, ptr, t.data_ptr())
            setattr(sh, strides, (ctypes.c_int64 * 3)(*t.stride()))
    if (k_scale_blk is None) != (v_scale_blk is None):
        raise ValueError("per-block scales: give both k_scale_blk and v_scale_blk, or neither")
    if k_scale_blk is not None:
        for t, ptr in ((k_scale_blk, "k_scale_blk"), (v_scale_blk, "v_scale_blk")):
            if t.dtype != torch.float32 or t.device != k_cache.device or \
                    tuple(t.shape) != (k_cache.shape[0], k_cache.shape[2]):
                raise ValueError("per-block scales must be float32 [num_blocks, H_kv] on the "
                                 "caches' device")
            setattr(sh, ptr, t.data_ptr())
            setattr(sh, ptr + "_stride", (ctypes.c_int64 * 2)(*t.stride()))
    return sh


def _check_attention(q, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, max_seqlen_q,
                     alibi_slopes, qq_bias, sinks, kv_scale, out, workspace):
    """What the library cannot see from the pointers of an attention call's tensors."""
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [total_q, H_q, D] and k_cache [blocks, block_size, H_kv, D]")
    dev, num_seqs = q.device, cu_seqlens_q.numel() - 1
    if k_cache.shape[3] != q.shape[2] or v_cache.shape != k_cache.shape:
        raise ValueError("q, k_cache and v_cache disagree on shape")
    if v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache disagree on dtype")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be contiguous and on q's device")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("seq_lens_k", seq_lens_k),
                    ("block_table", block_table)):
        if t.dtype != torch.int32 or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be a contiguous int32 tensor on q's device")
    if num_seqs < 0 or seq_lens_k.numel() < num_seqs or block_table.dim() < 1 or \
            block_table.numel() < num_seqs * block_table.shape[-1]:
        raise ValueError("seq_lens_k [S] and block_table [S, blocks] hold fewer sequences than "
                         "cu_seqlens_q [S + 1]")
    if qq_bias is not None and qq_bias.shape[0] < max_seqlen_q:
        raise ValueError("qq_bias needs at least max_seqlen_q rows")
    for name, t, n in (("alibi_slopes", alibi_slopes, q.shape[1]), ("sinks", sinks, q.shape[1]),
                       ("kv_scale", kv_scale, 2), ("qq_bias", qq_bias, 0)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or
                              t.device != dev or t.numel() < n):
            raise ValueError(f"{name} must be contiguous float32 on q's device"
                             + (f", {n} values" if n else ""))
    if out is not None and (out.numel() < q.numel() or not out.is_contiguous() or
                            out.device != dev):
        raise ValueError("out must be contiguous, on q's device and hold q's elements")
    if workspace is not None and (not workspace.is_contiguous() or workspace.device != dev):
        raise ValueError("workspace must be contiguous and on q's device")
    if not q.is_cuda:
        raise ValueError("q, k_cache and v_cache must be CUDA tensors")


def unified_attention(q, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, *,
                      max_seqlen_q: int, max_seqlen_k: int, scale: float | None = None,
                      softcap: float = 0.0, window_left: int = -1, alibi_slopes=None,
                      qq_bias=None, sinks=None, kv_scale=None, k_scale_tok=None,
                      v_scale_tok=None, k_scale_blk=None, v_scale_blk=None, out=None,
                      out_dtype=None, backend: str = "auto", num_splits: int = 0, workspace=None,
                      stream=None, events=None):
    """Paged varlen GQA attention on the GPU; returns ``out`` [total_q, H_q, D].

    q [total_q, H_q, D] f16/bf16; k_cache, v_cache [num_blocks, block_size, H_kv, D]
    f16/bf16/float8_e4m3fn/int8; cu_seqlens_q [S+1], seq_lens_k [S], block_table [S, max_blocks]
    int32; alibi_slopes / sinks [H_q] and qq_bias [rows, stride] float32; kv_scale float32[2]
    (k_scale, v_scale) for the fp8 cache, or k_scale_tok / v_scale_tok float32 [num_blocks,
    block_size, H_kv] (any strides) for per-token fp8 scales, or k_scale_blk / v_scale_blk
    float32 [num_blocks, H_kv] (any strides) for an fp8 or int8 cache with a scale for each
    block and kv-head (what :func:`append_kv` writes).  max_seqlen_q / max_seqlen_k are host
    ints.  All other tensors are contiguous (a q that :func:`append_kv` rotated in place inside
    a fused projection is not), on one device.
    """
    lib = _lib.load()
    _check_attention(q, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, max_seqlen_q,
                     alibi_slopes, qq_bias, sinks, kv_scale, out, workspace)
    total_q, hq, d = q.shape
    _, block_size, hkv, _ = k_cache.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _new((total_q, hq, d), out_dtype or q.dtype, q.device, stream)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sh = _shape(q, k_cache, block_table, cu_seqlens_q, max_seqlen_q, max_seqlen_k, qq_bias,
                _dtype_code(out), num_splits, workspace, events, k_scale_tok, v_scale_tok,
                k_scale_blk, v_scale_blk)
    rc = lib.ua_unified_attention(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(cu_seqlens_q), _ptr(seq_lens_k),
        _ptr(block_table), block_size, hq, hkv, d, float(scale), float(softcap or 0.0),
        int(window_left if window_left is not None else -1), _ptr(alibi_slopes), _ptr(qq_bias),
        _ptr(sinks), _dtype_code(k_cache), _ptr(kv_scale), BACKENDS[backend],
        ctypes.c_void_p(stream.cuda_stream), ctypes.byref(sh))
    if rc != 0:
        raise UaError(rc, "ua_unified_attention")
    return out


class PreparedAttention:
    """``unified_attention`` with its sizes and options marshalled once, for a loop that
    calls it again and again with the same shapes (a decode loop, a captured step).

    Built by :func:`prepare`.  Calling it passes new per-step tensors -- ``q``,
    ``cu_seqlens_q``, ``seq_lens_k``, ``block_table``, ``out`` -- each of the prepared one's
    shape, dtype and device (checked; if one is refused, none is taken); any left out, and
    ``stream``, keeps what was passed last.  The caches, the score features, the scales and the
    host sizes (``max_seqlen_q``/``max_seqlen_k``) stay as prepared.  Returns ``out``.
    """

    def __init__(self, lib, call, tensors, stream):
        self._lib = lib
        self._call = call
        self._ref = ctypes.byref(call)
        self._meta = {n: (t.shape, t.dtype, t.device) for n, t in tensors.items()}
        self._now = {n: (t, t.data_ptr(), t.shape) for n, t in tensors.items()}
        self._stream = stream
        self.out = tensors["out"]

    def _take(self, new):
        for name, t in new:
            if (t.shape, t.dtype, t.device) != self._meta[name] or not t.is_contiguous():
                raise ValueError(f"{name}: shape, dtype, device or layout differs from the "
                                 "prepared call")
        for name, t in new:
            setattr(self._call, name, t.data_ptr())
            self._now[name] = (t, t.data_ptr(), t.shape)

    def __call__(self, q=None, cu_seqlens_q=None, seq_lens_k=None, block_table=None, out=None,
                 stream=None):
        now = self._now
        new = None
        for name, t in (("q", q), ("cu_seqlens_q", cu_seqlens_q), ("seq_lens_k", seq_lens_k),
                        ("block_table", block_table), ("out", out)):
            if t is None:
                continue
            kept, ptr, shape = now[name]
            if t is not kept or t.data_ptr() != ptr or t.shape != shape or not t.is_contiguous():
                new = new or []
                new.append((name, t))
        if new:
            self._take(new)
        if stream is not None:
            self._stream = stream
        rc = self._lib.ua_unified_attention_call(self._ref, self._stream.cuda_stream)
        if rc != 0:
            raise UaError(rc, "ua_unified_attention")
        return now["out"][0]


def prepare(q, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, *, max_seqlen_q: int,
            max_seqlen_k: int, scale: float | None = None, softcap: float = 0.0,
            window_left: int = -1, alibi_slopes=None, qq_bias=None, sinks=None, kv_scale=None,
            k_scale_tok=None, v_scale_tok=None, k_scale_blk=None, v_scale_blk=None, out=None,
            out_dtype=None, backend: str = "auto", num_splits: int = 0, workspace=None,
            stream=None) -> PreparedAttention:
    """Validate and marshal a ``unified_attention`` call once (same arguments); the
    returned :class:`PreparedAttention` makes the call with new per-step tensors."""
    lib = _lib.load()
    _check_attention(q, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, max_seqlen_q,
                     alibi_slopes, qq_bias, sinks, kv_scale, out, workspace)
    total_q, hq, d = q.shape
    _, block_size, hkv, _ = k_cache.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _new((total_q, hq, d), out_dtype or q.dtype, q.device, stream)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sh = _shape(q, k_cache, block_table, cu_seqlens_q, max_seqlen_q, max_seqlen_k, qq_bias,
                _dtype_code(out), num_splits, workspace, None, k_scale_tok, v_scale_tok,
                k_scale_blk, v_scale_blk)
    call = _lib.UaAttention(
        *(0 if t is None else t.data_ptr()
          for t in (q, k_cache, v_cache, out, cu_seqlens_q, seq_lens_k, block_table, alibi_slopes,
                    qq_bias, sinks, kv_scale)),
        ctypes.pointer(sh), block_size, hq, hkv, d, float(scale), float(softcap or 0.0),
        int(window_left if window_left is not None else -1), _dtype_code(k_cache),
        BACKENDS[backend])
    tensors = {"q": q, "cu_seqlens_q": cu_seqlens_q, "seq_lens_k": seq_lens_k,
               "block_table": block_table, "out": out}
    prep = PreparedAttention(lib, call, tensors, stream)
    # the caches, score features and scales the prepared call points at stay alive with it
    prep._static = (k_cache, v_cache, alibi_slopes, qq_bias, sinks, kv_scale, k_scale_tok,
                    v_scale_tok, k_scale_blk, v_scale_blk, workspace)
    return prep


def rope_table(max_position: int, rot_dim: int, *, base: float = 10000.0, inv_freq=None,
               device="cuda") -> torch.Tensor:
    """The rotation table of :func:`append_kv`: float32 [max_position, rot_dim], row p the
    cosines of p * f for the rot_dim / 2 frequencies f, then the sines.  f is
    base^(-2 i / rot_dim), or ``inv_freq`` (rot_dim / 2 values, for scaled variants).  The
    angles are taken in 64 bits: fp32 products are off by whole radians at far positions."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be a positive even number")
    if inv_freq is None:
        i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
        inv_freq = base ** (-2.0 * i / rot_dim)
    else:
        inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64, device=device)
        if tuple(inv_freq.shape) != (rot_dim // 2,):
            raise ValueError("inv_freq must hold rot_dim / 2 frequencies")
    a = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * inv_freq
    return torch.cat([torch.cos(a), torch.sin(a)], dim=1).to(torch.float32)


def _rows3(name, t, total_q, d, dtype, device):
    if t.dim() != 3 or t.shape[0] != total_q or t.shape[2] != d:
        raise ValueError(f"{name} must be [total_q, heads, head_dim]")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must have k's dtype and device")
    if t.stride(2) != 1 or t.stride(0) % 8 or t.stride(1) % 8:
        raise ValueError(f"{name}: the head dim must be contiguous, the other strides "
                         "multiples of 8 elements")


def _append_call(k, v, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, max_seqlen_q,
                 q, q_out, cos_sin, positions, axis_of, interleaved, kv_scale, k_scale_tok,
                 v_scale_tok, k_scale_blk, v_scale_blk, stream):
    """Checks the tensors of an append_kv call; returns its UaAppend and what it points at."""
    if k.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("k must be [total_q, H_kv, D] and k_cache [blocks, block_size, H_kv, D]")
    total_q, hkv, d = k.shape
    num_blocks, block_size = k_cache.shape[:2]
    dev = k.device
    if not k.is_cuda:
        raise ValueError("k must be a CUDA tensor")
    if v_cache.shape != k_cache.shape or tuple(k_cache.shape[2:]) != (hkv, d):
        raise ValueError("k, k_cache and v_cache disagree on shape")
    if v.shape != k.shape:
        raise ValueError("k and v disagree on shape")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_contiguous() or t.dtype != k_cache.dtype or t.device != dev:
            raise ValueError(f"{name} must be contiguous, on k's device, of the caches' dtype")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("seq_lens_k", seq_lens_k),
                    ("block_table", block_table)):
        if t.dtype != torch.int32 or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be a contiguous int32 tensor on k's device")
    num_seqs = cu_seqlens_q.numel() - 1
    if num_seqs < 0 or seq_lens_k.numel() != num_seqs or block_table.dim() != 2 or \
            block_table.shape[0] != num_seqs:
        raise ValueError("cu_seqlens_q [S + 1], seq_lens_k [S] and block_table [S, blocks] "
                         "disagree on the number of sequences")
    _rows3("k", k, total_q, d, k.dtype, dev)
    _rows3("v", v, total_q, d, k.dtype, dev)
    a = _lib.UaAppend()
    if q is not None:
        _rows3("q", q, total_q, d, k.dtype, dev)
        if q_out is None:
            q_out = _new(tuple(q.shape), q.dtype, dev, stream)
        _rows3("q_out", q_out, total_q, d, k.dtype, dev)
        if q_out.shape != q.shape:
            raise ValueError("q and q_out disagree on shape")
        a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
        a.q_stride = (ctypes.c_int64 * 2)(*q.stride()[:2])
        a.q_out_stride = (ctypes.c_int64 * 2)(*q_out.stride()[:2])
        a.num_q_heads = q.shape[1]
    elif q_out is not None:
        raise ValueError("q_out without q")
    a.k, a.v = k.data_ptr(), v.data_ptr()
    a.k_stride = (ctypes.c_int64 * 2)(*k.stride()[:2])
    a.v_stride = (ctypes.c_int64 * 2)(*v.stride()[:2])
    a.k_cache, a.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    a.cu_seqlens_q, a.seq_lens_k = cu_seqlens_q.data_ptr(), seq_lens_k.data_ptr()
    a.block_table = block_table.data_ptr()
    axes = None
    a.n_axes = 1
    if cos_sin is not None:
        if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.device != dev or \
                not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous float32 [max_position, rot_dim] tensor "
                             "on k's device (see rope_table)")
        a.cos_sin = cos_sin.data_ptr()
        a.max_position, a.rot_dim = cos_sin.shape
        if a.rot_dim % 16 or not 0 < a.rot_dim <= d:
            raise ValueError("rot_dim must be a multiple of 16 within 16 .. head_dim")
    elif positions is not None or axis_of is not None:
        raise ValueError("positions and axis_of need cos_sin")
    if positions is not None:
        if positions.dtype != torch.int32 or positions.device != dev or \
                positions.dim() not in (1, 2) or positions.shape[-1] != total_q or \
                (positions.numel() and positions.stride(-1) != 1):
            raise ValueError("positions must be int32 [total_q] or [axes, total_q] on k's device")
        if positions.dim() == 2:
            a.n_axes = positions.shape[0]
            a.positions_stride = positions.stride(0)
        a.positions = positions.data_ptr()
    if axis_of is not None:
        axes = bytes(axis_of)
        if len(axes) != a.rot_dim // 2 or (axes and max(axes) >= a.n_axes):
            raise ValueError("axis_of names an axis of positions for each of the rot_dim / 2 "
                             "frequencies")
    elif a.n_axes > 1:
        raise ValueError("positions of several axes need axis_of")
    if axes is not None:
        axes = ctypes.create_string_buffer(axes, len(axes))
        a.axis_of = ctypes.addressof(axes)
    if kv_scale is not None:
        if kv_scale.dtype != torch.float32 or kv_scale.device != dev or kv_scale.numel() != 2 or \
                not kv_scale.is_contiguous():
            raise ValueError("kv_scale must be float32 [2] on k's device")
        a.kv_scale = kv_scale.data_ptr()
    for form, ks, vs, shape in (("tok", k_scale_tok, v_scale_tok, (num_blocks, block_size, hkv)),
                                ("blk", k_scale_blk, v_scale_blk, (num_blocks, hkv))):
        if (ks is None) != (vs is None):
            raise ValueError(f"give both k_scale_{form} and v_scale_{form}, or neither")
        if ks is None:
            continue
        for n, t in (("k", ks), ("v", vs)):
            if t.dtype != torch.float32 or t.device != dev or tuple(t.shape) != shape:
                raise ValueError(f"{n}_scale_{form} must be float32 {list(shape)} on k's device")
            setattr(a, f"{n}_scale_{form}", t.data_ptr())
            setattr(a, f"{n}_scale_{form}_stride",
                    (ctypes.c_int64 * len(shape))(*t.stride()))
    a.num_seqs, a.total_q, a.max_seqlen_q = num_seqs, total_q, int(max_seqlen_q)
    a.max_blocks_per_seq, a.num_blocks, a.block_size = block_table.shape[1], num_blocks, block_size
    a.num_kv_heads, a.head_dim = hkv, d
    a.dtype, a.kv_dtype = _dtype_code(k), _dtype_code(k_cache)
    a.interleaved = 1 if interleaved else 0
    keep = dict(k=k, v=v, q=q, q_out=q_out, cu_seqlens_q=cu_seqlens_q, seq_lens_k=seq_lens_k,
                block_table=block_table, positions=positions)
    static = (k_cache, v_cache, cos_sin, axes, kv_scale, k_scale_tok, v_scale_tok, k_scale_blk,
              v_scale_blk)
    return a, keep, static


class PreparedAppend:
    """``append_kv`` with its checks made and its sizes marshalled once, for a loop that calls
    it with the same shapes (a decode loop, a captured step).

    Built by :func:`prepare_append`.  Calling it passes the step's tensors -- ``k``, ``v``,
    ``q``, ``q_out``, ``cu_seqlens_q``, ``seq_lens_k``, ``block_table``, ``positions`` -- each
    of the prepared one's shape, strides, dtype and device (checked; if one is refused, none is
    taken); any left out, and ``stream``, keeps what was passed last.  The caches, the table and
    the scales stay as prepared.  Returns ``q_out``.
    """

    def __init__(self, lib, call, keep, static, stream):
        self._lib = lib
        self._call = call
        self._ref = ctypes.byref(call)
        self._static = static
        self._meta = {n: (t.shape, t.stride(), t.dtype, t.device)
                      for n, t in keep.items() if t is not None}
        # the tensors passed last: one passed again, as most are, costs four comparisons
        self._now = {n: (None, 0, None, None) if t is None else
                     (t, t.data_ptr(), t.shape, t.stride()) for n, t in keep.items()}
        self._device = keep["k"].device.index
        self._one_device = torch.cuda.device_count() == 1
        self._stream = stream

    def _take(self, new):
        for name, t in new:
            if (t.shape, t.stride(), t.dtype, t.device) != self._meta.get(name):
                raise ValueError(f"{name}: shape, strides, dtype or device differs from the "
                                 "prepared call")
        for name, t in new:
            setattr(self._call, name, t.data_ptr())
            self._now[name] = (t, t.data_ptr(), t.shape, t.stride())

    def __call__(self, k=None, v=None, q=None, q_out=None, cu_seqlens_q=None, seq_lens_k=None,
                 block_table=None, positions=None, stream=None):
        now = self._now
        new = None
        for name, t in (("k", k), ("v", v), ("q", q), ("q_out", q_out),
                        ("cu_seqlens_q", cu_seqlens_q), ("seq_lens_k", seq_lens_k),
                        ("block_table", block_table), ("positions", positions)):
            if t is None:
                continue
            kept, ptr, shape, stride = now[name]
            if t is not kept or t.data_ptr() != ptr or t.shape != shape or t.stride() != stride:
                new = new or []
                new.append((name, t))
        if new:
            self._take(new)
        if stream is not None:
            self._stream = stream
        handle = self._stream.cuda_stream
        if self._one_device or torch.cuda.current_device() == self._device:
            rc = self._lib.ua_append_kv(self._ref, handle)
        else:
            with torch.cuda.device(self._device):
                rc = self._lib.ua_append_kv(self._ref, handle)
        if rc != 0:
            raise UaError(rc, "ua_append_kv")
        return now["q_out"][0]


def prepare_append(k, v, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, *,
                   max_seqlen_q: int, q=None, q_out=None, cos_sin=None, positions=None,
                   axis_of=None, interleaved: bool = False, kv_scale=None, k_scale_tok=None,
                   v_scale_tok=None, k_scale_blk=None, v_scale_blk=None,
                   stream=None) -> PreparedAppend:
    """Check and marshal an ``append_kv`` call once (same arguments); the returned
    :class:`PreparedAppend` makes the call with new per-step tensors."""
    lib = _lib.load()
    call, keep, static = _append_call(
        k, v, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, max_seqlen_q, q, q_out,
        cos_sin, positions, axis_of, interleaved, kv_scale, k_scale_tok, v_scale_tok,
        k_scale_blk, v_scale_blk, stream)
    if stream is None:
        stream = torch.cuda.current_stream(k.device)
    return PreparedAppend(lib, call, keep, static, stream)


def append_kv(k, v, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, *,
              max_seqlen_q: int, q=None, q_out=None, cos_sin=None, positions=None, axis_of=None,
              interleaved: bool = False, kv_scale=None, k_scale_tok=None, v_scale_tok=None,
              k_scale_blk=None, v_scale_blk=None, stream=None):
    """Append new keys and values to the paged cache, rotating keys (and queries) by position.

    k, v [total_q, H_kv, D] f16/bf16 (any token and head strides that are multiples of 8, so
    slices of a fused projection go in as they are); token i of sequence b is written at cache
    position seq_lens_k[b] - q_len + i through the block table, with the caches, cu_seqlens_q,
    seq_lens_k (lengths with the new tokens) and block_table of :func:`unified_attention`.

    Rotation: ``cos_sin`` float32 [max_position, rot_dim] (:func:`rope_table`) turns the first
    rot_dim elements of every k and q head; pairs are (f, f + rot_dim / 2), or with
    ``interleaved`` (2f, 2f + 1).  A token's angle is taken at its cache position, or at
    ``positions`` int32 [total_q], or, with several axes (time, height, width), at positions
    [axes, total_q] with ``axis_of``: the axis of each of the rot_dim / 2 frequencies, e.g.
    [0] * 16 + [1] * 24 + [2] * 24.  ``q`` [total_q, H_q, D] is rotated into ``q_out`` (new
    unless given; may be q itself, else overlaps none of q, k and v), which is returned.

    Scales of an 8-bit cache, one form: ``kv_scale`` float32 [2] (e4m3, per tensor, read);
    k_scale_tok / v_scale_tok float32 [blocks, block_size, H_kv] (e4m3, per token, written);
    k_scale_blk / v_scale_blk float32 [blocks, H_kv] (e4m3 or int8, one for each block and
    head, updated: a block's scale grows with its tokens, and the codes it holds are rounded
    again when it does).  include/ua.h has the arithmetic and what is left unwritten.
    """
    lib = _lib.load()
    call, keep, _static = _append_call(
        k, v, k_cache, v_cache, cu_seqlens_q, seq_lens_k, block_table, max_seqlen_q, q, q_out,
        cos_sin, positions, axis_of, interleaved, kv_scale, k_scale_tok, v_scale_tok,
        k_scale_blk, v_scale_blk, stream)
    if stream is None:
        stream = torch.cuda.current_stream(k.device)
    with torch.cuda.device(k.device):
        rc = lib.ua_append_kv(ctypes.byref(call), ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise UaError(rc, "ua_append_kv")
    return keep["q_out"]


def plan(*, num_seqs, total_q, max_seqlen_q, max_seqlen_k, block_size, num_q_heads,
         num_kv_heads, head_dim, window_left=-1, kv_dtype=UA_DT_BF16, q_dtype=None,
         backend="auto", num_splits=0, num_sms=0, max_blocks_per_seq=1, num_blocks=1,
         per_token_scales=False, per_block_scales=False):
    """The dispatcher's decision for these sizes (host only; no GPU needed when num_sms > 0).
    per_token_scales: plan for an fp8 call with per-token K/V scales (the dispatcher only
    tests the scale pointers for null; this passes a placeholder that is never read);
    per_block_scales: for an fp8 call with per-block scales (an int8 one always has them)."""
    lib = _lib.load()
    sh = _lib.UaShape()
    if per_token_scales:
        sh.k_scale_tok = sh.v_scale_tok = 256
    if per_block_scales or kv_dtype == UA_DT_I8:
        sh.k_scale_blk = sh.v_scale_blk = 256
    sh.num_seqs, sh.total_q = num_seqs, total_q
    sh.max_seqlen_q, sh.max_seqlen_k = max_seqlen_q, max_seqlen_k
    sh.max_blocks_per_seq, sh.num_blocks = max_blocks_per_seq, num_blocks
    sh.q_dtype = q_dtype if q_dtype is not None else (
        UA_DT_BF16 if kv_dtype in (UA_DT_F8E4M3, UA_DT_I8) else kv_dtype)
    sh.out_dtype = sh.q_dtype
    sh.num_splits = num_splits
    pl = _lib.UaPlan()
    rc = lib.ua_plan(ctypes.byref(sh), block_size, num_q_heads, num_kv_heads, head_dim,
                     window_left, kv_dtype, BACKENDS[backend], num_sms, ctypes.byref(pl))
    if rc != 0:
        raise UaError(rc, "ua_plan")
    return {f: getattr(pl, f) for f, _ in pl._fields_}


def device_status(stream=None) -> int:
    """Synchronise the stream and return the kernels' device check status (ua_status_t)."""
    lib = _lib.load()
    stream = stream or torch.cuda.current_stream()
    st = ctypes.c_int(0)
    rc = lib.ua_device_status(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(st))
    if rc != 0:
        raise UaError(rc, "ua_device_status")
    return st.value


def device_status_reset(stream=None) -> None:
    lib = _lib.load()
    stream = stream or torch.cuda.current_stream()
    rc = lib.ua_device_status_reset(ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise UaError(rc, "ua_device_status_reset")
