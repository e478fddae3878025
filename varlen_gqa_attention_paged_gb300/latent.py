"""Latent attention: append to a latent cache, attention over it (absorbed form, drafted trees
included) and over expanded keys and values.  The public names are the package's own."""
from __future__ import annotations

import ctypes
import math

import torch

from . import UaError, _dtype_code, _hold, _lib, _new


def _strides(t, n):
    return (ctypes.c_int64 * n)(*t.stride()[:n])


def _ints(name, t, dev):
    if t.dtype != torch.int32 or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous int32 tensor on the call's device")


def _half_cuda(name, t):
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"unsupported dtype {t.dtype}: {name} must be float16 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _batch(cu_seqlens_q, seq_lens_k, block_table, dev):
    """Checks the batch's index tensors; returns the number of sequences."""
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("seq_lens_k", seq_lens_k),
                    ("block_table", block_table)):
        _ints(name, t, dev)
    n = cu_seqlens_q.numel() - 1
    if n < 0 or seq_lens_k.numel() != n or block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError("cu_seqlens_q [S + 1], seq_lens_k [S] and block_table [S, blocks] "
                         "disagree on the number of sequences")
    return n


def _rows(name, t, shape, dtype, dev, strides=True):
    """A tensor of this shape whose last dim is contiguous, the others' strides multiples of 8."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype or t.device != dev:
        raise ValueError(f"{name} must have the call's dtype and device")
    if not strides:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.shape[-1] > 1 and t.stride(-1) != 1 or \
            any(n > 1 and (s % 8 or s < 0) for s, n in zip(t.stride()[:-1], t.shape[:-1])):
        raise ValueError(f"{name}: the last dim must be contiguous, the other strides multiples "
                         "of 8 elements")


def _out(out, shape, like, out_dtype, stream):
    if out is None:
        return _new(shape, out_dtype or like.dtype, like.device, stream)
    if tuple(out.shape) != tuple(shape) or not out.is_contiguous() or out.device != like.device:
        raise ValueError(f"out must be contiguous {list(shape)} on q's device")
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out and out_dtype disagree")
    return out


def _handle(stream, index):
    """The handle of a stream, or of the device's current one (whose object costs 3 us)."""
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


class _Prepared:
    """A call with its checks made and its sizes marshalled once; its steps pass new tensors of
    the prepared ones' shapes, strides, dtypes and device.  As long as no stream was passed, a step
    goes to the stream that is current when it is made."""

    def __init__(self, what, call, tensors, static, stream, made=()):
        self._what = what
        self._entry = getattr(_lib.load(), what)
        self._call = call
        self._ref = ctypes.byref(call)
        self._static = static
        self._names = tuple(tensors)
        self._meta = {n: (t.shape, t.stride(), t.dtype, t.device)
                      for n, t in tensors.items() if t is not None}
        # the tensors passed last, and where they were
        self._now = {n: (t, 0 if t is None else t.data_ptr()) for n, t in tensors.items()}
        dev = next(t.device for t in tensors.values() if t is not None)
        self._device = dev.index
        self._one_device = torch.cuda.device_count() == 1
        self._stream = stream   # passed last, if one was
        # the results that the preparation allocated, while they are the ones in use, and the last
        # stream that they are held for
        self._made = {n: tensors[n] for n in made if tensors[n] is not None}
        self._used = _handle(stream, self._device)

    def _step(self, passed, stream):
        now = self._now
        new = None
        for name, t in zip(self._names, passed):
            if t is None:
                continue
            kept, at = now[name]
            meta = self._meta.get(name)
            # (the layout of a tensor that is passed again may have changed in place)
            if meta is None or t.shape != meta[0] or t.stride() != meta[1] or \
                    (t is not kept and (t.dtype != meta[2] or t.device != meta[3])):
                raise ValueError(f"{name}: shape, strides, dtype or device differs from the "
                                 "prepared call")
            ptr = t.data_ptr()
            if t is not kept or ptr != at:
                new = new or []
                new.append((name, t, ptr, at))
        if stream is None:
            stream = self._stream
        handle = _handle(stream, self._device)
        if new:
            for name, _, ptr, at in new:
                if ptr != at:
                    setattr(self._call, name, ptr)
        if self._one_device or torch.cuda.current_device() == self._device:
            rc = self._entry(self._ref, handle)
        else:
            with torch.cuda.device(self._device):
                rc = self._entry(self._ref, handle)
        if rc != 0:     # (none is taken if one was refused, here or above)
            for name, _, _, at in new or ():
                setattr(self._call, name, at)
            raise UaError(rc, self._what)
        if new:
            for name, t, ptr, _ in new:
                now[name] = (t, ptr)
                self._made.pop(name, None)
        self._stream = stream
        if handle != self._used:
            self._used = handle
            for t in self._made.values():
                _hold(t, stream, handle)

    def _last(self, name):
        return self._now[name][0]


# ------------------------------------------------------------------ the append

class PreparedAppendLatent(_Prepared):
    """``append_latent`` for a loop with fixed shapes, built by :func:`prepare_append_latent`.
    Calling it passes the step's tensors (checked; if one is refused, none is taken); any left
    out, and ``stream``, keeps what was passed last (no stream yet: the current one).  The cache,
    the norm's weight and the table stay as prepared.  Returns ``q_rope_out``."""

    def __call__(self, latent=None, k_rope=None, q_rope=None, q_rope_out=None, cu_seqlens_q=None,
                 seq_lens_k=None, block_table=None, positions=None, stream=None):
        self._step((latent, k_rope, q_rope, q_rope_out, cu_seqlens_q, seq_lens_k, block_table,
                    positions), stream)
        return self._last("q_rope_out")


def _append_call(latent, k_rope, cache, cu_seqlens_q, seq_lens_k, block_table, norm_weight,
                 norm_eps, q_rope, q_rope_out, cos_sin, positions, interleaved, stream):
    if latent.dim() != 2 or k_rope.dim() != 2 or cache.dim() != 3:
        raise ValueError("latent must be [total_q, L], k_rope [total_q, R] and cache "
                         "[blocks, block_size, L + R]")
    _half_cuda("latent", latent)
    dev, dt = latent.device, latent.dtype
    total_q, width = latent.shape
    rope = k_rope.shape[1]
    _rows("latent", latent, (total_q, width), dt, dev)
    _rows("k_rope", k_rope, (total_q, rope), dt, dev)
    _rows("cache", cache, (cache.shape[0], cache.shape[1], width + rope), dt, dev, strides=False)
    num_seqs = _batch(cu_seqlens_q, seq_lens_k, block_table, dev)
    a = _lib.UaAppendLatent()
    a.latent, a.k_rope, a.cache = latent.data_ptr(), k_rope.data_ptr(), cache.data_ptr()
    a.latent_stride, a.k_rope_stride = latent.stride(0), k_rope.stride(0)
    if q_rope is not None:
        if q_rope.dim() != 3:
            raise ValueError("q_rope must be [total_q, H, R]")
        shape = (total_q, q_rope.shape[1], rope)
        _rows("q_rope", q_rope, shape, dt, dev)
        if q_rope_out is None:
            q_rope_out = _new(shape, dt, dev, stream)
        _rows("q_rope_out", q_rope_out, shape, dt, dev)
        if q_rope_out.data_ptr() == q_rope.data_ptr() and any(
                n > 1 and x != y for n, x, y in zip(shape, q_rope.stride(), q_rope_out.stride())):
            raise ValueError("q_rope_out in q_rope's place must have its strides")
        a.q_rope, a.q_rope_out = q_rope.data_ptr(), q_rope_out.data_ptr()
        a.q_rope_stride, a.q_rope_out_stride = _strides(q_rope, 2), _strides(q_rope_out, 2)
        a.num_heads = q_rope.shape[1]
    elif q_rope_out is not None:
        raise ValueError("q_rope_out without q_rope")
    if norm_weight is not None:
        if tuple(norm_weight.shape) != (width,) or not norm_weight.is_contiguous() or \
                norm_weight.dtype not in (dt, torch.float32) or norm_weight.device != dev:
            raise ValueError("norm_weight must be contiguous [L] of latent's dtype or float32, on "
                             "latent's device")
        a.norm_weight, a.norm_dtype = norm_weight.data_ptr(), _dtype_code(norm_weight)
        a.norm_eps = float(norm_eps)
    if cos_sin is not None:
        if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.shape[1] != rope or \
                cos_sin.device != dev or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous float32 [max_position, R] tensor on "
                             "latent's device (see rope_table)")
        a.cos_sin, a.max_position = cos_sin.data_ptr(), cos_sin.shape[0]
    if positions is not None:
        if cos_sin is None:
            raise ValueError("positions need cos_sin")
        _ints("positions", positions, dev)
        if tuple(positions.shape) != (total_q,):
            raise ValueError("positions must be int32 [total_q]")
        a.positions = positions.data_ptr()
    a.cu_seqlens_q, a.seq_lens_k = cu_seqlens_q.data_ptr(), seq_lens_k.data_ptr()
    a.block_table = block_table.data_ptr()
    a.num_seqs, a.total_q, a.max_blocks_per_seq = num_seqs, total_q, block_table.shape[1]
    a.num_blocks, a.block_size = cache.shape[:2]
    a.latent_dim, a.rope_dim, a.dtype = width, rope, _dtype_code(latent)
    a.interleaved = 1 if interleaved else 0
    tensors = dict(latent=latent, k_rope=k_rope, q_rope=q_rope, q_rope_out=q_rope_out,
                   cu_seqlens_q=cu_seqlens_q, seq_lens_k=seq_lens_k, block_table=block_table,
                   positions=positions)
    return a, tensors, (cache, norm_weight, cos_sin)


def append_latent(latent, k_rope, cache, cu_seqlens_q, seq_lens_k, block_table, *,
                  norm_weight=None, norm_eps: float = 1e-6, q_rope=None, q_rope_out=None,
                  cos_sin=None, positions=None, interleaved: bool = False, stream=None):
    """Append new tokens to a paged latent cache, normalised and rotated on the way.

    latent [total_q, L] (L 128, 256 or 512) and k_rope [total_q, R] (R a multiple of 16 up to 64)
    f16/bf16, any row strides that are multiples of 8 (the two parts of a down-projection go in
    as they are); cache [num_blocks, block_size, L + R]; token i of sequence b is written at
    cache position seq_lens_k[b] - q_len + i (lengths with the new tokens) through the block
    table.  ``norm_weight`` [L] (latent's dtype or float32) normalises the latents by their root
    mean square; without it they are stored as they are.  ``cos_sin`` float32 [max_position, R]
    (:func:`rope_table`) rotates k_rope, and ``q_rope`` [total_q, H, R] into ``q_rope_out`` (new
    unless given; may be q_rope itself or the rope part of the absorbed queries), at a token's
    cache position or at ``positions`` int32 [total_q].  Returns ``q_rope_out``.
    """
    return prepare_append_latent(
        latent, k_rope, cache, cu_seqlens_q, seq_lens_k, block_table, norm_weight=norm_weight,
        norm_eps=norm_eps, q_rope=q_rope, q_rope_out=q_rope_out, cos_sin=cos_sin,
        positions=positions, interleaved=interleaved, stream=stream)()


def prepare_append_latent(latent, k_rope, cache, cu_seqlens_q, seq_lens_k, block_table, *,
                          norm_weight=None, norm_eps: float = 1e-6, q_rope=None, q_rope_out=None,
                          cos_sin=None, positions=None, interleaved: bool = False,
                          stream=None) -> PreparedAppendLatent:
    """Check and marshal an :func:`append_latent` call once (same arguments); the returned
    :class:`PreparedAppendLatent` makes the call with new per-step tensors."""
    call, tensors, static = _append_call(
        latent, k_rope, cache, cu_seqlens_q, seq_lens_k, block_table, norm_weight, norm_eps,
        q_rope, q_rope_out, cos_sin, positions, interleaved, stream)
    made = ("q_rope_out",) if q_rope_out is None else ()
    return PreparedAppendLatent("ua_append_latent", call, tensors, static, stream, made)


# ------------------------------------------------------------------ absorbed attention

class PreparedLatentAttention(_Prepared):
    """``latent_attention`` for a loop with fixed shapes, built by
    :func:`prepare_latent_attention`.  Calling it passes the step's tensors (checked; if one is
    refused, none is taken); any left out, and ``stream``, keeps what was passed last (no stream
    yet: the current one).  The cache, the sizes and the workspace stay as prepared.  Returns
    ``out``, or ``(out, lse)``."""

    def __call__(self, q=None, cu_seqlens_q=None, seq_lens_k=None, block_table=None,
                 tree_mask=None, out=None, lse=None, stream=None):
        self._step((q, cu_seqlens_q, seq_lens_k, block_table, tree_mask, out, lse), stream)
        out, lse = self._last("out"), self._last("lse")
        return out if lse is None else (out, lse)


def _attention_call(q, cache, cu_seqlens_q, seq_lens_k, block_table, rope_dim, scale, max_seqlen_q,
                    max_seqlen_k, tree_mask, out, out_dtype, return_lse, workspace, stream):
    if q.dim() != 3 or cache.dim() != 3:
        raise ValueError("q must be [total_q, H, L + R] and cache [blocks, block_size, L + R]")
    _half_cuda("q", q)
    dev, dt = q.device, q.dtype
    total_q, heads, width = q.shape
    _rows("q", q, (total_q, heads, width), dt, dev, strides=False)
    _rows("cache", cache, (cache.shape[0], cache.shape[1], width), dt, dev, strides=False)
    num_seqs = _batch(cu_seqlens_q, seq_lens_k, block_table, dev)
    latent = width - int(rope_dim)
    a = _lib.UaLatent()
    if tree_mask is not None:
        if tree_mask.dtype != torch.int32 or tree_mask.dim() != 2 or tree_mask.device != dev or \
                tree_mask.shape[0] != total_q or \
                (tree_mask.shape[1] > 1 and tree_mask.stride(1) != 1):
            raise ValueError("tree_mask must be int32 [total_q, words] on q's device (see "
                             "tree_mask())")
        if 32 * tree_mask.shape[1] < int(max_seqlen_q):
            raise ValueError("tree_mask needs a bit for each of max_seqlen_q tokens")
        a.tree_mask, a.tree_words = tree_mask.data_ptr(), tree_mask.shape[1]
        a.tree_mask_stride = tree_mask.stride(0)
    out = _out(out, (total_q, heads, max(latent, 0)), q, out_dtype, stream)
    lse = _new((total_q, heads), torch.float32, dev, stream) if return_lse else None
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError("workspace must be contiguous and on q's device")
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.q, a.cache, a.out = q.data_ptr(), cache.data_ptr(), out.data_ptr()
    if lse is not None:
        a.lse = lse.data_ptr()
    a.cu_seqlens_q, a.seq_lens_k = cu_seqlens_q.data_ptr(), seq_lens_k.data_ptr()
    a.block_table = block_table.data_ptr()
    a.num_seqs, a.total_q = num_seqs, total_q
    a.max_seqlen_q, a.max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    a.max_blocks_per_seq = block_table.shape[1]
    a.num_blocks, a.block_size = cache.shape[:2]
    a.num_heads, a.latent_dim, a.rope_dim = heads, latent, int(rope_dim)
    a.dtype, a.out_dtype, a.scale = _dtype_code(q), _dtype_code(out), float(scale)
    tensors = dict(q=q, cu_seqlens_q=cu_seqlens_q, seq_lens_k=seq_lens_k, block_table=block_table,
                   tree_mask=tree_mask, out=out, lse=lse)
    return a, tensors, (cache, workspace)


def latent_attention(q, cache, cu_seqlens_q, seq_lens_k, block_table, *, scale: float,
                     max_seqlen_q: int, max_seqlen_k: int, rope_dim: int = 64, tree_mask=None,
                     out=None, out_dtype=None, return_lse: bool = False, workspace=None,
                     stream=None):
    """Attention over a paged latent cache with absorbed projections; returns ``out``
    [total_q, H, L], or ``(out, lse)``.

    q [total_q, H, L + R] f16/bf16: each head's query in the latent space (the key up-projection
    applied to it), then its rope part; cache [num_blocks, block_size, L + R] as
    :func:`append_latent` fills it: every head attends with [c | r] as keys and c as values.
    scale is the model's (1 / sqrt of its head's width before absorption).  Causal by default;
    with ``tree_mask`` int32 [total_q, words] (:func:`tree_mask`) a token sees the cached prefix
    and those of its sequence's new tokens whose bits are set.  lse float32 [total_q, H] is the
    log of each row's sum of exponentials (-inf where it saw no key; its out is 0).
    """
    return prepare_latent_attention(
        q, cache, cu_seqlens_q, seq_lens_k, block_table, scale=scale, max_seqlen_q=max_seqlen_q,
        max_seqlen_k=max_seqlen_k, rope_dim=rope_dim, tree_mask=tree_mask, out=out,
        out_dtype=out_dtype, return_lse=return_lse, workspace=workspace, stream=stream)()


def prepare_latent_attention(q, cache, cu_seqlens_q, seq_lens_k, block_table, *, scale: float,
                             max_seqlen_q: int, max_seqlen_k: int, rope_dim: int = 64,
                             tree_mask=None, out=None, out_dtype=None, return_lse: bool = False,
                             workspace=None, stream=None) -> PreparedLatentAttention:
    """Check and marshal a :func:`latent_attention` call once (same arguments); the returned
    :class:`PreparedLatentAttention` makes the call with new per-step tensors."""
    call, tensors, static = _attention_call(
        q, cache, cu_seqlens_q, seq_lens_k, block_table, rope_dim, scale, max_seqlen_q,
        max_seqlen_k, tree_mask, out, out_dtype, return_lse, workspace, stream)
    made = ("out", "lse") if out is None else ("lse",)
    return PreparedLatentAttention("ua_latent_attention", call, tensors, static, stream, made)


def latent_workspace_bytes(prepared: PreparedLatentAttention) -> int:
    """Bytes of scratch that a prepared call needs on its device: 0, or what ``workspace``
    has to hold where one is given."""
    with torch.cuda.device(prepared._device):  # noqa: SLF001
        return _lib.load().ua_latent_workspace_bytes(prepared._ref)  # noqa: SLF001


# ------------------------------------------------------------------ drafted trees

def tree_mask(parents, cu_seqlens_q, seq_lens_k, *, max_seqlen_q: int, mask=None, positions=None,
              stream=None):
    """Masks and positions of drafted trees; returns ``(mask, positions)``.

    parents int32 [total_q]: each new token's parent as an index among its sequence's new tokens,
    below its own; -1 for none.  mask int32 [total_q, ceil(max_seqlen_q / 32)] (new unless given):
    bit j of a token's row says that new token j is the token itself or one of its ancestors;
    positions int32 [total_q]: the cached length before the new tokens plus the token's depth,
    which :func:`append_latent` and :func:`append_kv` rotate by.  max_seqlen_q is at most 4096.
    """
    lib = _lib.load()
    if not parents.is_cuda:
        raise ValueError("parents must be a CUDA tensor")
    dev, i32 = parents.device, torch.int32
    given = (parents, cu_seqlens_q, seq_lens_k) if positions is None else \
        (parents, cu_seqlens_q, seq_lens_k, positions)
    for t in given:
        if t.dtype != i32 or t.dim() != 1 or t.device != dev or not t.is_contiguous():
            raise ValueError("parents, cu_seqlens_q, seq_lens_k and positions must be contiguous "
                             "int32 vectors on one device")
    total_q, num_seqs = parents.numel(), cu_seqlens_q.numel() - 1
    if num_seqs < 0 or seq_lens_k.numel() != num_seqs or \
            (positions is not None and positions.numel() != total_q):
        raise ValueError("parents [total_q], cu_seqlens_q [S + 1], seq_lens_k [S] and positions "
                         "[total_q] disagree")
    need = max(1, (int(max_seqlen_q) + 31) // 32)
    if mask is None:
        mask = _new((total_q, need), i32, dev, stream)
    rows, words = mask.shape if mask.dim() == 2 else (-1, 0)
    step, inner = mask.stride() if rows >= 0 else (0, 0)
    if mask.dtype != i32 or mask.device != dev or rows != total_q or words < need or \
            (words > 1 and inner != 1) or (rows > 1 and step < words):
        raise ValueError("mask must be int32 [total_q, words], 32 words >= max_seqlen_q, on "
                         "parents' device")
    if positions is None:
        positions = _new((total_q,), i32, dev, stream)
    handle = _handle(stream, dev.index)
    call = _lib.UaTree(parents.data_ptr(), cu_seqlens_q.data_ptr(), seq_lens_k.data_ptr(),
                       mask.data_ptr(), positions.data_ptr(), max(step, words), num_seqs, total_q,
                       int(max_seqlen_q), words)
    if torch.cuda.current_device() == dev.index:
        rc = lib.ua_tree_mask(ctypes.byref(call), handle)
    else:
        with torch.cuda.device(dev):
            rc = lib.ua_tree_mask(ctypes.byref(call), handle)
    if rc != 0:
        raise UaError(rc, "ua_tree_mask")
    return mask, positions


# ------------------------------------------------------------------ expanded attention

class PreparedLatentPrefill(_Prepared):
    """``latent_prefill`` for a loop with fixed shapes, built by :func:`prepare_latent_prefill`.
    Calling it passes the step's tensors (checked; if one is refused, none is taken); any left
    out, and ``stream``, keeps what was passed last (no stream yet: the current one).  Returns
    ``out``, or ``(out, lse)``."""

    def __call__(self, q=None, k_nope=None, k_rope=None, v=None, cu_seqlens_q=None,
                 cu_seqlens_k=None, out=None, lse=None, stream=None):
        self._step((q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, out, lse), stream)
        out, lse = self._last("out"), self._last("lse")
        return out if lse is None else (out, lse)


def _prefill_call(q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                  scale, out, out_dtype, return_lse, stream):
    if q.dim() != 3 or k_nope.dim() != 3 or k_rope.dim() != 2 or v.dim() != 3:
        raise ValueError("q must be [total_q, H, N + R], k_nope [total_k, H, N], k_rope "
                         "[total_k, R] and v [total_k, H, V]")
    _half_cuda("q", q)
    dev, dt = q.device, q.dtype
    total_q, heads, _ = q.shape
    total_k, rope = k_rope.shape
    nope, value = k_nope.shape[2], v.shape[2]
    _rows("q", q, (total_q, heads, nope + rope), dt, dev)
    _rows("k_nope", k_nope, (total_k, heads, nope), dt, dev)
    _rows("k_rope", k_rope, (total_k, rope), dt, dev)
    _rows("v", v, (total_k, heads, value), dt, dev)
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        _ints(name, t, dev)
    num_seqs = cu_seqlens_q.numel() - 1
    if num_seqs < 0 or cu_seqlens_k.numel() != num_seqs + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k [S + 1] disagree on the number of "
                         "sequences")
    if scale is None:
        scale = 1.0 / math.sqrt(nope + rope)
    out = _out(out, (total_q, heads, value), q, out_dtype, stream)
    lse = _new((total_q, heads), torch.float32, dev, stream) if return_lse else None
    a = _lib.UaLatentPrefill()
    a.q, a.k_nope, a.k_rope, a.v = (t.data_ptr() for t in (q, k_nope, k_rope, v))
    a.out = out.data_ptr()
    if lse is not None:
        a.lse = lse.data_ptr()
    a.cu_seqlens_q, a.cu_seqlens_k = cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr()
    a.q_stride, a.k_nope_stride, a.v_stride = _strides(q, 2), _strides(k_nope, 2), _strides(v, 2)
    a.k_rope_stride = k_rope.stride(0)
    a.num_seqs, a.total_q, a.total_k = num_seqs, total_q, total_k
    a.max_seqlen_q, a.max_seqlen_k, a.num_heads = int(max_seqlen_q), int(max_seqlen_k), heads
    a.nope_dim, a.rope_dim, a.value_dim = nope, rope, value
    a.dtype, a.out_dtype, a.scale = _dtype_code(q), _dtype_code(out), float(scale)
    tensors = dict(q=q, k_nope=k_nope, k_rope=k_rope, v=v, cu_seqlens_q=cu_seqlens_q,
                   cu_seqlens_k=cu_seqlens_k, out=out, lse=lse)
    return a, tensors, ()


def latent_prefill(q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int,
                   max_seqlen_k: int, scale: float | None = None, out=None, out_dtype=None,
                   return_lse: bool = False, stream=None):
    """Latent attention in its expanded form, for prompts; returns ``out`` [total_q, H, V], or
    ``(out, lse)``.

    q [total_q, H, N + R], k_nope [total_k, H, N] and v [total_k, H, V] (N and V 64 or 128) f16 or
    bf16, with any strides that are multiples of 8: k_nope and v may be the two parts of one
    up-projection.  k_rope [total_k, R] is every head's.  Causal, a sequence's last query at its
    last key (cu_seqlens_q, cu_seqlens_k int32 [S + 1]); scale defaults to 1 / sqrt(N + R).  lse
    float32 [total_q, H] is the log of each row's sum of exponentials (-inf where it saw no key;
    its out is 0).
    """
    return prepare_latent_prefill(
        q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
        max_seqlen_k=max_seqlen_k, scale=scale, out=out, out_dtype=out_dtype,
        return_lse=return_lse, stream=stream)()


def prepare_latent_prefill(q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, *,
                           max_seqlen_q: int, max_seqlen_k: int, scale: float | None = None,
                           out=None, out_dtype=None, return_lse: bool = False,
                           stream=None) -> PreparedLatentPrefill:
    """Check and marshal a :func:`latent_prefill` call once (same arguments); the returned
    :class:`PreparedLatentPrefill` makes the call with new per-step tensors."""
    call, tensors, static = _prefill_call(
        q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, out,
        out_dtype, return_lse, stream)
    made = ("out", "lse") if out is None else ("lse",)
    return PreparedLatentPrefill("ua_latent_prefill", call, tensors, static, stream, made)
