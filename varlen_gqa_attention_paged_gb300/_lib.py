"""ctypes declarations of the C ABI in include/ua.h (libua.so next to this file)."""
from __future__ import annotations

import ctypes
import os
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libua.so")

# ua_status_t
UA_OK, UA_ERR_INVALID_ARG, UA_ERR_UNSUPPORTED, UA_ERR_CUDA = 0, 1, 2, 3
UA_ERR_WORKSPACE, UA_ERR_DEVICE_CHECK, UA_ERR_TIMEOUT, UA_ERR_SCRATCH_LIMIT = 4, 5, 6, 7
UA_NOALLOC_SCRATCH_BYTES = 16 << 20
# ua_dtype_t
UA_DT_F16, UA_DT_BF16, UA_DT_F8E4M3, UA_DT_F32, UA_DT_I8 = 0, 1, 2, 3, 4
# ua_backend_t
UA_BACKEND_AUTO, UA_BACKEND_2D, UA_BACKEND_SPLIT = 0, 1, 2
# ua_path_t
UA_PATH_2D, UA_PATH_SPLIT = 1, 2

# every symbol include/ua.h declares
EXPORTS = ("ua_unified_attention", "ua_unified_attention_call", "ua_unified_attention_noalloc",
           "ua_append_kv", "ua_append_latent", "ua_latent_attention", "ua_latent_workspace_bytes",
           "ua_latent_prefill", "ua_tree_mask", "ua_plan", "ua_workspace_bytes", "ua_device_status",
           "ua_device_status_reset", "ua_shape_bytes", "ua_status_string", "ua_version")


class UaShape(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("max_seqlen_q", ctypes.c_int32),
        ("max_seqlen_k", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("qq_bias_stride", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("events", ctypes.c_void_p),
        ("k_scale_tok", ctypes.c_void_p),
        ("v_scale_tok", ctypes.c_void_p),
        ("k_scale_stride", ctypes.c_int64 * 3),
        ("v_scale_stride", ctypes.c_int64 * 3),
        ("k_scale_blk", ctypes.c_void_p),
        ("v_scale_blk", ctypes.c_void_p),
        ("k_scale_blk_stride", ctypes.c_int64 * 2),
        ("v_scale_blk_stride", ctypes.c_int64 * 2),
    ]


class UaAttention(ctypes.Structure):
    _fields_ = (
        [(n, ctypes.c_void_p) for n in (
            "q", "k_cache", "v_cache", "out", "cu_seqlens_q", "seq_lens_k", "block_table",
            "alibi_slopes", "qq_bias", "sinks", "kv_scale")] +
        [("shape", ctypes.POINTER(UaShape))] +
        [(n, ctypes.c_int32) for n in ("block_size", "num_q_heads", "num_kv_heads", "head_dim")] +
        [("scale", ctypes.c_float), ("softcap", ctypes.c_float)] +
        [(n, ctypes.c_int32) for n in ("window_left", "kv_dtype", "backend")])


class UaAppend(ctypes.Structure):
    _fields_ = (
        [(n, ctypes.c_void_p) for n in (
            "k", "v", "q", "q_out", "k_cache", "v_cache", "cu_seqlens_q", "seq_lens_k",
            "block_table", "cos_sin", "positions", "kv_scale", "k_scale_tok", "v_scale_tok",
            "k_scale_blk", "v_scale_blk")] +
        [(n, ctypes.c_int64 * 2) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride")] +
        [(n, ctypes.c_int64 * 3) for n in ("k_scale_tok_stride", "v_scale_tok_stride")] +
        [(n, ctypes.c_int64 * 2) for n in ("k_scale_blk_stride", "v_scale_blk_stride")] +
        [("positions_stride", ctypes.c_int64)] +
        [(n, ctypes.c_int32) for n in (
            "num_seqs", "total_q", "max_seqlen_q", "max_blocks_per_seq", "num_blocks",
            "block_size", "num_q_heads", "num_kv_heads", "head_dim", "dtype", "kv_dtype",
            "rot_dim", "max_position", "interleaved", "n_axes")] +
        [("axis_of", ctypes.c_void_p)])


class UaAppendLatent(ctypes.Structure):
    _fields_ = (
        [(n, ctypes.c_void_p) for n in (
            "latent", "k_rope", "q_rope", "q_rope_out", "cache", "cu_seqlens_q", "seq_lens_k",
            "block_table", "norm_weight", "cos_sin", "positions")] +
        [(n, ctypes.c_int64) for n in ("latent_stride", "k_rope_stride")] +
        [(n, ctypes.c_int64 * 2) for n in ("q_rope_stride", "q_rope_out_stride")] +
        [(n, ctypes.c_int32) for n in (
            "num_seqs", "total_q", "max_blocks_per_seq", "num_blocks", "block_size", "num_heads",
            "latent_dim", "rope_dim", "dtype", "norm_dtype", "max_position", "interleaved")] +
        [("norm_eps", ctypes.c_float)])


class UaTree(ctypes.Structure):
    _fields_ = (
        [(n, ctypes.c_void_p) for n in ("parents", "cu_seqlens_q", "seq_lens_k", "mask",
                                        "positions")] +
        [("mask_stride", ctypes.c_int64)] +
        [(n, ctypes.c_int32) for n in ("num_seqs", "total_q", "max_seqlen_q", "mask_words")])


class UaLatent(ctypes.Structure):
    _fields_ = (
        [(n, ctypes.c_void_p) for n in (
            "q", "cache", "out", "lse", "cu_seqlens_q", "seq_lens_k", "block_table", "tree_mask",
            "workspace")] +
        [("workspace_bytes", ctypes.c_size_t), ("tree_mask_stride", ctypes.c_int64)] +
        [(n, ctypes.c_int32) for n in (
            "num_seqs", "total_q", "max_seqlen_q", "max_seqlen_k", "max_blocks_per_seq",
            "num_blocks", "block_size", "num_heads", "latent_dim", "rope_dim", "dtype",
            "out_dtype", "tree_words")] +
        [("scale", ctypes.c_float)])


class UaLatentPrefill(ctypes.Structure):
    _fields_ = (
        [(n, ctypes.c_void_p) for n in (
            "q", "k_nope", "k_rope", "v", "out", "lse", "cu_seqlens_q", "cu_seqlens_k")] +
        [(n, ctypes.c_int64 * 2) for n in ("q_stride", "k_nope_stride", "v_stride")] +
        [("k_rope_stride", ctypes.c_int64)] +
        [(n, ctypes.c_int32) for n in (
            "num_seqs", "total_q", "total_k", "max_seqlen_q", "max_seqlen_k", "num_heads",
            "nope_dim", "rope_dim", "value_dim", "dtype", "out_dtype")] +
        [("scale", ctypes.c_float)])


class UaPlan(ctypes.Structure):
    _fields_ = [
        ("path", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("block_m", ctypes.c_int32),
        ("n_part", ctypes.c_int32),
        ("grid_x", ctypes.c_int32),
        ("grid_y", ctypes.c_int32),
        ("grid_z", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
        ("cluster_y", ctypes.c_int32),
        ("cluster_z", ctypes.c_int32),
        ("slot_per_seq", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_size_t),
    ]


_LOCK = threading.Lock()
_LIB = None


def load():
    """The loaded libua.so.  Raises if the CUDA library has not been built."""
    global _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build the CUDA library first "
                "(varlen_gqa_attention_paged_gb300.build.build()); there is no CPU fallback")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.ua_unified_attention.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32,
                                             f32, i32, vp, vp, vp, i32, vp, i32, vp,
                                             ctypes.POINTER(UaShape)]
        lib.ua_unified_attention.restype = ctypes.c_int
        lib.ua_unified_attention_noalloc.argtypes = lib.ua_unified_attention.argtypes
        lib.ua_unified_attention_noalloc.restype = ctypes.c_int
        lib.ua_unified_attention_call.argtypes = [ctypes.POINTER(UaAttention), vp]
        lib.ua_unified_attention_call.restype = ctypes.c_int
        lib.ua_append_kv.argtypes = [ctypes.POINTER(UaAppend), vp]
        lib.ua_append_kv.restype = ctypes.c_int
        lib.ua_plan.argtypes = [ctypes.POINTER(UaShape), i32, i32, i32, i32, i32, i32, i32, i32,
                                ctypes.POINTER(UaPlan)]
        lib.ua_plan.restype = ctypes.c_int
        lib.ua_workspace_bytes.argtypes = [ctypes.POINTER(UaShape), i32, i32, i32, i32, i32, i32,
                                           i32]
        lib.ua_workspace_bytes.restype = ctypes.c_size_t
        lib.ua_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
        lib.ua_device_status.restype = ctypes.c_int
        lib.ua_device_status_reset.argtypes = [vp]
        lib.ua_device_status_reset.restype = ctypes.c_int
        lib.ua_status_string.argtypes = [ctypes.c_int]
        lib.ua_status_string.restype = ctypes.c_char_p
        lib.ua_version.argtypes = []
        lib.ua_version.restype = ctypes.c_int
        _check_layout(lib)
        missing = [name for name in EXPORTS if not hasattr(lib, name)]
        if missing:
            raise RuntimeError(f"{LIB_PATH} lacks {missing[0]}: build it again "
                               "(varlen_gqa_attention_paged_gb300.build.build())")
        for name, struct in (("ua_append_latent", UaAppendLatent), ("ua_tree_mask", UaTree),
                             ("ua_latent_attention", UaLatent),
                             ("ua_latent_prefill", UaLatentPrefill)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [ctypes.POINTER(struct), vp], ctypes.c_int
        lib.ua_latent_workspace_bytes.argtypes = [ctypes.POINTER(UaLatent)]
        lib.ua_latent_workspace_bytes.restype = ctypes.c_size_t
        _LIB = lib
        return lib


def _check_layout(lib):
    """Raises if the library was built from another include/ua.h than these declarations."""
    try:
        size = lib.ua_shape_bytes
    except AttributeError:
        size = None
    if size is not None:
        size.argtypes, size.restype = [], ctypes.c_size_t
    if size is None or size() != ctypes.sizeof(UaShape):
        raise RuntimeError(f"{LIB_PATH} was built from another version of include/ua.h: build it "
                           "again (varlen_gqa_attention_paged_gb300.build.build())")
