"""ua_append_kv on the host: the binding's struct matches the header, and bad arguments are
refused before anything is launched."""
import ctypes
import os
import subprocess

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from varlen_gqa_attention_paged_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name,struct", [("ua_append_t", _lib.UaAppend),
                                         ("ua_attention_t", _lib.UaAttention)])
def test_struct_matches_the_header(name, struct, tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "ua.h"', "int main(void) {",
             f'printf("sizeof %zu 0\\n", sizeof({name}));']
    for f, _ in struct._fields_:
        lines.append(f'printf("{f} %zu %zu\\n", offsetof({name}, {f}), '
                     f"sizeof((({name}*)0)->{f}));")
    src, exe = tmp_path / "a.c", tmp_path / "a"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe),
                    str(src)], check=True)
    got = {}
    for ln in subprocess.run([str(exe)], check=True, capture_output=True,
                             text=True).stdout.splitlines():
        n, a, b = ln.split()
        got[n] = (int(a), int(b))
    assert got.pop("sizeof")[0] == ctypes.sizeof(struct)
    for f, _ in struct._fields_:
        desc = getattr(struct, f)
        assert got[f] == (desc.offset, desc.size), f


def test_the_struct_call_without_a_struct():
    assert _lib.load().ua_unified_attention_call(None, None) == _lib.UA_ERR_INVALID_ARG
    assert _lib.load().ua_unified_attention_call(_lib.UaAttention(), None) == \
        _lib.UA_ERR_INVALID_ARG


FAKE = 0x7f0000001000  # aligned, never dereferenced: every case fails validation first


def call(**over):
    a = _lib.UaAppend()
    for n in ("k", "v", "q", "q_out", "k_cache", "v_cache", "cu_seqlens_q", "seq_lens_k",
              "block_table", "cos_sin"):
        setattr(a, n, FAKE)
    for n in ("q_stride", "k_stride", "v_stride", "q_out_stride"):
        setattr(a, n, (ctypes.c_int64 * 2)(512, 64))
    a.num_seqs, a.total_q, a.max_seqlen_q, a.max_blocks_per_seq = 2, 6, 5, 3
    a.num_blocks, a.block_size, a.num_q_heads, a.num_kv_heads, a.head_dim = 8, 16, 4, 2, 64
    a.dtype, a.kv_dtype, a.rot_dim, a.max_position, a.n_axes = 1, 1, 64, 100, 1
    for k, v in over.items():
        setattr(a, k, v)
    return _lib.load().ua_append_kv(ctypes.byref(a), None)


INVALID, UNSUPPORTED = _lib.UA_ERR_INVALID_ARG, _lib.UA_ERR_UNSUPPORTED
AXES = (ctypes.c_uint8 * 32)(*([0] * 31 + [2]))


@pytest.mark.parametrize("over,code", [
    (dict(k=None), INVALID),
    (dict(v_cache=None), INVALID),
    (dict(seq_lens_k=None), INVALID),
    (dict(q_out=None), INVALID),
    (dict(q=None), INVALID),                                   # heads without q
    (dict(num_q_heads=0), INVALID),                            # q without heads
    (dict(k=FAKE + 8), INVALID),
    (dict(k_cache=FAKE + 4), INVALID),
    (dict(cos_sin=FAKE + 4), INVALID),
    (dict(cos_sin=None), INVALID),
    (dict(k_stride=(ctypes.c_int64 * 2)(512, 60)), INVALID),
    (dict(q_out_stride=(ctypes.c_int64 * 2)(-512, 64)), INVALID),
    (dict(q_out_stride=(ctypes.c_int64 * 2)(0, 64)), INVALID),  # overlapping outputs
    (dict(q_out_stride=(ctypes.c_int64 * 2)(248, 64)), INVALID),
    (dict(q_out_stride=(ctypes.c_int64 * 2)(64, 376)), INVALID),
    (dict(total_q=2 ** 31 - 1, block_size=1, kv_dtype=4, k_scale_blk=FAKE, v_scale_blk=FAKE,
          k_scale_blk_stride=(ctypes.c_int64 * 2)(2, 1),
          v_scale_blk_stride=(ctypes.c_int64 * 2)(2, 0)), INVALID),
    (dict(head_dim=96), INVALID),
    (dict(num_kv_heads=0), INVALID),
    (dict(block_size=0), INVALID),
    (dict(num_blocks=0), INVALID),
    (dict(total_q=-1), INVALID),
    (dict(rot_dim=24), INVALID),
    (dict(rot_dim=128), INVALID),
    (dict(max_position=0), INVALID),
    (dict(n_axes=0), INVALID),
    (dict(n_axes=5), INVALID),
    (dict(n_axes=2), INVALID),                                 # no positions
    (dict(n_axes=2, positions=FAKE), INVALID),                 # no axis_of
    (dict(n_axes=2, positions=FAKE, axis_of=ctypes.addressof(AXES)), INVALID),
    (dict(dtype=3), INVALID),
    (dict(kv_dtype=3), INVALID),
    (dict(kv_dtype=0), UNSUPPORTED),                           # bf16 k, f16 cache
    (dict(kv_scale=FAKE), INVALID),                            # 16-bit cache with a scale
    (dict(kv_dtype=2), INVALID),                               # e4m3 without scales
    (dict(kv_dtype=2, kv_scale=FAKE, k_scale_blk=FAKE, v_scale_blk=FAKE), INVALID),
    (dict(kv_dtype=2, k_scale_tok=FAKE), INVALID),
    (dict(kv_dtype=2, k_scale_tok=FAKE, v_scale_tok=FAKE,
          k_scale_tok_stride=(ctypes.c_int64 * 3)(32, 2, 1),
          v_scale_tok_stride=(ctypes.c_int64 * 3)(16, 2, 1)), INVALID),
    (dict(kv_dtype=2, k_scale_blk=FAKE), INVALID),
    (dict(kv_dtype=2, k_scale_blk=FAKE + 2, v_scale_blk=FAKE), INVALID),
    (dict(kv_dtype=4), INVALID),                               # int8 without scales
    (dict(kv_dtype=4, kv_scale=FAKE), INVALID),                # int8 goes by block scales only
    (dict(kv_dtype=4, k_scale_blk=FAKE, v_scale_blk=FAKE,
          k_scale_blk_stride=(ctypes.c_int64 * 2)(-1, 1)), INVALID),
])
def test_refused_before_any_launch(over, code):
    assert call(**over) == code


def test_an_empty_batch_is_a_no_op():
    assert call(total_q=0) == _lib.UA_OK
    assert call(num_seqs=0) == _lib.UA_OK
    assert _lib.load().ua_append_kv(None, None) == INVALID


def test_rope_table_holds_far_positions_exactly():
    t = ua.rope_table(200001, 32, device="cpu")
    f = torch.tensor([10000.0 ** (-2 * i / 32) for i in range(16)], dtype=torch.float64)
    a = 200000 * f
    # the angle itself is good to 2^-52 of 200000 radians in 64 bits, then one fp32 rounding
    assert (t[200000, :16].double() - torch.cos(a)).abs().max() <= 2.0 ** -25 + 1e-9
    assert (t[200000, 16:].double() - torch.sin(a)).abs().max() <= 2.0 ** -25 + 1e-9
    assert torch.equal(ua.rope_table(9, 32, inv_freq=f, device="cpu"),
                       ua.rope_table(9, 32, device="cpu"))
    with pytest.raises(ValueError):
        ua.rope_table(9, 31, device="cpu")
    with pytest.raises(ValueError):
        ua.rope_table(9, 32, inv_freq=f[:3], device="cpu")


def test_append_refuses_cpu_tensors():
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((2,), dtype=torch.int32)
    with pytest.raises(ValueError):
        ua.append_kv(k, k, c, c, i, i[:1], i.reshape(1, 2), max_seqlen_q=2)
