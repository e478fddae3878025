"""The latent entry points of the C ABI on the host: struct layouts, and arguments that are refused
before the GPU is touched."""
import ctypes
import os
import subprocess

import pytest

from varlen_gqa_attention_paged_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7f0000001000  # aligned, never dereferenced: every case fails validation first
INVALID, UNSUPPORTED = _lib.UA_ERR_INVALID_ARG, _lib.UA_ERR_UNSUPPORTED


def test_binding_structs_match_the_header_layout(tmp_path):
    structs = {"ua_append_latent_t": _lib.UaAppendLatent, "ua_tree_t": _lib.UaTree,
               "ua_latent_t": _lib.UaLatent, "ua_latent_prefill_t": _lib.UaLatentPrefill}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ua.h"', "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        for f, _ in py._fields_:
            lines.append(f'printf("{cname} {f} %zu %zu\\n", offsetof({cname}, {f}), '
                         f"sizeof((({cname}*)0)->{f}));")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe),
                    str(src)], check=True)
    got = {}
    for ln in subprocess.run([str(exe)], check=True, capture_output=True,
                             text=True).stdout.splitlines():
        parts = ln.split()
        got[(parts[0], parts[1])] = tuple(int(x) for x in parts[2:])
    for cname, py in structs.items():
        assert got[(cname, "sizeof")] == (ctypes.sizeof(py),), cname
        for f, _ in py._fields_:
            desc = getattr(py, f)
            assert got[(cname, f)] == (desc.offset, desc.size), (cname, f)


def make(struct, base, over):
    a = struct()
    for k, v in {**base, **over}.items():
        if isinstance(v, tuple):
            v = (ctypes.c_int64 * len(v))(*v)
        setattr(a, k, v)
    return a


def run(name, struct, base, over):
    return getattr(_lib.load(), name)(ctypes.byref(make(struct, base, over)), None)


APPEND = dict(latent=FAKE, k_rope=FAKE, q_rope=FAKE, q_rope_out=FAKE, cache=FAKE,
              cu_seqlens_q=FAKE, seq_lens_k=FAKE, block_table=FAKE, norm_weight=FAKE,
              cos_sin=FAKE, latent_stride=576, k_rope_stride=576, q_rope_stride=(1024, 64),
              q_rope_out_stride=(1024, 64), num_seqs=2, total_q=6, max_blocks_per_seq=3,
              num_blocks=8, block_size=16, num_heads=16, latent_dim=512, rope_dim=64, dtype=1,
              norm_dtype=1, max_position=100, norm_eps=1e-6)


@pytest.mark.parametrize("over", [
    dict(num_seqs=-1), dict(total_q=-1), dict(num_blocks=-1), dict(num_blocks=0),
    dict(max_blocks_per_seq=0), dict(block_size=0), dict(num_heads=-1), dict(latent_dim=64),
    dict(latent_dim=500), dict(rope_dim=0), dict(rope_dim=24), dict(rope_dim=80), dict(dtype=3),
    dict(dtype=2), dict(norm_dtype=0), dict(norm_dtype=4), dict(norm_eps=-1.0),
    dict(norm_eps=float("nan")), dict(norm_weight=FAKE + 2), dict(cos_sin=FAKE + 4),
    dict(max_position=0), dict(cos_sin=None, positions=FAKE), dict(positions=FAKE + 2),
    dict(latent=None), dict(k_rope=None), dict(cache=None), dict(cu_seqlens_q=None),
    dict(seq_lens_k=None), dict(block_table=None), dict(q_rope=None), dict(q_rope_out=None),
    dict(num_heads=0), dict(latent=FAKE + 2), dict(cache=FAKE + 8), dict(q_rope_out=FAKE + 4),
    dict(latent_stride=12), dict(k_rope_stride=-8), dict(q_rope_stride=(1024, 12)),
    # what is written may not overlap itself
    dict(q_rope_out_stride=(1024, 32)), dict(q_rope_out_stride=(0, 64)),
    dict(q_rope_out_stride=(64, 64)), dict(q_rope_out_stride=(512, 64)),
])
def test_append_refuses(over):
    assert run("ua_append_latent", _lib.UaAppendLatent, APPEND, over) == INVALID


LATENT = dict(q=FAKE, cache=FAKE, out=FAKE, cu_seqlens_q=FAKE, seq_lens_k=FAKE, block_table=FAKE,
              num_seqs=2, total_q=6, max_seqlen_q=5, max_seqlen_k=37, max_blocks_per_seq=3,
              num_blocks=8, block_size=16, num_heads=16, latent_dim=512, rope_dim=64, dtype=1,
              out_dtype=1, scale=0.1)


@pytest.mark.parametrize("over,code", [
    (dict(num_seqs=-1), INVALID), (dict(total_q=-2), INVALID), (dict(max_seqlen_q=-1), INVALID),
    (dict(max_seqlen_k=-1), INVALID), (dict(num_blocks=0), INVALID), (dict(block_size=0), INVALID),
    (dict(max_blocks_per_seq=0), INVALID), (dict(num_heads=0), INVALID),
    (dict(latent_dim=384), INVALID), (dict(rope_dim=8), INVALID), (dict(rope_dim=128), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=3), INVALID), (dict(out_dtype=4), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(cache=None), INVALID),
    (dict(out=None), INVALID), (dict(cu_seqlens_q=None), INVALID), (dict(seq_lens_k=None), INVALID),
    (dict(block_table=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(cache=FAKE + 8), INVALID),
    (dict(out=FAKE + 4), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(tree_mask=FAKE, tree_words=0), INVALID),
    (dict(tree_mask=FAKE, tree_words=1, max_seqlen_q=33), INVALID),
    (dict(tree_mask=FAKE, tree_words=1, tree_mask_stride=-1), INVALID),
    (dict(tree_mask=FAKE + 2, tree_words=1, tree_mask_stride=1), INVALID),
    # coordinates of 31 bits
    (dict(total_q=1 << 24, num_heads=128), UNSUPPORTED),
    (dict(num_blocks=1 << 26, block_size=64), UNSUPPORTED),
])
def test_attention_refuses(over, code):
    assert run("ua_latent_attention", _lib.UaLatent, LATENT, over) == code


PREFILL = dict(q=FAKE, k_nope=FAKE, k_rope=FAKE, v=FAKE, out=FAKE, cu_seqlens_q=FAKE,
               cu_seqlens_k=FAKE, q_stride=(3000, 192), k_nope_stride=(4096, 256),
               v_stride=(4096, 256), k_rope_stride=64, num_seqs=2, total_q=6, total_k=9,
               max_seqlen_q=5, max_seqlen_k=6, num_heads=16, nope_dim=128, rope_dim=64,
               value_dim=128, dtype=1, out_dtype=1, scale=0.1)


@pytest.mark.parametrize("over,code", [
    (dict(num_seqs=-1), INVALID), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID),
    (dict(num_heads=0), INVALID), (dict(nope_dim=96), INVALID), (dict(nope_dim=256), INVALID),
    (dict(value_dim=32), INVALID), (dict(rope_dim=0), INVALID), (dict(rope_dim=72), INVALID),
    (dict(dtype=2), INVALID), (dict(out_dtype=2), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(k_nope=None), INVALID),
    (dict(k_rope=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(cu_seqlens_q=None), INVALID), (dict(cu_seqlens_k=None), INVALID),
    (dict(q=FAKE + 2), INVALID), (dict(v=FAKE + 8), INVALID), (dict(lse=FAKE + 1), INVALID),
    (dict(q_stride=(3000, 100)), INVALID), (dict(q_stride=(0, 192)), INVALID),
    (dict(k_nope_stride=(4096, 0)), INVALID), (dict(v_stride=(-8, 256)), INVALID),
    (dict(k_rope_stride=0), INVALID), (dict(k_rope_stride=1 << 40), INVALID),
    (dict(total_q=1 << 30), UNSUPPORTED),
])
def test_prefill_refuses(over, code):
    assert run("ua_latent_prefill", _lib.UaLatentPrefill, PREFILL, over) == code


TREE = dict(parents=FAKE, cu_seqlens_q=FAKE, seq_lens_k=FAKE, mask=FAKE, positions=FAKE,
            mask_stride=1, num_seqs=2, total_q=6, max_seqlen_q=5, mask_words=1)


@pytest.mark.parametrize("over", [
    dict(num_seqs=-1), dict(total_q=-1), dict(max_seqlen_q=-1), dict(max_seqlen_q=4097),
    dict(max_seqlen_q=33), dict(mask_words=0), dict(mask_stride=0), dict(parents=None),
    dict(cu_seqlens_q=None), dict(seq_lens_k=None), dict(mask=None, positions=None),
    dict(parents=FAKE + 1), dict(mask=FAKE + 2), dict(positions=FAKE + 3),
])
def test_tree_refuses(over):
    assert run("ua_tree_mask", _lib.UaTree, TREE, over) == INVALID


def test_empty_batches_and_missing_calls():
    lib = _lib.load()
    for name, struct, base in (("ua_append_latent", _lib.UaAppendLatent, APPEND),
                               ("ua_latent_attention", _lib.UaLatent, LATENT),
                               ("ua_latent_prefill", _lib.UaLatentPrefill, PREFILL),
                               ("ua_tree_mask", _lib.UaTree, TREE)):
        assert run(name, struct, base, dict(total_q=0)) == _lib.UA_OK
        assert run(name, struct, base, dict(num_seqs=0)) == _lib.UA_OK
        assert getattr(lib, name)(None, None) == INVALID
    assert lib.ua_latent_workspace_bytes(None) == 0
