"""What unified_attention and prepare refuse of the tensors they are given, before any launch: a
wrong layout, device, type or size, which the library could not tell from a pointer.  (CPU tensors:
a call that passes every other check is refused last, for its device.)"""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua

BF, I32 = torch.bfloat16, torch.int32


def tensors():
    return dict(q=torch.zeros((6, 4, 64), dtype=BF),
                k_cache=torch.zeros((5, 16, 2, 64), dtype=BF),
                v_cache=torch.zeros((5, 16, 2, 64), dtype=BF),
                cu_seqlens_q=torch.zeros(3, dtype=I32), seq_lens_k=torch.zeros(2, dtype=I32),
                block_table=torch.zeros((2, 3), dtype=I32))


FUSED = torch.zeros((6, 8, 64), dtype=BF)
META = dict(device="meta")
BAD = [
    ("q must", dict(q=torch.zeros((6, 256), dtype=BF))),
    ("shape", dict(q=torch.zeros((6, 4, 128), dtype=BF))),
    ("shape", dict(v_cache=torch.zeros((4, 16, 2, 64), dtype=BF))),
    ("dtype", dict(v_cache=torch.zeros((5, 16, 2, 64), dtype=torch.int8))),
    ("q must", dict(q=FUSED[:, :4])),                        # a slice of a fused projection
    ("k_cache", dict(k_cache=torch.zeros((5, 2, 16, 64), dtype=BF).transpose(1, 2))),
    ("v_cache", dict(v_cache=torch.zeros((5, 16, 2, 64), dtype=BF, **META))),
    ("cu_seqlens_q", dict(cu_seqlens_q=torch.zeros(3, dtype=torch.int64))),
    ("seq_lens_k", dict(seq_lens_k=torch.zeros(2, dtype=I32, **META))),
    ("block_table", dict(block_table=torch.zeros((3, 2), dtype=I32).T)),
    ("block_table", dict(block_table=torch.zeros((2, 3), dtype=I32, **META))),
    ("sequences", dict(seq_lens_k=torch.zeros(1, dtype=I32))),
    ("sequences", dict(block_table=torch.zeros((1, 3), dtype=I32))),
    ("sequences", dict(block_table=torch.zeros((0, 3), dtype=I32))),
    ("qq_bias", dict(qq_bias=torch.zeros((2, 8)))),
    ("qq_bias", dict(qq_bias=torch.zeros((8, 8)).T[:, :7])),
    ("alibi_slopes", dict(alibi_slopes=torch.zeros(3))),
    ("alibi_slopes", dict(alibi_slopes=torch.zeros(4, **META))),
    ("sinks", dict(sinks=torch.zeros(4, dtype=BF))),
    ("kv_scale", dict(kv_scale=torch.zeros(2, **META))),
    ("kv_scale", dict(kv_scale=torch.zeros(1))),
    ("out", dict(out=torch.zeros((6, 4, 64), dtype=BF, **META))),
    ("out", dict(out=FUSED[:, :4])),
    ("out", dict(out=torch.zeros((5, 4, 64), dtype=BF))),
    ("workspace", dict(workspace=torch.zeros(1024, dtype=torch.uint8, **META))),
]


@pytest.mark.parametrize("call", [ua.unified_attention, ua.prepare], ids=["call", "prepare"])
@pytest.mark.parametrize("match,over", BAD, ids=[f"{i}-{m}" for i, (m, _) in enumerate(BAD)])
def test_refused(call, match, over):
    with pytest.raises(ValueError, match=match):
        call(**{**tensors(), **over}, max_seqlen_q=3, max_seqlen_k=40)


@pytest.mark.parametrize("call", [ua.unified_attention, ua.prepare], ids=["call", "prepare"])
def test_a_right_call_is_refused_for_its_device_only(call):
    more = dict(alibi_slopes=torch.zeros(4), sinks=torch.zeros(4), qq_bias=torch.zeros((3, 7)),
                kv_scale=torch.zeros(2), out=torch.zeros((6, 4, 64)),
                workspace=torch.zeros(64, dtype=torch.uint8))
    # and buffers that hold more than the call needs, or in another shape
    room = dict(alibi_slopes=torch.zeros(9), seq_lens_k=torch.zeros(4, dtype=I32),
                block_table=torch.zeros((4, 3), dtype=I32), out=torch.zeros((6, 256)))
    for over in ({}, room):
        with pytest.raises(ValueError, match="CUDA"):
            call(**{**tensors(), **more, **over}, max_seqlen_q=3, max_seqlen_k=40)
