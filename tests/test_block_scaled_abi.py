"""Block-scaled caches on the host: what the attention call refuses before any launch, and
that the dispatcher plans them."""
import ctypes

import pytest

import varlen_gqa_attention_paged_gb300 as ua
from tests.test_abi import FAKE, _plan, call
from varlen_gqa_attention_paged_gb300 import _lib

I8, F8 = _lib.UA_DT_I8, _lib.UA_DT_F8E4M3
BLK = dict(k_scale_blk=FAKE, v_scale_blk=FAKE)


@pytest.mark.parametrize("over", [
    dict(kv_dtype=I8),                                          # int8 without scales
    dict(kv_dtype=I8, k_scale_blk=FAKE),
    dict(kv_dtype=F8, v_scale_blk=FAKE),
    dict(kv_dtype=F8, **BLK, k_scale_tok=FAKE, v_scale_tok=FAKE),
    dict(kv_dtype=I8, **{**BLK, "v_scale_blk": FAKE + 2}),
    dict(kv_dtype=I8, **BLK, k_scale_blk_stride=(ctypes.c_int64 * 2)(-2, 1)),
    dict(kv_dtype=I8, **BLK, v_scale_blk_stride=(ctypes.c_int64 * 2)(2, -1)),
    dict(kv_dtype=I8, **BLK, d=96),
    dict(kv_dtype=I8, **BLK, num_blocks=0),
    dict(kv_dtype=5, **BLK),
])
def test_refused_before_any_launch(over):
    assert call(**over) == _lib.UA_ERR_INVALID_ARG


def test_an_empty_batch_is_a_no_op():
    assert call(total_q=0, kv_dtype=I8, **BLK) == _lib.UA_OK


def test_plans():
    # int8 plans like e4m3 with block scales, whether the placeholder scales are asked or not
    for kw in (dict(), dict(head_dim=256), dict(block_size=13), dict(max_seqlen_q=3),
               dict(num_seqs=5, total_q=18432, max_seqlen_q=4096, max_seqlen_k=18432,
                    window_left=-1)):
        assert _plan(kv_dtype=I8, **kw) == _plan(kv_dtype=F8, per_block_scales=True, **kw)
    with pytest.raises(ua.UaError):
        _plan(kv_dtype=7)
