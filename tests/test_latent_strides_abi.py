"""Strides of ua_append_latent, on the host.  (Without a GPU: the pointers are not real, so that a call
that passes every check must find no device.)"""
import pytest
import torch

from tests.test_latent_abi import APPEND, INVALID, run
from varlen_gqa_attention_paged_gb300 import _lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on these pointers")


def append(**over):
    return run("ua_append_latent", _lib.UaAppendLatent, APPEND, over)


@pytest.mark.parametrize("over", [
    dict(total_q=1, latent_stride=580, k_rope_stride=581, q_rope_stride=(9999, 64),
         q_rope_out_stride=(3, 64)),
    dict(total_q=1, latent_stride=-1, k_rope_stride=1, q_rope_stride=(1, 64)),
    dict(num_heads=1, q_rope_stride=(64, 5), q_rope_out_stride=(64, 1)),
    dict(total_q=1, num_heads=1, latent_stride=1, k_rope_stride=1, q_rope_stride=(1, 1),
         q_rope_out_stride=(1, 1)),
])
def test_strides_that_are_never_taken_may_be_anything(over):
    assert append(**over) == _lib.UA_ERR_CUDA


@pytest.mark.parametrize("over", [
    dict(total_q=1, q_rope_stride=(9999, 60)), dict(total_q=1, q_rope_out_stride=(8, 60)),
    dict(total_q=1, q_rope_out_stride=(9999, 32)), dict(num_heads=1, q_rope_stride=(60, 64)),
    dict(num_heads=1, q_rope_out_stride=(32, 64)), dict(total_q=2, latent_stride=580),
])
def test_strides_that_are_taken_are_checked(over):
    assert append(**over) == INVALID


@pytest.mark.parametrize("over", [
    dict(q_rope_out_stride=(576 * 16, 576)), dict(q_rope_stride=(2048, 128)),
    dict(q_rope_stride=(64, 384), q_rope_out_stride=(1024, 64)),
    dict(total_q=1, q_rope_out_stride=(1024, 128)), dict(num_heads=1, q_rope_stride=(2048, 64)),
])
def test_queries_in_place_keep_their_strides(over):
    """What a warp writes would lie where another is still to read."""
    assert append(**over) == INVALID
    assert append(**over, q_rope_out=(1 << 20) + APPEND["q_rope_out"]) == _lib.UA_ERR_CUDA


def test_queries_in_place_whose_other_stride_is_never_taken():
    assert append(total_q=1, q_rope_out_stride=(8, 64)) == _lib.UA_ERR_CUDA
    assert append(num_heads=1, q_rope_stride=(1024, 7)) == _lib.UA_ERR_CUDA
