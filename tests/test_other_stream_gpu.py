"""GPU: calls on a stream that is not the current one.  A result that the call allocates is not
handed out again, when its tensor is dropped, before that stream is done with it."""
from types import SimpleNamespace

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def calls():
    i = dict(dtype=torch.int32, device="cuda")
    x = torch.randn((3, 2, 64), device="cuda").to(BF)
    q = torch.randn((3, 8, 64), device="cuda").to(BF)
    cache = torch.zeros((4, 16, 2, 64), dtype=BF, device="cuda")
    args = (torch.arange(4, **i), torch.tensor([5, 9, 16], **i),
            torch.tensor([[0], [1], [2]], **i))
    table = ua.rope_table(64, 64)
    att = dict(max_seqlen_q=1, max_seqlen_k=16)
    app = dict(max_seqlen_q=1, q=q, cos_sin=table)
    return {
        "append_kv": lambda s: ua.append_kv(x, x, cache, cache.clone(), *args, stream=s, **app),
        "prepare_append": lambda s: ua.prepare_append(x, x, cache, cache.clone(), *args, stream=s,
                                                      **app)(),
        "unified_attention": lambda s: ua.unified_attention(q, cache, cache, *args, stream=s,
                                                            **att),
        "prepare": lambda s: ua.prepare(q, cache, cache, *args, stream=s, **att)(),
    }


@pytest.mark.parametrize("foreign", [False, True])
@pytest.mark.parametrize("name", ["append_kv", "prepare_append", "unified_attention", "prepare"])
def test_a_new_result_outlives_the_work_of_its_stream(name, foreign):
    call = calls()[name]
    side = torch.cuda.Stream()
    stream = SimpleNamespace(cuda_stream=side.cuda_stream) if foreign else side
    call(stream)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                    # about a tenth of a second
    out = call(stream)
    at, shape = out.data_ptr(), tuple(out.shape)
    del out
    held = [torch.empty(shape, dtype=BF, device="cuda") for _ in range(4)]
    assert not side.query()                               # the call's kernel is still to run
    assert at not in [t.data_ptr() for t in held]
    torch.cuda.synchronize()


def test_on_the_current_stream_memory_is_used_again():
    call = calls()["append_kv"]
    out = call(torch.cuda.current_stream())
    at, shape = out.data_ptr(), tuple(out.shape)
    del out
    assert torch.empty(shape, dtype=BF, device="cuda").data_ptr() == at
    torch.cuda.synchronize()
