"""The prepared latent calls' own bookkeeping, with a library that only notes what it is called
with."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from varlen_gqa_attention_paged_gb300 import _lib, latent

BF = torch.bfloat16
GIVEN, OTHER = SimpleNamespace(cuda_stream=11), SimpleNamespace(cuda_stream=12)


@pytest.fixture
def world(monkeypatch):
    """The current stream's handle, the library's calls and what its next ones return."""
    w = SimpleNamespace(current=7, calls=[], code=0)

    def entry(ref, stream):
        call = ref._obj
        w.calls.append(({n: getattr(call, n) for n, _ in call._fields_}, stream))
        return w.code

    lib = SimpleNamespace(ua_latent_attention=entry, ua_status_string=lambda c: b"refused")
    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "device", lambda i: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: SimpleNamespace(cuda_stream=w.current))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: w.current, raising=False)
    return w


def attention(stream=None):
    i = dict(dtype=torch.int32)
    t = dict(q=torch.zeros((4, 2, 576), dtype=BF), cu_seqlens_q=torch.zeros(3, **i),
             seq_lens_k=torch.zeros(2, **i), block_table=torch.zeros((2, 5), **i), tree_mask=None,
             out=torch.zeros((4, 2, 512), dtype=BF), lse=None)
    call = _lib.UaLatent(**{n: x.data_ptr() for n, x in t.items() if x is not None})
    return latent.PreparedLatentAttention("ua_latent_attention", call, t, (), stream), t


def test_a_call_without_a_stream_goes_to_the_current_one(world):
    """(As tree_mask() does, whose masks it reads.)"""
    step, _ = attention()
    for current in (7, 8, 7):
        world.current = current
        step()
        assert world.calls[-1][1] == current


def test_a_stream_passed_once_is_kept(world):
    step, _ = attention(GIVEN)
    for stream, want in ((None, 11), (OTHER, 12), (None, 12), (GIVEN, 11), (None, 11)):
        step(stream=stream)
        assert world.calls[-1][1] == want
    step, _ = attention()
    step(stream=OTHER)
    step()
    assert world.calls[-1][1] == 12
