"""The prepared latent calls' own bookkeeping, with a library that only notes what it is called
with."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from varlen_gqa_attention_paged_gb300 import _lib, latent

BF = torch.bfloat16
GIVEN, OTHER = SimpleNamespace(cuda_stream=11), SimpleNamespace(cuda_stream=12)


@pytest.fixture
def world(monkeypatch):
    """The current stream's handle, the library's calls and what its next ones return."""
    w = SimpleNamespace(current=7, calls=[], code=0, held=[])

    def entry(ref, stream):
        call = ref._obj
        w.calls.append(({n: getattr(call, n) for n, _ in call._fields_}, stream))
        return w.code

    lib = SimpleNamespace(ua_latent_attention=entry, ua_unified_attention_call=entry,
                          ua_append_kv=entry, ua_status_string=lambda c: b"refused")
    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "device", lambda i: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: SimpleNamespace(cuda_stream=w.current))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: w.current, raising=False)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda h, device=None: SimpleNamespace(cuda_stream=h))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: w.held.append((t.data_ptr(), s.cuda_stream)))
    return w


def attention(stream=None, **kw):
    i = dict(dtype=torch.int32)
    t = dict(q=torch.zeros((4, 2, 576), dtype=BF), cu_seqlens_q=torch.zeros(3, **i),
             seq_lens_k=torch.zeros(2, **i), block_table=torch.zeros((2, 5), **i), tree_mask=None,
             out=torch.zeros((4, 2, 512), dtype=BF), lse=None)
    call = _lib.UaLatent(**{n: x.data_ptr() for n, x in t.items() if x is not None})
    return latent.PreparedLatentAttention("ua_latent_attention", call, t, (), stream, **kw), t


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


def test_results_of_the_preparation_are_held_for_every_stream_that_writes_them(world):
    step, t = attention(made=("out",))
    at = t["out"].data_ptr()
    step()
    step(stream=SimpleNamespace(cuda_stream=7))         # the stream that it was made on
    assert world.held == []
    step(stream=OTHER)
    step()
    assert world.held == [(at, 12)]
    step, t = attention(made=("out",))
    world.held.clear()
    world.current = 8                                   # none passed: the current stream
    step()
    step()
    assert world.held == [(t["out"].data_ptr(), 8)]


def test_results_that_the_caller_passed_are_the_callers(world):
    step, t = attention()
    step(stream=OTHER)
    step, t = attention(made=("out",))
    step(out=torch.zeros_like(t["out"]), stream=OTHER)
    step(stream=GIVEN)
    assert world.held == []


def older():
    i = dict(dtype=torch.int32)
    t = dict(q=torch.zeros((4, 4, 64), dtype=BF), cu_seqlens_q=torch.zeros(3, **i),
             seq_lens_k=torch.zeros(2, **i), block_table=torch.zeros((2, 5), **i))
    x = torch.zeros((4, 4, 64), dtype=BF)
    made = torch.zeros_like(x)
    lib = _lib.load()
    a = ua.PreparedAttention(lib, _lib.UaAttention(), dict(t, out=made), GIVEN, made="out")
    b = ua.PreparedAppend(lib, _lib.UaAppend(), dict(t, k=x, v=x, q_out=made, positions=None), (),
                          GIVEN, made="q_out")
    return (a, "out", made), (b, "q_out", made)


def test_results_of_the_older_calls_are_held_too(world):
    for step, name, made in older():
        world.held.clear()
        step()
        assert world.held == []
        step(stream=OTHER)
        step()
        assert world.held == [(made.data_ptr(), 12)]
        step(**{name: torch.zeros_like(made)}, stream=GIVEN)
        assert len(world.held) == 1


def test_nothing_is_taken_that_the_library_refuses(world):
    """(It sees what the binding does not: a misaligned tensor.)"""
    step, t = attention(GIVEN)
    world.code = 1
    with pytest.raises(ua.UaError):
        step(q=torch.ones_like(t["q"]), out=torch.ones_like(t["out"]), stream=OTHER)
    world.code = 0
    assert step() is t["out"]
    call, stream = world.calls[-1]
    assert (call["q"], call["out"], stream) == (t["q"].data_ptr(), t["out"].data_ptr(), 11)
    q = torch.ones_like(t["q"])
    step(q=q)
    assert world.calls[-1][0]["q"] == q.data_ptr()
