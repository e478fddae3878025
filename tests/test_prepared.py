"""The prepared calls' own bookkeeping, with a library that only notes what it is called with."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from varlen_gqa_attention_paged_gb300 import _lib

BF = torch.bfloat16


class _Library:
    def __init__(self):
        self.calls = []

    def _note(self, ref, stream):
        call = ref._obj
        self.calls.append(({n: getattr(call, n) for n, _ in call._fields_}, stream))
        return 0

    ua_unified_attention_call = ua_append_kv = _note


def _tensors(rows=4, heads=4, d=64):
    i = dict(dtype=torch.int32)
    return dict(q=torch.zeros((rows, heads, d), dtype=BF), cu_seqlens_q=torch.zeros(3, **i),
                seq_lens_k=torch.zeros(2, **i), block_table=torch.zeros((2, 5), **i))


STREAM = SimpleNamespace(cuda_stream=11)
OTHER = SimpleNamespace(cuda_stream=12)


def attention():
    t = _tensors()
    t["out"] = torch.zeros_like(t["q"])
    lib = _Library()
    call = _lib.UaAttention(**{n: x.data_ptr() for n, x in t.items()})
    return ua.PreparedAttention(lib, call, t, STREAM), t, lib


@pytest.fixture
def append(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "device", lambda i: contextlib.nullcontext())
    t = _tensors()
    t.update(k=torch.zeros((4, 4, 64), dtype=BF), v=torch.zeros((4, 4, 64), dtype=BF),
             q_out=torch.zeros_like(t["q"]), positions=None)
    lib = _Library()
    call = _lib.UaAppend(**{n: x.data_ptr() for n, x in t.items() if x is not None})
    return ua.PreparedAppend(lib, call, t, (), STREAM), t, lib


def test_attention_takes_all_of_a_call_or_none():
    step, t, lib = attention()
    q = torch.ones_like(t["q"])
    with pytest.raises(ValueError, match="out"):
        step(q=q, out=t["out"].float())
    assert step() is t["out"]
    assert lib.calls[-1][0]["q"] == t["q"].data_ptr()
    assert step(q=q) is t["out"]
    assert lib.calls[-1][0]["q"] == q.data_ptr()


def test_append_takes_all_of_a_call_or_none(append):
    step, t, lib = append
    k, q = torch.ones_like(t["k"]), torch.ones_like(t["q"])
    for bad in (dict(block_table=t["block_table"].long()), dict(positions=t["seq_lens_k"]),
                dict(v=t["v"][:3])):
        with pytest.raises(ValueError, match=list(bad)[0]):
            step(k=k, q=q, **bad)
        assert step() is t["q_out"]
        assert lib.calls[-1][0]["k"] == t["k"].data_ptr()
        assert lib.calls[-1][0]["q"] == t["q"].data_ptr()
    step(k=k, q=q)
    assert (lib.calls[-1][0]["k"], lib.calls[-1][0]["q"]) == (k.data_ptr(), q.data_ptr())


def test_append_sees_strides_that_changed_in_place(append):
    step, t, lib = append
    step(k=t["k"])
    t["k"].transpose_(0, 1)                       # four tokens of four heads: the same shape
    with pytest.raises(ValueError, match="k: "):
        step(k=t["k"])
    assert len(lib.calls) == 1


def test_both_keep_the_stream_passed_last(append):
    for step, lib in (attention()[::2], append[::2]):
        for stream, want in ((None, 11), (OTHER, 12), (None, 12), (STREAM, 11)):
            step(stream=stream)
            assert lib.calls[-1][1] == want
