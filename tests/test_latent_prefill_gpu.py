"""Latent attention, expanded form, against the definition in 64 bits."""
import math

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def cum(n):
    return torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32)


def make(lens, h, nope=128, rope=64, value=128, dtype=BF, seed=0, pad_q=0, pad_k=0):
    g = torch.Generator().manual_seed(seed)
    cu_q, cu_k = cum([q for q, _ in lens]), cum([k for _, k in lens])
    tq, tk = int(cu_q[-1]) + pad_q, int(cu_k[-1]) + pad_k
    q = torch.randn((tq, h, nope + rope), generator=g).to(dtype)
    kv = torch.randn((tk, h, nope + value), generator=g).to(dtype)
    k_rope = torch.randn((tk, rope), generator=g).to(dtype)
    kv[int(cu_k[-1]):] = float("nan")       # rows behind the last sequence may hold anything
    k_rope[int(cu_k[-1]):] = float("nan")
    return q, kv[..., :nope], k_rope, kv[..., nope:], cu_q, cu_k


def run(t, **kw):
    d = []
    for i, x in enumerate(t):   # (.cuda() of a slice would lay it out again)
        if i in (1, 3):
            full = torch.empty((x.shape[0], x.shape[1], x.stride(1)), dtype=x.dtype, device="cuda")
            d.append(full[..., :x.shape[2]] if i == 1 else full[..., -x.shape[2]:])
            d[-1].copy_(x)
        else:
            d.append(x.cuda())
    n = [int((c[1:] - c[:-1]).max()) if c.numel() > 1 else 0 for c in (t[4], t[5])]
    return ua.latent_prefill(*d, **{**dict(max_seqlen_q=n[0], max_seqlen_k=n[1]), **kw})


def compare(t, scale=None, out_dtype=None, **kw):
    out, lse = run(t, scale=scale, out_dtype=out_dtype, return_lse=True, **kw)
    want, wlse, tol, ltol = ref.prefill(*t, scale or 1.0 / math.sqrt(t[0].shape[2]))
    end = int(t[4][-1])
    ref.check(out[:end], want[:end], tol[:end], out.dtype)
    ref.check(lse[:end], wlse[:end], ltol[:end], F32)
    assert ua.device_status() == 0


CASES = [
    ([(1, 1)], 1, 128, 64, 128, BF), ([(77, 77)], 16, 128, 64, 128, BF),
    ([(128, 128), (129, 129), (127, 127)], 4, 128, 64, 128, F16),
    ([(256, 256), (257, 300), (1, 500)], 3, 128, 64, 128, BF),
    ([(0, 5), (3, 0), (5, 2), (0, 0), (300, 290), (2, 2)], 5, 128, 64, 128, BF),
    ([(200, 700), (513, 513)], 2, 64, 32, 64, F16), ([(90, 400)], 3, 128, 16, 64, BF),
    ([(90, 400)], 3, 64, 48, 128, BF), ([(600, 1100)], 2, 128, 64, 128, F16),
    ([(3, 40)] * 70, 2, 128, 64, 128, BF),
]


@pytest.mark.parametrize("lens,h,nope,rope,value,dtype", CASES)
def test_prefill(lens, h, nope, rope, value, dtype):
    t = make(lens, h, nope, rope, value, dtype, pad_q=3, pad_k=5)
    compare(t)
    compare(t, out_dtype=F32, scale=0.2)


@pytest.mark.parametrize("lens,h,nope,rope,value,dtype", CASES + [
    ([(256, 900), (77, 129)], 20, 128, 64, 128, BF), ([(100, 1500)], 40, 64, 64, 64, F16),
    ([(64, 3000)], 16, 128, 64, 128, BF),
])
def test_prefill_by_parts(lens, h, nope, rope, value, dtype):
    """A bound of the key lengths that has a few CTAs share every q-block's keys, some with none."""
    t = make(lens, h, nope, rope, value, dtype, pad_q=3, pad_k=5)
    compare(t, max_seqlen_k=(1 << 31) - 1)
    compare(t, out_dtype=F32, scale=0.2, max_seqlen_k=(1 << 31) - 1)
    out = torch.full((t[0].shape[0], h, value), 7.0, dtype=dtype, device="cuda")
    compare(t, out=out, max_seqlen_k=(1 << 31) - 1)
    assert torch.all(out[-3:] == 7)


def test_steep_scores():
    t = make([(400, 900)], 2)
    t[0][...] = 0.5
    t[1][...] = (torch.arange(900) // 16 * 0.04)[:, None, None].to(BF)
    compare(t, scale=0.5, out_dtype=F32)


def test_rows_behind_the_batch_stay():
    t = make([(5, 9), (130, 130)], 2, pad_q=200)
    out = torch.full((335, 2, 128), 7.0, dtype=BF, device="cuda")
    run(t, out=out)
    assert torch.all(out[135:] == 7) and not torch.any(out[:135] == 7)
