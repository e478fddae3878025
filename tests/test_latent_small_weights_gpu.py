"""GPU: rows of one dominant key and many small ones, whose weights are below f16's normal range.

Bounds.  A weight's product with the values takes it in 16 bits: half a step of it (2^-11 f16, 2^-8
bf16), or, since the largest weight of a row is held at 2^7 or more in f16, an absolute 2^-25 / 2^7 =
2^-32 of the largest; in all n 2^-32 max |v| / sum.  Sums of weights and of products round once a
16-key step, 2^-23 relative; scores are sums of K products in fp32 (K 2^-24 of their magnitude), the
exponential adds 2^-18.
"""
import math

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: 2.0 ** -8, F16: 2.0 ** -11}
# a small key's score below the dominant one's, in nats: weights of 2^-24.8 (which half of f16's
# smallest step would round up to 2^-24), 2^-25.4 (down to 0), 2^-30.3
DROPS = [17.2, 17.6, 21.0]


def check(out, lse, n, drop, k, dtype):
    """n keys, the dominant one's value 0 and the others' 1."""
    w = math.exp(-drop)
    total = 1 + (n - 1) * w
    want = (n - 1) * w / total
    ds = k * 2.0 ** -24 * drop
    rel = HALF[dtype] + 2 * math.expm1(ds) + 2.0 ** -18 + n / 16 * 2.0 ** -23
    bound = want * rel + n * 2.0 ** -32 + 2.0 ** -24 * want
    err = float((out.double() - want).abs().max())
    assert err <= bound, f"{float(out.double().mean())} for {want}: off by {err}, bound {bound}"
    err = float((lse.double() - drop - math.log(total)).abs().max())
    assert err <= ds + 2.0 ** -18 + n / 16 * 2.0 ** -23 + 2.0 ** -21 * drop


def score(drop, dtype):
    """Factors of the dominant key's score, and the score that they give in this type."""
    a = torch.tensor(drop / 4).to(dtype)
    return a, 4.0 * float(a)


@pytest.mark.parametrize("drop", DROPS)
@pytest.mark.parametrize("dtype", [F16, BF])
@pytest.mark.parametrize("seqs,n,heads,latent", [
    (1, 60001, 16, 512), (1, 700, 16, 512), (28, 1000, 16, 256), (3, 9000, 128, 128)])
def test_absorbed(seqs, n, heads, latent, dtype, drop):
    """By even shares and by parts; the dominant key early, and last."""
    a, drop = score(drop, dtype)
    i = dict(dtype=torch.int32, device="cuda")
    pages = -(-n // 64)
    for at in (5, n - 1):
        cache = torch.zeros((pages, 64, latent + 64), dtype=dtype, device="cuda")
        cache[..., :latent] = 1
        cache[at // 64, at % 64, :latent] = 0
        cache[at // 64, at % 64, latent] = a
        q = torch.zeros((seqs, heads, latent + 64), dtype=dtype, device="cuda")
        q[..., latent] = 4
        out, lse = ua.latent_attention(
            q, cache, torch.arange(seqs + 1, **i), torch.full((seqs,), n, **i),
            torch.arange(pages, **i).repeat(seqs, 1), scale=1.0, max_seqlen_q=1, max_seqlen_k=n,
            out_dtype=F32, return_lse=True)
        check(out, lse, n, drop, latent + 64, dtype)


@pytest.mark.parametrize("drop", DROPS)
@pytest.mark.parametrize("dtype", [F16, BF])
@pytest.mark.parametrize("n,heads", [(30001, 2), (9000, 80)])
def test_expanded(n, heads, dtype, drop):
    """A q-block's keys in parts, and in one."""
    a, drop = score(drop, dtype)
    i = dict(dtype=torch.int32, device="cuda")
    for at in (5, n - 1):
        rope = torch.zeros((n, 64), dtype=dtype, device="cuda")
        rope[at, 0] = a
        kv = torch.zeros((n, heads, 256), dtype=dtype, device="cuda")
        kv[..., 128:] = 1
        kv[at, :, 128:] = 0
        q = torch.zeros((1, heads, 192), dtype=dtype, device="cuda")
        q[..., 128] = 4
        out, lse = ua.latent_prefill(
            q, kv[..., :128], rope, kv[..., 128:], torch.tensor([0, 1], **i),
            torch.tensor([0, n], **i), scale=1.0, max_seqlen_q=1, max_seqlen_k=n, out_dtype=F32,
            return_lse=True)
        check(out, lse, n, drop, 192, dtype)
