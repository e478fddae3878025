"""Latent attention, absorbed form, against the definition in 64 bits."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(lens, h, latent=512, rope=64, bs=64, dtype=BF, seed=0, pad=0, poison=True, **kw):
    g = torch.Generator().manual_seed(seed)
    cu, sl, bt, nb = ref.batch(lens, bs, seed, **kw)
    total = int(cu[-1]) + pad
    q = torch.randn((total, h, latent + rope), generator=g).to(dtype)
    cache = torch.randn((nb, bs, latent + rope), generator=g).to(dtype)
    if poison:  # slots that hold no key may hold anything
        used = torch.zeros(nb, bs, dtype=torch.bool)
        for b, (_, kv) in enumerate(lens):
            for j in range(kv):
                used[bt[b, j // bs], j % bs] = True
        cache[~used] = float("nan")
    return q, cache, cu, sl, bt


def sizes(cu, sl):
    q = int((cu[1:] - cu[:-1]).max()) if cu.numel() > 1 else 0
    return dict(max_seqlen_q=q, max_seqlen_k=int(sl.max()) if sl.numel() else 0)


def run(t, rope=64, scale=0.08, mask=None, **kw):
    q, cache, cu, sl, bt = (x.cuda() for x in t)
    return ua.latent_attention(q, cache, cu, sl, bt, scale=scale, rope_dim=rope,
                               tree_mask=None if mask is None else mask.cuda(),
                               **{**sizes(t[2], t[3]), **kw})


def compare(t, rope=64, scale=0.08, mask=None, out_dtype=None, **kw):
    q, cache, cu, sl, bt = t
    latent = q.shape[2] - rope
    out, lse = run(t, rope, scale, mask, out_dtype=out_dtype, return_lse=True, **kw)
    want, wlse, tol, ltol = ref.attend(q, cache, cu, sl, bt, latent, scale, mask)
    end = int(cu[-1])
    ref.check(out[:end], want[:end], tol[:end], out.dtype)
    ref.check(lse[:end], wlse[:end], ltol[:end], F32)
    assert ua.device_status() == 0
    return out


ONE = [(1, 1), (1, 2), (1, 63), (1, 64), (1, 65), (1, 127), (1, 200)]
CASES = [
    # lens, heads, latent, rope, block size, dtype
    ([(1, 1)], 1, 512, 64, 64, BF),
    ([(1, 64)], 16, 512, 64, 64, BF),
    ([(1, 700)], 16, 512, 64, 64, BF),
    ([(1, 1500)], 16, 512, 64, 16, F16),
    (ONE, 16, 512, 64, 64, BF),
    (ONE, 5, 256, 32, 8, F16),
    (ONE, 40, 128, 16, 24, BF),
    ([(1, 300), (1, 77)], 64, 512, 64, 32, F16),
    ([(1, 300), (1, 1029)], 128, 512, 64, 64, BF),
    ([(1, 333)], 128, 512, 48, 5, BF),
    ([(1, 130), (2, 70)], 3, 512, 64, 1, F16),
    ([(1, 90)], 7, 128, 64, 13, F16),
    # several new tokens, none, and more of them than keys
    ([(3, 500), (0, 40), (2, 2), (4, 4), (1, 0), (5, 3), (0, 0)], 16, 512, 64, 64, BF),
    ([(9, 140), (33, 33), (70, 400)], 20, 256, 64, 16, BF),
    ([(50, 50), (17, 90)], 128, 128, 32, 64, F16),
    ([(130, 260)], 2, 512, 64, 128, F16),
    ([(1, 4000), (1, 10), (1, 2500), (1, 1)], 16, 512, 64, 64, BF),
    ([(1, 37)] * 70, 16, 512, 64, 16, BF),
    ([(1, 9000)], 16, 512, 64, 64, BF), ([(2, 6000), (1, 40), (1, 5000)], 20, 256, 32, 32, F16),
    ([(1, 8000)], 128, 512, 64, 64, BF), ([(3, 7000)], 9, 128, 64, 16, BF),
]


@pytest.mark.parametrize("lens,h,latent,rope,bs,dtype", CASES)
def test_attention(lens, h, latent, rope, bs, dtype):
    t = make(lens, h, latent, rope, bs, dtype)
    compare(t, rope)
    compare(t, rope, out_dtype=F32)


FAR = (1 << 31) - 1   # a bound of the lengths that leaves a cluster a row tile no good


@pytest.mark.parametrize("lens,h,latent,rope,bs,dtype", CASES)
def test_attention_by_even_shares(lens, h, latent, rope, bs, dtype):
    t = make(lens, h, latent, rope, bs, dtype)
    compare(t, rope, out_dtype=F32, max_seqlen_k=FAR)


@pytest.mark.parametrize("lens,h,latent", [
    # row tiles of 64 token-heads, the keys of each in 1, 2, 4, 8, 4 and 8 parts, parts without keys,
    # clusters without a row tile
    ([(1, 300)] * 100, 16, 512),
    ([(1, 150), (0, 9), (1, 0)] * 17, 16, 512),
    ([(1, 333), (1, 70), (0, 100), (1, 64), (3, 3)] * 5, 16, 512),
    ([(5, 700), (1, 1), (2, 129)], 64, 512),
    ([(1, 200), (4, 66)], 7, 256),
    ([(2, 500), (31, 90)], 5, 128),
])
@pytest.mark.parametrize("masked", [False, True])
def test_attention_by_parts(lens, h, latent, masked):
    t = make(lens, h, latent, bs=16, pad=7)
    mask = None
    if masked:
        mask = torch.nn.functional.pad(masks(lens), (0, 0, 0, 7), value=-1)
    q, cache, cu, sl, bt = (x.cuda() for x in t)
    for far, whole in ((None, True), (FAR, False)):
        size = sizes(t[2], t[3])
        step = ua.prepare_latent_attention(
            q, cache, cu, sl, bt, scale=0.08, max_seqlen_q=size["max_seqlen_q"],
            max_seqlen_k=far or size["max_seqlen_k"])
        assert (ua.latent_workspace_bytes(step) == 0) == whole
    compare(t, mask=mask, out_dtype=F32)
    out = torch.full((q.shape[0], h, latent), 7.0, dtype=BF, device="cuda")
    compare(t, mask=mask, out=out)
    assert torch.all(out[-7:] == 7)     # rows behind the last sequence


def masks(lens, seed=0):
    """Random masks: not trees, rows that see nothing among them."""
    g = torch.Generator().manual_seed(seed)
    total, most = sum(q for q, _ in lens), max(q for q, _ in lens)
    bits = torch.rand((total, most), generator=g) < 0.4
    bits[::5] = False
    words = (most + 31) // 32
    b = torch.nn.functional.pad(bits, (0, 32 * words - most)).reshape(total, words, 32)
    v = (b.long() << torch.arange(32)).sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)


@pytest.mark.parametrize("lens,h,dtype", [
    ([(1, 100)], 16, BF), ([(17, 301), (3, 3), (64, 100)], 16, BF),
    ([(70, 70), (33, 129), (1, 65), (2, 1)], 5, F16), ([(100, 1000)], 40, BF),
])
def test_masks(lens, h, dtype):
    t = make(lens, h, dtype=dtype, bs=32)
    compare(t, mask=masks(lens), out_dtype=F32)


def test_trees_of_parents():
    lens = [(17, 301), (60, 500), (1, 9), (0, 3), (40, 40)]
    parents = ref.random_parents(lens)
    cu, sl, _, _ = ref.batch(lens, 64)
    mask, pos = ua.tree_mask(parents.cuda(), cu.cuda(), sl.cuda(), max_seqlen_q=60)
    wmask, wpos = ref.tree(parents, cu, sl, 2)
    assert torch.equal(mask.cpu(), wmask) and torch.equal(pos.cpu(), wpos)
    compare(make(lens, 8), mask=mask.cpu())


def test_steep_scores():
    """Scores that climb tile by tile, so that every tile moves the running max."""
    t = make([(1, 900), (2, 640)], 16, seed=3)
    q, cache = t[0], t[1]
    q[...] = 0.5
    for b, (_, kv) in enumerate([(1, 900), (2, 640)]):
        for j in range(kv):
            cache[t[4][b, j // 64], j % 64] = (j // 16) * 0.05
    compare(t, scale=0.3, out_dtype=F32)
