"""append_latent against the definition in 64 bits, and what it leaves as it was."""
import math

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(lens, h, latent=512, rope=64, bs=64, dtype=BF, seed=0, pad=0, norm=BF, table=True,
         own_positions=False):
    g = torch.Generator().manual_seed(seed)
    cu, sl, bt, nb = ref.batch(lens, bs, seed)
    total = int(cu[-1]) + pad
    down = torch.randn((total, latent + rope), generator=g)
    down *= torch.exp2(torch.randint(-6, 5, (total, 1), generator=g).float())
    down = down.to(dtype)
    t = dict(latent=down[:, :latent], k_rope=down[:, latent:], cu=cu, sl=sl, bt=bt,
             cache=torch.randn((nb, bs, latent + rope), generator=g).to(dtype),
             q=torch.randn((total, h, 24 + rope), generator=g).to(dtype)[..., 24:] if h else None,
             w=None if norm is None else (1 + 0.3 * torch.randn(latent, generator=g)).to(norm))
    most = max([kv for _, kv in lens] + [1]) + 30
    t["table"] = ua.rope_table(most, rope, device="cpu") if table else None
    t["pos"] = torch.randint(0, most, (total,), generator=g).to(torch.int32) \
        if own_positions else None
    return t


def place(t):
    """(row, sequence, cache position) of the tokens that are written."""
    for b in range(t["sl"].numel()):
        r0, r1, kv = int(t["cu"][b]), int(t["cu"][b + 1]), int(t["sl"][b])
        for r in range(r0, r1):
            if kv - (r1 - r) >= 0:
                yield r, b, kv - (r1 - r)


def turned(x, t, pos, interleaved):
    """x [..., R] in 64 bits, and the largest magnitude of each pair."""
    half = x.shape[-1] // 2
    cs = t["table"][pos].double()
    c, s = cs[:half], cs[half:]
    y, m = torch.empty_like(x), torch.empty_like(x)
    ia, ib = (slice(0, None, 2), slice(1, None, 2)) if interleaved else \
        (slice(0, half), slice(half, None))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    m[..., ia] = m[..., ib] = torch.maximum(a.abs(), b.abs())
    return y, m


def expected(t, eps, interleaved):
    """The cache and the queries, with the bounds of fp32 arithmetic: a rotation rounds two
    products and their sum (3 2^-24 of at most 2 max |a|, |b|); a norm the mean (a few 2^-24), its
    root and two products (8 2^-24 together)."""
    latent = t["latent"].shape[1]
    want, tol = t["cache"].double(), torch.zeros(t["cache"].shape, dtype=torch.float64)
    q = None if t["q"] is None else torch.full(t["q"].shape, 7.0, dtype=torch.float64)
    qtol = None if q is None else torch.zeros_like(q)
    done = torch.zeros(t["cache"].shape[:2], dtype=torch.bool)
    bs = t["cache"].shape[1]
    for r, b, at in place(t):
        pos = at if t["pos"] is None else int(t["pos"][r])
        x = t["latent"][r].double()
        e = 0.0
        if t["w"] is not None:
            x = x / math.sqrt(float(x.square().mean()) + eps) * t["w"].double()
            e = 8 * 2.0 ** -24
        k = t["k_rope"][r].double()
        ke = torch.zeros_like(k)
        if t["table"] is not None:
            k, m = turned(k, t, pos, interleaved)
            ke = 6 * 2.0 ** -24 * m
        blk = int(t["bt"][b, at // bs])
        want[blk, at % bs] = torch.cat([x, k])
        tol[blk, at % bs] = torch.cat([x.abs() * e, ke])
        done[blk, at % bs] = True
        if q is not None:
            q[r], m = (t["q"][r].double(), 0.0) if t["table"] is None else \
                turned(t["q"][r].double(), t, pos, interleaved)
            qtol[r] = 6 * 2.0 ** -24 * m
    return want, tol, done, q, qtol


def dev(t):
    return {k: v if v is None else v.cuda() for k, v in t.items()}


def run(t, interleaved=False, eps=1e-6, out=None, **kw):
    d = dev(t)
    if out is None and d["q"] is not None:
        out = torch.full(tuple(t["q"].shape), 7.0, dtype=t["q"].dtype, device="cuda")
    got = ua.append_latent(d["latent"], d["k_rope"], d["cache"], d["cu"], d["sl"], d["bt"],
                           norm_weight=d["w"], norm_eps=eps, q_rope=d["q"], q_rope_out=out,
                           cos_sin=d["table"], positions=d["pos"], interleaved=interleaved, **kw)
    return d["cache"], got


def compare(t, interleaved=False, eps=1e-6):
    cache, q = run(t, interleaved, eps)
    want, tol, done, wq, qtol = expected(t, eps, interleaved)
    dt = t["cache"].dtype
    assert torch.equal(cache.cpu()[~done], t["cache"][~done])   # nothing else is written
    ref.check(cache.cpu()[done], want[done], tol[done], dt)
    if wq is not None:
        ref.check(q, wq, qtol, dt)
    assert ua.device_status() == 0


CASES = [
    ([(1, 1)], 1, 512, 64, 64, BF), ([(1, 7), (1, 64), (1, 65)], 16, 512, 64, 64, BF),
    ([(5, 5), (0, 3), (3, 130), (2, 1)], 128, 512, 64, 16, F16),
    ([(40, 100)], 40, 256, 32, 5, BF), ([(33, 33)], 7, 128, 16, 1, F16),
    ([(9, 20)], 12, 512, 48, 24, BF), ([(1, 30)] * 70, 3, 256, 64, 64, F16),
    ([(600, 700)], 64, 512, 64, 64, BF), ([(20, 25)], 0, 512, 64, 64, BF),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,h,latent,rope,bs,dtype", CASES)
def test_append(lens, h, latent, rope, bs, dtype, interleaved):
    compare(make(lens, h, latent, rope, bs, dtype, norm=dtype), interleaved)


@pytest.mark.parametrize("kw", [dict(norm=None), dict(norm=F32), dict(table=False),
                                dict(own_positions=True), dict(norm=None, table=False), dict(pad=9)])
def test_options(kw):
    compare(make([(3, 70), (17, 17), (1, 5)], 16, seed=2, **kw), True, eps=0.5)


def test_tokens_at_negative_positions_and_rows_behind_the_batch_stay():
    t = make([(5, 2), (3, 3)], 4, pad=6)
    _, q = run(t)
    assert torch.all(q[:3] == 7) and torch.all(q[8:] == 7) and not torch.any(q[3:8] == 7)
    compare(t)


def test_queries_in_place_and_into_the_absorbed_queries():
    t = make([(3, 70), (17, 17)], 16)
    _, apart = run(t)
    d = dev(t)
    whole = torch.full((20, 16, 512 + 64), 3.0, dtype=BF, device="cuda")
    _, got = run(t, out=whole[..., 512:])
    assert torch.equal(got, apart) and torch.all(whole[..., :512] == 3)
    ua.append_latent(d["latent"], d["k_rope"], d["cache"], d["cu"], d["sl"], d["bt"],
                     q_rope=d["q"], q_rope_out=d["q"], cos_sin=d["table"])
    assert torch.equal(d["q"], apart)


def test_bad_blocks_and_positions_are_reported_and_not_written():
    ua.device_status_reset()
    t = make([(3, 70), (4, 4)], 4)
    t["bt"][1, 0] = t["cache"].shape[0]
    cache, q = run(t)
    assert ua.device_status() == 5
    ua.device_status_reset()
    want, tol, done, wq, qtol = expected({**t, "cu": t["cu"][:2], "sl": t["sl"][:1]}, 1e-6, False)
    assert torch.equal(cache.cpu()[~done], t["cache"][~done])
    ref.check(q[:3], wq[:3], qtol[:3], BF)
    t = make([(3, 70), (4, 4)], 4, own_positions=True)
    t["pos"][4] = t["table"].shape[0]
    t["pos"][5] = -1
    _, q = run(t)
    assert ua.device_status() == 5
    ua.device_status_reset()
    assert torch.all(q[4:6] == 7) and not torch.any(q[:4] == 7)
