"""Plain references of the latent operators, on the CPU in 64 bits, one sequence at a time (tests
only), and the bounds of what rounding may add to them.

Bounds.  A weight of the softmax is rounded to the call's type for its product with the values:
half a step (2^-8 bf16, 2^-11 f16) of each weight, so half * sum_j w_j |v_j| of the output; an f16
weight below 2^-14 keeps an absolute half step of 2^-25 (the largest weight is at least 1 before
the division, and the sum too).  A score is a sum of K products in fp32, each of which may round:
K 2^-24 scale sum |q k|, which moves a weight by that relative amount, and the row's sum too.  The
exponential and the sums add a few 2^-22; the result is rounded once to the output's type.
"""
import math

import torch

# Half a step relative to the value, and at least: f16's steps stay 2^-24 below 2^-14, where half of
# one (2^-25) is more than 2^-11 of the value.
LEAST = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def batch(lens, bs, seed=0, spare=3, extra_cols=1):
    """cu_seqlens_q, seq_lens_k, block table (unused entries -1) and blocks of a batch."""
    g = torch.Generator().manual_seed(seed)
    per = [math.ceil(kv / bs) for _, kv in lens]
    nb = sum(per) + spare
    perm = torch.randperm(nb, generator=g)
    bt = torch.full((len(lens), max(per + [0]) + extra_cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        bt[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    cu = torch.tensor([0] + torch.tensor([q for q, _ in lens]).cumsum(0).tolist(),
                      dtype=torch.int32)
    return cu, torch.tensor([kv for _, kv in lens], dtype=torch.int32), bt, nb


def rows_of(cache, bt, b, kv):
    bs = cache.shape[1]
    pages = bt[b, :math.ceil(kv / bs)].long()
    return cache[pages].flatten(0, 1)[:kv]


def softmax_rows(q, k, v, see, scale, half):
    """out, lse and their bounds: q [n, d], k [kv, d], v [kv, e], see [n, kv], in 64 bits."""
    n, kv = see.shape
    if kv == 0:
        return (torch.zeros(n, v.shape[1], dtype=torch.float64),
                torch.full((n,), -math.inf, dtype=torch.float64),
                torch.zeros(n, v.shape[1], dtype=torch.float64),
                torch.zeros(n, dtype=torch.float64))
    x = (q @ k.T * scale).masked_fill(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    none = top[:, 0] == -math.inf
    w = torch.exp(x - torch.where(none[:, None], 0.0, top))
    total = w.sum(-1, keepdim=True)
    w = torch.where(none[:, None], 0.0, w / torch.where(none[:, None], 1.0, total))
    lse = torch.where(none, -math.inf, top[:, 0] + torch.log(total[:, 0]))
    ds = (q.abs() @ k.abs().T * scale).masked_fill(~see, 0.0).amax(-1) * q.shape[1] * 2.0 ** -24
    a = w @ v.abs()
    tol = a * (half + 2.0 * torch.expm1(ds)[:, None] + 2.0 ** -18)
    if half == HALF[torch.float16]:
        tol = tol + see.sum(-1, keepdim=True) * 2.0 ** -25 * v.abs().amax()
    ltol = ds + 2.0 ** -18 + 2.0 ** -21 * torch.where(none, 0.0, lse).abs()
    return w @ v, lse, tol, ltol


def attend(q, cache, cu, sl, bt, latent, scale, mask=None):
    """The absorbed form: out, lse and their bounds (before the output's own rounding)."""
    out = torch.zeros(q.shape[0], q.shape[1], latent, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros(q.shape[:2], dtype=torch.float64)
    for b in range(sl.numel()):
        r0, n, kv = int(cu[b]), int(cu[b + 1] - cu[b]), int(sl[b])
        k = rows_of(cache, bt, b, kv).double()
        at = torch.arange(kv - n, kv)[:, None]
        j = torch.arange(kv)[None]
        if mask is None:
            see = j <= at
        else:
            bit = j - (kv - n)
            word = mask[r0:r0 + n].long()
            pick = word.gather(1, (bit.clamp(min=0) // 32).expand(n, -1)) if kv else word[:, :0]
            see = (bit < 0) | (((pick >> (bit % 32)) & 1) > 0)
        for h in range(q.shape[1]):
            got = softmax_rows(q[r0:r0 + n, h].double(), k, k[:, :latent], see, scale,
                               HALF[q.dtype])
            for t, x in zip((out, lse, tol, ltol), got):
                t[r0:r0 + n, h] = x
    return out, lse, tol, ltol


def prefill(q, k_nope, k_rope, v, cu_q, cu_k, scale):
    out = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros(q.shape[:2], dtype=torch.float64)
    for b in range(cu_q.numel() - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        n, kv = q1 - q0, k1 - k0
        see = torch.arange(kv)[None] <= torch.arange(kv - n, kv)[:, None]
        for h in range(q.shape[1]):
            k = torch.cat([k_nope[k0:k1, h], k_rope[k0:k1]], -1).double()
            got = softmax_rows(q[q0:q1, h].double(), k, v[k0:k1, h].double(), see, scale,
                               HALF[q.dtype])
            for t, x in zip((out, lse, tol, ltol), got):
                t[q0:q1, h] = x
    return out, lse, tol, ltol


def tree(parents, cu, sl, words):
    """mask (int32) and positions of drafted trees."""
    mask = torch.zeros(parents.numel(), words, dtype=torch.int64)
    pos = torch.zeros(parents.numel(), dtype=torch.int32)
    for b in range(sl.numel()):
        r0, n = int(cu[b]), int(cu[b + 1] - cu[b])
        line = []
        for i, p in enumerate(parents[r0:r0 + n].tolist()):
            line.append((line[p] if p >= 0 else []) + [i])
            for a in line[i]:
                mask[r0 + i, a // 32] |= 1 << (a % 32)
            pos[r0 + i] = int(sl[b]) - n + len(line[i]) - 1
    return torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32), pos


def random_parents(lens, seed=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, _ in lens:
        up = [-1 if i == 0 else int(torch.randint(-1 if i % 7 == 6 else 0, i, (1,), generator=g))
              for i in range(n)]
        out += up
    return torch.tensor(out, dtype=torch.int32)


def check(got, want, tol, dtype):
    """got within its bounds of want, its own rounding to dtype among them."""
    got = got.detach().cpu().double()
    bound = tol + (HALF[dtype] * (want.abs() + tol)).clamp(min=LEAST[dtype]) + 2.0 ** -24 * 1e-3
    inf = ~torch.isfinite(want)
    assert torch.equal(got[inf], want[inf])
    err = (got - want).abs()[~inf]
    over = err - bound[~inf] if bound.shape == want.shape else err - bound
    assert not err.isnan().any()
    assert err.numel() == 0 or float(over.max()) <= 0, \
        f"off by {float(err.max()):.3e}, {float(over.max()):.3e} over its bound"
