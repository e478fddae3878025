"""Cases of the latent-attention operators, for measuring them.

A latent cache holds one vector for each token, shared by all heads: ``latent`` normalised
elements, which are keys and values at once, and ``rope`` rotated elements, which are keys only.
Four operators of a serving step on it, each in its plain form (``own`` false: elementary torch
operations in 32 bits) and as a user calls it (``own`` true: the package):

* ``append``: the step's latents are normalised (RMS) and its rope keys rotated on their way into
  the paged cache, the queries' rope parts rotated beside them.
* ``decode``: the absorbed form.  Queries are in the latent space already (the key
  up-projection is applied to them), and every head attends over the cached vectors themselves.
* ``tree``: the same for a tree of drafted tokens in each sequence: from every token's parent
  the masks and positions, then attention in which a drafted token sees the cached prefix, its
  ancestors and itself.
* ``prefill``: the expanded form: keys and values of every head, from the up-projection, and the
  shared rope keys; causal attention over ragged prompts, with their log-sums where asked.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program has in hand before the
call, ``run()`` makes one pass, ``work()`` counts what the pass cannot do without and
``exact()`` is the definition in 64 bits, one sequence at a time.
"""
import math

import torch

own = False

_DEV = "cuda"
_HALF = {"bf16": torch.bfloat16, "f16": torch.float16}
_BASE = 10000.0
_EPS = 1e-6


def _case(name, op, nseq, q, kv, **over):
    c = dict(name=name, op=op, nseq=nseq, q=q, kv=kv, ragged=False, h=16, latent=512, rope=64,
             bs=64, dtype="bf16", nope=128, value=128, lse=False, interleaved=False)
    c.update(over)
    return c


def listed():
    return [
        # one decode step of a batch of 32: every sequence adds its newest token
        _case("append_step", "append", 32, 1, 2500, ragged=True),
        # prompts of a prefill step, all heads of a model with many
        _case("append_prompts", "append", 4, 2048, 2048, h=64, interleaved=True),
        # a ragged step of a small model: short latents, small pages
        _case("append_small", "append", 7, 300, 900, ragged=True, h=40, latent=256, rope=32,
              bs=16, dtype="f16"),
        # one token of one short conversation, heads of one shard: the smallest attention call
        _case("decode_one", "decode", 1, 1, 700),
        # decode of a large ragged batch, heads of one shard
        _case("decode_batch", "decode", 64, 1, 8191, ragged=True),
        # decode with all heads of a large model on the card
        _case("decode_wide", "decode", 32, 1, 6000, h=128),
        # chains of two drafted tokens behind long contexts
        _case("decode_drafts", "decode", 12, 3, 12001, ragged=True, h=64, bs=32, dtype="f16"),
        # two conversations with small draft trees
        _case("tree_small", "tree", 2, 17, 3001),
        # a batch of large draft trees
        _case("tree_large", "tree", 8, 60, 8192, ragged=True, h=32),
        # one short prompt
        _case("prefill_short", "prefill", 1, 77, 77),
        # ragged chunks behind prefixes whose keys and values were expanded again
        _case("prefill_chunks", "prefill", 5, 1901, 3001, ragged=True, h=8, dtype="f16", lse=True),
        # two long prompts
        _case("prefill_long", "prefill", 2, 8192, 8192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _case("", "append", 1, 1, 1, dtype=rng.choice(["bf16", "f16"]),
              ragged=rng.random() < 0.75, h=rng.choice([1, 5, 8, 16, 16, 32, 40, 64, 128]),
              latent=rng.choice([512, 512, 512, 256, 128]), rope=rng.choice([64, 64, 64, 32]),
              bs=rng.choice([64, 64, 32, 16, 24, 128, 5]))
    c["op"] = rng.choice(["append", "decode", "decode", "tree", "prefill", "prefill"])
    if c["op"] == "append":
        c["interleaved"] = rng.random() < 0.5
        c["h"] = min(c["h"], 64)
        if rng.random() < 0.4:                  # a decode step
            c["nseq"], c["q"] = _log_int(rng, 1, 128), rng.choice([1, 1, 2, 3])
        else:
            c["nseq"] = rng.randint(1, 6)
            c["q"] = max(1, _log_int(rng, 1, 8000) // c["nseq"])
        c["kv"] = c["q"] + rng.choice([0, rng.randint(0, 3000)])
    elif c["op"] == "prefill":
        c["nope"] = c["value"] = rng.choice([128, 128, 64])
        c["lse"] = rng.random() < 0.4
        c["h"] = min(c["h"], 32)
        c["nseq"] = rng.randint(1, 5)
        most = int(math.sqrt(1.5e9 / c["h"] / c["nseq"]))
        c["kv"] = _log_int(rng, 1, min(8000, most))
        c["q"] = max(1, c["kv"] - rng.choice([0, rng.randint(0, c["kv"])]))
    else:
        c["nseq"] = _log_int(rng, 1, 64)
        c["q"] = rng.choice([1, 1, 1, 2, 3]) if c["op"] == "decode" else rng.randint(2, 70)
        c["nseq"] = max(1, min(c["nseq"], 40000 // (c["h"] * c["q"])))
        rows = c["h"] * c["q"] * c["nseq"]
        most = min(16000, 4e5 / c["nseq"], 5e7 / rows)
        c["kv"] = c["q"] + _log_int(rng, 1, max(2, most))
    del c["name"]
    return c


# ------------------------------------------------------------------ the cases' shapes

def _lens(c):
    """(new tokens, cached tokens with them) of each sequence."""
    out = []
    for i in range(c["nseq"]):
        f = 1.0 - 0.8 * ((i * 0.6180339887) % 1.0) if c["ragged"] else 1.0
        q = max(1, int(c["q"] * f))
        out.append((q, q + int((c["kv"] - c["q"]) * f)))
    return out


def work(c):
    lens, h, l, r, bs = _lens(c), c["h"], c["latent"], c["rope"], c["bs"]
    tokens, keys = sum(q for q, _ in lens), sum(kv for _, kv in lens)
    if c["op"] == "append":
        b = tokens * ((l + r) * 4 + h * r * 4) + l * 2 + max(kv for _, kv in lens) * r * 4
        b += sum((kv + bs - 1) // bs - (kv - q) // bs for q, kv in lens) * 4
        return {"bytes": b, "flops": tokens * (4 * l + 3 * r * (h + 1))}
    pairs = sum(q * (kv - q) + q * (q + 1) // 2 for q, kv in lens)
    if c["op"] == "prefill":
        n, v = c["nope"], c["value"]
        b = 2 * (tokens * h * (n + r + v) + keys * (h * (n + v) + r))
        b += tokens * h * 4 if c["lse"] else 0
        return {"bytes": b, "flops": 2 * h * (n + r + v) * pairs}
    b = keys * (l + r) * 2 + tokens * h * (2 * l + r) * 2
    b += 4 * sum((kv + bs - 1) // bs for _, kv in lens)
    if c["op"] == "tree":       # only the pairs of a tree that its parents name, about
        b += tokens * (8 + 4 * ((max(q for q, _ in lens) + 31) // 32))
    return {"bytes": b, "flops": 2 * h * (2 * l + r) * pairs}


# ------------------------------------------------------------------ the inputs

def _angles(pos, rot):
    """Angles of positions, in 64 bits: pos * base^(-2 i / rot)."""
    i = torch.arange(rot // 2, device=pos.device, dtype=torch.float64)
    return pos.double()[..., None] * torch.exp(i * (-2.0 * math.log(_BASE) / rot))


def _parents(q, g):
    """Parents of a draft tree's q tokens in order: the first is the root; a later one hangs
    from one of the few before it, mostly, so that the tree is some branches wide."""
    back = 1 + (torch.rand(q, generator=g) ** 2 * 8).long()
    i = torch.arange(q)
    return torch.where(i == 0, torch.full_like(i, -1), (i - back).clamp(min=0)).int()


def prepare(c, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    lens, h, l, r, bs = _lens(c), c["h"], c["latent"], c["rope"], c["bs"]
    half = _HALF[c["dtype"]]
    tokens, keys = sum(q for q, _ in lens), sum(kv for _, kv in lens)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32)

    def offsets(n):
        return torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32,
                            device=_DEV)

    s = dict(c=c, lens=lens, cu=offsets([q for q, _ in lens]),
             sl=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=_DEV),
             max_q=max(q for q, _ in lens), max_k=max(kv for _, kv in lens))
    if c["op"] == "prefill":
        n, v = c["nope"], c["value"]
        s["cu_k"] = offsets([kv for _, kv in lens])
        s["q"] = randn(tokens, h, n + r).to(half)
        # the up-projection's output holds a token's keys and values, head by head
        s["kv"] = randn(keys, h, n + v).to(half)
        s["k_rope"] = (1.5 * randn(keys, r)).to(half)
        s["scale"] = 1.0 / math.sqrt(n + r)
        s["out"] = torch.empty((tokens, h, v), dtype=half, device=_DEV)
        if own:
            import varlen_gqa_attention_paged_gb300 as ua
            s["step"] = ua.prepare_latent_prefill(
                s["q"], s["kv"][..., :n], s["k_rope"], s["kv"][..., n:], s["cu"], s["cu_k"],
                max_seqlen_q=s["max_q"], max_seqlen_k=s["max_k"], scale=s["scale"], out=s["out"],
                return_lse=c["lse"])
        return s
    per = [(kv + bs - 1) // bs for _, kv in lens]
    nb = int(1.25 * sum(per)) + 1
    perm = torch.randperm(nb, generator=g, device=_DEV)
    s["bt"] = torch.zeros((len(lens), max(per)), dtype=torch.int32, device=_DEV)
    at = 0
    for i, n in enumerate(per):
        s["bt"][i, :n] = perm[at:at + n].to(torch.int32)
        at += n
    if c["op"] == "append":
        # the down-projection's output holds a token's latent and its rope key side by side
        down = randn(tokens, l + r)
        down[:, :l] *= 0.5 + torch.rand((tokens, 1), generator=g, device=_DEV)
        down = down.to(half)
        s["lat"], s["k_rope"] = down[:, :l], down[:, l:]
        s["weight"] = (1.0 + 0.1 * randn(l)).to(half)
        # heads of the query projection: the part that is not rotated, then the rope part
        s["q"] = randn(tokens, h, 128 + r).to(half)[..., 128:]
        # the absorbed queries, whose front another product fills
        s["q_out"] = torch.zeros((tokens, h, l + r), dtype=half, device=_DEV)[..., l:]
        s["cache"] = torch.zeros((nb, bs, l + r), dtype=half, device=_DEV)
        a = _angles(torch.arange(s["max_k"] + 64, device=_DEV), r)
        s["table"] = torch.cat([torch.cos(a), torch.sin(a)], -1).float()
        if own:
            import varlen_gqa_attention_paged_gb300 as ua
            s["step"] = ua.prepare_append_latent(
                s["lat"], s["k_rope"], s["cache"], s["cu"], s["sl"], s["bt"],
                norm_weight=s["weight"], norm_eps=_EPS, q_rope=s["q"], q_rope_out=s["q_out"],
                cos_sin=s["table"], interleaved=c["interleaved"])
        return s
    s["q"] = randn(tokens, h, l + r).to(half)
    s["cache"] = randn(nb, bs, l + r)
    s["cache"][..., l:] *= 1.5
    s["cache"] = s["cache"].to(half)
    s["scale"] = 1.0 / math.sqrt(128 + r)
    s["out"] = torch.empty((tokens, h, l), dtype=half, device=_DEV)
    if c["op"] == "tree":
        cpu = torch.Generator().manual_seed(seed)
        s["parents"] = torch.cat([_parents(q, cpu) for q, _ in lens]).to(_DEV)
        s["mask"] = torch.zeros((tokens, (s["max_q"] + 31) // 32), dtype=torch.int32, device=_DEV)
        s["pos"] = torch.zeros(tokens, dtype=torch.int32, device=_DEV)
    if own:
        import varlen_gqa_attention_paged_gb300 as ua
        s["step"] = ua.prepare_latent_attention(
            s["q"], s["cache"], s["cu"], s["sl"], s["bt"], rope_dim=r, scale=s["scale"],
            max_seqlen_q=s["max_q"], max_seqlen_k=s["max_k"], tree_mask=s.get("mask"),
            out=s["out"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["c"]["op"]
    if op == "append":
        if own:
            s["step"](latent=s["lat"], k_rope=s["k_rope"], q_rope=s["q"], q_rope_out=s["q_out"])
        else:
            _append(s)
        return {"q_rope": s["q_out"], "cache": s["cache"]}
    if op == "prefill":
        if own:
            n = s["c"]["nope"]
            got = s["step"](q=s["q"], k_nope=s["kv"][..., :n], k_rope=s["k_rope"],
                            v=s["kv"][..., n:], out=s["out"])
            out, lse = got if s["c"]["lse"] else (got, None)
        else:
            out, lse = _prefill(s)
        return {"out": out, "lse": lse} if s["c"]["lse"] else out
    if op == "tree":
        if own:
            import varlen_gqa_attention_paged_gb300 as ua
            ua.tree_mask(s["parents"], s["cu"], s["sl"], max_seqlen_q=s["max_q"], mask=s["mask"],
                         positions=s["pos"])
            s["step"](q=s["q"], out=s["out"], tree_mask=s["mask"])
        else:
            _tree_mask(s)
            s["out"] = _attend(s)
        return {"mask": s["mask"], "positions": s["pos"], "out": s["out"]}
    if own:
        s["step"](q=s["q"], out=s["out"])
    else:
        s["out"] = _attend(s)
    return s["out"]


def _places(s):
    """Of every new token: its sequence and its place in the cache."""
    cu, sl = s["cu"].long(), s["sl"].long()
    tok = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return seq, sl[seq] - cu[seq + 1] + tok


def _rotated(x, cos, sin, interleaved):
    x = x.float()
    half = x.shape[-1] // 2
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else \
        (slice(0, half), slice(half, None))
    y = torch.empty_like(x)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _append(s):
    c, l, r, bs = s["c"], s["c"]["latent"], s["c"]["rope"], s["c"]["bs"]
    seq, at = _places(s)
    blk = s["bt"].long()[seq, at // bs]
    cs = s["table"][at]
    cos, sin = cs[:, :r // 2], cs[:, r // 2:]
    x = s["lat"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * s["weight"].float()
    k = _rotated(s["k_rope"], cos, sin, c["interleaved"])
    s["cache"][blk, at % bs] = torch.cat([y, k], -1).to(s["cache"].dtype)
    s["q_out"].copy_(_rotated(s["q"], cos[:, None], sin[:, None], c["interleaved"]))


def _tree_mask(s):
    """Every token's ancestors: its parent's bits are joined as often as the tree may be deep."""
    seq, _ = _places(s)
    first = s["cu"].long()[seq]
    own_bit = torch.arange(first.numel(), device=_DEV) - first
    up = s["parents"].long()
    bits = torch.zeros((first.numel(), s["max_q"]), dtype=torch.bool, device=_DEV)
    bits.scatter_(1, own_bit[:, None], True)
    at, depth = up, torch.zeros_like(up)
    for _ in range(s["max_q"] - 1):
        has = at >= 0
        depth += has
        bits.scatter_(1, torch.where(has, at, own_bit)[:, None], True)
        at = torch.where(has, up[first + at.clamp(min=0)], at)
    words = torch.nn.functional.pad(bits, (0, -s["max_q"] % 32)).reshape(bits.shape[0], -1, 32)
    value = (words.long() << torch.arange(32, device=_DEV)).sum(-1)
    s["mask"].copy_(torch.where(value >= 1 << 31, value - (1 << 32), value))
    sl, cu = s["sl"].long(), s["cu"].long()
    s["pos"].copy_(sl[seq] - (cu[seq + 1] - cu[seq]) + depth)


def _attend(s):
    c, bt, cu, sl = s["c"], s["bt"].long(), s["cu"].long(), s["sl"].long()
    h, l = c["h"], c["latent"]
    n, mq = bt.shape[0], s["max_q"]
    k = s["cache"][bt].float().reshape(n, -1, l + c["rope"])         # [n, keys, width]
    i = torch.arange(mq, device=cu.device)
    rows = torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1)        # padded to max_q
    q = s["q"][rows].float().reshape(n, mq * h, -1)
    x = q @ k.transpose(1, 2)
    x *= s["scale"]
    x = x.reshape(n, mq, h, -1)
    j = torch.arange(x.shape[-1], device=cu.device)
    ctx = sl - cu[1:] + cu[:-1]
    if c["op"] == "tree":
        bit = j - ctx[:, None]                                       # [n, keys]
        new = (bit >= 0) & (j < sl[:, None])
        at = bit.clamp(0, mq - 1)
        word = s["mask"][rows].long().gather(2, (at // 32)[:, None].expand(-1, mq, -1))
        sees = (word >> (at % 32)[:, None]) & 1 > 0
        hide = ~((bit < 0)[:, None] | (new[:, None] & sees))
    else:
        hide = j > (ctx[:, None] + i)[..., None]                     # [n, max_q, keys]
    x.masked_fill_(hide[:, :, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    y = (x.reshape(n, mq * h, -1) @ k[..., :l]).reshape(n, mq, h, l) / total
    seq, _ = _places(s)
    row = torch.arange(seq.numel(), device=cu.device) - cu[seq]
    return y[seq, row].to(s["q"].dtype)


def _prefill(s):
    """One sequence after the other: ragged ones share no shape."""
    c = s["c"]
    n, r = c["nope"], c["rope"]
    out, lse = [], []
    q0 = k0 = 0
    for nq, nk in s["lens"]:
        q = s["q"][q0:q0 + nq].float().transpose(0, 1)               # [h, q, n + r]
        kv = s["kv"][k0:k0 + nk].float().permute(1, 2, 0)            # [h, n + v, k]
        x = q[..., :n] @ kv[:, :n]
        x += q[..., n:] @ s["k_rope"][k0:k0 + nk].float().T
        x *= s["scale"]
        j, i = torch.arange(nk, device=_DEV), torch.arange(nk - nq, nk, device=_DEV)
        x.masked_fill_(j > i[:, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x -= top
        x.exp_()
        total = x.sum(-1, keepdim=True)
        y = x @ kv[:, n:].transpose(1, 2) / total
        out.append(y.transpose(0, 1))
        lse.append((top + torch.log(total))[..., 0].T)
        q0, k0 = q0 + nq, k0 + nk
    return torch.cat(out).to(s["q"].dtype), torch.cat(lse)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "prefill": _exact_prefill}.get(c["op"], _exact_attend)(s)


def _exact_append(s):
    c, l, r, bs = s["c"], s["c"]["latent"], s["c"]["rope"], s["c"]["bs"]
    freq = torch.tensor([_BASE ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64,
                        device=_DEV)
    cache, qo = s["cache"].double(), torch.empty(s["q"].shape, dtype=torch.float64, device=_DEV)
    for b, (n, kv) in enumerate(s["lens"]):
        r0 = int(s["cu"][b])
        at = torch.arange(kv - n, kv, device=_DEV)
        z = torch.polar(torch.ones((), dtype=torch.float64, device=_DEV), at[:, None] * freq)

        def turn(x, z):
            x = x.double()
            pair = x.unflatten(-1, (-1, 2)) if c["interleaved"] else \
                x.unflatten(-1, (2, -1)).transpose(-1, -2)
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            return (w if c["interleaved"] else w.transpose(-1, -2)).flatten(-2)

        qo[r0:r0 + n] = turn(s["q"][r0:r0 + n], z[:, None])
        x = s["lat"][r0:r0 + n].double()
        norm = torch.sqrt(x.square().sum(-1, keepdim=True) / l + _EPS)
        page, slot = s["bt"][b, at // bs].long(), at % bs
        cache[page, slot, :l] = x / norm * s["weight"].double()
        cache[page, slot, l:] = turn(s["k_rope"][r0:r0 + n], z)
    return {"q_rope": qo, "cache": cache}


def _exact_attend(s):
    c, bs, l = s["c"], s["c"]["bs"], s["c"]["latent"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=_DEV)
    words, place = [], []
    for b, (n, kv) in enumerate(s["lens"]):
        r0 = int(s["cu"][b])
        pages = s["bt"][b, :(kv + bs - 1) // bs].long()
        k = s["cache"][pages].flatten(0, 1)[:kv].double()
        see = torch.ones((n, kv), dtype=torch.bool, device=_DEV)
        if c["op"] == "tree":
            line = []       # of every token, its line of descent
            for i, p in enumerate(s["parents"][r0:r0 + n].tolist()):
                line.append((line[p] if p >= 0 else []) + [i])
            pick = torch.zeros((n, n), dtype=torch.bool)
            for i, a in enumerate(line):
                pick[i, a] = True
                bits = sum(1 << x for x in a)
                word = [bits >> 32 * w & 0xffffffff for w in range(s["mask"].shape[1])]
                words.append([w - (w >> 31 << 32) for w in word])
                place.append(kv - n + len(a) - 1)
            see[:, kv - n:] = pick.to(_DEV)
        else:
            see = see.tril(kv - n)
        for h in range(c["h"]):
            x = (s["q"][r0:r0 + n, h].double() @ k.T) * s["scale"]
            out[r0:r0 + n, h] = torch.softmax(x.masked_fill(~see, -math.inf), -1) @ k[:, :l]
    if c["op"] != "tree":
        return out
    return {"mask": torch.tensor(words, dtype=torch.int32, device=_DEV),
            "positions": torch.tensor(place, dtype=torch.int32, device=_DEV), "out": out}


def _exact_prefill(s):
    c = s["c"]
    n = c["nope"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.empty(s["out"].shape[:2], dtype=torch.float64, device=_DEV)
    q0 = k0 = 0
    for nq, nk in s["lens"]:
        for h in range(c["h"]):
            k = torch.cat([s["kv"][k0:k0 + nk, h, :n], s["k_rope"][k0:k0 + nk]], -1).double()
            x = (s["q"][q0:q0 + nq, h].double() @ k.T) * s["scale"]
            hide = torch.ones_like(x, dtype=torch.bool).triu(nk - nq + 1)
            x = x.masked_fill(hide, -math.inf)
            lse[q0:q0 + nq, h] = torch.logsumexp(x, -1)
            out[q0:q0 + nq, h] = torch.softmax(x, -1) @ s["kv"][k0:k0 + nk, h, n:].double()
        q0, k0 = q0 + nq, k0 + nk
    return {"out": out, "lse": lse} if c["lse"] else out
