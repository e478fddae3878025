"""Cases of the cache-writing and 8-bit-cache operators, for measuring them.

Three operators of one serving step, each in its plain form (``own`` false: elementary
torch operations in 32 bits) and as a user calls it (``own`` true: the package):

* ``append``: new keys and values go into the paged cache at their sequence's end, the
  keys rotated by their position on the way, the queries rotated beside them.  The cache is
  16-bit, e4m3 with one scale a tensor, or e4m3 with one scale a token.  Positions have one
  axis (text) or three (time, height and width of image and video tokens).
* ``append`` into a cache held in 8 bits (``e4m3_blk``, ``i8_blk``) with one K and one V
  scale for each block of tokens and kv-head: a block's scale grows with its tokens, and the
  codes it already holds are rounded again when it does.
* ``attend``: attention over such a cache.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program has in hand before the
call, ``run()`` makes one pass, ``work()`` counts what the pass cannot do without and
``exact()`` is the definition in 64 bits, one sequence at a time.
"""
import math

import torch

own = False

_DEV = "cuda"
_QMAX = {"e4m3": 448.0, "i8": 127.0}
_LO, _HI = 2.0 ** -40, 2.0 ** 40        # the range of a block's or a token's scale
_HALF = {"bf16": torch.bfloat16, "f16": torch.float16}
_BASE = 10000.0


def _case(name, op, nseq, q, kv, **over):
    c = dict(name=name, op=op, nseq=nseq, q=q, kv=kv, ragged=False, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", cache="bf16", rot=0, interleaved=False, axes=1, window=0, sinks=False,
             softcap=0.0)
    c.update(over)
    return c


def listed():
    return [
        # one decode step of a small batch: every sequence adds its newest token
        _case("append_decode", "append", 8, 1, 6700, rot=128),
        # prompts of a prefill step
        _case("append_prompts", "append", 4, 4096, 4096, rot=128),
        # a ragged step of an fp8 server: 256-wide heads, half of each rotated, in pairs
        _case("append_fp8_d256", "append", 5, 1500, 2500, ragged=True, hq=24, hkv=4, d=256,
              cache="e4m3", rot=128, interleaved=True),
        # images among text: three position axes
        _case("append_axes", "append", 7, 700, 900, ragged=True, rot=128, axes=3),
        # video tokens, one scale a token
        _case("append_video_tok", "append", 2, 8192, 8192, dtype="f16", cache="e4m3_tok", rot=128,
              axes=3),
        # one decode step of a large batch over a block-scaled cache
        _case("append_blk_decode", "append", 64, 1, 1500, ragged=True, cache="e4m3_blk", rot=128),
        # chunks behind prefixes into an int8 cache, odd lengths
        _case("append_blk_chunks", "append", 6, 1999, 3001, ragged=True, cache="i8_blk", rot=128,
              bs=32),
        # one token of one short conversation: the smallest attention call
        _case("attend_one", "attend", 1, 1, 300, hq=16, hkv=2, d=64, cache="i8_blk"),
        # sliding-window decode with sinks, batch 8
        _case("attend_window_decode", "attend", 8, 1, 6700, cache="e4m3_blk", window=4096,
              sinks=True),
        # long decode of a large batch over int8
        _case("attend_long_decode", "attend", 48, 1, 8191, ragged=True, cache="i8_blk", bs=64),
        # prompts behind a prefix of the same length
        _case("attend_prompts", "attend", 2, 4096, 8192, cache="e4m3_blk"),
        # a ragged mix of chunks with 256-wide heads and a softcap, int8
        _case("attend_chunks_d256", "attend", 3, 1501, 2999, ragged=True, hq=24, hkv=4, d=256,
              cache="i8_blk", dtype="f16", softcap=30.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    c = _case("", "append", 1, 1, 1, hkv=hkv, hq=hkv * rng.choice([1, 2, 4, 6, 8]), d=d,
              bs=rng.choice([16, 16, 32, 64, 24]), dtype=rng.choice(["bf16", "f16"]),
              ragged=rng.random() < 0.75)
    if rng.random() < 0.55:
        c["cache"] = rng.choice([c["dtype"], "e4m3", "e4m3_tok", "e4m3_blk", "i8_blk", "i8_blk"])
        c["rot"] = rng.choice([d, d, d // 2])
        c["interleaved"] = rng.random() < 0.4
        c["axes"] = rng.choice([1, 3])
        tokens = _log_int(rng, 1, 12000)
    else:
        c["op"] = "attend"
        c["cache"] = rng.choice(["e4m3_blk", "i8_blk"])
        c["window"] = rng.choice([0, 0, rng.randint(100, 3000)])
        c["sinks"] = rng.random() < 0.3
        c["softcap"] = rng.choice([0.0, 0.0, 30.0])
        tokens = _log_int(rng, 1, 4000)
    if rng.random() < 0.4:                  # a decode step
        c["nseq"] = _log_int(rng, 1, 64)
        c["q"] = rng.choice([1, 1, 1, 2, 3])
        c["kv"] = max(c["q"], _log_int(rng, 1, 8000))
    else:
        c["nseq"] = min(tokens, rng.randint(1, 6))
        c["q"] = max(1, tokens // c["nseq"])
        c["kv"] = c["q"] + rng.choice([0, rng.randint(0, 2500)])
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


def _kind(c):
    """(code type or None, scale form) of the cache."""
    t, _, form = c["cache"].partition("_")
    return (t, form or "tensor") if t in _QMAX else (None, "")


def _sections(c):
    """Frequencies of each position axis: a quarter for time, the rest for height and width."""
    n = c["rot"] // 2
    if c["axes"] == 1:
        return [n]
    t = n // 4
    return [t, (n - t) // 2, n - t - (n - t) // 2]


def work(c):
    lens, d, hq, hkv, bs = _lens(c), c["d"], c["hq"], c["hkv"], c["bs"]
    t, form = _kind(c)
    esz = 1 if t else 2
    tokens = sum(q for q, _ in lens)
    if c["op"] == "append":
        pages = sum((kv + bs - 1) // bs - (kv - q) // bs for q, kv in lens)
        b = tokens * d * (2 * hkv * (2 + esz) + 2 * hq * 2)      # k, v in and out; q in and out
        b += pages * 4 + 2 * hkv * 4 * (tokens if form == "tok" else pages if form == "blk" else 0)
        b += max(kv for _, kv in lens) * c["rot"] * 4 * (1 if c["axes"] == 1 else 0)
        b += tokens * 4 * (c["axes"] if c["axes"] > 1 else 0)
        f = tokens * (hq + hkv) * c["rot"] * 3 + (tokens * 2 * hkv * d * 2 if t else 0)
        return {"bytes": b, "flops": f}
    keys = pairs = pages = 0
    for q, kv in lens:
        w = c["window"] or kv + 1
        first = max(0, kv - q + 1 - w)
        keys += kv - first
        pages += (kv + bs - 1) // bs - first // bs
        ctx = kv - q
        full = max(0, min(q, w - 1 - ctx))          # rows that see every key before them
        pairs += full * ctx + full * (full + 1) // 2 + (q - full) * w
    return {"bytes": keys * hkv * d * 2 + pages * (4 + 8 * hkv) + tokens * hq * d * 4,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the inputs

def _angles(pos, rot):
    """Angles of positions, in 64 bits: pos * base^(-2 i / rot)."""
    i = torch.arange(rot // 2, device=pos.device, dtype=torch.float64)
    return pos.double()[..., None] * torch.exp(i * (-2.0 * math.log(_BASE) / rot))


def _codes(x, t):
    if t == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.round(x).clamp(-127.0, 127.0).to(torch.int8)


def prepare(c, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    lens, d, hq, hkv, bs = _lens(c), c["d"], c["hq"], c["hkv"], c["bs"]
    half = _HALF[c["dtype"]]
    t, form = _kind(c)
    tokens = sum(q for q, _ in lens)
    per = [(kv + bs - 1) // bs for _, kv in lens]
    nb = int(1.25 * sum(per)) + 1

    def randn(*shape):
        return torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32)

    perm = torch.randperm(nb, generator=g, device=_DEV)
    bt = torch.zeros((len(lens), max(per)), dtype=torch.int32, device=_DEV)
    at = 0
    for i, n in enumerate(per):
        bt[i, :n] = perm[at:at + n].to(torch.int32)
        at += n
    cu = torch.tensor([0] + torch.tensor([q for q, _ in lens]).cumsum(0).tolist(),
                      dtype=torch.int32, device=_DEV)
    s = dict(c=c, lens=lens, bt=bt, cu=cu, t=t, form=form,
             sl=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=_DEV),
             max_q=max(q for q, _ in lens), max_k=max(kv for _, kv in lens))
    # keys with a few strong channels, as rotated keys have
    gain = 1.0 + 3.0 * (torch.rand(d, generator=g, device=_DEV) < 0.06).float()
    full = (nb, bs, hkv, d)
    if c["op"] == "append":
        # one projection's output holds q, k and v of a token side by side
        qkv = randn(tokens, hq + 2 * hkv, d)
        qkv[:, :hq + hkv] *= gain
        qkv = qkv.to(half)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty((tokens, hq, d), dtype=half, device=_DEV)
        if t is None:
            s["kc"], s["vc"] = torch.zeros(full, dtype=half, device=_DEV), \
                torch.zeros(full, dtype=half, device=_DEV)
        else:
            s["kc"], s["vc"] = (_codes(randn(*full) * (0.25 * _QMAX[t]), t) for _ in range(2))
        if form == "tensor":
            s["kv_scale"] = torch.tensor([16.0 / 448.0, 5.0 / 448.0], device=_DEV)
        elif form == "tok":
            s["ks"], s["vs"] = (torch.ones(full[:3], device=_DEV) for _ in range(2))
        elif form == "blk":     # blocks in use: their tokens' scales, some to be outgrown
            s["ks"], s["vs"] = ((0.3 + 0.9 * torch.rand((nb, hkv), generator=g, device=_DEV)) *
                                (m / _QMAX[t]) for m in (12.0, 4.0))
        # the rotation's table, and the tokens' positions: the cache's, or a grid of images
        pmax = s["max_k"] + 64
        a = _angles(torch.arange(pmax, device=_DEV), c["rot"])
        s["table"] = torch.cat([torch.cos(a), torch.sin(a)], -1).float()
        s["axis_of"] = [x for x, n in enumerate(_sections(c)) for _ in range(n)]
        if c["axes"] > 1:
            p = torch.cat([torch.arange(kv - q, kv, device=_DEV) for q, kv in lens])
            w = 24 + seed % 17
            s["pos"] = torch.stack([p // (w * w), p // w % w, p % w]).to(torch.int32)
        else:
            s["pos"] = None
    else:
        s["q"] = randn(tokens, hq, d).to(half)
        s["out"] = torch.empty((tokens, hq, d), dtype=half, device=_DEV)
        lift = 0.5 + torch.rand((2, nb, 1, hkv, 1), generator=g, device=_DEV)
        for n, (x, y) in enumerate((("kc", "ks"), ("vc", "vs"))):
            f = randn(*full) * lift[n]
            if n == 0:
                f *= gain
            scale = f.abs().amax((1, 3)) * (1.0 / _QMAX[t])
            s[x], s[y] = _codes(f / scale[:, None, :, None], t), scale
        s["sinks"] = randn(hq) if c["sinks"] else None
    if own:
        import varlen_gqa_attention_paged_gb300 as ua
        if c["op"] == "append":
            s["step"] = ua.prepare_append(
                s["k"], s["v"], s["kc"], s["vc"], s["cu"], s["sl"], s["bt"],
                max_seqlen_q=s["max_q"], q=s["q"], q_out=s["q_out"], cos_sin=s["table"],
                positions=s["pos"], axis_of=s["axis_of"] if c["axes"] > 1 else None,
                interleaved=c["interleaved"], kv_scale=s.get("kv_scale"),
                **({"k_scale_tok": s["ks"], "v_scale_tok": s["vs"]} if form == "tok" else
                   {"k_scale_blk": s["ks"], "v_scale_blk": s["vs"]} if form == "blk" else {}))
        else:
            s["step"] = ua.prepare(
                s["q"], s["kc"], s["vc"], s["cu"], s["sl"], s["bt"], max_seqlen_q=s["max_q"],
                max_seqlen_k=s["max_k"], softcap=c["softcap"],
                window_left=c["window"] - 1 if c["window"] else -1, sinks=s["sinks"],
                k_scale_blk=s["ks"], v_scale_blk=s["vs"], out=s["out"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if s["c"]["op"] == "append":
        if own:
            s["step"](q=s["q"], k=s["k"], v=s["v"], q_out=s["q_out"])
        else:
            _append(s)
        out = {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}
        if s["form"] in ("tok", "blk"):
            out["k_scale"], out["v_scale"] = s["ks"], s["vs"]
        return out
    if own:
        s["step"](q=s["q"], out=s["out"])
    else:
        s["out"] = _attend(s)
    return s["out"]


def _rotated(s, x, cos, sin):
    """x with its first `rot` elements of every head rotated in pairs, in 32 bits: each
    product and each sum rounded."""
    rot = s["c"]["rot"]
    x = x.float()
    y = x.clone()
    if s["c"]["interleaved"]:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    else:
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _append(s):
    c, bs, t, form = s["c"], s["c"]["bs"], s["t"], s["form"]
    bt, cu, sl = s["bt"].long(), s["cu"].long(), s["sl"].long()
    tok = torch.arange(s["k"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    at = sl[seq] - cu[seq + 1] + tok
    blk, slot = bt[seq, at // bs], at % bs
    half = c["rot"] // 2
    if s["pos"] is None:
        cs = s["table"][at]
        cos, sin = cs[:, None, :half], cs[:, None, half:]
    else:
        axis = torch.tensor(s["axis_of"], device=cu.device)
        p = s["pos"].long()[axis].T                                  # [tokens, half]
        i = torch.arange(half, device=cu.device)
        cos, sin = s["table"][p, i][:, None], s["table"][p, i + half][:, None]
    s["q_out"].copy_(_rotated(s, s["q"], cos, sin))
    k, v = _rotated(s, s["k"], cos, sin), s["v"].float()
    if t is None:
        s["kc"][blk, slot], s["vc"][blk, slot] = k.to(s["kc"].dtype), v.to(s["vc"].dtype)
    elif form == "tensor":
        inv = 1.0 / s["kv_scale"]
        s["kc"][blk, slot], s["vc"][blk, slot] = _codes(k * inv[0], t), _codes(v * inv[1], t)
    elif form == "tok":
        _append_tok(s["kc"], s["ks"], k, blk, slot, t)
        _append_tok(s["vc"], s["vs"], v, blk, slot, t)
    else:
        _append_blk(s["kc"], s["ks"], k, blk, slot, s, t)
        _append_blk(s["vc"], s["vs"], v, blk, slot, s, t)


def _append_tok(cache, scales, x, blk, slot, t):
    """Every token and head by its own largest magnitude."""
    scale = (x.abs().amax(-1) * (1.0 / _QMAX[t])).clamp(_LO, _HI)
    cache[blk, slot] = _codes(x * (1.0 / scale)[..., None], t)
    scales[blk, slot] = scale


def _append_blk(cache, scales, x, blk, slot, s, t):
    """Every block and head by its tokens' largest magnitude: the scale of a block that holds
    tokens already only grows, and its codes are then rounded again."""
    nb, bs, hkv, d = cache.shape
    cu, sl = s["cu"].long(), s["sl"].long()
    ctx = sl - (cu[1:] - cu[:-1])                                    # tokens held before
    first = s["bt"].long().gather(1, (ctx // bs)[:, None])[:, 0]     # the block they end in
    held = torch.arange(bs, device=cu.device)[None] < (ctx % bs)[:, None]
    where = blk[:, None].expand(-1, hkv)
    top = torch.zeros((nb, hkv), device=x.device)
    top = top.scatter_reduce(0, where, x.abs().amax(-1), "amax")
    new = (top * (1.0 / _QMAX[t])).clamp(_LO, _HI)
    old = scales[first].clamp(_LO, _HI)
    new[first] = torch.where(held[:, :1], torch.maximum(new[first], old), new[first])
    codes = cache[first]
    ratio = (old / new[first])[:, None, :, None]
    again = _codes(codes.float() * ratio, t)
    raw = torch.uint8
    cache.view(raw)[first] = torch.where(held[:, :, None, None], again.view(raw), codes.view(raw))
    touched = torch.zeros((nb, hkv), device=x.device).scatter(0, where, 1.0) > 0
    scales.copy_(torch.where(touched, new, scales))
    cache[blk, slot] = _codes(x * (1.0 / new)[blk][..., None], t)


def _attend(s):
    c, bt, cu, sl = s["c"], s["bt"].long(), s["cu"].long(), s["sl"].long()
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    n, m = bt.shape
    grp = hq // hkv

    def gather(cache, scales):
        x = cache[bt].float() * scales[bt][:, :, None, :, None]
        return x.reshape(n, -1, hkv, d).transpose(1, 2)              # [n, hkv, keys, d]

    k, v = gather(s["kc"], s["ks"]), gather(s["vc"], s["vs"])
    i = torch.arange(s["max_q"], device=cu.device)
    rows = torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1)        # padded to max_q
    q = s["q"][rows].float().reshape(n, -1, hkv, grp, d).permute(0, 2, 3, 1, 4)
    x = q.reshape(n, hkv, -1, d) @ k.transpose(2, 3)
    x *= 1.0 / math.sqrt(d)
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    x = x.reshape(n, hkv, grp, s["max_q"], -1)
    j = torch.arange(x.shape[-1], device=cu.device)
    pos = (sl - cu[1:] + cu[:-1])[:, None] + i                       # [n, max_q]
    hide = (j > pos[..., None]) | (j >= sl[:, None, None])
    if c["window"]:
        hide |= j <= pos[..., None] - c["window"]
    x.masked_fill_(hide[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    if c["sinks"]:
        sink = s["sinks"].reshape(hkv, grp, 1, 1)
        top = torch.maximum(top, sink)
    x -= top
    x.exp_()
    total = x.sum(-1, keepdim=True)
    if c["sinks"]:
        total = total + torch.exp(sink - top)
    y = x.reshape(n, hkv, -1, x.shape[-1]) @ v
    y = y.reshape(n, hkv, grp, -1, d) / total
    seq = torch.searchsorted(cu[1:], torch.arange(s["q"].shape[0], device=cu.device), right=True)
    row = torch.arange(s["q"].shape[0], device=cu.device) - cu[seq]
    return y.permute(0, 3, 1, 2, 4)[seq, row].reshape(-1, hq, d).to(s["q"].dtype)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return _exact_append(s) if c["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    c, t, form = s["c"], s["t"], s["form"]
    bs, rot = c["bs"], c["rot"]
    freq = [_BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    freq = torch.tensor(freq, dtype=torch.float64, device=_DEV)
    axis = torch.tensor(s["axis_of"], device=_DEV)
    qo = torch.empty(s["q"].shape, dtype=torch.float64, device=_DEV)
    kc, vc = s["kc"].double(), s["vc"].double()
    ks, vs = (s[x].double() if form in ("tok", "blk") else None for x in ("ks", "vs"))
    for b, (n, kv) in enumerate(s["lens"]):
        r0, ctx = int(s["cu"][b]), kv - n
        at = torch.arange(ctx, kv, device=_DEV)
        p = s["pos"][:, r0:r0 + n].double() if s["pos"] is not None else at.double()[None]
        z = torch.polar(torch.ones((), dtype=torch.float64, device=_DEV),
                        p[axis].T * freq)[:, None]

        def turn(x):
            x = x[r0:r0 + n].double()
            head = x[..., :rot]
            pair = head.unflatten(-1, (-1, 2)) if c["interleaved"] else \
                head.unflatten(-1, (2, -1)).transpose(-1, -2)
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            w = w if c["interleaved"] else w.transpose(-1, -2)
            return torch.cat([w.flatten(-2), x[..., rot:]], -1)

        qo[r0:r0 + n] = turn(s["q"])
        blk, slot = s["bt"][b, at // bs].long(), at % bs
        for i, (x, cache, scales) in enumerate(((turn(s["k"]), kc, ks),
                                                (s["v"][r0:r0 + n].double(), vc, vs))):
            if t is None:
                cache[blk, slot] = x
            elif form == "tensor":
                cache[blk, slot] = _exact_codes(x / s["kv_scale"][i].double(), t)
            elif form == "tok":
                scale = (x.abs().amax(-1) / _QMAX[t]).clamp(_LO, _HI)
                scales[blk, slot] = scale
                cache[blk, slot] = _exact_codes(x / scale[..., None], t)
            else:
                for page in range(ctx // bs, (kv - 1) // bs + 1):
                    lo, hi = max(ctx, page * bs), min(kv, (page + 1) * bs)
                    y, phys, keep = x[lo - ctx:hi - ctx], int(s["bt"][b, page]), lo - page * bs
                    scale = (y.abs().amax((0, 2)) / _QMAX[t]).clamp(_LO, _HI)
                    if keep:
                        before = scales[phys].clamp(_LO, _HI)
                        scale = torch.maximum(scale, before)
                        cache[phys, :keep] = _exact_codes(
                            cache[phys, :keep] * (before / scale)[:, None], t)
                    scales[phys] = scale
                    cache[phys, keep:keep + hi - lo] = _exact_codes(y / scale[:, None], t)
    out = {"q": qo, "k_cache": None if t == "i8" else kc, "v_cache": None if t == "i8" else vc}
    if ks is not None:
        out["k_scale"], out["v_scale"] = ks, vs
    return out


def _exact_codes(x, t):
    """The nearest code, ties to even: steps of 1, or of e4m3's 2^-3 below each power of two
    (2^-9 below 2^-6)."""
    x = x.clamp(-_QMAX[t], _QMAX[t])
    if t == "i8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(x / step) * step


def _exact_attend(s):
    c, bs = s["c"], s["c"]["bs"]
    grp = c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=_DEV)
    for b, (n, kv) in enumerate(s["lens"]):
        pages = s["bt"][b, :(kv + bs - 1) // bs].long()
        r0 = int(s["cu"][b])
        at = torch.arange(kv - n, kv, device=_DEV)[:, None]
        j = torch.arange(kv, device=_DEV)[None]
        see = j <= at
        if c["window"]:
            see &= at - j < c["window"]
        for g in range(c["hkv"]):
            k, v = ((s[x][pages, :, g].double() * s[y][pages, g].double()[:, None, None])
                    .flatten(0, 1)[:kv] for x, y in (("kc", "ks"), ("vc", "vs")))
            for h in range(g * grp, (g + 1) * grp):
                x = s["q"][r0:r0 + n, h].double() @ k.T / math.sqrt(c["d"])
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                x = x.masked_fill(~see, -math.inf)
                if c["sinks"]:
                    sink = s["sinks"][h].double().expand(n, 1)
                    w = torch.softmax(torch.cat([x, sink], -1), -1)[:, :-1]
                else:
                    w = torch.softmax(x, -1)
                out[r0:r0 + n, h] = w @ v
    return out
