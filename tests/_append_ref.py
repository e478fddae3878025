"""Plain reference of append_kv, on the CPU, one token and one block at a time (tests only).

``append(case, f)`` works in the float type ``f``: float64 is the definition; float32 rounds
every product, sum, reciprocal and quotient on its own, as the operator promises to, and
gives its codes and scales bit for bit.
"""
import math
from dataclasses import dataclass, field

import torch

import varlen_gqa_attention_paged_gb300 as ua

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
LO, HI = 2.0 ** -40, 2.0 ** 40


@dataclass
class Case:
    lens: list                      # [(q_len, kv_len), ...]
    hq: int = 8
    hkv: int = 2
    d: int = 64
    bs: int = 16
    dtype: torch.dtype = torch.bfloat16
    cache: torch.dtype = None       # None: dtype
    form: str = ""                  # scales: "", "tensor", "tok", "blk"
    rot: int = 0
    interleaved: bool = False
    axes: int = 1
    own_positions: bool = False
    pad: int = 0                    # rows behind the last sequence
    with_q: bool = True
    seed: int = 0
    fused: bool = True              # q, k, v are slices of one projection
    scale_strides: bool = False     # scales in a buffer laid out head first
    max_position: int = 0
    t: dict = field(default_factory=dict)

    def __str__(self):
        n = "" if self.cache is None else f"-{str(self.cache).split('.')[-1]}-{self.form}"
        return (f"{str(self.dtype).split('.')[-1]}{n}-d{self.d}-bs{self.bs}-r{self.rot}"
                f"{'i' if self.interleaved else ''}-a{self.axes}-{self.hq}x{self.hkv}-s{self.seed}"
                f"-n{len(self.lens)}")


def make(c: Case):
    """CPU tensors of a case, in c.t."""
    g = torch.Generator().manual_seed(c.seed)
    total = sum(q for q, _ in c.lens)
    rows = total + c.pad
    per = [max(1, math.ceil(kv / c.bs)) for _, kv in c.lens]
    nb = sum(per) + 3
    qkv = torch.randn((rows, c.hq + 2 * c.hkv, c.d), generator=g)
    qkv *= torch.exp2(torch.randint(-3, 4, (rows, c.hq + 2 * c.hkv, 1), generator=g).float())
    qkv = qkv.to(c.dtype)
    parts = [qkv[:, :c.hq], qkv[:, c.hq:c.hq + c.hkv], qkv[:, c.hq + c.hkv:]]
    if not c.fused:
        parts = [p.contiguous() for p in parts]
    t = dict(q=parts[0], k=parts[1], v=parts[2])
    cache = c.cache or c.dtype
    full = (nb, c.bs, c.hkv, c.d)
    for n in ("k_cache", "v_cache"):
        x = torch.randn(full, generator=g)
        if cache == torch.int8:
            t[n] = (x * 40).round().clamp(-127, 127).to(torch.int8)
        elif cache == torch.float8_e4m3fn:
            t[n] = (x * 100).clamp(-448, 448).to(cache)
        else:
            t[n] = x.to(cache)
    perm = torch.randperm(nb, generator=g)
    t["block_table"] = torch.full((len(c.lens), max(per) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        t["block_table"][b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    t["cu_seqlens_q"] = torch.tensor([0] + torch.tensor([q for q, _ in c.lens]).cumsum(0).tolist(),
                                     dtype=torch.int32)
    t["seq_lens_k"] = torch.tensor([kv for _, kv in c.lens], dtype=torch.int32)
    if c.form == "tensor":
        t["kv_scale"] = torch.tensor([0.043, 0.017])
    elif c.form:
        shape = full[:3] if c.form == "tok" else (nb, c.hkv)
        for n in ("k", "v"):
            s = torch.exp2(torch.rand(shape, generator=g) * 6 - 3) * (3.0 / QMAX[cache])
            if c.scale_strides:
                s = s.movedim(-1, 0).contiguous().movedim(0, -1)
            t[f"{n}_scale_{c.form}"] = s
    if c.rot:
        most = c.max_position or max([kv for _, kv in c.lens] + [1]) + 40
        t["cos_sin"] = ua.rope_table(most, c.rot, device="cpu")
        if c.axes > 1:
            t["positions"] = torch.randint(0, most, (c.axes, rows), generator=g).to(torch.int32)
            t["axis_of"] = torch.randint(0, c.axes, (c.rot // 2,), generator=g).tolist()
        elif c.own_positions:
            t["positions"] = torch.randint(0, most, (rows,), generator=g).to(torch.int32)
    c.t = t
    return c


def _turn(x, c, t, pos, f):
    """One token's heads [h, d], rotated in the float type f."""
    x = x.to(f)
    if not c.rot:
        return x
    half = c.rot // 2
    p = [int(pos)] * half
    if "positions" in t:
        own = t["positions"].reshape(c.axes, -1)
        p = [int(own[a, t["_row"]]) for a in t.get("axis_of", [0] * half)]
    cs = torch.stack([t["cos_sin"][p[i], i] for i in range(half)]).to(f)
    sn = torch.stack([t["cos_sin"][p[i], half + i] for i in range(half)]).to(f)
    ia = torch.arange(half) * (2 if c.interleaved else 1)
    ib = ia + (1 if c.interleaved else half)
    a, b = x[:, ia], x[:, ib]
    y = x.clone()
    y[:, ia] = a * cs - b * sn
    y[:, ib] = b * cs + a * sn
    return y


def codes(x, dtype):
    if dtype == torch.int8:
        return x.round().clamp(-127, 127)
    return x.clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).to(x.dtype)


def append(c: Case, f):
    """What the call leaves, in the float type f: q_out, the caches as values of f (16-bit:
    unrounded) and the scales."""
    t = dict(c.t)
    q_out = torch.full(t["q"].shape, float("nan"), dtype=f)
    cache = c.cache or c.dtype
    out = dict(q_out=q_out, k_cache=t["k_cache"].to(f), v_cache=t["v_cache"].to(f))
    for n in ("k", "v"):
        if c.form in ("tok", "blk"):
            out[f"{n}_scale"] = t[f"{n}_scale_{c.form}"].to(f).clone()
    one = torch.ones((), dtype=f)
    inv_q = (one / QMAX.get(cache, 1.0)).to(f)
    for b, (n, kv) in enumerate(c.lens):
        r0, ctx = int(t["cu_seqlens_q"][b]), kv - n
        new = {}                                   # block -> [(slot, k, v)]
        for i in range(n):
            pos = ctx + i
            if pos < 0:
                continue
            t["_row"] = r0 + i
            q_out[r0 + i] = _turn(t["q"][r0 + i], c, t, pos, f)
            blk = int(t["block_table"][b, pos // c.bs])
            new.setdefault(blk, []).append((pos % c.bs, _turn(t["k"][r0 + i], c, t, pos, f),
                                            t["v"][r0 + i].to(f)))
        for blk, rows in new.items():
            for w, name in ((1, "k"), (2, "v")):
                dst = out[f"{name}_cache"][blk]
                x = torch.stack([r[w] for r in rows])              # [rows, h, d]
                slots = [r[0] for r in rows]
                if not c.form:
                    dst[slots] = x
                elif c.form == "tensor":
                    dst[slots] = codes(x * (one / t["kv_scale"][w - 1].to(f)), cache)
                elif c.form == "tok":
                    s = (x.abs().amax(-1) * inv_q).clamp(LO, HI)
                    out[f"{name}_scale"][blk, slots] = s
                    dst[slots] = codes(x * (one / s)[..., None], cache)
                else:
                    s = (x.abs().amax((0, 2)) * inv_q).clamp(LO, HI)
                    held = slots[0]                # earlier tokens of the same sequence
                    if held:
                        old = out[f"{name}_scale"][blk].clamp(LO, HI)
                        s = torch.maximum(s, old)
                        again = codes(dst[:held] * (old / s)[None, :, None], cache)
                        grew = (s > old)[None, :, None]
                        dst[:held] = torch.where(grew, again, dst[:held])
                    out[f"{name}_scale"][blk] = s
                    dst[slots] = codes(x * (one / s)[..., None], cache)
    return out
