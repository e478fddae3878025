"""GPU: append_kv and unified_attention together, as a serving loop runs them.

Prompts in chunks, then single tokens, some of the steps as one captured graph that is
replayed on new values.  The reference keeps its own caches on the CPU: each step's tokens are
rotated and appended by the plain fp32 definition, whose 16-bit queries, cache bits, codes and
scales the operator gives bit for bit; the attention is a dense 64-bit softmax over what those
caches stand for.

Bar of the fp32 output: weights are rounded to u = 2^-11 of themselves where the products run
in f16 (f16 caches and 8-bit codes) and 2^-8 in bf16, which moves a weighted mean by at most
u max |v|; scores are off by at most e = scale 2^-16 max|q| max_j sum_d |k_jd|, which moves the
quotient by twice that; 2^-17 covers the fp32 exponentials and sums.
"""
import math

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _append_ref as R
from tests._dense import dense_attention

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
BF, F16 = torch.bfloat16, torch.float16

CHUNKS = [[130, 40, 1, 7, 0], [61, 1, 1, 300, 5], [1, 1, 17, 1, 0]]
DECODE = 5


class Loop:
    def __init__(self, hq, hkv, d, bs, dtype, cache, form, rot, axes, interleaved, seed):
        self.cfg = dict(hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype, cache=cache, form=form, rot=rot,
                        axes=axes, interleaved=interleaved)
        self.seed = seed
        self.kv = [0] * len(CHUNKS[0])
        self.most = [sum(c[b] for c in CHUNKS) + DECODE for b in range(len(self.kv))]
        c = R.make(R.Case([(0, m) for m in self.most], seed=seed, max_position=1000, **self.cfg))
        self.names = [n for n in ("k_cache", "v_cache", "k_scale_tok", "v_scale_tok",
                                  "k_scale_blk", "v_scale_blk") if n in c.t]
        self.state = {n: c.t[n] for n in self.names}
        self.fixed = {n: c.t[n] for n in ("block_table", "cos_sin")}
        self.axis_of = c.t.get("axis_of")
        self.dev = {n: x.cuda() for n, x in {**self.state, **self.fixed}.items()}

    def tokens(self, lens):
        """A step's rows and lengths, on the CPU."""
        self.seed += 1
        self.kv = [a + n for a, n in zip(self.kv, lens)]
        c = R.make(R.Case(list(zip(lens, self.kv)), seed=self.seed, max_position=1000,
                          **self.cfg))
        c.t.update({**self.state, **self.fixed})
        if self.axis_of is not None:
            c.t["axis_of"] = self.axis_of
        return c

    def step_args(self, c):
        return {n: c.t[n].cuda() for n in ("q", "k", "v", "cu_seqlens_q", "seq_lens_k",
                                           "positions") if n in c.t}

    def append_kw(self, s):
        kw = {n: self.dev[n] for n in self.names if "scale" in n}
        kw.update(cos_sin=self.dev["cos_sin"], interleaved=self.cfg["interleaved"])
        if "positions" in s:
            kw.update(positions=s["positions"], axis_of=self.axis_of)
        return kw

    def attend_kw(self):
        return {**{n: self.dev[n] for n in self.names if "scale" in n},
                "scale": 1.0 / math.sqrt(self.cfg["d"])}

    def check(self, c, q_out, out):
        """Moves the reference on by the step and compares."""
        form, dt = self.cfg["form"], self.cfg["dtype"]
        new = R.append(c, torch.float32)
        for n in self.names:
            want = new[n] if "cache" in n else new[n[0] + "_scale"]
            self.state[n] = want.to(self.state[n].dtype)
            assert torch.equal(self.dev[n].cpu().float(), self.state[n].float()), n
        total = int(c.t["cu_seqlens_q"][-1])
        q = new["q_out"][:total].to(dt)
        assert torch.equal(q_out[:total].cpu(), q)
        vals = []
        for n in ("k", "v"):
            x = self.state[f"{n}_cache"].double()
            if form == "tok":
                x = x * self.state[f"{n}_scale_tok"].double()[..., None]
            if form == "blk":
                x = x * self.state[f"{n}_scale_blk"].double()[:, None, :, None]
            vals.append(x)
        scale = 1.0 / math.sqrt(self.cfg["d"])
        bt = self.fixed["block_table"]
        want = torch.from_numpy(dense_attention(q, *vals, c.t["cu_seqlens_q"],
                                                c.t["seq_lens_k"], bt, scale=scale))
        own = bt[bt >= 0].long()
        k, v = vals[0][own], vals[1][own]
        e = scale * 2.0 ** -16 * float(q.abs().max()) * float(k.abs().sum(-1).max())
        u = 2.0 ** -8 if self.cfg["cache"] is None and dt == BF else 2.0 ** -11
        room = float(v.abs().max()) * (u + 2 * e + 2.0 ** -17)
        err = float((out[:total].cpu().double() - want).abs().max())
        assert err <= room, f"max abs err {err:.3e}, bar {room:.3e}"


CASES = [
    (8, 2, 128, 16, BF, I8, "blk", 128, 1, False),
    (8, 2, 128, 16, BF, E4M3, "blk", 128, 3, False),
    (6, 2, 64, 32, F16, I8, "blk", 32, 1, True),
    (16, 1, 256, 64, BF, E4M3, "blk", 64, 1, False),
    (4, 4, 256, 16, F16, I8, "blk", 256, 4, True),
    (8, 2, 128, 16, BF, E4M3, "tok", 64, 1, False),
    (8, 2, 128, 16, BF, None, "", 128, 3, False),
    (8, 8, 64, 24, F16, None, "", 64, 1, True),
]


def ids(c):
    return f"{c[0]}x{c[1]}-d{c[2]}-bs{c[3]}-{str(c[5] or c[4]).split('.')[-1]}{c[6]}-a{c[8]}"


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_append_then_attend(case):
    loop = Loop(*case, seed=3)
    for lens in CHUNKS:
        c = loop.tokens(lens)
        s = loop.step_args(c)
        q = torch.empty_like(s["q"])
        got = ua.append_kv(s["k"], s["v"], loop.dev["k_cache"], loop.dev["v_cache"],
                           s["cu_seqlens_q"], s["seq_lens_k"], loop.dev["block_table"],
                           max_seqlen_q=max(lens), q=s["q"], q_out=q, **loop.append_kw(s))
        assert got is q
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        ua.unified_attention(q, loop.dev["k_cache"], loop.dev["v_cache"], s["cu_seqlens_q"],
                             s["seq_lens_k"], loop.dev["block_table"], max_seqlen_q=max(lens),
                             max_seqlen_k=max(loop.kv), out=out, **loop.attend_kw())
        torch.cuda.synchronize()
        loop.check(c, q, out)

    # single tokens: both calls in one graph, on a stream of its own, replayed on new values
    ones = [1] * len(loop.kv)
    c = loop.tokens(ones)
    s = loop.step_args(c)
    q = torch.empty_like(s["q"])
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    put = ua.prepare_append(s["k"], s["v"], loop.dev["k_cache"], loop.dev["v_cache"],
                            s["cu_seqlens_q"], s["seq_lens_k"], loop.dev["block_table"],
                            max_seqlen_q=1, q=s["q"], q_out=q, stream=stream,
                            **loop.append_kw(s))
    read = ua.prepare(q, loop.dev["k_cache"], loop.dev["v_cache"], s["cu_seqlens_q"],
                      s["seq_lens_k"], loop.dev["block_table"], max_seqlen_q=1,
                      max_seqlen_k=max(loop.most), out=out, stream=stream, **loop.attend_kw())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        put()
        read()
    graph.replay()
    torch.cuda.synchronize()
    loop.check(c, q, out)
    for _ in range(DECODE - 1):
        c = loop.tokens(ones)
        for n, x in loop.step_args(c).items():
            s[n].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        loop.check(c, q, out)
