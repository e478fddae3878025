"""GPU: long prompts whose scores run into the thousands (ALiBi far from the chunk's first token),
on every tensor-memory prefill kernel, against sampled rows of a dense 64-bit softmax.

The bar of the fp32 output: out = sum w v / sum w with weights off by u relatively (2^-11 where
P is f16, 2^-8 where it is bf16) moves by at most u max |v|; a score off by e moves the quotient
by at most twice e max |v|.  e has two parts: the products' (scale 2^-16 max|q| max_j sum_d |k_jd|:
fp32 sums of up to 256 products), and the bias': slope times distance, added in fp32, is rounded
three times at its magnitude A = slope q_len (half a step: 2^-24 A each); the softmax's factor
and subtraction are one FMA whose own rounding is relative to the small difference.  2^-17 covers
the exponential and the sums."""
import math

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
BF, F16 = torch.bfloat16, torch.float16
SLOPES = (0.84, 0.0625)
Q = 6500
BS = 16


def build(d, kind, seed, window, hq=2, hkv=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = math.ceil(Q / BS) + 2
    half = F16 if kind == "f16" else BF
    q = (torch.randn((Q, hq, d), generator=g, device="cuda")).to(half)
    k, v = (torch.randn((nb, BS, hkv, d), generator=g, device="cuda") for _ in range(2))
    kw = {}
    if kind in ("e4m3", "e4m3_blk", "i8_blk"):
        if kind == "e4m3":
            kw["kv_scale"] = torch.tensor([0.02, 0.015], device="cuda")
            ks, vs = (kw["kv_scale"][i].expand(nb, hkv) for i in range(2))
        else:
            qmax = 127.0 if kind == "i8_blk" else 448.0
            ks, vs = (x.abs().amax((1, 3)) / qmax for x in (k, v))
            kw.update(k_scale_blk=ks, v_scale_blk=vs)
        k, v = (x / s[:, None, :, None] for x, s in ((k, ks), (v, vs)))
        k, v = ((x.round().clamp(-127, 127).to(I8) if kind == "i8_blk" else
                 x.clamp(-448, 448).to(E4M3)) for x in (k, v))
        kd, vd = (x.double() * s.double()[:, None, :, None] for x, s in ((k, ks), (v, vs)))
    else:
        k, v = k.to(half), v.to(half)
        kd, vd = k.double(), v.double()
    bt = torch.randperm(nb, generator=g, device="cuda")[None].to(torch.int32)
    i = dict(dtype=torch.int32, device="cuda")
    args = (q, k, v, torch.tensor([0, Q], **i), torch.tensor([Q], **i), bt.contiguous())
    kw.update(alibi_slopes=torch.tensor(SLOPES[:hq], device="cuda"), window_left=window)
    flat = [x[bt[0].long()].flatten(0, 1)[:Q] for x in (kd, vd)]
    return args, kw, flat


def sampled(q, flat, window, scale):
    rows = torch.cat([torch.arange(0, Q, 61), torch.arange(Q - 40, Q)]).cuda()
    k, v = flat
    want = torch.empty((len(rows), q.shape[1], q.shape[2]), dtype=torch.float64, device="cuda")
    j = torch.arange(Q, device="cuda")
    for h in range(q.shape[1]):
        slope = float(torch.tensor(SLOPES[h]))          # as the kernel has it, in 32 bits
        x = scale * (q[rows, h].double() @ k[:, h].T) + slope * j.double()
        hide = j > rows[:, None]
        if window >= 0:
            hide |= j < rows[:, None] - window
        want[:, h] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v[:, h]
    return rows, want


CASES = [(256, "e4m3_blk"), (256, "i8_blk"), (256, "bf16"), (256, "f16"), (256, "e4m3"),
         (128, "e4m3_blk"), (128, "i8_blk"), (128, "bf16"), (128, "f16"), (128, "e4m3"),
         (64, "e4m3_blk"), (64, "i8_blk"), (64, "bf16"), (64, "f16"), (64, "e4m3")]


@pytest.mark.parametrize("window", [-1, 900])
@pytest.mark.parametrize("backend", ["2d", "split"])
@pytest.mark.parametrize("d,kind", CASES)
def test_alibi_far_from_the_first_token(d, kind, backend, window):
    args, kw, flat = build(d, kind, d + len(kind), window)
    q, k, v = args[:3]
    plan = ua.plan(num_seqs=1, total_q=Q, max_seqlen_q=Q, max_seqlen_k=Q, block_size=BS,
                   num_q_heads=2, num_kv_heads=2, head_dim=d, window_left=window,
                   kv_dtype=ua._DTYPES[k.dtype], q_dtype=ua._DTYPES[q.dtype], backend=backend,
                   num_blocks=k.shape[0], per_block_scales=kind.endswith("blk"))
    assert plan["kernel"] == 8                                   # one q tile a CTA
    scale = 0.25 / math.sqrt(d)
    ua.device_status_reset()
    out = ua.unified_attention(*args, max_seqlen_q=Q, max_seqlen_k=Q, scale=scale,
                               out_dtype=torch.float32, backend=backend, **kw)
    rows, want = sampled(q, flat, window, scale)
    assert ua.device_status() == 0
    e = scale * 2.0 ** -16 * float(q.abs().max()) * float(flat[0].abs().sum(-1).max())
    e += 3.0 * SLOPES[0] * Q * 2.0 ** -24
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    room = float(flat[1].abs().max()) * (u + 2.0 * e + 2.0 ** -17)
    err = (out[rows].double() - want).abs().amax((1, 2))
    assert float(err.max()) <= room, (float(err.max()), room, int(rows[err.argmax()]))
