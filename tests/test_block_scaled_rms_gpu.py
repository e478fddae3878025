"""GPU: attention over block-scaled caches, the rms of the error against the rms of the output.

An output is a mean of n values of either sign, so its size falls as 1 / sqrt(n), and so must the
error's; a bound by the largest value would not see one that does not.  What the kernels may lose,
relative to the output's rms, for scores of a few units and values whose signs do not follow the
weights:
  * each weight is rounded to f16 for P V: uniform within half a step, so 2^-11 / sqrt(3) of a
    weight at most (at the bottom of its binade) in the rms, and the same in a sum of independent
    terms.  A tile whose maximum grows rounds its first keys' weights twice: few of n;
  * 2^-13 for all else: scores (q as e4m3 terms keeps 2^-17 of its largest value, 2^-15 in the
    rms of a score here), the approximate exponential, logarithm and reciprocal (2^-22 each), and
    the fp32 sums of P V, whose roundings are independent (2^-24 of a running sum that exceeds
    the result by sqrt(n / 64) at most where int8 codes carry an offset that is taken off again
    every few tiles).
The reference is a dense 64-bit softmax over the dequantised cache, on sampled rows."""
import math

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
BF, F16 = torch.bfloat16, torch.float16
BAR = 2.0 ** -11 / math.sqrt(3.0) + 2.0 ** -13


def build(seqs, hq, hkv, d, bs, code, q_dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = [math.ceil(kv / bs) for _, kv in seqs]
    nb = sum(per) + 1
    total = sum(q for q, _ in seqs)
    q = torch.randn((total, hq, d), generator=g, device="cuda").to(q_dtype)
    qmax = 127.0 if code == I8 else 448.0
    lift = torch.exp2(2.0 * torch.rand((2, nb, 1, hkv, 1), generator=g, device="cuda") - 1.0)
    caches, scales = [], []
    for i in range(2):
        x = torch.randn((nb, bs, hkv, d), generator=g, device="cuda") * lift[i]
        s = x.abs().amax((1, 3)) / qmax
        x = x / s[:, None, :, None]
        caches.append(x.round().to(I8) if code == I8 else x.clamp(-448, 448).to(E4M3))
        scales.append(s)
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    bt = torch.zeros((len(seqs), max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        bt[b, :n] = perm[at:at + n]
        at += n
    i = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + torch.tensor([n for n, _ in seqs]).cumsum(0).tolist(), **i)
    return q, caches, scales, cu, torch.tensor([kv for _, kv in seqs], **i), bt


def errors(seqs, q, caches, scales, bt, bs, out):
    """Per sequence: the error's rms over the output's, over sampled rows."""
    hq, d = q.shape[1:]
    hkv = caches[0].shape[2]
    worst, r0 = 0.0, 0
    for b, (n, kv) in enumerate(seqs):
        rows = torch.unique(torch.linspace(0, n - 1, min(n, 24)).long()).cuda()
        pages = bt[b, :math.ceil(kv / bs)].long()
        pos = kv - n + rows
        hide = torch.arange(kv, device="cuda") > pos[:, None]
        num = den = 0.0
        for h in range(hkv):
            k, v = ((c[pages, :, h].double() * s[pages, h].double()[:, None, None])
                    .flatten(0, 1)[:kv] for c, s in zip(caches, scales))
            for x in range(h * hq // hkv, (h + 1) * hq // hkv):
                s = q[r0 + rows, x].double() @ k.T / math.sqrt(d)
                want = torch.softmax(s.masked_fill(hide, -math.inf), -1) @ v
                num += float(((out[r0 + rows, x].double() - want) ** 2).sum())
                den += float((want ** 2).sum())
        worst = max(worst, math.sqrt(num / den))
        r0 += n
    return worst


LONG = [(1, 9000), (1, 4001), (1, 8191)]
FORMS = {
    # name: (sequences, query heads, kv-heads, head dims, page, call options, plan's kernel)
    "pair": (LONG, 8, 2, (64, 128), 16, dict(backend="2d"), 64),
    "pair_split": (LONG, 8, 2, (64, 128), 32, dict(backend="split", num_splits=6), 64),
    "eight_rows": (LONG * 30, 24, 3, (64, 128, 256), 64, dict(backend="2d"), 2),
    "wide": (LONG, 24, 3, (64, 128, 256), 16, dict(backend="2d"), 32),
    "share": ([(1, 500 + 1301 * i % 8000) for i in range(40)], 32, 8, (64, 128, 256), 16, {}, 128),
    "sixteen_rows": (LONG, 32, 2, (64, 128, 256), 16, dict(backend="2d"), 1),
    "odd_pages": (LONG, 8, 2, (64, 128, 256), 24, dict(backend="2d"), 1),
    "one_tile": ([(100, 9000), (33, 4001)], 8, 2, (64, 128, 256), 16, dict(backend="2d"), 8),
    "two_tiles": ([(5000, 9000), (6000, 6000)], 32, 8, (64, 128), 16, {}, 16),
    "odd_prompts": ([(100, 9000), (33, 4001)], 8, 2, (64, 128, 256), 40, dict(backend="2d"), 4),
    "longest": ([(1, 131072)], 8, 2, (64, 128), 64, dict(backend="2d"), 64),
    "longest_wide": ([(1, 131072)], 8, 1, (128, 256), 64, dict(backend="2d"), 32),
}


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("form,d", [(n, d) for n, f in FORMS.items() for d in f[3]])
def test_the_error_falls_as_the_output_does(form, d, code):
    seqs, hq, hkv, _, bs, opt, kernel = FORMS[form]
    q_dtype = BF if d == 128 else F16
    q, caches, scales, cu, sl, bt = build(seqs, hq, hkv, d, bs, code, q_dtype, d + len(form))
    mq, mk = max(n for n, _ in seqs), max(kv for _, kv in seqs)
    plan = ua.plan(num_seqs=len(seqs), total_q=q.shape[0], max_seqlen_q=mq, max_seqlen_k=mk,
                   block_size=bs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                   kv_dtype=ua._DTYPES[code], q_dtype=ua._DTYPES[q_dtype], per_block_scales=True,
                   num_blocks=caches[0].shape[0], max_blocks_per_seq=bt.shape[1], **opt)
    assert plan["kernel"] == kernel
    ua.device_status_reset()
    out = ua.unified_attention(q, *caches, cu, sl, bt, max_seqlen_q=mq, max_seqlen_k=mk,
                               k_scale_blk=scales[0], v_scale_blk=scales[1],
                               out_dtype=torch.float32, **opt)
    err = errors(seqs, q, caches, scales, bt, bs, out)
    assert ua.device_status() == 0
    print(f"{form} d{d} {err:.2e}")
    assert err <= BAR, f"rms error {err:.2e} of the output's rms, bar {BAR:.2e}"
