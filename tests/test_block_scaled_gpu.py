"""GPU: attention over e4m3 and int8 caches with a scale for each block and kv-head, against a
dense 64-bit softmax over the dequantised cache.

Slots that no sequence owns are poisoned (e4m3 NaN codes, int8 -128, NaN scales of unused
blocks).  The bar, for the fp32 output: with weights w and values v, out = sum w v / sum w.
The kernels round each weight to f16 (half a step: 2^-11 of it), so the sum moves by at most
2^-11 max |v|; a score is off by at most e = scale 2^-16 max|q| max_j sum_d |k_jd| (q as e4m3
terms keeps 2^-17 of its row's largest magnitude; fp32 sums of up to 256 products lose
256 * 2^-24 = 2^-16 at most of the same sum), which moves a weight by the factor e^e and the
quotient by twice that.  Softcap, ALiBi and QQ-bias terms are O(10) numbers in fp32: 2^-17
covers their roundings and the exponential's.
"""
import ctypes
import math

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
import workloads as W
from tests._dense import dense_attention

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
BF, F16 = torch.bfloat16, torch.float16
QMAX = {E4M3: 448.0, I8: 127.0}


def make(seqs, *, hq=8, hkv=2, d=128, bs=16, q_dtype=BF, code=E4M3, seed=0, pad_rows=0,
         scale_spread=0.0, v_gain=1.0, q_gain=1.0, sinks=False, alibi=False, qq_bias=False,
         softcap=0.0, window=None):
    g = torch.Generator().manual_seed(seed)
    per = [math.ceil(kv / bs) for _, kv in seqs]
    nb = sum(per) + 3
    total = sum(q for q, _ in seqs)
    t = {"q": (torch.randn((total + pad_rows, hq, d), generator=g) * q_gain).to(q_dtype)}
    perm = torch.randperm(nb, generator=g)
    bt = torch.zeros((len(seqs), max(per + [1])), dtype=torch.int32)
    used = torch.zeros((nb, bs), dtype=torch.bool)
    at = 0
    for b, n in enumerate(per):
        bt[b, :n] = perm[at:at + n].to(torch.int32)
        for i in range(n):
            used[perm[at + i], :min(bs, seqs[b][1] - i * bs)] = True
        at += n
    t["block_table"] = bt
    for n, gain in (("k", 1.0), ("v", v_gain)):
        x = torch.randn((nb, bs, hkv, d), generator=g) * gain
        if n == "v" and scale_spread:
            x *= torch.exp2((torch.rand((nb, 1, hkv, 1), generator=g) * 2 - 1) * scale_spread)
        s = x.abs().amax((1, 3)) / QMAX[code]
        y = x / s[:, None, :, None]
        t[f"{n}_cache"] = y.round().to(I8) if code == I8 else y.clamp(-448, 448).to(E4M3)
        t[f"{n}_cache"].view(torch.uint8)[~used] = 0x80 if code == I8 else 0x7F
        s[~used.any(1)] = float("nan")
        # K's scales as they are, V's laid out head first
        t[f"{n}_scale_blk"] = s if n == "k" else s.T.contiguous().T
    t["cu_seqlens_q"] = torch.tensor([0] + torch.tensor([q for q, _ in seqs]).cumsum(0).tolist(),
                                     dtype=torch.int32)
    t["seq_lens_k"] = torch.tensor([kv for _, kv in seqs], dtype=torch.int32)
    t["sinks"] = torch.randn((hq,), generator=g) if sinks else None
    t["alibi_slopes"] = W.alibi_slopes(hq) if alibi else None
    mq = max(q for q, _ in seqs)
    t["qq_bias"] = torch.randn((mq, mq + 3), generator=g) * 0.1 if qq_bias else None
    opt = dict(softcap=softcap, window_left=window - 1 if window else -1)
    return dict(t=t, opt=opt, seqs=seqs, scale=1.0 / math.sqrt(d), used=used)


def dequantised(c):
    """The caches' values in 64 bits (unused slots: 0)."""
    out = []
    for n in ("k", "v"):
        s = c["t"][f"{n}_scale_blk"].double()
        x = c["t"][f"{n}_cache"].double() * s[:, None, :, None]
        out.append(torch.where(c["used"][:, :, None, None], x, torch.zeros_like(x)))
    return out


def reference(c, kv=None):
    t = c["t"]
    k, v = kv or dequantised(c)
    qq = t["qq_bias"]
    return dense_attention(t["q"], k, v, t["cu_seqlens_q"], t["seq_lens_k"], t["block_table"],
                           scale=c["scale"], sinks=t["sinks"], alibi_slopes=t["alibi_slopes"],
                           qq_bias=qq, qq_bias_stride=None if qq is None else qq.shape[1],
                           **c["opt"])


def bar(c, kv=None):
    k, v = kv or dequantised(c)
    e = c["scale"] * 2.0 ** -16 * float(c["t"]["q"].abs().max()) * float(k.abs().sum(-1).max())
    return float(v.abs().max()) * (2.0 ** -11 + 2.0 * e + 2.0 ** -17)


def on_gpu(c):
    return {n: None if x is None else x.cuda() for n, x in c["t"].items()}


def run(c, d=None, out_dtype=torch.float32, fn=ua.unified_attention, max_k=None, **kw):
    d = d or on_gpu(c)
    rows, hq, dim = d["q"].shape
    out = torch.full((rows, hq, dim), 7.0, dtype=out_dtype, device="cuda")
    args = (d["q"], d["k_cache"], d["v_cache"], d["cu_seqlens_q"], d["seq_lens_k"],
            d["block_table"])
    got = fn(*args, max_seqlen_q=max(q for q, _ in c["seqs"]),
             max_seqlen_k=max_k or max(kv for _, kv in c["seqs"]), scale=c["scale"], out=out,
             **{n: d[n] for n in ("k_scale_blk", "v_scale_blk", "sinks", "alibi_slopes",
                                  "qq_bias")}, **c["opt"], **kw)
    if fn is ua.prepare:
        return got
    torch.cuda.synchronize()
    return got


def check(c, out, kv=None):
    want = torch.from_numpy(reference(c, kv))
    total = int(c["t"]["cu_seqlens_q"][-1])
    got = out[:total].cpu().double()
    assert torch.isfinite(got).all()
    err, room = float((got - want[:total]).abs().max()), bar(c, kv)
    assert err <= room, f"max abs err {err:.3e}, bar {room:.3e}"
    assert (out[total:] == 7.0).all()


def planned(c, max_k=None, **kw):
    t = c["t"]
    code = ua._DTYPES[t["k_cache"].dtype]
    nb, bs, hkv, d = t["k_cache"].shape
    return ua.plan(num_seqs=len(c["seqs"]), total_q=t["q"].shape[0],
                   max_seqlen_q=max(q for q, _ in c["seqs"]),
                   max_seqlen_k=max_k or max(kv for _, kv in c["seqs"]), block_size=bs,
                   num_q_heads=t["q"].shape[1], num_kv_heads=hkv, head_dim=d,
                   window_left=c["opt"]["window_left"], kv_dtype=code,
                   q_dtype=ua._DTYPES[t["q"].dtype], max_blocks_per_seq=t["block_table"].shape[1],
                   num_blocks=nb, per_block_scales=True, **kw)


DECODE = [(1, 1), (1, 16), (1, 17), (1, 300), (0, 40), (1, 1025), (1, 0)]
CHUNKS = [(1, 1), (37, 37), (129, 400), (0, 7), (1, 90), (64, 65), (5, 2)]
SHAPES = {
    # one to four rows a kv-head, an even number of kv-heads; an odd one; five to eight rows
    "decode4": dict(seqs=DECODE, hq=16, hkv=4),
    "decode3_odd": dict(seqs=DECODE, hq=9, hkv=3),
    "decode8": dict(seqs=DECODE, hq=16, hkv=2),
    "decode_many": dict(seqs=[(1, 20 + 31 * i) for i in range(30)], hq=32, hkv=8),
    # nine to sixteen rows, several tokens
    "decode16": dict(seqs=DECODE, hq=32, hkv=2),
    "drafts": dict(seqs=[(3, 50), (2, 700), (3, 3), (1, 4)], hq=8, hkv=2),
    "chunks": dict(seqs=CHUNKS, hq=8, hkv=2),
    "chunks_g3": dict(seqs=CHUNKS, hq=6, hkv=2),
    "one_head": dict(seqs=[(200, 333)], hq=1, hkv=1),
}
ODD_PAGES = {"decode4": 13, "decode8": 1, "chunks": 24, "drafts": 40, "one_head": 7}
FEATURES = {
    "plain": {},
    "window_sinks": dict(window=100, sinks=True),
    "capped": dict(softcap=20.0, alibi=True, qq_bias=True, sinks=True),
}


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("feat", FEATURES)
@pytest.mark.parametrize("shape", SHAPES)
def test_block_scales_match_the_definition(shape, feat, d, code):
    seed = d + len(shape) + len(feat)
    c = make(**SHAPES[shape], **FEATURES[feat], d=d, code=code, seed=seed, pad_rows=seed % 3,
             q_dtype=BF if seed % 2 else F16, bs=(16, 32, 64)[seed % 3], scale_spread=3.0)
    ua.device_status_reset()
    check(c, run(c))
    assert ua.device_status() == 0


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("shape", ODD_PAGES)
def test_block_scales_with_any_block_size(shape, d, code):
    c = make(**SHAPES[shape], d=d, code=code, seed=d, bs=ODD_PAGES[shape], sinks=True,
             scale_spread=3.0)
    check(c, run(c))


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("shape", ["decode4", "decode3_odd", "decode16", "chunks"])
@pytest.mark.parametrize("splits", [2, 7, 20])
def test_block_scales_split(shape, splits, code):
    """Every merge: in the cluster, and (20 partitions, or chunks) through the scratch; some
    partitions of the short sequences hold no key, and partition 0 the sink."""
    c = make(**SHAPES[shape], code=code, sinks=True, seed=splits, scale_spread=3.0)
    check(c, run(c, backend="split", num_splits=splits))


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("shape", ["decode4", "decode8", "decode16", "chunks"])
def test_block_scales_far_from_one(shape, d, code):
    """Values of 2^-36, and of 2^30, with sinks of ordinary size: what counts is relative."""
    for gain in (2.0 ** -30, 2.0 ** 38):
        c = make(**SHAPES[shape], d=d, code=code, v_gain=gain, sinks=True, seed=3)
        s = c["t"]["v_scale_blk"]
        assert ((s >= 2.0 ** -40) & (s <= 2.0 ** 40) | s.isnan()).all()
        check(c, run(c))


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("shape", ["decode4", "decode8", "decode16", "chunks"])
def test_block_scales_far_apart(shape, code):
    """Blocks whose V scales differ by up to 2^40."""
    c = make(**SHAPES[shape], code=code, scale_spread=20.0, sinks=True, seed=4)
    check(c, run(c))


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
def test_scales_outside_the_range_are_taken_at_its_ends(code):
    c = make([(1, 40), (1, 33)], hq=8, hkv=2, code=code, seed=5)
    for n in ("k", "v"):
        s = c["t"][f"{n}_scale_blk"]
        s[c["t"]["block_table"][1, 0]] = 0.0
        s[c["t"]["block_table"][1, 1]] = 1e-30
    d = on_gpu(c)
    for n in ("k", "v"):
        c["t"][f"{n}_scale_blk"] = c["t"][f"{n}_scale_blk"].clamp(2.0 ** -40, 2.0 ** 40)
    check(c, run(c, d))


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("shape", ["decode4", "decode16", "chunks"])
def test_16bit_outputs(shape, code):
    for dt in (BF, F16):
        c = make(**SHAPES[shape], code=code, q_dtype=dt, seed=6)
        want = torch.from_numpy(reference(c))
        got = run(c, out_dtype=dt).cpu().double()
        room = bar(c) + torch.finfo(dt).eps / 2 * want.abs()
        assert ((got - want).abs() <= room).all()


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("shape,splits", [("decode4", 0), ("decode16", 20), ("chunks", 3)])
def test_prepared_captured_and_twice_the_same(shape, splits, code):
    c = make(**SHAPES[shape], code=code, sinks=True, seed=8)
    d = on_gpu(c)
    stream = torch.cuda.Stream()
    need = planned(c, backend="split" if splits else "auto", num_splits=splits)["workspace_bytes"]
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    step = run(c, d, fn=ua.prepare, stream=stream, workspace=ws,
               backend="split" if splits else "auto", num_splits=splits)
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    once = step.out.clone()
    check(c, once)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    step.out.fill_(7.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, once)


LONG = {
    # two q tiles a CTA (at head_dim <= 128), ragged sequence ends, a chunk behind a prefix
    "prompts": dict(seqs=[(1500, 1500), (1000, 1600), (300, 300), (3, 700)], hq=16, hkv=8),
    "g3": dict(seqs=[(1400, 1400), (900, 1000), (129, 129)], hq=24, hkv=8),
}
HARD = {
    # scores of a few units; scores whose maximum climbs all along a row's walk, with each feature
    "plain": dict(),
    "steep": dict(q_gain=6.0),
    "steep_window": dict(q_gain=6.0, window=300, sinks=True),
    "steep_capped": dict(q_gain=6.0, softcap=40.0, alibi=True, sinks=True),
    "biased": dict(qq_bias=True, window=500),
}


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("feat", HARD)
@pytest.mark.parametrize("shape", LONG)
def test_block_scaled_prompts(shape, feat, d, code):
    seed = d + len(shape) + len(feat)
    c = make(**LONG[shape], **HARD[feat], d=d, code=code, seed=seed, pad_rows=1,
             q_dtype=BF if seed % 2 else F16, bs=(16, 48, 64)[seed % 3], scale_spread=3.0)
    if d <= 128:
        assert planned(c)["kernel"] == 16
    ua.device_status_reset()
    check(c, run(c))
    assert ua.device_status() == 0


RAGGED = {
    # many sequences of very different lengths, idle slots among them; a batch of 200 short
    # ones (more than a CTA's threads); one long sequence in many ranges; two heads a CTA, one,
    # and eight rows a kv-head
    "ragged": dict(seqs=[(1, 1 + 97 * i * i % 2600) for i in range(37)] + [(0, 0), (0, 9), (1, 0)],
                   hq=32, hkv=8),
    "many": dict(seqs=[(int(i % 5 != 0), 1 + i % 130) for i in range(200)], hq=8, hkv=2),
    "long": dict(seqs=[(1, 3), (1, 9000), (1, 64), (1, 65)] + [(1, 5 + i) for i in range(60)],
                 hq=4, hkv=2),
    "rows8": dict(seqs=[(2, 2 + 211 * i % 1000) for i in range(25)], hq=12, hkv=3),
    "rows5": dict(seqs=[(1, 1 + 211 * i % 1000) for i in range(60)], hq=10, hkv=2),
}


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("feat", FEATURES)
@pytest.mark.parametrize("shape,d", [(n, d) for n in RAGGED for d in (64, 128)] +
                         [("rows5", 256), ("rows8", 256)])
def test_an_even_share_of_ragged_batches(shape, feat, d, code):
    """Decode batches whose bound on kv_len makes the dispatcher cut all keys into equal ranges."""
    seed = d + len(shape) + len(feat)
    c = make(**RAGGED[shape], **FEATURES[feat], d=d, code=code, seed=seed, pad_rows=2,
             q_dtype=BF if seed % 2 else F16, bs=(16, 32, 64)[seed % 3], scale_spread=3.0)
    c["opt"]["window_left"] = 1500 if c["opt"]["window_left"] >= 0 else -1
    max_k = 40000 if c["opt"]["window_left"] < 0 else None
    if max_k or shape == "ragged":
        assert planned(c, max_k)["kernel"] == 128
    ua.device_status_reset()
    d_ = on_gpu(c)
    out = run(c, d_, max_k=max_k)
    check(c, out)
    assert torch.equal(out, run(c, d_, max_k=max_k))
    assert ua.device_status() == 0


def test_an_even_share_captured_on_a_poisoned_workspace():
    """The scratch needs no clearing, and a replayed call takes the lengths it finds."""
    c = make(**RAGGED["ragged"], d=128, code=I8, seed=5, sinks=True)
    d = on_gpu(c)
    plan = planned(c, 40000)
    assert plan["kernel"] == 128
    ws = torch.full((plan["workspace_bytes"],), 0xFF, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    step = run(c, d, fn=ua.prepare, max_k=40000, workspace=ws, stream=stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    graph.replay()
    torch.cuda.synchronize()
    check(c, step.out)
    # other lengths (all within the first ones' blocks) in the captured tensor
    c["seqs"] = [(q, kv if kv < 2 else 1 + kv // 3) for q, kv in c["seqs"]]
    c["t"]["seq_lens_k"] = torch.tensor([kv for _, kv in c["seqs"]], dtype=torch.int32)
    d["seq_lens_k"].copy_(c["t"]["seq_lens_k"])
    ws.fill_(0x7F)
    graph.replay()
    torch.cuda.synchronize()
    check(c, step.out)
    with pytest.raises(ua.UaError):
        run(c, d, max_k=40000, workspace=ws[:1024])


def test_an_even_share_of_lengths_above_the_bound():
    """max_seqlen_k only chooses the plan: a kv_len far above it is right too."""
    c = make([(1, 300)] * 239 + [(1, 60000)], hq=8, hkv=1, d=64, code=I8, seed=5)
    d = on_gpu(c)
    assert planned(c, 2000)["kernel"] == 128
    ua.device_status_reset()
    check(c, run(c, d, max_k=2000))
    assert ua.device_status() == 0


def test_a_bad_block_counts_as_zero():
    """A block id outside the cache: its keys score 0 with value 0, the status word says so."""
    for shape in (dict(seqs=[(1, 60), (1, 20)], hq=8, hkv=2),
                  dict(seqs=[(40, 60), (3, 20)], hq=8, hkv=2)):
        for code in (E4M3, I8):
            c = make(**shape, code=code, seed=9)
            d = on_gpu(c)
            d["block_table"][0, 1] = 10 ** 6
            kv = [x.clone() for x in dequantised(c)]
            for x in kv:
                x[c["t"]["block_table"][0, 1]] = 0.0
            ua.device_status_reset()
            out = run(c, d)
            assert ua.device_status() == ua._lib.UA_ERR_DEVICE_CHECK
            ua.device_status_reset()
            check(c, out, kv)


def test_refusals():
    c = make(DECODE, hq=8, hkv=2, code=I8, seed=1)
    d = on_gpu(c)

    def call(err, **over):
        kw = {n: d[n] for n in ("q", "k_cache", "v_cache", "cu_seqlens_q", "seq_lens_k",
                                "block_table", "k_scale_blk", "v_scale_blk")}
        kw.update(max_seqlen_q=1, max_seqlen_k=1025)
        kw.update(over)
        with pytest.raises(err):
            ua.unified_attention(**kw)

    call(ValueError, v_scale_blk=None)
    call(ValueError, k_scale_blk=d["k_scale_blk"].double())
    call(ValueError, k_scale_blk=d["k_scale_blk"][:, :1])
    call(ValueError, k_scale_blk=d["k_scale_blk"].cpu())
    call(ua.UaError, k_scale_blk=None, v_scale_blk=None)                 # int8 without scales
    e = {n: torch.zeros(d[n].shape, device="cuda").to(E4M3) for n in ("k_cache", "v_cache")}
    call(ua.UaError, k_scale_blk=None, v_scale_blk=None, **e)            # e4m3 without scales
    tok = torch.ones(d["k_cache"].shape[:3], device="cuda")
    call(ua.UaError, k_scale_tok=tok, v_scale_tok=tok, **e)              # two forms of scales
    assert ua.device_status() == 0


def test_block_scales_with_a_16bit_cache_are_refused():
    c = make(DECODE, hq=8, hkv=2, code=I8, seed=1)
    d = on_gpu(c)
    for n in ("k_cache", "v_cache"):
        d[n] = d[n].to(BF)
    with pytest.raises(ua.UaError):
        run(c, d)
    assert ua.device_status() == 0


def test_the_prepared_tensors_are_checked_again():
    """A tensor resized in place is not taken for the one that was prepared."""
    c = make(DECODE, hq=8, hkv=2, code=I8, seed=1)
    d = on_gpu(c)
    step = run(c, d, fn=ua.prepare)
    step(q=d["q"])
    d["seq_lens_k"].resize_(1)
    with pytest.raises(ValueError):
        step(seq_lens_k=d["seq_lens_k"])


@pytest.mark.parametrize("shape,max_k", [("ragged", 8192), ("long", 40000), ("rows8", 40000)])
def test_an_even_share_fits_the_fixed_scratch(shape, max_k):
    """The entry point that never allocates takes even-share plans: their scratch grows with the
    tokens and the ranges, not with their product."""
    c = make(**RAGGED[shape], d=128, code=I8, seed=3, sinks=True)
    d = on_gpu(c)
    assert planned(c, max_k)["kernel"] == 128
    out = torch.full(tuple(d["q"].shape), 7.0, dtype=torch.float32, device="cuda")
    sh = ua._shape(d["q"], d["k_cache"], d["block_table"], d["cu_seqlens_q"],
                   max(q for q, _ in c["seqs"]), max_k, None, ua.UA_DT_F32, 0, None, None,
                   k_scale_blk=d["k_scale_blk"], v_scale_blk=d["v_scale_blk"])
    p = ua._ptr
    _, bs, hkv, dim = d["k_cache"].shape
    rc = ua._lib.load().ua_unified_attention_noalloc(
        p(d["q"]), p(d["k_cache"]), p(d["v_cache"]), p(out), p(d["cu_seqlens_q"]),
        p(d["seq_lens_k"]), p(d["block_table"]), bs, d["q"].shape[1], hkv, dim, c["scale"], 0.0,
        -1, None, None, p(d["sinks"]), ua.UA_DT_I8, None, ua.UA_BACKEND_AUTO,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), ctypes.byref(sh))
    assert rc == 0
    torch.cuda.synchronize()
    check(c, out)
    big = ua.plan(num_seqs=60, total_q=60, max_seqlen_q=1, max_seqlen_k=131072, block_size=64,
                  num_q_heads=64, num_kv_heads=8, head_dim=128, kv_dtype=ua.UA_DT_I8,
                  num_blocks=1 << 19, max_blocks_per_seq=2048)
    assert big["kernel"] == 128
    assert big["workspace_bytes"] <= ua._lib.UA_NOALLOC_SCRATCH_BYTES


def test_two_even_shares_at_once():
    """Two streams, a workspace each (the library's own is one a stream)."""
    cs = [make(**RAGGED["ragged"], d=128, code=k, seed=8 + i) for i, k in enumerate((I8, E4M3))]
    ds = [on_gpu(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    steps = [run(c, d, fn=ua.prepare, max_k=40000, stream=s) for c, d, s in zip(cs, ds, streams)]
    for _ in range(20):
        for step in steps:
            step()
    torch.cuda.synchronize()
    for c, step in zip(cs, steps):
        check(c, step.out)


@pytest.mark.parametrize("bs", [64, 24])
@pytest.mark.parametrize("shape,max_k", [("decode4", None), ("chunks", None), ("ragged", 40000)])
def test_blocks_past_32_bits_of_a_large_cache(shape, max_k, bs):
    """Blocks that lie past 2^32 bytes of the cache, with the scales of all its blocks."""
    c = make(**{**(RAGGED if shape == "ragged" else SHAPES)[shape], "bs": bs}, d=128, code=I8,
             seed=2)
    d = on_gpu(c)
    nb, _, hkv, dim = d["k_cache"].shape
    first = 2 ** 32 // (bs * hkv * dim) + 1
    for n in ("k", "v"):
        cache = torch.zeros((first + nb, bs, hkv, dim), dtype=I8, device="cuda")
        cache[first:] = d[f"{n}_cache"]
        scales = torch.full((first + nb, hkv), float("nan"), device="cuda")
        scales[first:] = d[f"{n}_scale_blk"]
        d[f"{n}_cache"], d[f"{n}_scale_blk"] = cache, scales
    d["block_table"] += first
    check(c, run(c, d, max_k=max_k))
