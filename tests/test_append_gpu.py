"""GPU: append_kv against its plain reference.

8-bit caches: codes and scales equal the fp32 reference's bit for bit (every operation of
the operator rounds on its own), slots, blocks and scales that no new token reaches keep
their bits, and what the codes stand for lies within half a step of the 64-bit definition.
16-bit caches and rotated queries: within half a unit of the type (eps / 2 relative) plus the
fp32 arithmetic's error: two products and a sum, each off by at most 2^-24 of its magnitude,
with |cos|, |sin| <= 1, so below 2^-22 (|a| + |b|) for a pair (a, b).
"""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _append_ref as R

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
BF, F16 = torch.bfloat16, torch.float16


def to_dev(c):
    """The case's tensors on the GPU with their strides kept (slices of one projection stay
    slices); the caches are copies."""
    d = {}
    for n, x in c.t.items():
        if isinstance(x, torch.Tensor):
            base = x._base if x._base is not None else x
            d[n] = base.cuda().as_strided(x.shape, x.stride(), x.storage_offset())
        else:
            d[n] = x
    return d


def kwargs(c, d):
    kw = {n: d[n] for n in ("cos_sin", "positions", "axis_of", "kv_scale", "k_scale_tok",
                            "v_scale_tok", "k_scale_blk", "v_scale_blk") if n in d}
    kw.update(max_seqlen_q=max([q for q, _ in c.lens] + [0]), interleaved=c.interleaved)
    if c.with_q:
        kw["q"] = d["q"]
    return kw


ARGS = ("k", "v", "k_cache", "v_cache", "cu_seqlens_q", "seq_lens_k", "block_table")


def run(c, d, **over):
    kw = kwargs(c, d)
    kw.update(over)
    if c.with_q and "q_out" not in kw:
        kw["q_out"] = torch.full(tuple(d["q"].shape), 7.0, dtype=c.dtype, device="cuda")
    out = ua.append_kv(*(d[n] for n in ARGS), **kw)
    torch.cuda.synchronize()
    return out


def bits(x):
    return x.contiguous().view(torch.uint8 if x.element_size() == 1 else
                               torch.int16 if x.element_size() == 2 else torch.int32).cpu()


def check(c, d, q_out):
    want64, want32 = R.append(c, torch.float64), R.append(c, torch.float32)
    half_step = torch.finfo(c.dtype).eps / 2
    if c.with_q:
        w = want64["q_out"]
        live = ~w.isnan().any(-1).any(-1)
        got = q_out.cpu().double()
        room = 2.0 ** -22 * 2 * c.t["q"].double().abs().amax(-1, keepdim=True)
        err = (got - w).abs() - half_step * w.abs() - room
        assert (err[live] <= 0).all(), f"q: {err[live].max():.2e} over"
        assert (got[~live] == 7.0).all()                     # rows of no token stay
    for n in ("k", "v"):
        before, after = c.t[f"{n}_cache"], d[f"{n}_cache"].cpu()
        w64, w32 = want64[f"{n}_cache"], want32[f"{n}_cache"]
        if not c.form:
            changed = (w64 != before.double()).any(-1)
            room = 2.0 ** -22 * 2 * float(c.t[n].double().abs().max())
            err = (after.double() - w64).abs() - half_step * w64.abs() - room
            assert (err[changed] <= 0).all()
            assert torch.equal(bits(after)[~changed], bits(before)[~changed])
            continue
        assert torch.equal(after.float(), w32), f"{n}: {(after.float() != w32).sum()} codes"
        untouched = (w32 == before.float()).all(-1)
        assert torch.equal(bits(after)[untouched], bits(before)[untouched])
        if c.form != "tensor":
            s = d[f"{n}_scale_{c.form}"].cpu()
            assert torch.equal(s, want32[f"{n}_scale"])
            rel = (s.double() / want64[f"{n}_scale"] - 1).abs().max()
            assert rel <= 2.0 ** -21                          # fp32 rounding of the rotation


ODD = [(1, 37), (5, 18), (0, 9), (16, 16), (33, 33), (1, 1), (7, 103), (0, 0), (2, 17)]

CASES = []
for i, (cache, form) in enumerate([(None, ""), (E4M3, "tensor"), (E4M3, "tok"), (E4M3, "blk"),
                                   (I8, "blk")]):
    for d in (64, 128, 256):
        for dt in (BF, F16):
            s = 10 * i + d // 64 + (dt == F16)
            CASES.append(R.Case(ODD, d=d, dtype=dt, cache=cache, form=form, seed=s,
                                rot=(d, d // 2, 16)[s % 3], interleaved=bool(s % 2),
                                axes=(1, 3, 4)[(s // 2) % 3], pad=s % 4,
                                hq=(8, 5, 2)[s % 3], hkv=(2, 5, 1)[s % 3],
                                bs=(16, 16, 32, 64, 13, 1)[s % 6], fused=s % 3 != 0,
                                scale_strides=s % 2 == 1))
            CASES.append(R.Case(ODD, d=d, dtype=dt, cache=cache, form=form, seed=s + 100, rot=0,
                                hq=4, hkv=4, bs=(128, 24, 16)[s % 3], with_q=s % 2 == 0))


@pytest.mark.parametrize("c", CASES, ids=str)
def test_append_matches_the_reference(c):
    R.make(c)
    d = to_dev(c)
    ua.device_status_reset()
    check(c, d, run(c, d))
    assert ua.device_status() == 0


DECODE = [(1, 1 + 53 * i % 211) for i in range(70)] + [(0, 12), (1, 16), (1, 17)]


@pytest.mark.parametrize("cache,form", [(None, ""), (E4M3, "tensor"), (E4M3, "tok"),
                                        (E4M3, "blk"), (I8, "blk")])
@pytest.mark.parametrize("bs", [16, 48])
def test_append_decode_step(cache, form, bs):
    c = R.make(R.Case(DECODE, hq=32, hkv=8, d=128, bs=bs, cache=cache, form=form, rot=128,
                      seed=bs))
    d = to_dev(c)
    check(c, d, run(c, d))


@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 5000)], [(1200, 1203)], [(3, 3)] * 40,
                                  [(0, 0), (0, 5), (1, 8)]], ids=str)
@pytest.mark.parametrize("cache,form", [(None, ""), (I8, "blk")])
def test_append_lengths(lens, cache, form):
    c = R.make(R.Case(lens, hq=4, hkv=1, d=128, cache=cache, form=form, rot=64, seed=5))
    d = to_dev(c)
    check(c, d, run(c, d))


@pytest.mark.parametrize("cache,form", [(None, ""), (I8, "blk")])
def test_append_thousands_of_sequences(cache, form):
    """The search for a token's and a page's sequence in several rounds, empty ones between."""
    lens = [((3 * i * i) % 4 if i % 7 else 0, 1 + i % 23) for i in range(2100)]
    lens = [(min(q, kv), kv) for q, kv in lens] + [(0, 5)] * 40
    c = R.make(R.Case(lens, hq=2, hkv=1, d=64, bs=16, cache=cache, form=form, rot=64, seed=4))
    d = to_dev(c)
    check(c, d, run(c, d))


@pytest.mark.parametrize("cache,form", [(None, ""), (E4M3, "tok"), (I8, "blk")])
def test_tokens_before_the_cache_are_skipped(cache, form):
    """kv_len < q_len (a padded slot): the tokens at negative positions write nothing."""
    c = R.make(R.Case([(1, 0), (6, 4), (2, 2), (40, 3)], cache=cache, form=form, rot=64, seed=9))
    d = to_dev(c)
    check(c, d, run(c, d))
    assert ua.device_status() == 0


@pytest.mark.parametrize("cache,form", [(E4M3, "blk"), (I8, "blk")])
def test_block_scale_extremes(cache, form):
    """Zeros, and magnitudes past both ends of the scales' range."""
    c = R.make(R.Case([(16, 16), (3, 20), (16, 16), (16, 16)], cache=cache, form=form, seed=3))
    c.t["k"][:16] = 0.0
    c.t["v"][:16] = 0.0
    c.t["k"][19:35] *= 2.0 ** -60
    c.t["v"][35:] = (c.t["v"][35:].float() * 2.0 ** 60).to(c.dtype)
    d = to_dev(c)
    check(c, d, run(c, d))
    assert torch.equal(d["k_scale_blk"].cpu()[int(c.t["block_table"][0, 0])],
                       torch.full((c.hkv,), 2.0 ** -40))


@pytest.mark.parametrize("cache,form", [(None, ""), (E4M3, "blk"), (I8, "blk")])
def test_append_twice_is_the_same(cache, form):
    c = R.make(R.Case(ODD, cache=cache, form=form, rot=64, seed=4))
    d = to_dev(c)
    run(c, d)
    once = {n: bits(d[n]) for n in ("k_cache", "v_cache")}
    run(c, d)
    for n, x in once.items():
        assert torch.equal(bits(d[n]), x)


def test_queries_in_place_and_without_rotation():
    for rot in (0, 64):
        c = R.make(R.Case(ODD, rot=rot, seed=6))
        d = to_dev(c)
        out = run(c, d, q_out=d["q"])
        assert out is d["q"]
        check(c, d, out)


def test_bad_blocks_are_not_written():
    for cache, form in ((None, ""), (E4M3, "tok"), (I8, "blk")):
        c = R.make(R.Case([(4, 20), (4, 4)], cache=cache, form=form, rot=64, seed=7))
        d = to_dev(c)
        before = {n: bits(d[n]) for n in ("k_cache", "v_cache")}
        d["block_table"][0, 1] = c.t["k_cache"].shape[0]
        d["block_table"][1, 0] = -5
        ua.device_status_reset()
        out = run(c, d)
        assert ua.device_status() == ua._lib.UA_ERR_DEVICE_CHECK
        for n, x in before.items():
            assert torch.equal(bits(d[n]), x)
        assert torch.isfinite(out.float()).all() and not (out == 7.0).all(-1).any()
        ua.device_status_reset()


def test_positions_outside_the_table_skip_their_token():
    for cache, form in ((None, ""), (E4M3, "tok"), (I8, "blk")):
        c = R.make(R.Case([(4, 4), (3, 35)], cache=cache, form=form, rot=64, own_positions=True,
                          seed=8))
        d = to_dev(c)
        d["positions"][1] = -1
        d["positions"][5] = c.t["cos_sin"].shape[0]
        before = {n: d[n].clone() for n in ("k_cache", "v_cache")}
        ua.device_status_reset()
        out = run(c, d)
        assert ua.device_status() == ua._lib.UA_ERR_DEVICE_CHECK
        ua.device_status_reset()
        assert (out[[1, 5]] == 7.0).all() and not (out[[0, 2, 3, 4, 6]] == 7.0).all(-1).any()
        blk = int(c.t["block_table"][0, 0])
        for n, x in before.items():
            assert torch.equal(bits(d[n][blk, 1]), bits(x[blk, 1]))
            assert not torch.equal(bits(d[n][blk, 0]), bits(x[blk, 0]))


def test_prepared_and_captured():
    """A prepared call on another stream, captured, replayed on new tensors' values."""
    c = R.make(R.Case([(1, 5 + 7 * i) for i in range(9)], hq=8, hkv=4, d=128, cache=I8, form="blk",
                      rot=128, seed=11))
    d = to_dev(c)
    first = {n: d[n].clone() for n in ("k_cache", "v_cache", "k_scale_blk", "v_scale_blk")}
    q_out = torch.full(tuple(d["q"].shape), 7.0, dtype=c.dtype, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    step = ua.prepare_append(*(d[n] for n in ARGS), q_out=q_out, stream=stream, **kwargs(c, d))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for n, x in first.items():
        d[n].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    check(c, d, q_out)
    # new values in the captured tensors
    c2 = R.make(R.Case(c.lens, hq=8, hkv=4, d=128, cache=I8, form="blk", rot=128, seed=12))
    d2 = to_dev(c2)
    for n in ("q", "k", "v", "k_cache", "v_cache", "k_scale_blk", "v_scale_blk", "block_table"):
        d[n].copy_(d2[n])
    graph.replay()
    torch.cuda.synchronize()
    check(c2, d, q_out)
    # and the prepared call with other tensors, eagerly
    d3 = to_dev(c)
    q3 = torch.full_like(q_out, 7.0)
    for n, x in first.items():
        d[n].copy_(x)
    stream.wait_stream(torch.cuda.current_stream())
    out = step(q=d3["q"], k=d3["k"], v=d3["v"], block_table=d3["block_table"], q_out=q3)
    torch.cuda.synchronize()
    assert out is q3
    check(c, d, q3)
    with pytest.raises(ValueError):
        step(k=d3["k"][:-1])
    with pytest.raises(ValueError):
        step(positions=torch.zeros(9, dtype=torch.int32, device="cuda"))


def test_a_large_cache_is_addressed_in_64_bits():
    """A block past 2^31 elements and one past 2^32 bytes of the cache."""
    nb, bs, hkv, d = 1 << 18, 16, 8, 128                     # 2^32 elements
    kc = torch.zeros((nb, bs, hkv, d), dtype=I8, device="cuda")
    vc = torch.zeros((nb, bs, hkv, d), dtype=I8, device="cuda")
    ks = torch.ones((nb, hkv), device="cuda")
    vs = torch.ones((nb, hkv), device="cuda")
    k = torch.randn((3, hkv, d), device="cuda").to(BF)
    v = torch.randn((3, hkv, d), device="cuda").to(BF)
    i32 = dict(dtype=torch.int32, device="cuda")
    bt = torch.tensor([[nb - 1], [nb // 2 + 1], [1]], **i32)
    ua.append_kv(k, v, kc, vc, torch.arange(4, **i32), torch.tensor([1, 3, 16], **i32), bt,
                 max_seqlen_q=1, k_scale_blk=ks, v_scale_blk=vs)
    torch.cuda.synchronize()
    for b, slot in ((0, 0), (1, 2), (2, 15)):
        blk = int(bt[b, 0])
        for x, cache, scales in ((k, kc, ks), (v, vc, vs)):
            got = cache[blk, slot].double() * scales[blk].double()[:, None]
            step = scales[blk].double()[:, None]
            # half a step, and the fp32 product with the reciprocal: 127 * 2^-23 of one
            assert ((got - x[b].double()).abs() <= step * (0.5 + 127 * 2.0 ** -22)).all()
    assert int((kc[:1] != 0).sum()) == 0
    assert int((kc != 0).any(-1).any(-1).sum()) == 3


def test_refusals():
    c = R.make(R.Case([(4, 20), (4, 4)], cache=I8, form="blk", rot=64, axes=3, seed=7))
    d = to_dev(c)

    def call(err, **over):
        a = {n: d[n] for n in ARGS} | kwargs(c, d) | over
        pos = [a.pop(n) for n in ARGS]
        with pytest.raises(err):
            ua.append_kv(*pos, **a)

    call(ValueError, k=d["k"].cpu())
    call(ValueError, v=d["v"][:, :1])
    call(ValueError, k=d["k"].transpose(1, 2).contiguous().transpose(1, 2))
    call(ValueError, v=d["v"].to(F16))
    call(ValueError, k_cache=d["k_cache"][:, :, :1])
    call(ValueError, v_cache=d["v_cache"].to(BF))
    call(ValueError, block_table=d["block_table"].long())
    call(ValueError, seq_lens_k=d["seq_lens_k"][:1])
    call(ValueError, cos_sin=d["cos_sin"][:, :40].contiguous())
    call(ValueError, cos_sin=d["cos_sin"].double())
    call(ValueError, cos_sin=None)
    call(ValueError, axis_of=None)
    call(ValueError, axis_of=[0] * 31)
    call(ValueError, axis_of=[3] * 32)
    call(ValueError, positions=d["positions"].long())
    call(ValueError, positions=d["positions"][:, :-1])
    call(ValueError, v_scale_blk=None)
    call(ValueError, k_scale_blk=d["k_scale_blk"][:-1])
    call(ua.UaError, k_scale_blk=None, v_scale_blk=None)         # int8 needs block scales
    call(ua.UaError, kv_scale=torch.ones(2, device="cuda"))      # two forms of scales
    bf = {n: torch.zeros(d[n].shape, dtype=BF, device="cuda") for n in ("k_cache", "v_cache")}
    call(ua.UaError, **bf)                                       # scales with a 16-bit cache
    f16 = {n: torch.zeros(d[n].shape, dtype=F16, device="cuda") for n in ("k_cache", "v_cache")}
    call(ua.UaError, k_scale_blk=None, v_scale_blk=None, **f16)  # bf16 k, f16 cache
    call(ValueError, q=None, q_out=d["q"])
    call(ValueError, q_out=d["q"][:, :1])
    # outputs that overlap themselves: one row for all tokens, one scale for all heads
    call(ua.UaError, q_out=torch.empty_like(d["q"][:1]).expand_as(d["q"]))
    call(ua.UaError, q_out=torch.empty_like(d["q"][:, :1]).expand_as(d["q"]))
    for n in ("k_scale_blk", "v_scale_blk"):
        call(ua.UaError, **{n: d[n][:, :1].contiguous().expand(-1, d[n].shape[1])})
        call(ua.UaError, **{n: d[n][:1].contiguous().expand_as(d[n])})
    assert ua.device_status() == 0
