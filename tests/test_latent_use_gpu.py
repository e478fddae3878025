"""The latent operators as a program uses them: together, prepared, captured, on other streams, at
the edges of their sizes, and called wrongly."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
L, R, N, V = 512, 64, 128, 128


def batch(lens, bs=64, seed=0, **kw):
    cu, sl, bt, nb = ref.batch(lens, bs, seed, **kw)
    return cu.cuda(), sl.cuda(), bt.cuda(), nb


def most(lens):
    return dict(max_seqlen_q=max(q for q, _ in lens), max_seqlen_k=max(k for _, k in lens))


def rand(*shape, dtype=BF, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def check_attention(q, cache, cu, sl, bt, out, lse=None, scale=0.08, mask=None):
    cpu = [x.cpu() for x in (q, cache, cu, sl, bt)]
    want, wlse, tol, ltol = ref.attend(*cpu, q.shape[2] - R, scale,
                                       None if mask is None else mask.cpu())
    end = int(cu[-1])
    ref.check(out[:end], want[:end], tol[:end], out.dtype)
    if lse is not None:
        ref.check(lse[:end], wlse[:end], ltol[:end], F32)


# ------------------------------------------------------------------ together

class Layer:
    """Heads whose up-projections pick elements of the latent, so that both forms have the same
    keys and values to the bit."""

    def __init__(self, h, seed=0):
        self.h = h
        at = torch.arange(128)
        self.k_of = torch.stack([(37 * i + at) % L for i in range(h)]).cuda()
        self.v_of = torch.stack([(53 * i + 11 + at) % L for i in range(h)]).cuda()

    def expand(self, c):        # [t, L] -> [t, H, N + V]
        return torch.cat([c[:, self.k_of], c[:, self.v_of]], -1)

    def absorb(self, q):        # [t, H, N + R] -> [t, H, L + R]
        out = torch.zeros((q.shape[0], self.h, L + R), dtype=q.dtype, device="cuda")
        out[..., :L].scatter_(2, self.k_of.expand(q.shape[0], -1, -1), q[..., :N])
        out[..., L:] = q[..., N:]
        return out

    def values(self, o):        # [t, H, L] -> [t, H, V]
        return o.gather(2, self.v_of.expand(o.shape[0], -1, -1))


def latents_of(cache, bt, b, kv):
    bs = cache.shape[1]
    return cache[bt[b, :(kv + bs - 1) // bs].long()].flatten(0, 1)[:kv]


@pytest.mark.parametrize("dtype", [BF, F16])
def test_prompts_then_tokens_then_a_tree(dtype):
    h, table = 8, ua.rope_table(400, R)
    layer, lens = Layer(h), [37, 5, 130]
    cache = torch.full((12, 64, L + R), float("nan"), dtype=dtype, device="cuda")
    bt = torch.randperm(12, generator=torch.Generator().manual_seed(1))[:12].reshape(3, 4)
    bt = bt.int().cuda()
    w = 1 + 0.2 * rand(L, seed=9, dtype=F32)
    scale = (N + R) ** -0.5
    for step in range(5):
        new = lens if step == 0 else [6, 4, 9] if step == 4 else [1, 1, 1]
        have = [n if step == 0 else kv + n for kv, n in zip(lens, new)]
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist()).int().cuda()
        sl, total = torch.tensor(have).int().cuda(), sum(new)
        down, q = rand(total, L + R, dtype=dtype, seed=step), rand(total, h, N + R, dtype=dtype,
                                                                   seed=50 + step)
        mask = positions = None
        if step == 4:
            parents = ref.random_parents([(n, 0) for n in new], seed=3).cuda()
            mask, positions = ua.tree_mask(parents, cu, sl, max_seqlen_q=9)
        ua.append_latent(down[:, :L], down[:, L:], cache, cu, sl, bt, norm_weight=w,
                         q_rope=q[..., N:], q_rope_out=q[..., N:], cos_sin=table,
                         positions=positions)
        sizes = dict(max_seqlen_q=max(new), max_seqlen_k=max(have))
        rows = torch.cat([latents_of(cache, bt, b, kv) for b, kv in enumerate(have)])
        kv = layer.expand(rows[:, :L])
        cu_k = torch.tensor([0] + torch.tensor(have).cumsum(0).tolist()).int().cuda()
        absorbed = layer.absorb(q)
        out = ua.latent_attention(absorbed, cache, cu, sl, bt, scale=scale, tree_mask=mask, **sizes)
        check_attention(absorbed, cache, cu, sl, bt, out, scale=scale, mask=mask)
        if mask is None:        # the expanded form has the same numbers to work on
            exp = ua.latent_prefill(q, kv[..., :N], rows[:, L:].contiguous(), kv[..., N:], cu, cu_k,
                                    **sizes)
            want, _, tol, _ = ref.prefill(*(x.cpu() for x in (q, kv[..., :N], rows[:, L:],
                                                              kv[..., N:], cu, cu_k)), scale)
            ref.check(exp, want, tol, dtype)
            # (the absorbed scores sum L + R products, of which L - N are zeros)
            ref.check(layer.values(out), want, 3 * tol, dtype)
            lens = have
    assert ua.device_status() == 0


# ------------------------------------------------------------------ prepared and captured

def step_of(lens, h=16, bs=64, seed=0, **kw):
    cu, sl, bt, nb = batch(lens, bs, seed)
    total = sum(q for q, _ in lens)
    q, cache = rand(total, h, L + R, seed=seed), rand(nb, bs, L + R, seed=seed + 1)
    step = ua.prepare_latent_attention(q, cache, cu, sl, bt, scale=0.08, **most(lens), **kw)
    return step, (q, cache, cu, sl, bt)


def test_prepared_steps_take_new_tensors_or_none():
    step, (q, cache, cu, sl, bt) = step_of([(1, 700), (1, 130)], return_lse=True)
    out, lse = step()
    check_attention(q, cache, cu, sl, bt, out, lse)
    q2, sl2 = rand(2, 16, L + R, seed=7), torch.tensor([500, 90]).int().cuda()
    out2 = torch.empty_like(out)
    got, lse = step(q=q2, seq_lens_k=sl2, out=out2)
    assert got is out2
    check_attention(q2, cache, cu, sl2, bt, out2, lse)
    before = out2.clone()
    for bad in (dict(q=q2[:1]), dict(q=q2.half()), dict(seq_lens_k=sl2.long()),
                dict(out=torch.empty_like(out).transpose(0, 1)), dict(tree_mask=sl2),
                dict(q=rand(2, 16, L + R, seed=8), seq_lens_k=sl2[:1])):
        with pytest.raises(ValueError, match="prepared call"):
            step(**bad)
    step()          # none of a refused call's tensors was taken
    assert torch.equal(out2, before)


def test_results_are_the_same_every_time():
    step, _ = step_of([(1, 4000), (1, 10), (1, 2500), (3, 900)])
    first = step().clone()
    for _ in range(5):
        assert torch.equal(step(), first)


def captured(run):
    return captured_on(torch.cuda.Stream(priority=-1), run)


def captured_on(stream, run):
    with torch.cuda.stream(stream):
        run(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run(stream)
    torch.cuda.synchronize()
    return graph


def test_a_captured_step_follows_the_lengths():
    h, lens = 16, [(1, 60), (1, 700)]
    cu, sl, bt, nb = batch([(1, 100), (1, 800)])
    sl.copy_(torch.tensor([60, 700]))
    cache, table = rand(nb, 64, L + R), ua.rope_table(900, R)
    down, q = rand(2, L + R, seed=2), rand(2, h, L + R, seed=3)
    raw = rand(2, h, R, seed=4)
    out = torch.empty((2, h, L), dtype=BF, device="cuda")

    def run(stream):
        ua.append_latent(down[:, :L], down[:, L:], cache, cu, sl, bt, q_rope=raw,
                         q_rope_out=q[..., L:], cos_sin=table, stream=stream)
        ua.latent_attention(q, cache, cu, sl, bt, scale=0.08, max_seqlen_q=1, max_seqlen_k=800,
                            out=out, stream=stream)

    graph = captured(run)
    for step in range(4):
        sl.copy_(torch.tensor([61 + step, 701 + 9 * step]))
        down.copy_(rand(2, L + R, seed=20 + step))
        graph.replay()
        torch.cuda.synchronize()
        check_attention(q, cache, cu, sl, bt, out)
    assert ua.device_status() == 0


BOTH = pytest.mark.parametrize("lens", [    # even shares with scratch; a cluster a row tile
    [(1, 6000), (2, 3000)], [(1, 700), (2, 300), (1, 64)]])


@BOTH
def test_two_graphs_of_one_stream_run_side_by_side(lens):
    steps = [step_of(lens, seed=s) for s in (0, 10)]
    assert (ua.latent_workspace_bytes(steps[0][0]) == 0) == (lens[0][1] == 700)
    want = [s[0]().clone() for s in steps]
    stream = torch.cuda.Stream(priority=-1)
    graphs = []
    for s, _ in steps:
        s(stream=stream)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s(stream=stream)
        graphs.append(g)
    for s, _ in steps:
        s._last("out").zero_()
    sides = [torch.cuda.Stream(priority=-1), torch.cuda.Stream(priority=-1)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    for (s, _), w in zip(steps, want):
        assert torch.equal(s._last("out"), w)


@BOTH
def test_two_streams_at_once(lens):
    steps = [step_of(lens, seed=s) for s in (0, 10)]
    want = [s[0]().clone() for s in steps]
    sides = [torch.cuda.Stream(priority=-1), torch.cuda.Stream(priority=-1)]
    torch.cuda.synchronize()
    for _ in range(20):
        for (s, _), side in zip(steps, sides):
            s(stream=side)
    torch.cuda.synchronize()
    for (s, _), w in zip(steps, want):
        assert torch.equal(s._last("out"), w)


@pytest.mark.parametrize("q_len,k_len,h", [(64, 2000, 16), (700, 700, 8), (900, 900, 40)])
def test_captured_prefills_on_two_streams(q_len, k_len, h):
    """Four CTAs a q-block's keys, two or four, and one; both graphs at once, again and again."""
    cu = torch.tensor([0, q_len], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, k_len], dtype=torch.int32, device="cuda")
    sides, calls = [torch.cuda.Stream(priority=-1) for _ in range(2)], []
    for seed, side in enumerate(sides):
        q, kv = rand(q_len, h, N + R, seed=seed), rand(k_len, h, N + V, seed=seed + 5)
        args = (q, kv[..., :N], rand(k_len, R, seed=seed + 9), kv[..., N:], cu, cu_k)
        out = torch.zeros((q_len, h, V), dtype=BF, device="cuda")
        calls.append((args, out, captured_on(side, lambda s: ua.latent_prefill(
            *args, max_seqlen_q=q_len, max_seqlen_k=k_len, out=out, stream=s))))
    torch.cuda.synchronize()
    for _, out, _ in calls:
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for (_, _, graph), side in zip(calls, sides):
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for args, out, _ in calls:
        want, _, tol, _ = ref.prefill(*(x.cpu() for x in args), (N + R) ** -0.5)
        ref.check(out, want, tol, BF)
    assert ua.device_status() == 0


def test_a_workspace_of_the_caller():
    lens = [(1, 3000), (1, 5000)]
    step, tensors = step_of(lens)
    want = step().clone()
    need = ua.latent_workspace_bytes(step)
    for n, ok in ((need, True), (need - 16, False)):
        own = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        got = ua.prepare_latent_attention(*tensors, scale=0.08, workspace=own, **most(lens))
        if ok:
            assert torch.equal(got(), want)
        else:
            with pytest.raises(ua.UaError) as e:
                got()
            assert e.value.code == 4


# ------------------------------------------------------------------ edges

def test_rows_behind_the_batch_stay():
    cu, sl, bt, nb = batch([(1, 3000), (3, 70)])
    q, cache = rand(9, 16, L + R), rand(nb, 64, L + R)
    out = torch.full((9, 16, L), 7.0, dtype=BF, device="cuda")
    ua.latent_attention(q, cache, cu, sl, bt, scale=0.08, max_seqlen_q=3, max_seqlen_k=3000, out=out)
    assert torch.all(out[4:] == 7)
    check_attention(q, cache, cu, sl, bt, out)
    mask = torch.full((9, 1), 7, dtype=torch.int32, device="cuda")
    pos = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    ua.tree_mask(torch.zeros(9, dtype=torch.int32, device="cuda") - 1, cu, sl, max_seqlen_q=3,
                 mask=mask, positions=pos)
    assert torch.all(mask[4:] == 7) and torch.all(pos[4:] == 7)
    assert mask[:4, 0].tolist() == [1, 1, 2, 4] and pos[:4].tolist() == [2999, 67, 67, 67]


def test_many_sequences_with_and_without_keys():
    g = torch.Generator().manual_seed(5)
    lens = [(int(torch.randint(0, 3, (1,), generator=g)), int(torch.randint(0, 200, (1,), generator=g)))
            for _ in range(300)]
    step, (q, cache, cu, sl, bt) = step_of(lens, h=5, bs=16)
    check_attention(q, cache, cu, sl, bt, step())


def test_sizes_that_are_larger_than_the_lengths():
    """max_seqlen_q and max_seqlen_k are bounds: a captured step keeps the largest."""
    lens = [(1, 90), (1, 300)]
    step, (q, cache, cu, sl, bt) = step_of(lens)
    want = step().clone()
    for mq, mk in ((1, 100000), (64, 300), (500, 5000)):
        out = ua.latent_attention(q, cache, cu, sl, bt, scale=0.08, max_seqlen_q=mq, max_seqlen_k=mk)
        check_attention(q, cache, cu, sl, bt, out)
    assert torch.equal(step(), want)


def test_blocks_past_32_bits_of_a_large_cache():
    nb, bs = 62000, 64                          # 2.3e9 elements
    cache = torch.zeros((nb, bs, L + R), dtype=BF, device="cuda")
    bt = torch.tensor([[nb - 1, 3, nb - 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    sl = torch.tensor([150], dtype=torch.int32, device="cuda")
    down, q = rand(150, L + R), rand(1, 16, L + R, seed=1)
    ua.append_latent(down[:, :L], down[:, L:], cache, cu, sl, bt)
    rows = torch.cat([cache[nb - 1], cache[3], cache[nb - 2]])[:150]
    assert torch.equal(rows, down)
    assert not torch.any(cache[4:nb - 2])
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = ua.latent_attention(q, cache, one, sl, bt, scale=0.08, max_seqlen_q=1, max_seqlen_k=150)
    small = torch.cat([cache[nb - 2:], cache[3:4]])
    check_attention(q, small, one, sl, torch.tensor([[1, 2, 0]], dtype=torch.int32), out)


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_blocks_count_as_zeros_and_are_reported(bad):
    ua.device_status_reset()
    step, (q, cache, cu, sl, bt) = step_of([(1, 300), (1, 200)])
    bt[0, 2] = bad
    out = step()
    assert ua.device_status() == 5
    ua.device_status_reset()
    zeros = torch.cat([cache, torch.zeros_like(cache[:1])])
    bt[0, 2] = cache.shape[0]
    check_attention(q, zeros, cu, sl, bt, out)


def test_tables_that_are_too_short_are_reported():
    ua.device_status_reset()
    step, (q, cache, cu, sl, bt) = step_of([(1, 64), (1, 60)])
    step(seq_lens_k=torch.tensor([64, 500]).int().cuda())
    assert ua.device_status() == 5
    ua.device_status_reset()


def test_bad_parents_count_as_roots_and_are_reported():
    ua.device_status_reset()
    cu, sl = torch.tensor([0, 4]).int().cuda(), torch.tensor([10]).int().cuda()
    mask, pos = ua.tree_mask(torch.tensor([-1, 1, 0, -5]).int().cuda(), cu, sl, max_seqlen_q=4)
    assert ua.device_status() == 5
    ua.device_status_reset()
    assert mask[:, 0].tolist() == [1, 2, 5, 8] and pos.tolist() == [6, 6, 7, 6]


@pytest.mark.parametrize("n", [1, 32, 33, 1000])
def test_deep_trees(n):
    """A chain: every token sees all before it, which is the causal mask."""
    cu, sl = torch.tensor([0, n]).int(), torch.tensor([n + 7]).int()
    parents = torch.arange(-1, n - 1, dtype=torch.int32)
    mask, pos = ua.tree_mask(parents.cuda(), cu.cuda(), sl.cuda(), max_seqlen_q=n)
    wmask, wpos = ref.tree(parents, cu, sl, (n + 31) // 32)
    assert torch.equal(mask.cpu(), wmask) and torch.equal(pos.cpu(), wpos)
    if n <= 33:
        cu, sl, bt, nb = batch([(n, n + 7)])
        q, cache = rand(n, 3, L + R), rand(nb, 64, L + R)
        a, b = (ua.latent_attention(q, cache, cu, sl, bt, scale=0.08, max_seqlen_q=n,
                                    max_seqlen_k=n + 7, tree_mask=m) for m in (None, mask))
        assert torch.equal(a, b)


def test_masks_in_a_wider_buffer():
    lens = [(40, 300), (3, 9)]
    cu, sl, bt, nb = batch(lens)
    q, cache = rand(43, 4, L + R), rand(nb, 64, L + R)
    wide = torch.full((43, 5), -1, dtype=torch.int32, device="cuda")
    mask, _ = ua.tree_mask(ref.random_parents(lens).cuda(), cu, sl, max_seqlen_q=40, mask=wide[:, 1:3])
    assert torch.all(wide[:, 0] == -1) and torch.all(wide[:, 3:] == -1)
    out = ua.latent_attention(q, cache, cu, sl, bt, scale=0.08, tree_mask=mask, **most(lens))
    check_attention(q, cache, cu, sl, bt, out, mask=mask)


def test_nan_in_a_key_reaches_its_rows():
    step, (q, cache, cu, sl, bt) = step_of([(1, 300), (1, 200)])
    cache[bt[0, 1], 5, 10] = float("nan")
    out = step()
    assert torch.all(out[0].isnan().any(-1)) and not torch.any(out[1].isnan())


# ------------------------------------------------------------------ called wrongly

def test_refusals_of_the_binding():
    lens = [(2, 70), (1, 9)]
    cu, sl, bt, nb = batch(lens)
    q, cache = rand(3, 4, L + R), rand(nb, 64, L + R)
    good = dict(q=q, cache=cache, cu_seqlens_q=cu, seq_lens_k=sl, block_table=bt, scale=0.1,
                max_seqlen_q=2, max_seqlen_k=70)
    ua.latent_attention(**good)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]), dict(q=q.transpose(0, 1)),
                dict(cache=cache.half()), dict(cache=cache[..., :-8]), dict(cache=cache[:, ::2]),
                dict(cu_seqlens_q=cu.long()), dict(seq_lens_k=sl[:1]), dict(block_table=bt[0]),
                dict(block_table=bt.cpu()), dict(out=torch.empty_like(q)),
                dict(out=torch.empty(3, 4, L, device="cuda"), out_dtype=BF),
                dict(tree_mask=torch.zeros(3, 1, device="cuda")),
                dict(tree_mask=torch.zeros(2, 1, dtype=torch.int32, device="cuda")),
                dict(tree_mask=torch.zeros(3, 1, dtype=torch.int32, device="cuda"),
                     max_seqlen_q=33)):
        with pytest.raises((ValueError, TypeError)):
            ua.latent_attention(**{**good, **bad})
    for bad, code in ((dict(rope_dim=8), 1), (dict(rope_dim=32), 1), (dict(scale=0.0), 1),
                      (dict(scale=float("inf")), 1)):
        with pytest.raises(ua.UaError) as e:
            ua.latent_attention(**{**good, **bad})
        assert e.value.code == code

    down, qr = rand(3, L + R), rand(3, 4, R)
    table = ua.rope_table(100, R)
    good = dict(latent=down[:, :L], k_rope=down[:, L:], cache=cache, cu_seqlens_q=cu, seq_lens_k=sl,
                block_table=bt, q_rope=qr, cos_sin=table)
    ua.append_latent(**good)
    for bad in (dict(latent=down[:, :L].float()), dict(latent=down[:2, :L]), dict(k_rope=down[:, 1:65]),
                dict(k_rope=down[:, L:].half()), dict(cache=cache[..., 8:]), dict(q_rope=None, q_rope_out=qr),
                dict(q_rope=qr[:2]), dict(q_rope_out=qr.transpose(0, 1)),
                dict(q_rope_out=torch.empty(3, 4, 40, dtype=BF, device="cuda")),
                dict(norm_weight=torch.ones(L)), dict(norm_weight=torch.ones(L, dtype=F16, device="cuda")),
                dict(cos_sin=table.half()), dict(cos_sin=table[:, :32]),
                dict(cos_sin=None, positions=sl), dict(positions=sl)):
        if "k_rope" in bad and bad["k_rope"].dtype == BF:    # the last dim is not 16-byte aligned
            with pytest.raises(ua.UaError):
                ua.append_latent(**{**good, **bad})
            continue
        with pytest.raises((ValueError, TypeError)):
            ua.append_latent(**{**good, **bad})

    kv, kr, qq = rand(79, 4, N + V), rand(79, R), rand(3, 4, N + R)
    cu_k = torch.tensor([0, 70, 79]).int().cuda()
    good = dict(q=qq, k_nope=kv[..., :N], k_rope=kr, v=kv[..., N:], cu_seqlens_q=cu,
                cu_seqlens_k=cu_k, max_seqlen_q=2, max_seqlen_k=70)
    ua.latent_prefill(**good)
    for bad in (dict(q=qq.float()), dict(q=qq[..., :-16]), dict(k_nope=kv[:, :2, :N]),
                dict(v=kv[:70, :, N:]), dict(k_rope=kr.half()), dict(k_rope=kr[:, ::2]),
                dict(cu_seqlens_k=cu_k[:2]), dict(cu_seqlens_q=cu.long()),
                dict(out=torch.empty_like(qq))):
        with pytest.raises((ValueError, TypeError)):
            ua.latent_prefill(**{**good, **bad})
    for bad in (dict(scale=-1.0), dict(k_nope=kv[..., :N][:, :1].expand(-1, 4, -1))):
        with pytest.raises((ua.UaError, ValueError)):
            ua.latent_prefill(**{**good, **bad})

    parents = torch.tensor([-1, 0, -1]).int().cuda()
    ua.tree_mask(parents, cu, sl, max_seqlen_q=2)
    for bad in (dict(parents=parents.long()), dict(parents=parents.cpu()), dict(parents=parents[None]),
                dict(seq_lens_k=sl[:1]), dict(mask=torch.zeros(3, 1, device="cuda")),
                dict(mask=torch.zeros(2, 1, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            ua.tree_mask(**{**dict(parents=parents, cu_seqlens_q=cu, seq_lens_k=sl, max_seqlen_q=2),
                            **bad})
    with pytest.raises(ua.UaError):
        ua.tree_mask(parents, cu, sl, max_seqlen_q=5000)
    assert ua.device_status() == 0
