"""GPU: the latent calls where the current stream is not the one that they were prepared on, and
results that prepared calls write on several streams."""
from types import SimpleNamespace

import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _latent_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
LENS = [(17, 301), (40, 500), (1, 9)]


def tree_step():
    """A step over drafted trees, prepared on the current stream without one given."""
    g = torch.Generator().manual_seed(3)
    cu, sl, bt, nb = ref.batch(LENS, 64)
    q = torch.randn((58, 8, 576), generator=g).to(BF)
    cache = torch.randn((nb, 64, 576), generator=g).to(BF)
    parents = ref.random_parents(LENS)
    want = ref.attend(q, cache, cu, sl, bt, 512, 0.08, ref.tree(parents, cu, sl, 2)[0])
    cu, sl, parents = cu.cuda(), sl.cuda(), parents.cuda()
    mask = torch.zeros((58, 2), dtype=torch.int32, device="cuda")
    out = torch.zeros((58, 8, 512), dtype=BF, device="cuda")
    step = ua.prepare_latent_attention(q.cuda(), cache.cuda(), cu, sl, bt.cuda(), scale=0.08,
                                       max_seqlen_q=40, max_seqlen_k=500, tree_mask=mask, out=out)

    def run():
        ua.tree_mask(parents, cu, sl, max_seqlen_q=40, mask=mask)
        return step()

    torch.cuda.synchronize()
    return run, mask, out, lambda: ref.check(out, want[0], want[2], BF)


def test_masks_and_their_attention_on_another_current_stream():
    run, mask, out, check = tree_step()
    with torch.cuda.stream(torch.cuda.Stream(priority=-1)):
        torch.cuda._sleep(20_000_000)       # the masks are made some milliseconds later
        assert run() is out
    torch.cuda.synchronize()
    check()


def test_captured_without_a_stream_given():
    run, mask, out, check = tree_step()
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    mask.zero_()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check()
    assert ua.device_status() == 0


def prepared():
    """Prepared calls whose result the preparation allocates."""
    i = dict(dtype=torch.int32, device="cuda")
    x = torch.randn((3, 2, 64), device="cuda").to(BF)
    kv = torch.zeros((4, 16, 2, 64), dtype=BF, device="cuda")
    q, cache = torch.randn((3, 8, 576), device="cuda").to(BF), \
        torch.zeros((4, 16, 576), dtype=BF, device="cuda")
    cu, sl = torch.arange(4, **i), torch.tensor([5, 9, 16], **i)
    bt = torch.tensor([[0], [1], [2]], **i)
    e, r = torch.randn((3, 8, 256), device="cuda").to(BF), q[:, 0, :64].contiguous()
    one = dict(max_seqlen_q=1, max_seqlen_k=16)
    return {
        "append": lambda **k: ua.prepare_append_latent(
            q[:, 0, :512], q[:, 0, 512:], cache, cu, sl, bt, q_rope=q[..., 512:], **k),
        "attention": lambda **k: ua.prepare_latent_attention(
            q, cache, cu, sl, bt, scale=0.1, return_lse=True, **one, **k),
        "prefill": lambda **k: ua.prepare_latent_prefill(
            q[..., :192].contiguous(), e[..., :128], r, e[..., 128:], cu, cu, max_seqlen_q=1,
            max_seqlen_k=1, **k),
        "append_kv": lambda **k: ua.prepare_append(x, x, kv, kv.clone(), cu, sl, bt,
                                                   max_seqlen_q=1, q=x, **k),
        "unified_attention": lambda **k: ua.prepare(x, kv, kv, cu, sl, bt, **one, **k),
    }


# (append_kv and unified_attention keep the preparation's stream, not the current one)
@pytest.mark.parametrize("name,how", [(n, h) for n in ("append", "attention", "prefill") for h in (
    "a step's stream", "a foreign stream", "the current stream")] + [
    (n, h) for n in ("append_kv", "unified_attention") for h in (
        "a step's stream", "a foreign stream")])
def test_a_result_outlives_the_work_of_a_steps_stream(name, how):
    prepare = prepared()[name]
    side = torch.cuda.Stream(priority=-1)

    def other(step):
        if how == "the current stream":
            with torch.cuda.stream(side):
                return step()
        return step(stream=side if how == "a step's stream" else
                    SimpleNamespace(cuda_stream=side.cuda_stream))

    prepare()()
    other(prepare())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    step = prepare()
    step()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                    # about a tenth of a second
    out = other(step)
    outs = out if isinstance(out, tuple) else (out,)
    was = [(o.data_ptr(), tuple(o.shape), o.dtype) for o in outs]
    del out, outs, step
    held = [torch.empty(shape, dtype=dtype, device="cuda") for _, shape, dtype in was
            for _ in range(4)]
    assert not side.query()                               # the step's kernel is still to run
    assert not {at for at, _, _ in was} & {t.data_ptr() for t in held}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["append", "attention", "prefill"])
def test_results_of_the_preparation_in_a_capture(name):
    """Made outside the capture, written by its stream, read after replays, dropped in its time."""
    step = prepared()[name]()

    def outs():
        out = step()
        return out if isinstance(out, tuple) else (out,)

    want = [o.clone() for o in outs()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = outs()
    for o in got:
        o.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del graph, got, step
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert ua.device_status() == 0
