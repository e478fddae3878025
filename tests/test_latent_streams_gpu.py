"""GPU: the latent calls where the current stream is not the one that they were prepared on."""
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
