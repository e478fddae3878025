"""GPU: calls that need scratch, captured without a workspace of the caller's.  A capture needs no
call before it on its stream, and graphs captured on one stream have scratch of their own, so that
they may be replayed at the same time."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests.test_block_scaled_gpu import E4M3, I8, RAGGED, check, make, on_gpu, planned

pytestmark = pytest.mark.gpu
CASES = {
    # an even share of ragged lengths; partitions beyond a cluster's; a prompt's split
    "share": (dict(**RAGGED["ragged"]), 40000, {}),
    "merge": (dict(seqs=[(1, 900), (1, 2000), (1, 40)], hq=16, hkv=2), None,
              dict(backend="split", num_splits=24)),
    "prompt": (dict(seqs=[(60, 900), (33, 500)], hq=8, hkv=2), None,
               dict(backend="split", num_splits=4)),
}


def call(c, d, out, max_k, kw):
    return ua.unified_attention(
        *(d[n] for n in ("q", "k_cache", "v_cache", "cu_seqlens_q", "seq_lens_k", "block_table")),
        max_seqlen_q=max(q for q, _ in c["seqs"]),
        max_seqlen_k=max_k or max(kv for _, kv in c["seqs"]), scale=c["scale"], out=out,
        k_scale_blk=d["k_scale_blk"], v_scale_blk=d["v_scale_blk"], **kw)


def captured(name, code, seed, stream):
    shape, max_k, kw = CASES[name]
    c = make(**shape, code=code, seed=seed)
    assert planned(c, max_k, **kw)["workspace_bytes"] > 0
    d = on_gpu(c)
    out = torch.full(tuple(d["q"].shape), 7.0, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(c, d, out, max_k, kw)
    return c, d, out, graph


def warm():
    """One call of each case, on another stream: kernels loaded, tables looked up."""
    for name, (shape, max_k, kw) in CASES.items():
        c = make(**shape, code=I8, seed=1)
        d = on_gpu(c)
        call(c, d, torch.empty(tuple(d["q"].shape), device="cuda"), max_k, kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", CASES)
def test_a_stream_the_library_has_not_seen_is_captured(name):
    warm()
    c, _, out, graph = captured(name, I8, 2, torch.cuda.Stream())
    graph.replay()
    torch.cuda.synchronize()
    check(c, out)
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    check(c, out)


@pytest.mark.parametrize("name", CASES)
def test_two_graphs_of_one_stream_replay_at_once(name):
    warm()
    stream = torch.cuda.Stream()
    both = [captured(name, code, 3 + i, stream) for i, code in enumerate((I8, E4M3))]
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(40):
        for (_, _, _, graph), s in zip(both, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for c, _, out, _ in both:
        check(c, out)
    assert ua.device_status() == 0


def test_a_captured_graph_and_the_same_stream_eagerly():
    """The graph replayed on another stream while its capture stream runs the same call."""
    warm()
    stream = torch.cuda.Stream()
    c, d, out, graph = captured("share", I8, 5, stream)
    shape, max_k, kw = CASES["share"]
    c2 = make(**shape, code=E4M3, seed=6)
    d2, other = on_gpu(c2), torch.cuda.Stream()
    out2 = torch.full(tuple(d2["q"].shape), 7.0, device="cuda")
    torch.cuda.synchronize()
    for _ in range(40):
        with torch.cuda.stream(other):
            graph.replay()
        with torch.cuda.stream(stream):
            call(c2, d2, out2, max_k, kw)
    torch.cuda.synchronize()
    check(c, out)
    check(c2, out2)
