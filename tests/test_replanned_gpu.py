"""GPU: calls whose first plan cannot be launched.  A cache of 2^31 rows or more has no tensor map
with 32-bit row coordinates, so the dispatcher plans again for the kernel that needs none.  (The
sizes say so here; the block table names the few blocks there are.)"""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests._dense import dense_attention
from tests.test_block_scaled_gpu import E4M3, I8, bar, check, make, on_gpu, run

pytestmark = pytest.mark.gpu
SHAPES = {
    "rows64": [(16, 50), (3, 40), (16, 16), (1, 90), (0, 5), (9, 30)],    # one q-block a sequence
    "rows20": [(5, 50), (5, 40), (2, 16), (1, 90), (5, 7)],
    "prompts": [(40, 50), (70, 90), (3, 3)],
    "decode": [(1, 50), (1, 40), (0, 3), (1, 17)],
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("backend", ["2d", "auto"])
def test_block_scaled(shape, code, backend):
    c = make(SHAPES[shape], hq=8, hkv=2, code=code, seed=3, sinks=True)
    d = on_gpu(c)
    ua.device_status_reset()
    step = run(c, d, fn=ua.prepare, backend=backend)
    step._call.shape.contents.num_blocks = 1 << 27
    check(c, step())
    assert ua.device_status() == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 256])
def test_16bit(shape, d):
    c = make(SHAPES[shape], hq=8, hkv=2, d=d, q_dtype=torch.float16, seed=4)
    t = c["t"]
    kv = []
    for n in ("k", "v"):
        t[f"{n}_cache"] = torch.randn(t[f"{n}_cache"].shape,
                                      generator=torch.Generator().manual_seed(5)).half()
        t[f"{n}_scale_blk"] = None
        kv.append(t[f"{n}_cache"].double())
    out = torch.full(tuple(t["q"].shape), 7.0, device="cuda")
    step = run(c, on_gpu(c), fn=ua.prepare)
    step._call.shape.contents.num_blocks = 1 << 27
    ua.device_status_reset()
    got = step(out=out).cpu().double()
    assert ua.device_status() == 0
    want = torch.from_numpy(dense_attention(t["q"], *kv, t["cu_seqlens_q"], t["seq_lens_k"],
                                            t["block_table"], scale=c["scale"], **c["opt"]))
    assert float((got - want).abs().max()) <= bar(c, kv)
