"""GPU: batches with rows behind the last sequence.  Those rows of the output stay as they were,
whichever way the partitions of the others are merged, and whatever the scratch holds."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests._dense import dense_attention
from tests.test_block_scaled_gpu import E4M3, I8, bar, check, make, on_gpu, planned, run

pytestmark = pytest.mark.gpu
F16 = torch.float16
SHAPES = {
    "decode": dict(seqs=[(1, 300), (0, 40), (1, 17), (1, 0)], hq=16, hkv=4),
    "drafts": dict(seqs=[(3, 50), (2, 700), (3, 3)], hq=16, hkv=4),
    "chunks": dict(seqs=[(37, 37), (129, 400), (1, 90)], hq=8, hkv=2),
}
SPLITS = [0, 2, 7, 20]


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("bs", [16, 24])
@pytest.mark.parametrize("shape", SHAPES)
def test_block_scaled(shape, bs, splits, code):
    c = make(**SHAPES[shape], bs=bs, code=code, seed=splits, sinks=True, pad_rows=5)
    kw = dict(backend="split", num_splits=splits) if splits else {}
    ws = torch.full((planned(c, **kw)["workspace_bytes"] + 256,), 0x41, dtype=torch.uint8,
                    device="cuda")                     # partial sums of 12, not of nothing
    check(c, run(c, workspace=ws, **kw))


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("shape", SHAPES)
def test_16bit(shape, d, splits):
    c = make(**SHAPES[shape], d=d, q_dtype=F16, seed=splits, pad_rows=5)
    t, kv = c["t"], []
    for n in ("k", "v"):
        g = torch.Generator().manual_seed(d)
        t[f"{n}_cache"] = torch.randn(t[f"{n}_cache"].shape, generator=g).half()
        t[f"{n}_scale_blk"] = None
        kv.append(t[f"{n}_cache"].double())
    kw = dict(backend="split", num_splits=splits) if splits else {}
    ws = torch.full((64 << 20,), 0x41, dtype=torch.uint8, device="cuda")
    got = run(c, workspace=ws, **kw).cpu().double()
    total = int(t["cu_seqlens_q"][-1])
    want = torch.from_numpy(dense_attention(t["q"], *kv, t["cu_seqlens_q"], t["seq_lens_k"],
                                            t["block_table"], scale=c["scale"], **c["opt"]))
    assert float((got - want)[:total].abs().max()) <= bar(c, kv)
    assert (got[total:] == 7.0).all()
    assert ua.device_status() == 0
