"""GPU: the prefill kernels' walks, tile by tile: every number of key tiles, again and again while
another stream keeps the device busy, ends, and gives the same bits each time."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests.test_block_scaled_gpu import E4M3, F16, BF, I8, check, make, on_gpu, planned, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", [E4M3, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("capped", [False, True])
def test_walks_of_every_length_end(d, code, capped):
    """One q tile a CTA, 1 to 9 key tiles, under a load that delays warps and CTAs."""
    c = make([(20, 20 + 128 * i + 5 * i) for i in range(9)], hq=8, hkv=2, d=d, code=code,
             q_dtype=BF if capped else F16, softcap=20.0 if capped else 0.0, seed=d + capped)
    assert planned(c, backend="2d")["kernel"] == 8
    dev = on_gpu(c)
    ua.device_status_reset()
    first = run(c, dev, backend="2d")
    check(c, first)
    load = torch.empty(1 << 24, device="cuda")
    side = torch.cuda.Stream()
    outs = []
    for i in range(60):
        with torch.cuda.stream(side):
            load.mul_(1.0)
        outs.append(ua.unified_attention(
            *(dev[n] for n in ("q", "k_cache", "v_cache", "cu_seqlens_q", "seq_lens_k",
                               "block_table")),
            max_seqlen_q=20, max_seqlen_k=1084, scale=c["scale"], softcap=c["opt"]["softcap"],
            k_scale_blk=dev["k_scale_blk"], v_scale_blk=dev["v_scale_blk"], backend="2d",
            out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert ua.device_status() == 0
    for o in outs:
        assert torch.equal(o, first)
