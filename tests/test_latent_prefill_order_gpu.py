"""GPU: the expanded form where its q-blocks start by the length of their walks (at most 64 slots, more
CTAs than a device takes at once): every q-block is done, and by itself."""
import pytest
import torch

from tests.test_latent_prefill_gpu import compare, make

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("lens,h,dtype", [
    # ragged, the longest in front, an empty sequence, equal walks, slots that the next takes over
    ([(300, 900), (0, 40), (1, 700), (513, 513), (256, 256), (256, 256)], 32, BF),
    ([(5, 600), (0, 3), (70, 70), (257, 300)] * 10, 4, F16),     # 52 slots
    ([(6, 520)] + [(5, 9)] * 62, 3, BF),                         # 64 slots
    ([(5, 9)] * 62 + [(6, 520)], 3, BF),
    ([(6, 520)] + [(5, 9)] * 63, 3, BF),                         # 65: in reverse order
    ([(256, 600)] * 12, 16, BF),                                 # every other slot idle
    ([(0, 600), (0, 0), (1000, 1000), (0, 5), (3, 0), (9, 4)], 40, F16),
    ([(700, 100), (1, 513), (600, 1100)], 40, BF),               # more queries than keys
    ([(1025, 1500)], 31, BF),
])
def test_every_block_is_done(lens, h, dtype):
    t = make(lens, h, 128, 64, 128, dtype, pad_q=3, pad_k=5)
    compare(t, out_dtype=F32)
    out = torch.full((t[0].shape[0], h, 128), 7.0, dtype=dtype, device="cuda")
    compare(t, out=out)
    assert torch.all(out[-3:] == 7)
