"""GPU: rows whose keys many workers share, in batches where the row tiles are many (the merge kernel
that counts CTAs, not row tiles), against the definition in 64 bits."""
import pytest
import torch

from tests.test_latent_gpu import compare, make

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# (The parts are those of a device of 152 SMs; others cut the keys otherwise, and merge them as well.)
@pytest.mark.parametrize("lens,h,latent,rope,bs,dtype", [
    # at most 32 rows: a block a row, 125, 125, 125, 32, 71 and 40 parts of a row
    ([(1, 16000)] + [(1, 100)] * 15, 16, 512, 64, 64, BF),
    ([(1, 100)] * 15 + [(1, 16000)], 16, 256, 32, 16, F16),
    ([(1, 70)] * 9 + [(1, 16000)] + [(1, 64)] * 6, 16, 128, 64, 64, BF),
    ([(1, 4000)] + [(1, 100)] * 15, 16, 512, 64, 64, F16),
    ([(2, 9000)] + [(1, 64)] * 20, 9, 256, 64, 64, BF),
    ([(1, 5000)] + [(0, 9)] * 30, 32, 512, 64, 64, BF),
    # more rows: two warps a row, 71, and in pairs of row tiles 63 and 36 parts
    ([(1, 9000)] + [(1, 1)] * 12, 40, 512, 64, 64, BF),
    ([(1, 24000)] + [(1, 100)] * 5, 128, 512, 64, 64, BF),
    ([(1, 100)] * 5 + [(2, 20000)], 100, 256, 32, 64, F16),
    # 21 parts, the last of which has no key for the first rows
    ([(40, 2600)] + [(1, 100)] * 15, 1, 128, 64, 64, BF),
])
def test_rows_of_many_parts(lens, h, latent, rope, bs, dtype):
    t = make(lens, h, latent, rope, bs, dtype, pad=2)
    compare(t, rope, out_dtype=F32)
    out = torch.full((t[0].shape[0], h, latent), 7.0, dtype=dtype, device="cuda")
    compare(t, rope, out=out)
    assert torch.all(out[-2:] == 7)
