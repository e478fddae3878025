"""GPU: append_kv with a cu_seqlens_q that ends behind the inputs.  The tokens that the inputs hold
are appended as ever; the others are neither read (the rows behind the inputs hold values that
would show in every scale) nor written."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _append_ref as R
from tests.test_append_gpu import check, run, to_dev

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
FORMS = [(None, ""), (E4M3, "tensor"), (E4M3, "tok"), (E4M3, "blk"), (I8, "blk")]


def short(c, rows):
    """The case with its tensors cut to `rows` rows and its last sequences' tokens cut alike:
    the same tokens at the same places; and the whole case's lengths, on the GPU."""
    whole = to_dev(c)
    left, lens = rows, []
    for n, kv in c.lens:
        m = min(n, left)
        lens.append((m, kv - n + m))
        left -= m
    cut = R.Case(lens, **{f: getattr(c, f) for f in (
        "hq", "hkv", "d", "bs", "dtype", "cache", "form", "rot", "interleaved", "axes", "seed")})
    cut.t = dict(c.t)
    for n in ("q", "k", "v"):
        cut.t[n] = c.t[n][:rows]
        whole[n][rows:] = 1.0e4
        whole[n] = whole[n][:rows]
    if "positions" in c.t:
        cut.t["positions"] = c.t["positions"][..., :rows].contiguous()
        whole["positions"] = cut.t["positions"].cuda()
    cut.t["cu_seqlens_q"] = torch.tensor(
        [0] + torch.tensor([n for n, _ in lens]).cumsum(0).tolist(), dtype=torch.int32)
    return cut, whole


@pytest.mark.parametrize("cache,form", FORMS)
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("lens,rows", [([(20, 30), (70, 75)], 41), ([(20, 30), (70, 75)], 20),
                                       ([(20, 30), (70, 75), (9, 9)], 13),
                                       ([(1, 4 + i) for i in range(9)], 5)], ids=str)
def test_tokens_behind_the_inputs_are_skipped(lens, rows, axes, bs, cache, form):
    c = R.make(R.Case(lens, hq=4, hkv=2, d=128, bs=bs, cache=cache, form=form, rot=64, axes=axes,
                      seed=rows))
    cut, d = short(c, rows)
    ua.device_status_reset()
    check(cut, d, run(c, d))
    assert ua.device_status() == 0
