"""GPU: latent calls at the edges of what their arguments may be."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import test_append_latent_gpu as appended

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16
L, R = 512, 64


def rand(*shape, dtype=BF, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def batch(q_lens, kv_lens, cols=4):
    i = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), **i)
    n = len(q_lens)
    return cu, torch.tensor(kv_lens, **i), torch.arange(n * cols, **i).reshape(n, cols)


@pytest.mark.parametrize("tokens,heads", [(1, 16), (9, 1), (1, 1)])
def test_appended_rows_that_have_no_stride(tokens, heads):
    """One token, or one head: strides that are never taken, and are no multiples of 8."""
    args = batch([tokens], [tokens + 70])
    table = ua.rope_table(100, R)

    def run(down, q, out):
        cache = torch.zeros((4, 64, L + R), dtype=BF, device="cuda")
        got = ua.append_latent(down[:, :L], down[:, L:L + R], cache, *args, q_rope=q,
                               q_rope_out=out, cos_sin=table)
        return cache, got.clone()

    down, q = rand(tokens, L + R), rand(tokens, heads, R, seed=1)
    want = run(down, q, torch.zeros_like(q))
    wide = torch.zeros((tokens, 580 if tokens == 1 else 584), dtype=BF, device="cuda")
    wide[:, :L + R] = down
    q2 = torch.zeros(q.numel() + 3, dtype=BF, device="cuda")
    step = (heads * R + 3 if tokens == 1 else R * heads, R + 5 if heads == 1 else R, 1)
    q2, out = (q2.as_strided(q.shape, step), torch.zeros_like(q2).as_strided(q.shape, step))
    q2.copy_(q)
    got = run(wide, q2, out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ua.device_status() == 0


def test_a_step_with_a_misaligned_tensor_leaves_the_call_as_it_was():
    cu, sl, bt = batch([1, 1], [100, 200])
    q, cache = rand(2, 8, L + R), rand(8, 64, L + R, seed=1)
    step = ua.prepare_latent_attention(q, cache, cu, sl, bt, scale=0.1, max_seqlen_q=1,
                                       max_seqlen_k=200)
    want = step().clone()
    odd = torch.zeros(q.numel() + 1, dtype=BF, device="cuda")[1:].reshape(q.shape)
    with pytest.raises(ua.UaError) as e:
        step(q=odd, stream=torch.cuda.Stream(priority=-1))
    assert e.value.code == 1
    step._last("out").zero_()
    assert torch.equal(step(), want)


def test_a_step_in_place_with_other_strides_is_refused():
    """Prepared apart, where the strides may differ, and then given one memory for both."""
    args = batch([3, 2], [40, 90])
    down, cache = rand(5, L + R), torch.zeros((8, 64, L + R), dtype=BF, device="cuda")
    table = ua.rope_table(100, R)
    whole = rand(5, 16, 128 + R, seed=1)
    q = whole[..., 128:]
    step = ua.prepare_append_latent(down[:, :L], down[:, L:], cache, *args, q_rope=q, cos_sin=table)
    want = step().clone()
    before = whole.clone()
    room = whole.flatten()[128:128 + want.numel()].view(want.shape)     # q's address, its own strides
    assert room.data_ptr() == q.data_ptr()
    with pytest.raises(ua.UaError):
        step(q_rope_out=room)
    assert torch.equal(whole, before)
    same = ua.prepare_append_latent(down[:, :L], down[:, L:], cache, *args, q_rope=q,
                                    q_rope_out=torch.zeros_like(whole)[..., 128:], cos_sin=table)
    assert torch.equal(same(q_rope_out=q), want)
    assert torch.equal(whole[..., :128], before[..., :128])


@pytest.mark.parametrize("tokens", [404, 408, 480, 540, 544])
def test_appends_where_a_warp_takes_one_pass_and_where_four(tokens):
    """About as many warps as 152 SMs hold, with a pass of query heads each."""
    appended.compare(appended.make([(tokens, tokens + 5), (1, 70)], 64), True)
