"""GPU: latent calls at the edges of what their arguments may be."""
import pytest
import torch

import varlen_gqa_attention_paged_gb300 as ua
from tests import _latent_ref as ref
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


@pytest.mark.parametrize("most", [0, 1 << 20])
def test_prefill_of_no_keys_at_all(most):
    cu = torch.tensor([0, 3, 3, 200], dtype=torch.int32, device="cuda")
    q, kv = rand(200, 4, 128 + R), rand(0, 4, 256)
    out, lse = ua.latent_prefill(q, kv[..., :128], rand(0, R), kv[..., 128:], cu, torch.zeros_like(cu),
                                 max_seqlen_q=197, max_seqlen_k=most, return_lse=True,
                                 out=torch.full((200, 4, 128), 7.0, dtype=BF, device="cuda"))
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))
    assert ua.device_status() == 0


def test_sequences_that_share_blocks_and_slots_of_the_batch_that_are_empty():
    """A prefix in the tables of three sequences; sequences without tokens whose lengths are left over
    from before; both ways of cutting the keys."""
    lens = [(1, 300), (3, 290), (1, 256), (0, 999), (0, 70), (0, 1)]
    cu = torch.tensor([0, 1, 4, 5, 5, 5, 5]).int()
    sl = torch.tensor([k for _, k in lens]).int()
    bt = torch.tensor([[2, 0, 5, 1, 7], [2, 0, 5, 1, 3], [2, 0, 5, 1, -1]] + [[-1] * 5] * 3).int()
    q, cache = rand(9, 16, L + R), rand(8, 64, L + R, seed=1)
    want, wlse, tol, ltol = ref.attend(q.cpu(), cache.cpu(), cu[:4], sl[:3], bt[:3], L, 0.08)
    for most in (300, (1 << 31) - 1):
        out = torch.full((9, 16, L), 7.0, dtype=BF, device="cuda")
        out, lse = ua.latent_attention(q, cache, cu.cuda(), sl.cuda(), bt.cuda(), scale=0.08,
                                       max_seqlen_q=3, max_seqlen_k=most, out=out, return_lse=True)
        ref.check(out[:5], want[:5], tol[:5], BF)
        ref.check(lse[:5], wlse[:5], ltol[:5], torch.float32)
        assert torch.all(out[5:] == 7)
    assert ua.device_status() == 0
