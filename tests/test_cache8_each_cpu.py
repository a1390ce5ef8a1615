"""What the token-by-token attention tests can see (no GPU): their plain form
agrees with the other one, and losing or doubling a block breaks their bounds."""
import pytest
import torch

from tests import _cache8_each as each
from tests import _cache8_ref as ref


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("length,n,count,window,sinks", [(1, 1, 1, 0, 0), (300, 5, 3, 0, 0), (97, 40, 40, 20, 3), (5, 9, 9, 2, 1)])
def test_the_two_plain_forms_agree(dtype, length, n, count, window, sinks):
    g = gen(length)
    k, v = (torch.randn(2, length, 128, generator=g).to(dtype).double() for _ in range(2))
    q = torch.randn(6, n, 128, generator=g).to(dtype).double()
    u = torch.full((2, length), 2.0 ** -5, dtype=torch.float64)
    one, lim = each.attend(q, k, v, u, count, 0.09, window, sinks, dtype)
    two, _, _ = ref.attend(q, k, v, count, 0.09, window, sinks)
    assert (one - two).abs().max() <= 1e-12
    assert (lim[:, :count][two[:, :count] != 0] > 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("length", [9000, 20011, 40000])
def test_a_lost_or_doubled_block_is_seen(dtype, length):
    """Equal scores and values that name their block: every block matters."""
    v = each.one_hot(length, torch.float64)
    total, blocks = v.sum(0), v[:length // 16 * 16].view(-1, 16, 128).sum(1)
    want = total / length
    lim = each.one_hot_bound(want, dtype, length)
    for sign in (-1, 1):
        got = (total + sign * blocks) / (length + sign * 16)
        assert ((got - want).abs() > lim).any(1).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_lost_block_breaks_the_bound_of_single_outputs(dtype):
    """Ordinary rows of some hundreds of tokens: a lost block is far outside."""
    g = gen(3)
    length = 640
    k, v = (torch.randn(1, length, 128, generator=g).to(dtype).double() for _ in range(2))
    q = torch.randn(4, 1, 128, generator=g).to(dtype).double()
    u = torch.full((1, length), 2.0 ** -5, dtype=torch.float64)
    want, lim = each.attend(q, k, v, u, 1, 128 ** -0.5, 0, 0, dtype)
    for b in range(length // 16):
        keep = torch.ones(length, dtype=torch.bool)
        keep[16 * b:16 * b + 16] = False
        got, _ = each.attend(q, k[:, keep], v[:, keep], u[:, keep], 1, 128 ** -0.5, 0, 0, dtype)
        assert ((got - want).abs() > lim).any(-1).all(), b
