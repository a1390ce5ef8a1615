"""Rotary positions on the GPU against the 64-bit form."""
import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _cache8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def bound(want, size, dtype, far):
    """Both sides form a rate with a few fp64 roundings and this side's angle
    rounds once more: 8 * 2^-53 radians a position for rates up to 1. The fraction of a turn is cut at 2^-32 and rounded to fp32 (at most
    2^-25 of a turn in the argument of sincospi, which is two turns), the sine
    and cosine are good to 2 units (2^-23), the gain, two products and a sum
    round once each: 2^-24 of |x1| + |x2| a time. Then one rounding to dtype."""
    turn = 2 * 3.1416 * (2.0 ** -25 + 2.0 ** -32 + 2.0 ** -38) + far * 2.0 ** -50
    e = size * (turn + 2.0 ** -23 + 4 * 2.0 ** -24)
    return e + (want.abs() + e) * ref.half_step(dtype)


def check(got, x, positions, rates, gain, layout):
    want, size = ref.rope(x.cpu(), positions.cpu(), rates, gain, layout)
    err = (got.cpu().double() - want).abs()
    assert (err <= bound(want, size, got.dtype, positions.double().abs().max().item())).all(), f"off by {err.max():.3e}"


def inputs(b, h, hkv, n, dtype, seed=0, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(b, h, n, 128, generator=g).to(dtype).cuda()
    k = torch.randn(b, hkv, n, 128, generator=g).to(dtype).cuda() if hkv else None
    pos = torch.randint(0, far, (b, n), generator=g, dtype=torch.int32).cuda()
    return q, k, pos


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [2, 6, 16, 34, 48, 64, 96, 128])
@pytest.mark.parametrize("b,h,hkv,n", [(1, 1, 0, 1), (3, 5, 1, 7), (8, 32, 8, 1), (2, 8, 2, 257)])
def test_rope(dtype, layout, rd, b, h, hkv, n):
    q, k, pos = inputs(b, h, hkv, n, dtype)
    rates, gain = ref.rope_rates(rd)
    r = lkv.Rope(rotary_dim=rd, layout=layout)
    if hkv:
        q2, k2 = r.apply(q, pos, k)
        check(k2, k, pos, rates, gain, layout)
    else:
        q2 = r.apply(q, pos)
    check(q2, q, pos, rates, gain, layout)
    assert torch.equal(q2[..., rd:], q[..., rd:])
    # in place: the same bits
    r.apply(q, pos, k, q_out=q, k_out=k)
    assert torch.equal(q, q2) and (k is None or torch.equal(k, k2))


@pytest.mark.parametrize("kw", [
    dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=4.0, orig_len=4096)])
def test_rope_scaled_and_far(kw):
    """Stretched positions; positions at the ends of int32, and below zero."""
    q, k, pos = inputs(2, 4, 2, 50, torch.float32, seed=3)
    pos[0, :8] = torch.tensor([0, 1, 2**31 - 1, 2**31 - 2, -1, -2**31, 2**24 + 1, -12345], dtype=torch.int32)
    rates, gain = ref.rope_rates(128, **kw)
    q2, k2 = lkv.Rope(**kw).apply(q, pos, k)
    check(q2, q, pos, rates, gain, "half")
    check(k2, k, pos, rates, gain, "half")


def test_rope_more_heads_than_a_run_and_many_tokens():
    """Heads split over CTAs unevenly, and enough tokens that they are not."""
    for b, h, hkv, n in ((1, 37, 6, 3), (1, 3, 1, 20011)):
        q, k, pos = inputs(b, h, hkv, n, torch.bfloat16, seed=h)
        rates, gain = ref.rope_rates(128)
        q2, k2 = lkv.Rope().apply(q, pos, k)
        check(q2, q, pos, rates, gain, "half")
        check(k2, k, pos, rates, gain, "half")


def test_rope_captured_and_on_a_side_stream():
    q, k, pos = inputs(2, 4, 1, 5, torch.bfloat16, seed=9)
    r = lkv.Rope()
    want = r.apply(q, pos, k)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.apply(q, pos, k, q_out=qo, k_out=ko)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.apply(q, pos, k, q_out=qo, k_out=ko)
    pos += 17
    g.replay()
    want = r.apply(q, pos, k)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_rope_refuses():
    q, k, pos = inputs(2, 4, 2, 6, torch.bfloat16)
    r = lkv.Rope()
    with pytest.raises(ValueError):
        r.apply(q.transpose(1, 2).contiguous().transpose(1, 2), pos, k)  # strided
    with pytest.raises(ValueError):
        r.apply(q, pos[:, :5].contiguous(), k)
    with pytest.raises(TypeError):
        r.apply(q, pos.long(), k)
    with pytest.raises(TypeError):
        r.apply(q, pos, k.float())
    with pytest.raises(TypeError):
        r.apply(q.half(), pos)
    with pytest.raises(ValueError):
        r.apply(q, pos, k[:1])
    with pytest.raises(ValueError):
        r.apply(q, pos, k_out=k)
    with pytest.raises(ValueError):
        r.apply(q, pos.cpu(), k)
    flat = torch.zeros(q.numel() + 8, dtype=q.dtype, device="cuda")
    with pytest.raises(_lib.LKVError) as e:  # not 16-byte aligned
        r.apply(flat[1:1 + q.numel()].view(q.shape), pos)
    assert e.value.status == _lib.LKV_EINVAL
    with pytest.raises(_lib.LKVError):  # partly over its input
        r.apply(flat[:q.numel()].view(q.shape), pos, q_out=flat[8:].view(q.shape))
    assert r.apply(q[:0], pos[:0]).shape == (0, 4, 6, 128)
    assert r.apply(q[:, :, :0], pos[:, :0]).shape == (2, 4, 0, 128)
