"""Rotary positions on several axes against the 64-bit form."""
import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from tests import _cache8_ref as ref
from tests.test_gpu_rope import bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def check(got, x, positions, axes, rates, gain, layout):
    """Each axis's pairs on their own: rates of the others are 0, so that they stay."""
    want = size = None
    for a in set(axes):
        on = torch.tensor([v == a for v in axes])
        w, s = ref.rope(x.cpu(), positions[a].cpu(), torch.where(on, rates, 0.0), 1.0, layout)
        keep = torch.zeros(128, dtype=torch.bool)
        h = len(axes)
        keep[: 2 * h] = torch.cat((on, on)) if layout == "half" else on.repeat_interleave(2)
        want, size = (w, s) if want is None else (torch.where(keep, w, want), torch.where(keep, s, size))
    keep = torch.arange(128) >= 2 * len(axes)
    want, size = torch.where(keep, x.cpu().double(), want * gain), size * gain
    err = (got.cpu().double() - want).abs()
    assert (err <= bound(want, size, got.dtype, positions.double().abs().max().item())).all(), f"off by {err.max():.3e}"


def inputs(a, b, h, hkv, n, dtype, seed=0, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(b, h, n, 128, generator=g).to(dtype).cuda()
    k = torch.randn(b, hkv, n, 128, generator=g).to(dtype).cuda()
    return q, k, torch.randint(-far, far, (a, b, n), generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [8, 16, 34, 64, 96, 128])
@pytest.mark.parametrize("a", [1, 2, 3, 4])
@pytest.mark.parametrize("b,h,hkv,n", [(1, 1, 1, 1), (3, 5, 1, 7), (2, 8, 2, 257)])
def test_turns(dtype, layout, rd, a, b, h, hkv, n):
    q, k, pos = inputs(a, b, h, hkv, n, dtype)
    axes = [(i * 5 + i // 3) % a for i in range(rd // 2)]
    axes[-1] = a - 1
    r = lkv.Rope(rotary_dim=rd, layout=layout, axes=axes)
    rates, _ = ref.rope_rates(rd)
    q2, k2 = r.apply(q, pos, k)
    check(q2, q, pos, axes, rates, 1.0, layout)
    check(k2, k, pos, axes, rates, 1.0, layout)
    assert torch.equal(r.apply(q, pos), q2)
    r.apply(q, pos, k, q_out=q, k_out=k)  # in place: the same bits
    assert torch.equal(q, q2) and torch.equal(k, k2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("own_base", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=4.0, orig_len=4096)])
@pytest.mark.parametrize("sections", [(64,), (16, 24, 24), (2, 30, 31, 1), (32, 32)])
def test_sections(layout, own_base, kw, sections):
    if own_base and kw.get("scaling") == "ntk" and 1 in sections:
        pytest.skip("no pair to stretch")
    q, k, pos = inputs(len(sections), 2, 8, 2, 33, torch.float32, seed=1)
    r = lkv.Rope(layout=layout, sections=sections, own_base=own_base, **kw)
    rates, gain = ref.rope_rates(128, **kw)
    if own_base:
        rates = torch.cat([ref.rope_rates(2 * s, **kw)[0] for s in sections])
    axes = [a for a, s in enumerate(sections) for _ in range(s)]
    q2, k2 = r.apply(q, pos, k)
    check(q2, q, pos, axes, rates, gain, layout)
    check(k2, k, pos, axes, rates, gain, layout)


def test_equal_positions_are_one_axis():
    """Text: the same position on every axis gives the bits of the call with one."""
    for dtype in (torch.bfloat16, torch.float32):
        q, k, pos = inputs(1, 4, 8, 2, 129, dtype, seed=2, far=1 << 30)
        one = lkv.Rope(base=1e6).apply(q, pos[0].contiguous(), k)
        three = lkv.Rope(base=1e6, sections=(16, 24, 24)).apply(q, pos.expand(3, -1, -1).contiguous(), k)
        assert all(torch.equal(x, y) for x, y in zip(one, three))


def test_far_positions():
    q, k, _ = inputs(3, 1, 2, 1, 4, torch.float32, seed=3)
    pos = torch.tensor([[[0, 2 ** 31 - 1, -2 ** 31, 5]], [[2 ** 31 - 1, 0, 7, -1]], [[-2 ** 31, 3, 2 ** 30, 1]]], dtype=torch.int32, device="cuda")
    axes = [i % 3 for i in range(64)]
    rates, _ = ref.rope_rates(128, base=5e6)
    r = lkv.Rope(base=5e6, axes=axes)
    check(r.apply(q, pos), q, pos, axes, rates, 1.0, "half")


def test_graph_and_stream():
    q, k, pos = inputs(2, 2, 4, 1, 3, torch.bfloat16, seed=4)
    r = lkv.Rope(sections=(32, 32))
    want = r.apply(q, pos, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.apply(q, pos, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = r.apply(q, pos, k)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    pos += 1
    graph.replay()
    again = r.apply(q, pos, k)
    assert torch.equal(got[0], again[0]) and not torch.equal(got[0], want[0])


def test_refusals():
    q, k, pos = inputs(3, 2, 4, 1, 3, torch.bfloat16, seed=5)
    r = lkv.Rope(sections=(16, 24, 24))
    for bad in (pos[0].contiguous(), pos[:2], pos.long(), pos.cpu(), pos[:, :, :2].contiguous(), pos.transpose(1, 2)):
        with pytest.raises((ValueError, TypeError)):
            r.apply(q, bad, k)
    with pytest.raises(ValueError):
        lkv.Rope().apply(q, pos, k)
    with pytest.raises(ValueError, match="requires a gradient"):
        r.apply(q.clone().requires_grad_(), pos)
    for kw in (dict(sections=(16, 24)), dict(sections=(0, 64)), dict(sections=(65, -1)), dict(sections=(12, 13, 13, 13, 13)), dict(axes=[0] * 63), dict(axes=[4] * 64),
               dict(axes=[-1] + [0] * 63), dict(sections=(64,), axes=[0] * 64), dict(own_base=True), dict(own_base=True, axes=[0] * 64)):
        with pytest.raises(ValueError):
            lkv.Rope(**kw)
