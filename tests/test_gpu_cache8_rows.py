"""Attention of many rows over the 8-bit cache: prompts, chunks and batches of
drafts, at sizes that the kernel for many rows takes (a CTA a tile of 256 rows,
or streamed: all tiles' steps of 128 tokens shared out evenly), against the
plain 64-bit form with the bounds of the other attention tests."""
import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from tests.test_gpu_cache8 import FMTS, attend_case, check_attend, gen, i32, make, rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def many(seed, most):
    """64 lengths up to `most`: empty, single tokens, ends of blocks and of 128s."""
    some = [0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, most - 1, most]
    return some + torch.randint(1, most + 1, (64 - len(some),), generator=gen(seed)).tolist()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,n,window,sinks", [(8, 32, 0, 0), (3, 100, 0, 0), (1, 257, 0, 0), (16, 17, 0, 0), (128, 2, 0, 0), (4, 64, 1, 0),
                                                  (4, 64, 33, 17), (4, 70, 128, 1), (4, 70, 200, 300)])
def test_many_slices(fmt, group, n, window, sinks):
    attend_case(fmt, BF16, many(group, 300), 2, group, n, 320, seed=group + window, window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 5)])
def test_many_slices_padded(window, sinks):
    """Counts within and outside 0..n, above the length too: those rows are zero."""
    g = gen(5)
    counts = [-3, 0, 1, 31, 32, 33, 63, 64, 65, 1000] + torch.randint(0, 65, (54,), generator=g).tolist()
    lengths = many(6, 300)
    attend_case("int8", BF16, lengths, 2, 4, 64, 320, seed=6, counts=[min(c, n) if c < 64 else c for c, n in zip(counts, lengths)],
                window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lengths,h,group,n,window,sinks", [
    ([20001], 2, 4, 128, 0, 0), ([9000, 0, 1, 130, 20000, 8191], 1, 8, 100, 0, 0), ([12288, 12289], 3, 16, 33, 0, 0),
    ([30000, 5000], 2, 4, 200, 9000, 100), ([16000, 77, 16000], 1, 2, 300, 0, 0)])
def test_streamed(fmt, lengths, h, group, n, window, sinks):
    counts = [min(n, m) for m in lengths]
    attend_case(fmt, BF16, lengths, h, group, n, (max(lengths) + 15) // 16 * 16, seed=n, window=window, sinks=sinks, counts=counts)


def test_streamed_follows_lengths_not_the_bound():
    """The split is made for max_len (or the capacity), the work is the device's lengths'."""
    for lengths in ([300, 20000], [1, 2], [0, 0], [20000, 0]):
        attend_case("int8", BF16, lengths, 2, 4, 64, 20480, seed=11, counts=[min(64, m) for m in lengths])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lengths,h,n", [([2100], 1, 2100), ([4097, 3000], 2, 1500)])
def test_prompts_and_chunks(fmt, lengths, h, n):
    attend_case(fmt, BF16, lengths, h, 4, n, (max(lengths) + 15) // 16 * 16, seed=n, counts=[min(n, m) for m in lengths])


def jumps(b, h, group, n, length, seed):
    """Scores that climb: now and then a key along one query of its sequence,
    each louder than the last, so references move late, in either half of a
    step, for single rows and for all of them."""
    g = gen(seed)
    x, y = torch.randn(b, h, length, 128, generator=g), torch.randn(b, h, length, 128, generator=g)
    q = torch.randn(b, h * group, n, 128, generator=g)
    at = sorted(torch.randperm(length, generator=g)[:24].tolist())
    for i, t in enumerate(at):
        for s in range(b):
            for hh in range(h):
                r = int(torch.randint(0, n, (1,), generator=g))
                x[s, hh, t] = q[s, hh * group + i % group, r] * (1.0 + 0.5 * i)
    return q.to(BF16), x.to(BF16), y.to(BF16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("b,h,group,n,length", [(32, 2, 4, 64, 520), (1, 2, 4, 128, 16400)])
def test_references_move(fmt, b, h, group, n, length):
    q, x, y = jumps(b, h, group, n, length, seed=b + n)
    c, k, v = make(x, y, fmt, BF16, (length + 15) // 16 * 16, [length] * b)
    check_attend(c, k, v, [length] * b, q)
    check_attend(c, k, v, [length] * b, q, window=300, sinks=20)


def test_sizes_of_any_magnitude():
    for qs, ks, vs, scale in ((1e-20, 1e20, 1e10, None), (1e15, 1e-16, 1e-30, None), (1.0, 1.0, 1.0, -0.3), (1.0, 1.0, 1.0, 0.0)):
        g = gen(3)
        x, y = (torch.randn(64, 2, 300, 128, generator=g) * s for s in (ks, vs))
        q = torch.randn(64, 8, 64, 128, generator=g) * qs
        c, k, v = make(x.to(BF16), y.to(BF16), "int8", BF16, 304, [300] * 64)
        check_attend(c, k, v, [300] * 64, q.to(BF16), scale=scale)


def test_float32_many_rows():
    attend_case("int8", torch.float32, [300, 1, 0, 257] * 4, 2, 4, 64, 320, seed=13, counts=[64, 1, 0, 64] * 4)


@pytest.mark.parametrize("b,n,length", [(64, 64, 300), (1, 128, 20000)])
def test_repeats_captures_and_streams(b, n, length):
    """The same bits each time, captured and replayed with other lengths, and
    from two streams and two graphs at once."""
    g = gen(21)
    cap = (length + 15) // 16 * 16
    x, y = rows(g, b, 2, length, BF16), rows(g, b, 2, length, BF16)
    c, k, v = make(x, y, "int8", BF16, cap, [length] * b)
    qs = [torch.randn(b, 8, n, 128, generator=g).to(BF16).cuda() for _ in range(2)]
    want = [check_attend(c, k, v, [length] * b, q.cpu()) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.attend(qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    outs = [torch.zeros_like(q) for q in qs]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, q, out in zip(graphs, qs, outs):
        with torch.cuda.graph(graph):
            c.attend(q, out=out)
    for m in (1, length // 2, length):
        c.lengths.fill_(m)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], c.attend(qs[i]))
    for i in range(2):
        assert torch.equal(outs[i], want[i])
    c.check()


def test_rows_behind_a_sequence_and_garbage():
    """Codes, scales and tail rows past the length may hold anything."""
    g = gen(33)
    lengths = [100, 129, 16, 1] * 16
    x, y = rows(g, 64, 2, 150, BF16), rows(g, 64, 2, 150, BF16)
    q = torch.randn(64, 16, 32, 128, generator=g).to(BF16)
    counts = [min(32, m) for m in lengths]
    c, k, v = make(x, y, "e4m3", BF16, 256, lengths)
    want = check_attend(c, k, v, lengths, q, counts=counts)
    for i, m in enumerate(lengths):
        full = m // 16
        for codes, scale, tail in ((c.k_codes, c.k_scale, c.k_tail), (c.v_codes, c.v_scale, c.v_tail)):
            codes.view(torch.uint8)[i, :, full * 16:] = 0x7f  # a NaN of e4m3
            scale[i, :, full:] = float("nan")
            tail[i, :, (m - 1) % 16 + 1:] = float("inf")
    assert torch.equal(c.attend(q.cuda(), counts=i32(*counts)), want)


def test_refuses_sizes_past_32_bits():
    c = lkv.Cache8(batch=1, n_kv_heads=1, capacity=32, dtype=BF16)
    q = torch.zeros(1, 1, 1, 128, dtype=BF16, device="cuda")
    for kw in (dict(window=2 ** 32 + 5), dict(sinks=2 ** 31), dict(max_len=2 ** 40)):
        with pytest.raises(ValueError):
            c.attend(q, **kw)
    assert (c.attend(q, window=2 ** 31 - 1, sinks=2 ** 31 - 1, max_len=2 ** 31 - 1) == 0).all()


def test_outputs_without_the_short_allocation(monkeypatch):
    """A torch without it gives the same outputs, with the same layout."""
    from cluster_indexed_kv_gb300 import cache8
    g = gen(51)
    x, y = rows(g, 2, 2, 40, BF16), rows(g, 2, 2, 40, BF16)
    c, _, _ = make(x, y, "int8", BF16, 48, [40, 33])
    q = torch.randn(2, 8, 3, 128, generator=g).to(BF16).cuda()
    r, pos = lkv.Rope(), torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    k = q[:, :2].contiguous()

    def run():
        return [*c.read(40), c.attend(q), *r.apply(q, pos, k), r.apply(q, pos)]

    one = run()
    monkeypatch.setattr(cache8, "_empty_here", None)
    for a, b in zip(one, run()):
        assert torch.equal(a, b) and a.stride() == b.stride() and a.dtype == b.dtype and a.device == b.device
        assert a.is_contiguous()


@pytest.mark.parametrize("b,start,n,steps", [(1, 0, 6000, 12), (4, 8000, 1, 40), (16, 300, 48, 6)])
def test_calls_back_to_back(b, start, n, steps):
    """Rotate, write, attend and read in a row, each on what the one before it
    has just made: launches may overlap, accesses may not."""
    g = gen(61)
    total = start + n * steps + 16
    q = torch.randn(b, 8, n, 128, generator=g).to(BF16).cuda()
    k, v = (torch.randn(b, 2, n, 128, generator=g).to(BF16).cuda() for _ in range(2))
    k0, v0 = (torch.randn(b, 2, max(start, 1), 128, generator=g).to(BF16).cuda() for _ in range(2))
    r = lkv.Rope()

    def run(pause):
        c = lkv.Cache8(batch=b, n_kv_heads=2, capacity=(total + 15) // 16 * 16, dtype=BF16)
        got = []
        if start:
            c.write(k0, v0)
        x, y, z = q, k, v
        for i in range(steps):
            pos = (torch.arange(n, dtype=torch.int32, device="cuda") + c.lengths[:, None]).to(torch.int32)
            pause()
            x, y = r.apply(x, pos, y)
            pause()
            c.write(y, z)
            pause()
            x = c.attend(x, window=0 if i % 2 else 700, sinks=3)
            pause()
            y, z = c.read(n, first=c.lengths - n)
            pause()
            got.append(x)
        c.check()
        return got + [y, z, c.k_codes, c.k_tail, c.lengths]

    one = run(torch.cuda.synchronize)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            two = run(lambda: None)
        torch.cuda.synchronize()
        for a, b2 in zip(one, two):
            assert torch.equal(a.view(torch.uint8), b2.view(torch.uint8))
