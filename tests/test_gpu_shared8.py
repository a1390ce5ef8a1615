"""Attention behind shared prefixes: every output held to a bound of its own."""
import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _cache8_each as each
from tests import _cache8_ref as ref
from tests import _shared8_ref as sh
from tests.test_gpu_cache8 import DTYPES, FMTS, gen, i32, make, rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def cache(g, h, lengths, fmt, dtype, garbage=True, room=0):
    n = max(max(lengths), 1)
    x, y = rows(g, len(lengths), h, n, dtype), rows(g, len(lengths), h, n, dtype)
    return make(x, y, fmt, dtype, (n + 15) // 16 * 16 + room, lengths, g if garbage else None)


def check(c, p, prefix_of, lengths, prefix_lengths, q, *, counts=None, scale=None, max_len=0, got=None):
    """c and p: (Cache8, K's arrays, V's arrays)."""
    if got is None:
        got = c[0].attend_shared(q.cuda(), p[0], None if prefix_of is None else i32(*prefix_of), counts=None if counts is None else i32(*counts), scale=scale,
                                 max_len=max_len)
    n = q.shape[2]
    for b, length in enumerate(lengths):
        to = 0 if prefix_of is None else prefix_of[b]
        parts = [sh.sequence(*p[1:], to, prefix_lengths[to])] if 0 <= to < len(prefix_lengths) else []
        parts.append(sh.sequence(*c[1:], b, length))
        cnt = n if counts is None else min(max(counts[b], 0), n)
        want, lim = sh.attend(q[b].double(), parts, cnt, 128 ** -0.5 if scale is None else scale, q.dtype)
        err = (got[b].cpu().double() - want).abs()
        assert torch.isfinite(got[b]).all() and (err <= lim).all(), \
            f"sequence {b} behind {to}, {length} own tokens: off by {err.max():.3e}, {(err / lim.clamp_min(1e-300)).max():.2f} of the bound"
    return got


CASES = [  # prefixes' lengths, own lengths, prefix_of, KV heads, group, n
    ([1], [1], None, 1, 1, 1),
    ([16], [1, 2, 3], None, 2, 4, 1),
    ([777], [5, 16, 17, 200], None, 1, 2, 1),
    ([300, 33, 1], [40, 1, 64, 15, 90, 31], [0, 1, 0, 2, 0, -1], 2, 4, 3),
    ([0, 50], [7, 20, 3], [0, 1, 5], 2, 2, 2),
    ([64, 100], [12, 48, 13, 77, 12], [1, 0, 1, 1, 0], 3, 8, 12),
    ([2500], [30] * 9, None, 1, 4, 1),
    ([1000], [70, 65], None, 1, 4, 65),
    ([513, 40], [9] * 40, [b % 3 for b in range(40)], 1, 3, 2),
    ([130], [300, 150], None, 2, 16, 129),
    ([300], [20] * 16, None, 1, 1, 1),           # 16 rows, and 17
    ([300], [20] * 17, None, 1, 1, 1),
    ([300, 200], [20] * 7, [0, 1, 0, 1, 0, 1, 0], 2, 2, 4),   # 8 rows a sequence, and 9
    ([300, 200], [20] * 7, [0, 1, 0, 1, 0, 1, 0], 2, 3, 3),
    ([4000, 128, 127], [700, 256, 255, 129], [0, 1, 2, 0], 1, 128, 1),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES)
def test_shared(fmt, dtype, case):
    pre, own, to, h, group, n = case
    g = gen(len(own) * n)
    p, c = cache(g, h, pre, fmt, dtype), cache(g, h, own, fmt, dtype, room=32)
    q = torch.randn(len(own), h * group, n, 128, generator=g).to(dtype)
    got = check(c, p, to, own, pre, q)
    check(c, p, to, own, pre, q, max_len=max(own), scale=-0.2)
    again = c[0].attend_shared(q.cuda(), p[0], None if to is None else i32(*to))
    assert torch.equal(got, again)  # the same bits each time
    c[0].check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,group", [(1, 4), (4, 4), (40, 8)])
def test_counts_and_empty_sequences(dtype, n, group):
    """Padding is zero, whatever it holds; tokens of a sequence with fewer of its own than rows lie in the prefix."""
    pre, own, to = [100, 37, 0], [0, 1, 3, 50, 0, 20, 2, 5], [0, 1, 0, 0, -1, 1, 2, 0]
    g = gen(n)
    p, c = cache(g, 2, pre, "int8", dtype), cache(g, 2, own, "int8", dtype)
    q = torch.randn(8, 2 * group, n, 128, generator=g).to(dtype)
    for counts in (None, [n, 0, 1, n // 2, n, -3, n + 9, max(n - 1, 0)], [0] * 8):
        x = q.clone()
        if counts is not None:
            for b, cnt in enumerate(counts):
                x[b, :, max(cnt, 0):] = float("nan")
        got = c[0].attend_shared(x.cuda(), p[0], i32(*to), counts=None if counts is None else i32(*counts))
        check(c, p, to, own, pre, q, counts=counts, got=got)
        if counts is not None:
            for b, cnt in enumerate(counts):
                assert not got[b, :, max(cnt, 0):].any()


@pytest.mark.parametrize("fmt,dtype", [("int8", BF16), ("e4m3", F32)])
@pytest.mark.parametrize("pre,own,b,n", [(16 * 700 + 9, 16 * 5 + 3, 3, 1), (16 * 700 + 9, 16 * 5 + 3, 24, 2), (16 * 260, 16 * 130 + 1, 6, 30)])
def test_every_block_counts_once(fmt, dtype, pre, own, b, n):
    """Equal scores, and values that tell the blocks apart: the output of each row is a count of what it saw."""
    h, group = 2, 4
    zero = torch.zeros(1, h, pre, 128, dtype=dtype)
    p = make(zero, each.one_hot(pre, dtype).expand(1, h, -1, -1).contiguous(), fmt, dtype, (pre + 15) // 16 * 16, [pre])
    lengths = [own - i for i in range(b)]
    y = each.one_hot(own, dtype).flip(-1)
    c = make(torch.zeros(b, h, own, 128, dtype=dtype), y.expand(b, h, -1, -1).contiguous(), fmt, dtype, (own + 15) // 16 * 16, lengths)
    q = torch.randn(b, h * group, n, 128, generator=gen(b)).to(dtype)
    got = c[0].attend_shared(q.cuda(), p[0])
    for i, length in enumerate(lengths):
        vv = torch.cat((ref.values(*(t[0] for t in p[2]), pre), ref.values(*(t[i] for t in c[2]), length)), 1)[0]
        for r in range(n):
            seen = pre + length - n + r + 1
            want = vv[:seen].mean(0).expand(h * group, -1)
            err = (got[i, :, r].cpu().double() - want).abs()
            assert (err <= each.one_hot_bound(want, dtype, 2 * seen)).all(), (i, r, (err / want.clamp_min(1e-30)).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b", [3, 30])
def test_one_side_outweighs_the_other(dtype, b):
    """The prefix or the own tokens hold all the weight, or values of another size."""
    g = gen(b)
    for kx, ky, vx, vy in ((8.0, 0.1, 1, 1), (0.1, 8.0, 1, 1), (1, 1, 2.0 ** 40, 1), (1, 1, 1, 2.0 ** 40), (1, 1, 0, 1), (1, 1, 1, 0)):
        pre, own = [413], [50 + i for i in range(b)]
        x, y = (torch.randn(1, 2, 413, 128, generator=g) * s for s in (kx, vx))
        z, w = (torch.randn(b, 2, 90, 128, generator=g) * s for s in (ky, vy))
        p, c = make(x.to(dtype), y.to(dtype), "int8", dtype, 416, pre), make(z.to(dtype), w.to(dtype), "int8", dtype, 96, own)
        check(c, p, None, own, pre, torch.randn(b, 8, 2, 128, generator=g).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 20])
def test_a_bad_query_stays_alone(dtype, n):
    """NaN and infinities of one row give NaN in that row and nothing in the others, which share its tiles."""
    g = gen(3)
    pre, own = [500], [40] * 6
    p, c = cache(g, 2, pre, "int8", dtype), cache(g, 2, own, "int8", dtype)
    q = torch.randn(6, 8, n, 128, generator=g).to(dtype)
    want = c[0].attend_shared(q.cuda(), p[0])
    for bad in (float("nan"), float("inf")):
        x = q.clone()
        x[2, 3, n - 1, 5] = bad
        got = c[0].attend_shared(x.cuda(), p[0])
        assert got[2, 3, n - 1].isnan().all()
        got[2, 3, n - 1] = want[2, 3, n - 1]
        check(c, p, None, own, pre, q, got=got)


def test_a_prefix_in_the_cache_itself():
    g = gen(4)
    lengths = [333, 20, 5, 64]
    c = cache(g, 2, lengths, "int8", BF16)
    check(c, c, [-1, 0, 0, 3], lengths, lengths, torch.randn(4, 8, 1, 128, generator=g).to(BF16))


def test_lengths_out_of_range_are_cut():
    """What lies outside the arrays is not read."""
    g = gen(5)
    p, c = cache(g, 1, [64, 32], "int8", BF16, garbage=False), cache(g, 1, [48, 48, 48], "int8", BF16, garbage=False)
    q = torch.randn(3, 4, 1, 128, generator=g).to(BF16)
    p[0].lengths.copy_(i32(1 << 30, -5))
    c[0].lengths.copy_(i32(-1, 2 ** 31 - 1, 48))
    check(c, p, [0, 0, -1], [0, 48, 48], [64, 0], q, got=c[0].attend_shared(q.cuda(), p[0], i32(0, 0, 1)))
    c[0].check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_prefixes(dtype):
    """As many prefixes as sequences, some without a sequence."""
    g = gen(6)
    b = 70
    pre = [16 + 5 * i for i in range(b)]
    own = [3 + i % 20 for i in range(b)]
    to = [(i * 31 + 7) % b if i % 5 else (i * 13) % b for i in range(b)]
    p, c = cache(g, 1, pre, "e4m3", dtype), cache(g, 1, own, "e4m3", dtype)
    check(c, p, to, own, pre, torch.randn(b, 2, 1, 128, generator=g).to(dtype))


@pytest.mark.parametrize("n", [1, 17])
def test_the_most_sequences_and_prefixes(n):
    g = gen(7)
    b = 1024
    pre, own, to = [17] * b, [n + 1] * b, [(i * 5) % b if i % 3 else 7 for i in range(b)]
    p, c = cache(g, 1, pre, "int8", BF16), cache(g, 1, own, "int8", BF16)
    q = torch.randn(b, 1, n, 128, generator=g).to(BF16)
    got = c[0].attend_shared(q.cuda(), p[0], i32(*to))
    for i in range(0, b, 41):
        want, lim = sh.attend(q[i].double(), [sh.sequence(*p[1:], to[i], 17), sh.sequence(*c[1:], i, n + 1)], n, 128 ** -0.5, BF16)
        assert ((got[i].cpu().double() - want).abs() <= lim).all(), i
    more = lkv.Cache8(batch=1025, n_kv_heads=1, capacity=16, dtype=BF16)
    with pytest.raises(_lib.LKVError):
        c[0].attend_shared(q.cuda(), more)
    with pytest.raises(_lib.LKVError):
        more.attend_shared(torch.zeros(1025, 1, n, 128, dtype=BF16, device="cuda"), p[0])


@pytest.mark.parametrize("n", [1, 9, 20])
def test_offsets_past_32_bits(n):
    """A prefix whose codes take over 2^32 bytes: the heads at its end, attended and taken."""
    h, length = 136, (1 << 18) - 5
    capacity = 1 << 18
    g = torch.Generator(device="cuda").manual_seed(n)
    codes = [torch.randint(-127, 128, (1, h, capacity, 128), dtype=torch.int8, device="cuda", generator=g) for _ in range(2)]
    scale = [torch.full((1, h, capacity // 16), 2.0 ** -7, device="cuda") for _ in range(2)]
    tail = [torch.randn(1, h, 16, 128, device="cuda", generator=g).to(BF16) for _ in range(2)]
    p = lkv.Cache8.from_tensors(*codes, *scale, *tail, i32(length))
    c = cache(gen(n), h, [n + 3, n], "int8", BF16)
    q = torch.randn(2, h * 4, n, 128, generator=gen(n)).to(BF16)
    got = c[0].attend_shared(q.cuda(), p)
    for x in (0, h - 1):
        k, v = ([t[:, x:x + 1].cpu() for t in (codes[i], scale[i], tail[i])] for i in (0, 1))
        one, two = ([t[:, x:x + 1] for t in y] for y in c[1:])
        for b, own in enumerate((n + 3, n)):
            want, lim = sh.attend(q[b, 4 * x:4 * x + 4].double(), [sh.sequence(k, v, 0, length), sh.sequence(one, two, b, own)], n, 128 ** -0.5, BF16)
            assert ((got[b, 4 * x:4 * x + 4].cpu().double() - want).abs() <= lim).all(), (x, b)
    if n > 1:
        return
    d = lkv.Cache8(batch=1, n_kv_heads=h, capacity=capacity, dtype=BF16)
    d.take(p, lengths=i32(length - 16))
    for x in (0, h - 1):
        for y, z in ((d.k_codes, codes[0]), (d.v_codes, codes[1])):
            assert torch.equal(y[0, x, :length // 16 * 16 - 16], z[0, x, :length // 16 * 16 - 16])
    blocks = torch.arange(1, capacity // 16 - 1, 2, dtype=torch.int32, device="cuda").expand(1, h, -1).contiguous()
    kept = blocks.shape[2]
    d.keep(blocks, i32(kept))
    for x in (0, h - 1):
        for y, z in ((d.k_codes, codes[0]), (d.v_codes, codes[1])):
            assert torch.equal(y[0, x, :kept * 16].view(kept, 2048), z[0, x].view(-1, 2048)[blocks[0, x].long()])
    d.check()
    c[0].check()


@pytest.mark.parametrize("n", [1, 20])
def test_captured_with_lengths_that_change(n):
    """A graph follows the lengths, prefix_of and counts on the device; a second one runs on another stream meanwhile."""
    g = gen(8)
    b = 12
    graphs = []
    for k in range(2):
        p, c = cache(g, 2, [900, 400], "int8", BF16), cache(g, 2, [n + 3 * i for i in range(b)], "int8", BF16)
        q, to = torch.randn(b, 8, n, 128, generator=g).to(BF16).cuda(), i32(*[i % 2 for i in range(b)])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c[0].attend_shared(q, p[0], to)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = c[0].attend_shared(q, p[0], to)
        graphs.append((graph, p, c, q, to, out, side))
    for turn in range(4):
        for graph, p, c, q, to, out, side in graphs:
            q.normal_()
            to.random_(-1, 2)
            p[0].lengths.copy_(i32(900 - 100 * turn, 33 * turn))
            c[0].lengths.copy_(i32(*[max(n, n + 3 * i - turn) for i in range(b)]))
        torch.cuda.synchronize()
        for graph, *_, side in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for graph, p, c, q, to, out, side in graphs:
            # bits: a length cut without a take leaves rows of the tail that nobody wrote, NaN here
            assert torch.equal(out.view(torch.int16), c[0].attend_shared(q, p[0], to).view(torch.int16))
            c[0].check()


def test_refusals():
    g = gen(9)
    p, c = cache(g, 2, [40], "int8", BF16)[0], cache(g, 2, [5, 6], "int8", BF16)[0]
    q = torch.randn(2, 8, 1, 128, generator=g).to(BF16).cuda()
    for kw in (dict(h=3), dict(fmt="e4m3"), dict(dtype=F32)):
        a = dict(h=2, fmt="int8", dtype=BF16) | kw
        with pytest.raises(_lib.LKVError):
            c.attend_shared(q, cache(g, a["h"], [40], a["fmt"], a["dtype"])[0])
    for bad in (i32(0), i32(0, 0, 0), torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises((ValueError, TypeError)):
            c.attend_shared(q, p, bad)
    for bad in (q[:1], q.float(), q.cpu(), q[..., :64], q.transpose(0, 1), q[:, :3].contiguous()):
        with pytest.raises((ValueError, TypeError)):
            c.attend_shared(bad, p)
    with pytest.raises(TypeError):
        c.attend_shared(q, p._view)
    with pytest.raises(ValueError, match="requires a gradient"):
        c.attend_shared(q.clone().requires_grad_(), p)
    for kw in (dict(scale=float("nan")), dict(scale=3e38)):
        with pytest.raises(_lib.LKVError):
            c.attend_shared(q, p, **kw)
    for kw in (dict(max_len=-1), dict(max_len=2 ** 32)):
        with pytest.raises((_lib.LKVError, ValueError)):
            c.attend_shared(q, p, **kw)
    with pytest.raises(_lib.LKVError):
        c.attend_shared(q, p, out=q)
    assert c.attend_shared(torch.empty(2, 8, 0, 128, dtype=BF16, device="cuda"), p).shape == (2, 8, 0, 128)
    c.check()


@pytest.mark.parametrize("fmt,dtype", [("int8", BF16), ("e4m3", F32)])
def test_many_samples_of_one_prompt(fmt, dtype):
    """The calls together, as a server makes them: a prompt with positions on three axes goes into a prefix cache; samples
    step behind it; beams change places, drafts are given up; the result is that of each sample's rows read back."""
    g = gen(10)
    b, h, group, n = 4, 2, 2, 75
    rope = lkv.Rope(base=1e6, sections=(16, 24, 24))
    prefix = lkv.Cache8(batch=1, n_kv_heads=h, capacity=96, dtype=dtype, fmt=fmt)
    own = lkv.Cache8(batch=b, n_kv_heads=h, capacity=64, dtype=dtype, fmt=fmt)
    k, v = (torch.randn(1, h, n, 128, generator=g).to(dtype).cuda() for _ in range(2))
    i = torch.arange(n, device="cuda")
    grid = torch.stack((i // 25, i // 5 % 5, i % 5)).to(torch.int32).view(3, 1, n)
    _, k = rope.apply(k, grid, k)
    prefix.write(k, v)
    kk, vv = prefix.read(n)
    mine = None  # what the own cache held before a call, read back
    for step in range(30):
        at = torch.full((3, b, 1), 25 + step, dtype=torch.int32, device="cuda")
        q = torch.randn(b, h * group, 1, 128, generator=g).to(dtype).cuda()
        kn, vn = (torch.randn(b, h, 1, 128, generator=g).to(dtype).cuda() for _ in range(2))
        q, kn = rope.apply(q, at, kn)
        own.write(kn, vn)
        out = own.attend_shared(q, prefix)
        ko, vo = own.read(64)
        lengths = own.lengths.tolist()
        for x in range(b):
            assert torch.equal(ko[x, :, lengths[x] - 1], kn[x, :, 0]) or lengths[x] % 16 == 0
            ks = torch.cat((kk[0], ko[x, :, :lengths[x]]), 1).double().repeat_interleave(group, 0)
            vs = torch.cat((vv[0], vo[x, :, :lengths[x]]), 1).double().repeat_interleave(group, 0)
            want = torch.softmax(q[x].double() @ ks.transpose(1, 2) * 128 ** -0.5, -1) @ vs
            # rows read back are rounded to the type once, so scores are off by half a step of |q k|; weights as in the bounds above
            size = (q[x].double().abs() @ ks.abs().transpose(1, 2)).max().item() * 128 ** -0.5
            half = ref.half_step(dtype)
            d = size * (half + 2.0 ** -17) + (2 * size + 16) * 2.0 ** -22
            weights = 2.0 ** -11 + 2.0 ** -24 if dtype == BF16 else 2.0 ** -23
            lim = vs.abs().max().item() * (torch.expm1(torch.tensor(2 * d)).item() + half + 2 * weights + 80 * 2.0 ** -23)
            assert ((out[x].double() - want).abs() <= lim + (want.abs() + lim) * half).all(), (step, x)
        if step % 5 == 4:
            order = [(x * 3 + step) % b if x else 2 for x in range(b)]
            own.take(sequences=i32(*order))
            mine = own.read(64)
            assert own.lengths.tolist() == [lengths[x] for x in order]
            assert torch.equal(mine[0], ko[order]) and torch.equal(mine[1], vo[order])
        if step % 7 == 6:
            mine, before = own.read(64), own.lengths.tolist()
            own.take(lengths=own.lengths - 3)
            now = own.read(64)
            for x in range(b):
                m = before[x] - 3
                assert torch.equal(now[0][x, :, :m], mine[0][x, :, :m]) and not now[0][x, :, m:].any()
    kept = i32(*[x // 16 for x in own.lengths.tolist()])
    blocks = torch.arange(4, dtype=torch.int32, device="cuda").expand(b, h, 4).contiguous()
    before = own.read(64)
    own.keep(blocks, kept)  # everything stays
    assert all(torch.equal(x, y) for x, y in zip(before, own.read(64)))
    own.check()
    prefix.check()


@pytest.mark.parametrize("b,n", [(120, 3), (90, 3), (120, 2), (60, 4), (60, 5)])
def test_own_tokens_of_some_rows(b, n):
    """8 to 20 rows a sequence, of more sequences and fewer: either kernel takes their own tokens."""
    own = [1 + 7 * i % 30 for i in range(b)]
    g = gen(b + n)
    p, c = cache(g, 2, [300, 70], "int8", BF16), cache(g, 2, own, "int8", BF16)
    to = [i % 2 for i in range(b)]
    q = torch.randn(b, 8, n, 128, generator=g).to(BF16)
    check(c, p, to, own, [300, 70], q)
    counts = [i % (n + 1) for i in range(b)]
    check(c, p, to, own, [300, 70], q, counts=counts, max_len=max(own))
    c[0].check()


@pytest.mark.parametrize("fmt,dtype,b,n", [("int8", BF16, 4, 1), ("e4m3", F32, 3, 2), ("int8", BF16, 40, 1), ("e4m3", BF16, 12, 3)])
def test_steps_in_a_row(fmt, dtype, b, n):
    """Writes and attentions by turns with nothing between them: each sees what was written before it, and no later."""
    g = gen(b)
    pre = [700, 20]
    p, c = cache(g, 2, pre, fmt, dtype), cache(g, 2, [33] * b, fmt, dtype, room=96)
    to = i32(*[i % 2 for i in range(b)])
    d = c[0]
    steps = [torch.randn(3, b, 8, n, 128, generator=g).to(dtype).cuda() for _ in range(12)]
    start = [t.clone() for t in (d.k_codes.view(torch.int8), d.v_codes.view(torch.int8), d.k_scale, d.v_scale, d.k_tail, d.v_tail, d.lengths)]
    got = []
    for apart in (False, True):
        for t, x in zip((d.k_codes.view(torch.int8), d.v_codes.view(torch.int8), d.k_scale, d.v_scale, d.k_tail, d.v_tail, d.lengths), start):
            t.copy_(x)
        torch.cuda.synchronize()
        outs = []
        for x in steps:
            d.write(x[1, :, :2].contiguous(), x[2, :, :2].contiguous())
            if apart:
                torch.cuda.synchronize()
            outs.append(d.attend_shared(x[0], p[0], to))
            if apart:
                torch.cuda.synchronize()
        got.append(outs)
    for x, y in zip(*got):
        assert torch.equal(x, y)
    d.check()


@pytest.mark.parametrize("fmt,dtype", [("int8", BF16), ("e4m3", F32)])
@pytest.mark.parametrize("pre,b,h", [
    ([2000, 16, 700, 1, 9000], 4, 2), ([17] * 40 + [3000], 41, 1), ([16 * 16 * 9], 4, 2), ([16 * 16 * 9 + 1], 4, 2), ([16 * 16 * 200], 2, 1), ([48], 3, 5)])
def test_few_rows_of_uneven_prefixes(fmt, dtype, pre, b, h):
    """Tiles of 16 rows: short prefixes beside long ones, and one whose blocks are shared evenly, or not quite."""
    g = gen(len(pre) + b)
    own = [1 + 5 * i % 40 for i in range(b)]
    p, c = cache(g, h, pre, fmt, dtype), cache(g, h, own, fmt, dtype)
    to = [(i * 3 + 4) % len(pre) for i in range(b)]
    q = torch.randn(b, 2 * h, 1, 128, generator=g).to(dtype)
    check(c, p, to, own, pre, q)
    check(c, p, to, own, pre, q, max_len=40)
    c[0].check()


@pytest.mark.parametrize("fmt,dtype,b,own,n", [
    ("int8", BF16, 4, 33, 1), ("int8", BF16, 3, 700, 1), ("e4m3", BF16, 2, 5000, 2), ("e4m3", F32, 3, 33, 2), ("int8", F32, 2, 2000, 4),
    ("int8", BF16, 40, 33, 1), ("e4m3", BF16, 9, 300, 2), ("int8", BF16, 6, 40, 20)])
def test_own_tokens_taken_again(fmt, dtype, b, own, n):
    """The first kernel's word for what was written before the call comes late: the second takes the own tokens again, of
    every step what was written before it, and the bits are those of a word in time."""
    g = gen(b + own)
    p, c = cache(g, 2, [700, 20], fmt, dtype), cache(g, 2, [max(own - 3 * i, 1) for i in range(b - 1)] + [0], fmt, dtype, room=96)
    to = i32(*[i % 3 - 1 for i in range(b)])
    d = c[0]
    steps = [torch.randn(3, b, 8, n, 128, generator=g).to(dtype).cuda() for _ in range(3)]
    start = [t.clone() for t in (d.k_codes.view(torch.int8), d.v_codes.view(torch.int8), d.k_scale, d.v_scale, d.k_tail, d.v_tail, d.lengths)]
    got = []
    for late in (False, True):
        for t, x in zip((d.k_codes.view(torch.int8), d.v_codes.view(torch.int8), d.k_scale, d.v_scale, d.k_tail, d.v_tail, d.lengths), start):
            t.copy_(x)
        _lib.lkv_diag_shared_late(late)
        try:
            outs = []
            for x in steps:
                d.write(x[1, :, :2].contiguous(), x[2, :, :2].contiguous())
                outs.append(d.attend_shared(x[0], p[0], to))
        finally:
            _lib.lkv_diag_shared_late(False)
        torch.cuda.synchronize()
        got.append(outs)
    for x, y in zip(*got):
        assert torch.equal(x, y)
    d.check()


@pytest.mark.parametrize("fmt,pre,b,h,group,n,step", [
    ("int8", [20 + i % 300 for i in range(200)], 200, 2, 2, 1, 0), ("e4m3", [20 + i % 300 for i in range(200)], 200, 2, 2, 1, 1),
    ("int8", [300] * 100, 100, 2, 2, 20, 0), ("int8", [40000, 64], 40, 2, 4, 2, 3), ("int8", [700], 8, 2, 4, 64, 1)])
def test_a_wait_that_gives_up(fmt, pre, b, h, group, n, step):
    """Products that never come: the waits for them end, every tile and part of the call is told of all the same (the second
    kernel finds its way by them), the call is reported, and the next one is right."""
    g = gen(b + n + step)
    own = [n + i % 40 for i in range(b)]
    p, c = cache(g, h, pre, fmt, BF16)[0], cache(g, h, own, fmt, BF16)[0]
    to = i32(*[i % len(pre) for i in range(b)])
    q = torch.randn(b, h * group, n, 128, generator=g).to(BF16).cuda()
    want = c.attend_shared(q, p, to)
    c.check()
    R = n * group
    listed = [-(-sum(x % len(pre) == y for x in range(b)) * R // 128) * h for y in range(len(pre))] + ([-(-R // 128) * h] * b if R > 16 else [])
    most = (-(-b * R // 128) + min(len(pre), b)) * h + (b * h * -(-R // 128) if R > 16 else 0)
    bytes_ = _lib.lkv_cache8_attend_shared_workspace(c._at, p._at, group, n, 0)
    ws = torch.zeros(bytes_, dtype=torch.uint8, device="cuda")  # a tile that is not told of: no parts
    tiles_at = 16 + 16 * b
    parts_at = tiles_at + (8 * most + 15) // 16 * 16
    ws[parts_at:] = 255  # a part that is not told of: NaN
    _lib.lkv_diag_shared_hold(step, 1_000_000)
    try:
        _lib._check(_lib.load().lkv_cache8_attend_shared(c._at, p._at, to.data_ptr(), q.data_ptr(), group, n, None, 128 ** -0.5, 0,
                                                         torch.empty_like(q).data_ptr(), ws.data_ptr(), bytes_, torch.cuda.current_stream().cuda_stream), None)
    finally:
        _lib.lkv_diag_shared_hold(-1)
    with pytest.raises(_lib.LKVError) as e:
        c.check()
    assert e.value.status == _lib.LKV_ETIMEOUT
    tiles = ws[tiles_at:tiles_at + 8 * sum(listed)].view(torch.int32).view(-1, 2).cpu()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (tiles[:, 0] >= 0).all() and (tiles[:, 1] >= 1).all() and (tiles.sum(1) <= sms).all()
    parts = ws[parts_at:].view(torch.float32).view(-1, 128 * 131).cpu()
    for t, (first, count) in enumerate(tiles.tolist()):
        assert not parts[first + t:first + t + count, 128 * 128:128 * 130].isnan().any(), t
    assert torch.equal(c.attend_shared(q, p, to), want)
    c.check()


def test_a_call_that_does_not_come_to_the_step():
    """... has waited for nothing that did not come: it is right."""
    g = gen(11)
    p, c = cache(g, 2, [5000, 64], "int8", BF16)[0], cache(g, 2, [2 + i for i in range(40)], "int8", BF16)[0]
    to, q = i32(*[i % 2 for i in range(40)]), torch.randn(40, 8, 2, 128, generator=g).to(BF16).cuda()
    want = c.attend_shared(q, p, to)
    _lib.lkv_diag_shared_hold(40, 1_000_000)
    try:
        assert torch.equal(c.attend_shared(q, p, to), want)
    finally:
        _lib.lkv_diag_shared_hold(-1)
    c.check()


def test_a_wait_that_gives_up_refuses_limits():
    for limit in (0, -1, 1_000_000_001):
        with pytest.raises(_lib.LKVError):
            _lib.lkv_diag_shared_hold(0, limit)
    _lib.lkv_diag_shared_hold(-1, 0)


@pytest.mark.parametrize("dtype,b,n", [(BF16, 4, 1), (F32, 2, 1), (F32, 3, 4), (BF16, 9, 1)])
def test_one_cache_behind_prefixes_of_several_capacities(dtype, b, n):
    """Prompts of different lengths in caches of their own, by turns behind one cache, in either order."""
    g = gen(b)
    h, group = 8, 4
    lengths = [20 + i for i in range(b)]
    prompts = [cache(g, h, [length], "int8", dtype, room=room) for length, room in ((500, 32768 - 512), (2040, 0), (512, 0))]
    q = torch.randn(b, h * group, n, 128, generator=g).to(dtype)
    for order in ((0, 1, 2), (2, 1, 0)):
        c = cache(gen(b + 1), h, lengths, "int8", dtype, room=256 - 32)
        for x in order:
            check(c, prompts[x], None, lengths, [(500, 2040, 512)[x]], q)
        sizes = {_lib.lkv_cache8_attend_shared_workspace(c[0]._at, prompts[x][0]._at, group, n, 0) for x in order}
        assert len(sizes) == 1


@pytest.mark.parametrize("dtype,b,n", [(BF16, 4, 1), (BF16, 1, 1), (F32, 2, 1), (F32, 4, 4)])
def test_a_short_prefix_in_a_large_cache(dtype, b, n):
    """The split goes by the prefix cache's capacity: what it holds may be a small part of that, or nothing."""
    g = gen(b)
    lengths = [20 + i for i in range(b)]
    q = torch.randn(b, 32, n, 128, generator=g).to(dtype)
    c = cache(g, 8, lengths, "int8", dtype, room=64)
    for pre in (0, 1, 100, 1000):
        check(c, cache(g, 8, [pre], "int8", dtype, room=32768), None, lengths, [pre], q)
    c[0].check()
