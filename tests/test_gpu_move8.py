"""Taking and keeping tokens of the 8-bit cache: every bit of what it holds after."""
import random
import subprocess
import sys

import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _move8_ref as mv
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def upload(cache):
    (k, v), lengths = cache
    t = [x.cuda() for x in (k[0], v[0], k[1], v[1], k[2], v[2])]
    return lkv.Cache8.from_tensors(*t, torch.tensor(lengths, dtype=torch.int32).cuda())


def download(c):
    return [(c.k_codes.cpu(), c.k_scale.cpu(), c.k_tail.cpu()), (c.v_codes.cpu(), c.v_scale.cpu(), c.v_tail.cpu())], c.lengths.tolist()


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32).cuda()


def checked(c, bad):
    if bad:
        with pytest.raises(_lib.LKVError):
            c.check()
    c.check()
    assert not c._ticket.any()


TYPES = [("int8", BF16), ("e4m3", BF16), ("int8", F32), ("e4m3", F32)]


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("b,sources,h,n", [(1, 1, 1, 1), (3, 2, 2, 40), (5, 1, 8, 700), (40, 7, 1, 95), (2, 33, 3, 2049)])
def test_take_from_another_cache(fmt, dtype, b, sources, h, n):
    r = random.Random(b * n)
    have = [max(0, n - r.randrange(0, 1 + n // 2) * (s > 0)) for s in range(sources)]
    room = (n + 47) // 16 * 16
    src, dst = mv.filled(sources, h, room, fmt, dtype, have, 1), mv.filled(b, h, room - 16, fmt, dtype, [r.randrange(0, n + 1) for _ in range(b)], 2)
    s, d = upload(src), upload(dst)
    for turn in range(3):
        to = None if turn == 0 and b <= sources else [r.randrange(-1, sources) for _ in range(b)]
        some = to if to is not None else list(range(b))
        lengths = None if turn == 1 else [r.randrange(0, have[x] + 1) if x >= 0 else -5 for x in some]
        want, bad = mv.take(dst, src, to, lengths)
        assert not bad
        d.take(s, ints(to), ints(lengths))
        mv.same(download(d), want)
        checked(d, bad)
        dst = download(d)
    mv.same(download(s), src)


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("b,h,n", [(1, 1, 30), (2, 3, 64), (6, 2, 333), (33, 1, 170), (300, 1, 50), (1024, 1, 33)])
def test_take_within_a_cache(fmt, dtype, b, h, n):
    """Any order at once: rotations, copies, cuts; what others held before the call."""
    r = random.Random(b + n)
    have = [r.randrange(0, n + 1) for _ in range(b)]
    c = mv.filled(b, h, (n + 31) // 16 * 16, fmt, dtype, have, 3)
    d = upload(c)
    for turn in range(4):
        to = [None, [(i + 1) % b for i in range(b)], [r.randrange(-1, b) for _ in range(b)], [i // 2 for i in range(b)]][turn]
        some = to if to is not None else list(range(b))
        lengths = None if turn == 1 else [r.randrange(0, c[1][x] + 1) if x >= 0 else 0 for x in some]
        want, bad = mv.take(c, c, to, lengths)
        assert not bad
        d.take(sequences=ints(to), lengths=ints(lengths))
        mv.same(download(d), want)
        checked(d, bad)
        c = download(d)


@pytest.mark.parametrize("b,h,n", [(24, 2, 6000), (200, 2, 2500), (520, 1, 1100)])
def test_take_within_a_cache_of_narrow_columns(b, h, n):
    """Many sequences of many blocks: a block's bytes are several CTAs' work, which
    its scale and the tails made of it must not depend on."""
    r = random.Random(b)
    have = [r.randrange(n - 400, n + 1) for _ in range(b)]
    d = lkv.Cache8(batch=b, n_kv_heads=h, capacity=(n + 31) // 16 * 16, dtype=BF16, fmt="int8")
    g = torch.Generator(device="cuda").manual_seed(b)
    for x in (d.k_codes, d.v_codes):
        x.copy_(torch.randint(-127, 128, x.shape, device="cuda", generator=g))
    for x in (d.k_scale, d.v_scale, d.k_tail, d.v_tail):
        x.copy_(torch.rand(x.shape, device="cuda", generator=g) + .01)
    d.lengths.copy_(ints(have))
    c = download(d)
    for turn in range(4):
        to = [(i + 1 + turn) % b for i in range(b)] if turn % 2 == 0 else [r.randrange(b) for _ in range(b)]
        lengths = [c[1][x] if r.random() < .3 else r.randrange(c[1][x] // 2, c[1][x] + 1) for x in to]
        want, bad = mv.take(c, c, to, lengths)
        assert not bad
        d.take(sequences=ints(to), lengths=ints(lengths))
        mv.same(download(d), want)
        checked(d, bad)
        c = download(d)


@pytest.mark.parametrize("inside", [False, True])
def test_take_of_what_is_not_there(inside):
    """Such sequences are left as they are, the others are not."""
    c = mv.filled(6, 2, 64, "int8", BF16, [20, 33, 0, 64, 17, 5], 4)
    src = c if inside else mv.filled(4, 2, 128, "int8", BF16, [20, 128, 0, 64], 5)
    d = upload(c)
    s = None if inside else upload(src)
    cases = [([0, 9, 2, 3, 4, -2], [20, 1, 0, 10, 3, 1]), ([1, 1, 1, 1, 1, 1], [-1, 2 ** 31 - 1, 200, -2 ** 31, 30, 10]), ([3, 3, 1, 0, -1, 2], [65, 64, 66, 21, 7, 1])]
    for to, lengths in cases:
        now = download(d)
        want, bad = mv.take(now, now if inside else src, to, lengths)
        assert bad
        d.take(s, ints(to), ints(lengths))
        mv.same(download(d), want)
        checked(d, bad)


def test_take_of_each_ones_own_from_a_smaller_cache():
    """Without a list, sequences that the source does not have are refused."""
    src, dst = mv.filled(2, 1, 64, "int8", BF16, [50, 3], 1), mv.filled(4, 1, 64, "int8", BF16, [3, 4, 5, 6], 2)
    s, d = upload(src), upload(dst)
    want, bad = mv.take(dst, src, None, None)
    assert bad == {2, 3}
    d.take(s)
    mv.same(download(d), want)
    checked(d, bad)


def test_take_past_the_capacity_is_reported_as_that():
    src, dst = mv.filled(1, 1, 64, "int8", BF16, [50], 1), mv.filled(2, 1, 32, "int8", BF16, [3, 4], 2)
    s, d = upload(src), upload(dst)
    d.take(s, ints([0, 0]), ints([50, 32]))
    with pytest.raises(_lib.LKVError) as e:
        d.check()
    assert e.value.status == _lib.LKV_ECAPACITY
    assert d.lengths.tolist() == [3, 32]


@pytest.mark.parametrize("fmt,dtype", TYPES)
def test_a_cut_sequence_goes_on(fmt, dtype):
    """Cut back inside an older block, then written to: as if the rows read back had been written."""
    c = mv.filled(2, 2, 128, fmt, dtype, [100, 96], 6)
    d = upload(c)
    k0, v0 = d.read(100)
    d.take(lengths=ints([37, 48]))
    k1, v1 = d.read(48)
    for x, y in ((k0, k1), (v0, v1)):
        assert torch.equal(x[0, :, :37], y[0, :, :37]) and torch.equal(x[1, :, :48], y[1, :, :48]) and not y[0, :, 37:].any()
    new = torch.randn(2, 2, 20, 128, device="cuda").to(dtype)
    d.write(new, new)
    other = lkv.Cache8(batch=2, n_kv_heads=2, capacity=128, dtype=dtype, fmt=fmt)
    other.take(d, lengths=ints([32, 48]))
    both = torch.cat((k0[:1, :, 32:37], new[:1]), 2), torch.cat((v0[:1, :, 32:37], new[:1]), 2)
    pad = torch.zeros(1, 2, 25, 128, device="cuda", dtype=dtype)
    rest = new[1:], new[1:]
    other.write(*(torch.cat((x, torch.cat((y, pad[:, :, :5]), 2))) for x, y in zip(both, rest)), counts=ints([25, 20]))
    assert d.lengths.tolist() == other.lengths.tolist() == [57, 68]
    for x, y in zip(d.read(80), other.read(80)):
        assert torch.equal(x, y)
    for x, y in ((d.k_tail, other.k_tail), (d.v_tail, other.v_tail)):
        assert torch.equal(x[0, :, :9], y[0, :, :9]) and torch.equal(x[1, :, :4], y[1, :, :4])
    d.check()
    other.check()


@pytest.mark.parametrize("fmt,dtype", TYPES)
@pytest.mark.parametrize("b,h,n", [(1, 1, 16), (1, 2, 2047), (3, 8, 300), (9, 4, 1000), (70, 3, 64)])
@pytest.mark.parametrize("inside", [False, True])
def test_keep(fmt, dtype, b, h, n, inside):
    r = random.Random(n)
    have = [max(0, n - 7 * x if x % 2 else n // 16 * 16 - 16 * (x // 2)) for x in range(b)]
    room = (n + 31) // 16 * 16
    src = mv.filled(b, h, room, fmt, dtype, have, 7)
    s = upload(src)
    for turn in range(3):
        c = mv.filled(b, h, room, fmt, dtype, [r.randrange(0, n + 1) for _ in range(b)], 8)
        if inside:
            c = src = download(s)
        d = s if inside else upload(c)
        full = [x // 16 for x in src[1]]
        counts = [r.choice([-1, 0, f, r.randrange(0, f + 1), r.randrange(0, f + 1), r.randrange(0, f + 1)]) for f in full]
        m = max(max(counts), 1) + turn
        blocks = [[sorted(r.sample(range(f), max(k, 0))) + [-9] * (m - max(k, 0)) for _ in range(h)] for f, k in zip(full, counts)]
        want, bad = mv.keep(c, src, blocks, counts)
        assert not bad
        d.keep(ints(blocks), ints(counts), None if inside else s)
        mv.same(download(d), want)
        checked(d, bad)


@pytest.mark.parametrize("inside", [False, True])
def test_keep_of_what_is_not_there(inside):
    """A bad list of one head leaves the whole sequence as it is."""
    src = mv.filled(8, 2, 96, "e4m3", BF16, [96, 90, 50, 33, 96, 96, 16, 0], 9)
    c = src if inside else mv.filled(8, 2, 64, "e4m3", BF16, [1, 2, 3, 64, 5, 6, 7, 8], 10)
    s = upload(src)
    d = s if inside else upload(c)
    ok = [0, 1, 2, 3, 4, 5]
    blocks = [[ok, ok], [ok, [0, 2, 1, 3, 4, 4]], [[0, 1, 3, 4, 5, 6], [0, 1, 2, 0, 0, 0]], [[-1, 1, 0, 0, 0, 0], ok], [ok, [0, 1, 1, 2, 3, 4]], [ok, ok],
              [ok, ok], [ok, ok]]
    counts = [7, 5, 3, 2, 3, 2 ** 31 - 1, -2, 1]
    want, bad = mv.keep(c, src, blocks, counts)
    assert bad == {0, 1, 2, 3, 4, 5, 6, 7}
    d.keep(ints(blocks), ints(counts), None if inside else s)
    mv.same(download(d), want)
    checked(d, bad)
    counts = [4, 2, 2, -1, 2, 6, 1, 0]
    want, bad = mv.keep(download(d), src, blocks, counts)
    assert bad == ({5} if not inside else set())  # past the smaller cache's capacity
    d.keep(ints(blocks), ints(counts), None if inside else s)
    mv.same(download(d), want)
    checked(d, bad)


def test_no_lists_and_no_tokens():
    c = mv.filled(2, 2, 32, "int8", BF16, [5, 16], 11)
    d = upload(c)
    d.keep(torch.empty(2, 2, 0, dtype=torch.int32, device="cuda"), ints([0, 0]))
    assert d.lengths.tolist() == [5, 0]
    d.take(lengths=ints([0, 0]))
    assert d.lengths.tolist() == [0, 0]
    d.check()


def test_captured_and_replayed_on_another_stream():
    """A beam step (order, then write) as a graph, replayed: what the calls one by one do."""
    c = mv.filled(6, 2, 256, "int8", BF16, [30, 31, 32, 33, 34, 35], 12)
    d, e = upload(c), upload(c)
    order = ints([1, 1, 0, 5, 4, 2])
    k, v = (torch.randn(6, 2, 1, 128, device="cuda").to(BF16) for _ in range(2))

    def step(x):
        x.take(sequences=order)
        x.write(k, v)

    warm = upload(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d)
    for i in range(20):
        k.normal_()
        v.normal_()
        order.random_(0, 6)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        step(e)
        mv.same(download(d), download(e))
    d.check()
    e.check()


def test_refusals():
    c = mv.filled(2, 2, 64, "int8", BF16, [20, 33], 13)
    d, same_arrays = upload(c), None
    for kw in (dict(h=3), dict(fmt="e4m3"), dict(dtype=F32)):
        a = dict(h=2, fmt="int8", dtype=BF16) | kw
        other = upload(mv.filled(2, a["h"], 64, a["fmt"], a["dtype"], [3, 4], 14))
        with pytest.raises(_lib.LKVError):
            d.take(other)
        with pytest.raises(_lib.LKVError):
            d.keep(torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda"), ints([0, 0]), other)
    other = upload(mv.filled(3, 2, 64, "int8", BF16, [3, 4, 5], 14))
    with pytest.raises(_lib.LKVError):
        d.keep(torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda"), ints([0, 0]), other)
    same_arrays = lkv.Cache8.from_tensors(d.k_codes, other.v_codes[:2], d.k_scale, d.v_scale, d.k_tail, d.v_tail, d.lengths)
    part = lkv.Cache8.from_tensors(other.k_codes[:2], d.v_codes, other.k_scale[:2], other.v_scale[:2], other.k_tail[:2], other.v_tail[:2], other.lengths[:2])
    for x in (same_arrays, part):
        with pytest.raises(_lib.LKVError):
            d.take(x)
    for bad in (ints([0]), ints([0, 1, 1]), torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises((ValueError, TypeError)):
            d.take(sequences=bad)
        with pytest.raises((ValueError, TypeError)):
            d.take(lengths=bad)
        with pytest.raises((ValueError, TypeError)):
            d.keep(torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda"), bad)
    for bad in (torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, 1, device="cuda"),
                [[1]]):
        with pytest.raises((ValueError, TypeError)):
            d.keep(bad, ints([0, 0]))
    with pytest.raises(TypeError):
        d.take(d._view)
    with pytest.raises(_lib.LKVError):
        d.take(lengths=d.lengths)  # what the call writes is none of its inputs
    large = lkv.Cache8(batch=1025, n_kv_heads=1, capacity=16, dtype=BF16)
    with pytest.raises(_lib.LKVError):
        large.take()
    lkv.Cache8(batch=1025, n_kv_heads=1, capacity=16, dtype=BF16).take(large)
    mv.same(download(d), c)
    d.check()


@pytest.mark.parametrize("b,h,n", [(300, 2, 150), (345, 2, 150), (1024, 2, 100)])
def test_take_within_a_cache_where_fewer_ctas_fit(b, h, n):
    """The tables of many sequences leave room for two CTAs an SM in place of three."""
    r = random.Random(b)
    have = [r.randrange(n - 60, n + 1) for _ in range(b)]
    c = mv.filled(b, h, (n + 31) // 16 * 16, "int8", BF16, have, 5)
    d = upload(c)
    for to in ([(i * 7 + 3) % b for i in range(b)], [i - i % 64 for i in range(b)]):
        lengths = [c[1][x] if i % 3 else c[1][x] - r.randrange(40) for i, x in enumerate(to)]
        want, bad = mv.take(c, c, to, lengths)  # some are cut to less than nothing: those stay
        d.take(sequences=ints(to), lengths=ints(lengths))
        mv.same(download(d), want)
        checked(d, bad)
        c = download(d)


# An own cache, a prefix cache, queries and what the calls make of them, once in
# torch's context and once in another one on the same device.
OTHER_CONTEXT = '''
import ctypes as C
import torch
import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _move8_ref as mv
from tests.conftest import ROOT
from tests.test_gpu_move8 import upload

lkv.build()
cu = C.CDLL("libcuda.so.1")


def ok(e):
    assert e == 0, e


def arrays(c):
    return [c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail, c.lengths, c._ticket]


class There:
    """A tensor's bytes in the context that is current."""
    def __init__(self, t):
        self.host = t.detach().cpu().contiguous().flatten().view(torch.uint8)
        self.at = C.c_uint64()
        ok(cu.cuMemAlloc_v2(C.byref(self.at), C.c_size_t(self.host.numel())))
        ok(cu.cuMemcpyHtoD_v2(self.at, C.c_void_p(self.host.data_ptr()), C.c_size_t(self.host.numel())))

    def back(self):
        got = torch.empty_like(self.host)
        ok(cu.cuMemcpyDtoH_v2(C.c_void_p(got.data_ptr()), self.at, C.c_size_t(got.numel())))
        return got


def view(c, at):
    return _lib.lkv_cache8(c.batch, c.n_kv_heads, c.capacity, c._view.dtype, c._view.code, 0, *[x.at.value for x in at])


def calls(L, own, prefix, q, out, ws, ws_bytes, group, n, order, blocks, counts, spare):
    """Attention behind the prefixes, sequences put in order, blocks kept and copied."""
    for status in (L.lkv_cache8_attend_shared(own, prefix, None, q, group, n, None, 0.1, 0, out, ws, ws_bytes, None),
                   L.lkv_cache8_take(own, None, order, None, ws, ws_bytes, None),
                   L.lkv_cache8_keep(spare, own, blocks, 1, counts, None), L.lkv_cache8_take(spare, own, order, None, None, 0, None)):
        assert status == 0, _lib.lkv_last_error(None)


for dtype, b, n in ((torch.bfloat16, 2, 1), (torch.bfloat16, 6, 1), (torch.bfloat16, 3, 20), (torch.float32, 3, 1)):
    h, group = 2, 4
    made = [mv.filled(k, h, 96, "int8", dtype, [70 - i for i in range(k)], seed) for k, seed in ((b, 1), (1, 2), (b, 3))]
    caches = [upload(x) for x in made]
    q = torch.randn(b, h * group, n, 128).to(dtype).cuda()
    order = torch.tensor([(i + 1) % b for i in range(b)], dtype=torch.int32).cuda()
    blocks, counts = torch.ones(b, h, 1, dtype=torch.int32).cuda(), torch.ones(b, dtype=torch.int32).cuda()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    L = _lib.load()
    torch.cuda.synchronize()
    ctx, dev = C.c_void_p(), C.c_int()
    ok(cu.cuDeviceGet(C.byref(dev), 0))
    start, more = [[x.cpu() for x in arrays(c)] for c in caches], [x.cpu() for x in (q, out, order, blocks, counts)]
    calls(L, caches[0]._at, caches[1]._at, q.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(), group, n, order.data_ptr(), blocks.data_ptr(),
          counts.data_ptr(), caches[2]._at)
    torch.cuda.synchronize()
    want = [x.cpu().flatten().view(torch.uint8) for c in caches for x in arrays(c)] + [out.cpu().flatten().view(torch.uint8)]
    ok(cu.cuCtxCreate_v2(C.byref(ctx), 0, dev))
    there = [[There(x) for x in s] for s in start]
    views = [view(c, at) for c, at in zip(caches, there)]
    tq, to, tr, tb, tc = (There(x) for x in more)
    tw = There(torch.zeros(64 << 20, dtype=torch.uint8))
    at = [C.addressof(v) for v in views]
    calls(L, at[0], at[1], tq.at.value, to.at.value, tw.at.value, 64 << 20, group, n, tr.at.value, tb.at.value, tc.at.value, at[2])
    ok(cu.cuCtxSynchronize())
    got = [x.back() for s in there for x in s] + [to.back()]
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    ok(cu.cuCtxDestroy_v2(ctx))
    assert out.any()
print("same in both")
'''


def test_another_context_on_the_device():
    """What a kernel has been allowed in one context holds in another: the same bits in both."""
    r = subprocess.run([sys.executable, "-c", OTHER_CONTEXT], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "same in both" in r.stdout, r.stdout + r.stderr
