"""The 8-bit cache on the GPU: writing, reading back and attending, against
plain 64-bit forms."""
import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _cache8_ref as ref

pytestmark = pytest.mark.gpu

FMTS, DTYPES = ["int8", "e4m3"], [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(g, b, h, n, dtype):
    """Rows with a few large channels, a zero block and a tiny one now and then."""
    x = torch.randn(b, h, n, 128, generator=g)
    x[..., ::17] *= 8
    if n >= 48:
        x[:, 0, 16:32] = 0
        x[:, 0, 32:48] *= 2.0 ** -60
    return x.to(dtype)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(x, y, fmt, dtype, capacity, lengths, garbage=None):
    """A cache that holds rows x and y [B, H, n, 128] (CPU), and its CPU arrays."""
    k, v = (ref.held(z, fmt, dtype, capacity, lengths, garbage) for z in (x, y))
    c = lkv.Cache8.from_tensors(k[0].cuda(), v[0].cuda(), k[1].cuda(), v[1].cuda(), k[2].cuda(), v[2].cuda(),
                                i32(*lengths))
    return c, k, v


def same_state(c, k, v, lengths):
    """The cache's arrays hold exactly what the definition gives: codes and
    scales of full blocks, tails of the last one, lengths."""
    assert c.lengths.tolist() == list(lengths)
    for codes, scale, tail, want in ((c.k_codes, c.k_scale, c.k_tail, k), (c.v_codes, c.v_scale, c.v_tail, v)):
        for b, n in enumerate(lengths):
            full, last = n // 16, (n - 1) // 16 * 16
            got, exp = (x.view(torch.int8)[b, :, :full * 16] for x in (codes.cpu(), want[0]))
            assert torch.equal(got, exp), f"codes of sequence {b} differ"
            assert torch.equal(scale[b, :, :full].cpu(), want[1][b, :, :full])
            if n:
                assert torch.equal(tail[b, :, :n - last].cpu(), want[2][b, :, :n - last])


# ---------------------------------------------------------------- write

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("chunks", [[1] * 35, [16, 16], [5, 20, 7, 1, 100], [133], [15, 1, 17, 31, 48]])
def test_write_in_chunks(fmt, dtype, chunks):
    """However the tokens are split over calls, the cache holds the same codes,
    and those of the definition, bit for bit."""
    b, h, n = 2, 3, sum(chunks)
    g = gen(n)
    x, y = rows(g, b, h, n, dtype), rows(g, b, h, n, dtype)
    c = lkv.Cache8(batch=b, n_kv_heads=h, capacity=160, dtype=dtype, fmt=fmt)
    at = 0
    for m in chunks:
        c.write(x[:, :, at:at + m].contiguous().cuda(), y[:, :, at:at + m].contiguous().cuda())
        at += m
    c.check()
    same_state(c, ref.held(x, fmt, dtype, 160, [n] * b), ref.held(y, fmt, dtype, 160, [n] * b), [n] * b)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_write_decides_ties_exactly(fmt, dtype):
    """Values on and next to the halfway points between two codes."""
    top = ref.TOP[fmt]
    g = gen(5)
    n = 64
    x = torch.zeros(1, 2, n, 128, dtype=torch.float64)
    for h in range(2):
        for blk in range(n // 16):
            amax = [1.0, 127.0, 3.7109375, 448.0][blk] * (1 if h == 0 else 0.4375)
            if fmt == "int8":
                mid = torch.arange(2048, dtype=torch.float64) % 127 + 0.5
            else:
                code = torch.arange(126, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
                mid = ((code[1:] + code[:-1]) / 2)[torch.arange(2048) % 125]
            z = mid * amax / top * torch.where(torch.rand(2048, generator=g) < 0.5, -1.0, 1.0)
            z = z.to(dtype)
            step = (torch.randint(-2, 3, (2048,), generator=g)).to(torch.int16 if dtype == torch.bfloat16 else torch.int32)
            z = (z.view(step.dtype) + step).view(dtype)  # up to two units off the rounded halfway point
            z = torch.where(torch.isfinite(z) & (z.abs().double() <= amax), z, torch.zeros_like(z))
            z[7] = amax
            x[0, h, blk * 16:(blk + 1) * 16] = z.double().view(16, 128)
    x = x.to(dtype)
    c = lkv.Cache8(batch=1, n_kv_heads=2, capacity=n, dtype=dtype, fmt=fmt)
    c.write(x.cuda(), x.cuda())
    want = ref.held(x, fmt, dtype, n, [n])
    same_state(c, want, want, [n])
    c.check()


def test_write_extremes():
    """Blocks of denormal and of the largest values."""
    for dtype in DTYPES:
        for fmt in FMTS:
            x = torch.randn(1, 1, 64, 128, generator=gen(2))
            x[:, :, :16] *= 1e-39
            x[:, :, 16:32] *= 1e-44
            x[:, :, 32:48] = x[:, :, 32:48].clamp(-3, 3) * 1e38
            x[:, :, 48:] *= 2.0 ** -101
            x = x.to(dtype)
            c = lkv.Cache8(batch=1, n_kv_heads=1, capacity=64, dtype=dtype, fmt=fmt)
            c.write(x.cuda(), x.cuda())
            want = ref.held(x, fmt, dtype, 64, [64])
            same_state(c, want, want, [64])


def test_write_ragged_counts_and_start():
    """Counts of 0 and fewer than n; starts that take tokens back."""
    dtype, fmt, b, h = torch.bfloat16, "int8", 5, 2
    g = gen(11)
    old = [40, 33, 16, 0, 47]
    x, y = rows(g, b, h, 64, dtype), rows(g, b, h, 64, dtype)
    c = lkv.Cache8(batch=b, n_kv_heads=h, capacity=112, dtype=dtype, fmt=fmt)
    c.write(x.cuda(), y.cuda(), counts=i32(*old))
    same_state(c, ref.held(x, fmt, dtype, 112, old), ref.held(y, fmt, dtype, 112, old), old)
    z, w = rows(g, b, h, 21, dtype), rows(g, b, h, 21, dtype)
    start, counts = [40, 32, 5, 0, 34], [21, 1, 21, 0, 13]
    c.write(z.cuda(), w.cuda(), start=i32(*start), counts=i32(*counts))
    c.check()
    new = [s + m if m else o for s, m, o in zip(start, counts, old)]
    for t, add in ((x, z), (y, w)):
        t.resize_(b, h, 64, 128)
        for i in range(b):
            t[i, :, start[i]:start[i] + counts[i]] = add[i, :, :counts[i]]
    same_state(c, ref.held(x, fmt, dtype, 112, new), ref.held(y, fmt, dtype, 112, new), new)


def test_write_take_back_one_after_a_full_block():
    """The tail keeps a block that has just been filled: its last tokens can be replaced."""
    x = rows(gen(1), 1, 1, 32, torch.float32)
    c = lkv.Cache8(batch=1, n_kv_heads=1, capacity=48, dtype=torch.float32, fmt="int8")
    c.write(x.cuda(), x.cuda())
    y = rows(gen(2), 1, 1, 3, torch.float32)
    c.write(y.cuda(), y.cuda(), start=i32(29))
    c.check()
    x[:, :, 29:] = y
    want = ref.held(x, "int8", torch.float32, 48, [32])
    same_state(c, want, want, [32])


def test_write_refused_on_the_device_leaves_the_sequence():
    dtype = torch.bfloat16
    x = rows(gen(3), 4, 2, 40, dtype)
    for start, counts, n, status in (([40, 41, 40, 40], [1] * 4, 1, _lib.LKV_EINVAL),     # beyond the length
                                     ([40, 40, 20, 40], [1] * 4, 1, _lib.LKV_EINVAL),     # inside an older block
                                     ([40, 40, 40, -16], [1] * 4, 1, _lib.LKV_EINVAL),
                                     ([40] * 4, [2, 3, 2, 2], 2, _lib.LKV_EINVAL),        # more than n
                                     ([40] * 4, [2, 2, -1, 2], 2, _lib.LKV_EINVAL),
                                     ([40] * 4, [8, 9, 1, 0], 9, _lib.LKV_ECAPACITY)):
        c = lkv.Cache8(batch=4, n_kv_heads=2, capacity=48, dtype=dtype, fmt="e4m3")
        c.write(x.cuda(), x.cuda())
        z = rows(gen(4), 4, 2, n, dtype)
        c.write(z.cuda(), z.cuda(), start=i32(*start), counts=i32(*counts))
        ok = [(s == 40 and 0 <= m <= n and s + m <= 48) for s, m in zip(start, counts)]
        assert not all(ok)
        new = [s + m if o else 40 for s, m, o in zip(start, counts, ok)]
        full = torch.cat((x, torch.zeros(4, 2, 8, 128, dtype=dtype)), 2)
        for i in range(4):
            if ok[i]:
                full[i, :, 40:40 + counts[i]] = z[i, :, :counts[i]]
        want = ref.held(full, "e4m3", dtype, 48, new)
        same_state(c, want, want, new)
        with pytest.raises(_lib.LKVError) as e:
            c.check()
        assert e.value.status == status
        c.check()  # reported once


def test_write_not_finite():
    """NaN is held as 0, an infinity as the largest finite value; reported."""
    for dtype in DTYPES:
        x = rows(gen(8), 1, 2, 40, dtype)
        x[0, 0, 3, 5], x[0, 1, 20, 0], x[0, 1, 35, 127], x[0, 0, 36, 1] = float("nan"), float("inf"), float("-inf"), float("nan")
        c = lkv.Cache8(batch=1, n_kv_heads=2, capacity=48, dtype=dtype, fmt="int8")
        c.write(x.cuda(), x.cuda())
        big = torch.finfo(dtype).max
        clean = torch.nan_to_num(x.double(), nan=0.0, posinf=big, neginf=-big).to(dtype)
        want = ref.held(clean, "int8", dtype, 48, [40])
        same_state(c, want, want, [40])
        with pytest.raises(_lib.LKVError) as e:
            c.check()
        assert e.value.status == _lib.LKV_EINVAL and "NaN" in str(e.value)


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,first", [(1, [0, 0, 0, 0]), (80, None), (37, [0, 15, 31, 60]), (16, [64, 16, 2**31 - 8, -5])])
def test_read(fmt, dtype, n, first):
    lengths = [70, 16, 0, 63]
    g = gen(6)
    x, y = rows(g, 4, 2, 70, dtype), rows(g, 4, 2, 70, dtype)
    c, k, v = make(x, y, fmt, dtype, 96, lengths, garbage=g)
    got = c.read(n, first=None if first is None else i32(*first))
    for out, arr in zip(got, (k, v)):
        for b in range(4):
            held = ref.values(arr[0][b], arr[1][b], arr[2][b], lengths[b])
            want = torch.zeros(2, n, 128, dtype=torch.float64)
            f = 0 if first is None else first[b]
            for r in range(n):
                if 0 <= f + r < lengths[b]:
                    want[:, r] = held[:, f + r]
            err = (out[b].cpu().double() - want).abs()
            # the product rounds to fp32, then to dtype
            assert (err <= want.abs() * (2.0 ** -24 + ref.half_step(dtype) * (1 + 2.0 ** -24))).all()


def test_read_feeds_an_index_build():
    """The layout is Context.build_index's: an index built from the cache is
    the one built from the same values."""
    b, h, n = 1, 2, 600
    g = gen(12)
    x, y = rows(g, b, h, n, torch.bfloat16), rows(g, b, h, n, torch.bfloat16)
    c = lkv.Cache8(batch=b, n_kv_heads=h, capacity=608, dtype=torch.bfloat16, fmt="int8")
    c.write(x.cuda(), y.cuda())
    k, v = c.read(n)
    ctx = lkv.Context(batch=b, n_layers=1, n_kv_heads=h, group=4, dtype=torch.bfloat16, local_buf=8, max_clusters=16,
                      max_prefill=n, max_steps=4, max_budget=64)
    ctx.build_index(0, k, v, 16, 3, 1)
    one = [ctx.get_index(0, 0, i, n) for i in range(h)]
    kc, vc, _ = k.clone(), v.clone(), c.check()
    ctx.build_index(0, kc, vc, 16, 3, 1)
    for i in range(h):
        two = ctx.get_index(0, 0, i, n)
        assert (one[i]["assign"] == two["assign"]).all() and (one[i]["centroids"] == two["centroids"]).all()
        assert len(set(one[i]["assign"].tolist())) > 4
    ctx.close()


# ---------------------------------------------------------------- attend

def check_attend(c, k, v, lengths, q, *, counts=None, scale=None, window=0, sinks=0, max_len=0, out=None):
    got = c.attend(q.cuda(), counts=None if counts is None else i32(*counts), scale=scale, window=window, sinks=sinks,
                   max_len=max_len, out=out)
    n = q.shape[2]
    for b, length in enumerate(lengths):
        kk, vv = (ref.values(a[0][b], a[1][b], a[2][b], length) for a in (k, v))
        cnt = n if counts is None else min(max(counts[b], 0), n)
        want, size, vmax = ref.attend(q[b].double(), kk, vv, cnt, 128 ** -0.5 if scale is None else scale, window, sinks)
        err = (got[b].cpu().double() - want).abs()
        lim = ref.attend_bound(want, q.dtype, size, vmax, length)
        assert torch.isfinite(got[b]).all() and (err <= lim).all(), \
            f"sequence {b} of length {length}: off by {err.max():.3e}, {(err / lim.clamp_min(1e-300)).max():.2f} of the bound"
    return got


def attend_case(fmt, dtype, lengths, h, group, n, capacity, seed=0, **kw):
    g = gen(seed)
    b = len(lengths)
    top = max(max(lengths), 1)
    x, y = rows(g, b, h, top, dtype), rows(g, b, h, top, dtype)
    c, k, v = make(x, y, fmt, dtype, capacity, lengths, garbage=g)
    q = torch.randn(b, h * group, n, 128, generator=g).to(dtype)
    return check_attend(c, k, v, lengths, q, **kw)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group,n", [(4, 1), (1, 1), (8, 1), (3, 1), (16, 1), (4, 2), (2, 5), (1, 9), (4, 21)])
def test_attend(fmt, dtype, group, n):
    attend_case(fmt, dtype, [1, 15, 16, 17, 0, 31, 32, 100, 257, 300], 2, group, n, 320, seed=group + n)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (33, 17), (64, 40), (100, 1000), (319, 2), (320, 1),
                                          (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_attend_window_and_sinks(fmt, dtype, window, sinks, n):
    attend_case(fmt, dtype, [2, 16, 47, 100, 257, 305], 1, 4, n, 320, seed=window % 97 + sinks % 89, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attend_padded_rows(dtype):
    """Padded batches: rows at or past a sequence's count are zero, and the
    others are its last tokens. Counts outside 0..n are clamped."""
    attend_case("int8", dtype, [40, 100, 0, 7, 33, 64], 2, 4, 6, 112, seed=4, counts=[6, 1, 0, 3, 9, -2])
    attend_case("e4m3", dtype, [40, 100, 0, 7, 33, 64], 2, 2, 30, 112, seed=5, counts=[30, 1, 5, 30, 0, 17], window=8, sinks=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
def test_attend_long(fmt, dtype):
    """Long sequences, split over many CTAs, ragged; any bound max_len gives the same."""
    lengths = [20011, 1, 5000, 16384]
    for max_len in (0, 20011, 100):
        attend_case(fmt, dtype, lengths, 1, 4, 1, 20480, seed=7, max_len=max_len)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attend_prompt(dtype):
    """A whole prompt over its own cache, and a chunk behind earlier tokens."""
    attend_case("int8", dtype, [300, 257], 2, 4, 300, 320, seed=8)
    attend_case("e4m3", dtype, [700, 450], 1, 2, 333, 704, seed=9, window=50, sinks=3)
    attend_case("e4m3", dtype, [1000], 1, 8, 129, 1008, seed=10)


def test_attend_sharp_and_flat():
    """One token far above the rest, first, last and inside; and equal scores."""
    for dtype in DTYPES:
        for hot in (0, 5, 511, 600, 640):
            g = gen(hot)
            x, y = torch.randn(1, 1, 641, 128, generator=g), torch.randn(1, 1, 641, 128, generator=g)
            q = torch.randn(1, 4, 1, 128, generator=g)
            x[0, 0, hot] = q[0, 1, 0] * 20
            c, k, v = make(x.to(dtype), y.to(dtype), "int8", dtype, 656, [641])
            check_attend(c, k, v, [641], q.to(dtype))
        y = torch.randn(1, 2, 200, 128, generator=gen(1)).to(dtype)
        c, k, v = make(torch.zeros_like(y), y, "e4m3", dtype, 208, [200])
        check_attend(c, k, v, [200], torch.randn(1, 8, 3, 128, generator=gen(2)).to(dtype))


def test_attend_scales():
    """Queries, keys and values of any size, and a negative and a zero scale."""
    for dtype in DTYPES:
        for qs, ks, vs, scale in ((1e-20, 1e20, 1e10, None), (1e15, 1e-16, 1e-30, None), (1.0, 1.0, 1.0, -0.3), (1.0, 1.0, 1.0, 0.0),
                                  (1e-38, 1.0, 1e30, 1.0)):
            g = gen(3)
            x, y = (torch.randn(1, 1, 75, 128, generator=g) * s for s in (ks, vs))
            q = torch.randn(1, 2, 2, 128, generator=g) * qs
            c, k, v = make(x.to(dtype), y.to(dtype), "int8", dtype, 80, [75])
            check_attend(c, k, v, [75], q.to(dtype), scale=scale)


def test_attend_repeats_and_captures():
    """The same bits each time; a captured call follows the device's lengths;
    outputs on a side stream."""
    g = gen(21)
    x, y = rows(g, 2, 2, 3000, torch.bfloat16), rows(g, 2, 2, 3000, torch.bfloat16)
    c, k, v = make(x, y, "int8", torch.bfloat16, 3008, [3000, 2500])
    q = torch.randn(2, 8, 1, 128, generator=g).bfloat16().cuda()
    want = c.attend(q)
    for _ in range(5):
        assert torch.equal(c.attend(q), want)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.attend(q, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(q, out=out)
    for lengths in ([17, 1], [2999, 2496], [3000, 2500]):
        c.lengths.copy_(i32(*lengths))
        graph.replay()
        assert torch.equal(out, c.attend(q))
    assert torch.equal(out, want)


def test_attend_two_streams_at_once():
    g = gen(22)
    x, y = rows(g, 1, 4, 9000, torch.bfloat16), rows(g, 1, 4, 9000, torch.bfloat16)
    c, k, v = make(x, y, "e4m3", torch.bfloat16, 9008, [9000])
    qs = [torch.randn(1, 16, 1, 128, generator=g).bfloat16().cuda() for _ in range(2)]
    want = [c.attend(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.attend(qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_offsets_past_32_bits():
    """Codes whose byte offsets pass 2^32: the second KV head of a long
    capacity, its rows near the end, written, read and attended."""
    cap, n = 1 << 25, 100
    c = lkv.Cache8(batch=1, n_kv_heads=2, capacity=cap, dtype=torch.bfloat16, fmt="int8")
    at = cap - 104
    c.lengths.fill_(at)
    g = gen(31)
    x, y = rows(g, 1, 2, n, torch.bfloat16), rows(g, 1, 2, n, torch.bfloat16)
    at16 = at // 16 * 16
    c.write(x.cuda(), y.cuda(), start=i32(at16))
    c.check()
    assert c.lengths.tolist() == [at16 + n]
    k, v = c.read(n, first=i32(at16))
    wk, wv = ref.held(x, "int8", torch.bfloat16, 112, [n]), ref.held(y, "int8", torch.bfloat16, 112, [n])
    for out, w in ((k, wk), (v, wv)):
        want = ref.values(w[0][0], w[1][0], w[2][0], n)
        assert ((out[0].cpu().double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23)).all()
    q = torch.randn(1, 8, 1, 128, generator=g).bfloat16()
    got = c.attend(q.cuda(), window=64)
    want, size, vmax = ref.attend(q[0].double(), *(ref.values(w[0][0], w[1][0], w[2][0], n) for w in (wk, wv)), 1, 128 ** -0.5, 64, 0)
    assert ((got[0].cpu().double() - want).abs() <= ref.attend_bound(want, torch.bfloat16, size, vmax, n)).all()


def test_refusals():
    c = lkv.Cache8(batch=2, n_kv_heads=2, capacity=32, dtype=torch.bfloat16, fmt="int8")
    x = torch.zeros(2, 2, 4, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 8, 1, 128, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: c.write(x.float(), x.float()), lambda: c.attend(q.float()), lambda: c.write(x, x, start=torch.zeros(2, device="cuda")),
                 lambda: c.attend(q, counts=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: c.write(x, x[:, :, :2]), lambda: c.write(x[:1], x[:1]), lambda: c.write(x.cpu(), x.cpu()),
                 lambda: c.write(x.transpose(2, 3), x), lambda: c.write(x, x, start=i32(0)), lambda: c.attend(q[:, :7]),
                 lambda: c.attend(q[:, :0]), lambda: c.attend(q[..., :64]), lambda: c.attend(q, out=q[:, :4]), lambda: c.read(4, k_out=x, v_out=x[:, :1]),
                 lambda: c.attend(q.expand(2, 8, 2, 128))):
        with pytest.raises(ValueError):
            call()
    flat = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: c.attend(flat[1:1 + q.numel()].view(q.shape)), lambda: c.attend(q, out=q), lambda: c.attend(q, window=-1),
                 lambda: c.attend(q, scale=float("nan")), lambda: c.read(4, k_out=x, v_out=x), lambda: c.write(x, x, start=c.lengths),
                 lambda: c.attend(q, sinks=-1)):
        with pytest.raises(_lib.LKVError) as e:
            call()
        assert e.value.status == _lib.LKV_EINVAL
    assert c.read(0)[0].shape == (2, 2, 0, 128)
    assert c.attend(q[:, :, :0].contiguous()).shape == (2, 8, 0, 128)
    c.write(x[:, :, :0].contiguous(), x[:, :, :0].contiguous())
    assert (c.attend(q) == 0).all()  # empty sequences
    c.check()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 4)])
def test_serving_steps(fmt, dtype, window, sinks):
    """A prompt, then steps, as a server runs them: rotate q and k, write k and
    v, attend; the steps from one captured graph. Every output against the
    64-bit form on the values that the cache then holds."""
    b, h, group, n0, steps = 2, 2, 4, 37, 24
    g = gen(40)
    r = lkv.Rope(base=10000.0)
    rates, gain = ref.rope_rates(128)
    c = lkv.Cache8(batch=b, n_kv_heads=h, capacity=96, dtype=dtype, fmt=fmt)
    k0, v0 = rows(g, b, h, n0, dtype), rows(g, b, h, n0, dtype)
    q0 = torch.randn(b, h * group, n0, 128, generator=g).to(dtype)
    pos = torch.arange(n0, dtype=torch.int32).repeat(b, 1)
    qr, kr = r.apply(q0.cuda(), pos.cuda(), k0.cuda())
    counts = [n0, n0 - 5]
    c.write(kr, v0.cuda(), counts=i32(*counts))
    krows, vrows = kr.cpu(), v0

    def held(lengths):
        return ref.held(krows, fmt, dtype, 96, lengths), ref.held(vrows, fmt, dtype, 96, lengths)

    k, v = held(counts)
    same_state(c, k, v, counts)
    check_attend(c, k, v, counts, qr.cpu(), counts=counts, window=window, sinks=sinks)
    q1 = torch.zeros(b, h * group, 1, 128, dtype=dtype, device="cuda")
    k1, v1 = (torch.zeros(b, h, 1, 128, dtype=dtype, device="cuda") for _ in range(2))
    at = torch.zeros(b, 1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q1)

    def step():
        at.copy_(c.lengths.view(b, 1))
        qq, kk = r.apply(q1, at, k1)
        c.write(kk, v1)
        c.attend(qq, window=window, sinks=sinks, out=out)
        return qq, kk

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qq, kk = step()
    lengths = list(counts)
    krows, vrows = (torch.cat((z, torch.zeros(b, h, steps, 128, dtype=dtype)), 2) for z in (krows, vrows))
    for _ in range(steps):
        a = torch.randn(b, h * group, 1, 128, generator=g).to(dtype)
        kn, vn = rows(g, b, h, 1, dtype), rows(g, b, h, 1, dtype)
        q1.copy_(a)
        k1.copy_(kn)
        v1.copy_(vn)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(b):
            krows[i, :, lengths[i]] = kk[i, :, 0].cpu()
            vrows[i, :, lengths[i]] = vn[i, :, 0]
        want, size = ref.rope(kn, torch.tensor(lengths)[:, None], rates, gain, "half")
        assert ((kk.cpu().double() - want).abs() <= size * 2.0 ** -20 + want.abs() * ref.half_step(dtype) * (1 + 2.0 ** -8)).all()
        lengths = [x + 1 for x in lengths]
        k, v = held(lengths)
        same_state(c, k, v, lengths)
        for i in range(b):
            kk64, vv64 = (ref.values(z[0][i], z[1][i], z[2][i], lengths[i]) for z in (k, v))
            want, size, vmax = ref.attend(qq[i].cpu().double(), kk64, vv64, 1, 128 ** -0.5, window, sinks)
            err = (out[i].cpu().double() - want).abs()
            assert (err <= ref.attend_bound(want, dtype, size, vmax, lengths[i])).all()
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lengths,h,group,n,window,sinks", [
    ([9000], 1, 4, 1, 0, 0), ([7001, 1, 0, 6000], 2, 1, 1, 0, 0), ([40000, 3], 1, 4, 4, 0, 0), ([12000, 11984], 1, 8, 2, 6000, 20),
    ([5000, 5001, 4999, 17], 40, 1, 1, 0, 0)])
def test_attend_streamed(dtype, fmt, lengths, h, group, n, window, sinks):
    """Few or uneven tiles of long sequences: shared evenly by many CTAs and
    joined, the empty ones among them; the same bits each time."""
    g = gen(50)
    b, top = len(lengths), max(lengths)
    x, y = (rows(g, b, 1, top, dtype).expand(b, h, top, 128) for _ in range(2))
    c, k, v = make(x, y, fmt, dtype, (top + 31) // 16 * 16, lengths, garbage=g)
    view = c._view
    need = _lib.lkv_cache8_attend_workspace(c._at, group, n, window, sinks, 0)
    assert need > 0 and view.batch == b, "not a streamed call: the case does not test what it is for"
    q = torch.randn(b, h * group, n, 128, generator=g).to(dtype)
    heads = [0, h // 2, h - 1]
    got = c.attend(q.cuda(), window=window, sinks=sinks)
    for i, length in enumerate(lengths):
        for j in heads:
            kk, vv = (ref.values(a[0][i, j:j + 1], a[1][i, j:j + 1], a[2][i, j:j + 1], length) for a in (k, v))
            want, size, vmax = ref.attend(q[i, j * group:(j + 1) * group].double(), kk, vv, n, 128 ** -0.5, window, sinks)
            err = (got[i, j * group:(j + 1) * group].cpu().double() - want).abs()
            lim = ref.attend_bound(want, dtype, size, vmax, length)
            assert (err <= lim).all(), f"sequence {i}, head {j}: off by {err.max():.3e}, {(err / lim.clamp_min(1e-300)).max():.2f} of the bound"
    for _ in range(3):
        assert torch.equal(c.attend(q.cuda(), window=window, sinks=sinks), got)
    # a workspace that is too small, or none, is refused
    L, out, qc = _lib.load(), torch.empty_like(q, device="cuda"), q.cuda()
    for ws, size in ((None, 0), (out.data_ptr(), need), (torch.empty(need, dtype=torch.uint8, device="cuda").data_ptr(), need - 1)):
        assert L.lkv_cache8_attend(c._at, qc.data_ptr(), group, n, None, 1.0, window, sinks, 0, out.data_ptr(), ws, size, None) == _lib.LKV_EINVAL
