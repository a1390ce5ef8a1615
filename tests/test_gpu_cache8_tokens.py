"""Attention over the 8-bit cache, token by token: every output held to a bound
of its own, outputs that show a token lost or counted twice, and V units of any
size beside one another."""
import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _cache8_each as each
from tests import _cache8_ref as ref
from tests.test_gpu_cache8 import DTYPES, FMTS, gen, i32, make, rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def check_each(c, k, v, lengths, q, *, counts=None, scale=None, window=0, sinks=0, max_len=0):
    got = c.attend(q.cuda(), counts=None if counts is None else i32(*counts), scale=scale, window=window, sinks=sinks, max_len=max_len)
    n = q.shape[2]
    for b, length in enumerate(lengths):
        kk, vv = (ref.values(a[0][b], a[1][b], a[2][b], length) for a in (k, v))
        cnt = n if counts is None else min(max(counts[b], 0), n)
        want, lim = each.attend(q[b].double(), kk, vv, each.units(v[1][b], v[2][b], length), cnt, 128 ** -0.5 if scale is None else scale,
                                window, sinks, q.dtype)
        err = (got[b].cpu().double() - want).abs()
        assert torch.isfinite(got[b]).all() and (err <= lim).all(), \
            f"sequence {b} of length {length}: off by {err.max():.3e}, {(err / lim.clamp_min(1e-300)).max():.2f} of the bound"


# ---------------------------------------------------------------- V units

# A V scale of 0 stands for values of 0 whatever the codes are: by the
# definition of reading back, code * scale.

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,n", [(3, 1), (64, 64)])
def test_scale_of_zero_over_codes(fmt, dtype, b, n):
    """In a cache made elsewhere; the many rows of 64 sequences go to their own kernel (bf16)."""
    g = gen(b)
    lengths = [200, 217, 96][:b] if b < 4 else torch.randint(70, 220, (b,), generator=g).tolist()
    x, y = (torch.randn(b, 2, 224, 128, generator=g).to(dtype) for _ in range(2))
    k, v = (ref.held(z, fmt, dtype, 224, lengths) for z in (x, y))
    v[1][:, 0, 1] = 0
    v[1][:, 1, 2:5] = 0
    k[1][:, 1, 3] = 0
    c = lkv.Cache8.from_tensors(*(t.cuda() for pair in zip(k, v) for t in pair), i32(*lengths))
    q = torch.randn(b, 8, n, 128, generator=g).to(dtype)
    check_each(c, k, v, lengths, q)
    check_each(c, k, v, lengths, q, window=60, sinks=20)
    if b < 4:  # every V scale: nothing but the tail is left
        v[1][:] = 0
        c.v_scale.zero_()
        check_each(c, k, v, lengths, q)


@pytest.mark.parametrize("fmt", FMTS)
def test_written_values_whose_scale_rounds_to_zero(fmt):
    """fp32 values so small that amax / 127 rounds to 0 beside ordinary ones: read and attended alike."""
    x = torch.randn(1, 2, 100, 128, generator=gen(4))
    x[:, :, 16:48] = x[:, :, 16:48].clamp(-2, 2) * 1e-44
    c = lkv.Cache8(batch=1, n_kv_heads=2, capacity=112, dtype=torch.float32, fmt=fmt)
    c.write(x.cuda(), x.cuda())
    arrays = ref.held(x, fmt, torch.float32, 112, [100])
    assert (arrays[1][:, :, 1:3] == 0).all()
    assert (c.read(100)[1][:, :, 16:48] == 0).all()
    check_each(c, arrays, arrays, [100], torch.randn(1, 8, 2, 128, generator=gen(5)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("at,order,less", [(300, 40, 60), (300, 60, 30), (300, 20, 300), (511, 40, 50), (2, 80, 100), ("tail", 40, 60),
                                           ("tail", 30, 35), ("tail", 80, 70)])
def test_a_block_of_far_larger_values(dtype, fmt, at, order, less):
    """One block, or the tail, holds values 2^order times the others' in tokens
    that weigh 2^-less: what the other tokens before and after it add stays."""
    n = 8192 + 5
    x, y = torch.zeros(1, 1, n, 128), torch.randn(1, 1, n, 128, generator=gen(at if at != "tail" else 7)).abs() + 0.5
    big = slice(n - 5, n) if at == "tail" else slice(16 * at, 16 * at + 16)
    x[..., big, 0] = -1.0
    y[..., big, :] *= 2.0 ** order
    q = torch.zeros(1, 2, 1, 128)
    q[..., 0] = round(less * 0.6931471805599453 * 128 ** 0.5)
    c, k, v = make(x.to(dtype), y.to(dtype), fmt, dtype, 8208, [n])
    for max_len in (16, 0):  # one CTA, and as many as the call would take
        check_each(c, k, v, [n], q.to(dtype), max_len=max_len)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("at,order,less", [(100, 40, 60), (100, 60, 30), (2, 80, 100), ("tail", 40, 60), ("tail", 80, 70)])
def test_many_rows_some_of_which_see_far_larger_values(dtype, at, order, less):
    """The same for 64 tokens' rows: the tail's tokens are not seen by all of them, nor is the block by those of a window."""
    n, count = 4096 + 5, 64
    x, y = torch.zeros(1, 1, n, 128), torch.randn(1, 1, n, 128, generator=gen(6)).abs() + 0.5
    big = slice(n - 5, n) if at == "tail" else slice(16 * at, 16 * at + 16)
    x[..., big, 0] = -1.0
    y[..., big, :] *= 2.0 ** order
    q = torch.zeros(1, 4, count, 128)
    q[..., 0] = round(less * 0.6931471805599453 * 128 ** 0.5)
    c, k, v = make(x.to(dtype), y.to(dtype), "int8", dtype, 4112, [n])
    check_each(c, k, v, [n], q.to(dtype))
    check_each(c, k, v, [n], q.to(dtype), window=n - 16 * 101 - 30, sinks=64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_units_that_climb(dtype):
    """V units that rise by 2^7 every 64 blocks, over 2^84 in all, under weights
    that fall as fast, or slower, or faster, or rise."""
    n = 13 * 1024 - 3
    block = torch.arange(n) // 1024
    y = (torch.randn(1, 1, n, 128, generator=gen(1)).abs() + 0.5) * 2.0 ** (7.0 * block - 40)[:, None]
    for step in (7, 5, 6.5, 8, 2, -2):
        x = torch.zeros(1, 1, n, 128)
        x[..., 0] = -block.float()
        q = torch.zeros(1, 1, 1, 128)
        q[..., 0] = round(step * 0.6931471805599453 * 128 ** 0.5)
        c, k, v = make(x.to(dtype), y.to(dtype), "int8", dtype, 13 * 1024, [n])
        for max_len in (16, 0):
            check_each(c, k, v, [n], q.to(dtype), max_len=max_len)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("less", [20, 31, 40, 60])
def test_one_token_far_above(dtype, less):
    """A token of no value holds nearly all of the weight: the output is what
    the 2^-less of the others sum to (fp32 to all of its bits)."""
    n = 30000
    y = torch.randn(1, 1, n, 128, generator=gen(9)).abs() + 0.5
    y[:, :, 5] = 0
    x = torch.zeros(1, 1, n, 128)
    x[:, :, 5, 0] = 1.0
    q = torch.zeros(1, 3, 1, 128)
    q[..., 0] = round(less * 0.6931471805599453 * 128 ** 0.5)
    c, k, v = make(x.to(dtype), y.to(dtype), "int8", dtype, 30016, [n])
    for max_len in (16, 0):
        check_each(c, k, v, [n], q.to(dtype), max_len=max_len)


# ---------------------------------------------------------------- every output by itself

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,h,group,n,window,sinks", [
    ([1, 17, 300, 640, 0], 2, 4, 1, 0, 0), ([333, 64, 500], 2, 3, 5, 0, 0), ([700, 650], 1, 8, 3, 100, 20), ([400, 31] * 32, 2, 4, 30, 0, 0),
    ([260, 400] * 32, 2, 2, 64, 90, 5), ([900], 2, 4, 300, 0, 0)])
def test_every_output(fmt, dtype, lengths, h, group, n, window, sinks):
    g = gen(sum(lengths) + n)
    b, top = len(lengths), max(lengths)
    x, y = rows(g, b, h, top, dtype), rows(g, b, h, top, dtype)
    c, k, v = make(x, y, fmt, dtype, (top + 15) // 16 * 16, lengths, garbage=g)
    q = torch.randn(b, h * group, n, 128, generator=g).to(dtype)
    check_each(c, k, v, lengths, q, window=window, sinks=sinks, counts=[min(n, m) for m in lengths])


# ---------------------------------------------------------------- tokens counted

COUNTED = [([40000, 3, 20011], 1, 4, 1, 0, 0), ([9000], 1, 1, 1, 0, 0), ([131000], 2, 4, 1, 0, 0), ([33001, 32964] * 4, 8, 4, 1, 0, 0),
           ([30000, 29000], 2, 8, 2, 9000, 100), ([5000, 4999, 17, 0], 40, 1, 1, 0, 0), ([2100, 1033] * 8, 8, 2, 1, 1024, 4),
           ([20001], 2, 4, 128, 0, 0), ([9000, 130, 20000], 1, 8, 100, 0, 0), ([30000, 5000], 2, 4, 200, 9000, 100), ([700, 640] * 32, 2, 4, 64, 0, 0),
           ([1000, 555] * 32, 2, 4, 64, 300, 20)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,h,group,n,window,sinks", COUNTED)
def test_blocks_are_counted_once(fmt, dtype, lengths, h, group, n, window, sinks):
    """Equal scores and values that name their block: an output is the count of
    the visible tokens of its blocks times their height, over the count of all."""
    if dtype == torch.float32 and n * group * len(lengths) * h > 4096:
        pytest.skip("fp32 has one kernel: its other cases take it")
    b, top = len(lengths), max(lengths)
    y = each.one_hot(top, dtype).expand(b, h, top, 128)
    c, k, v = make(torch.zeros(1, 1, top, 128, dtype=dtype).expand(b, h, top, 128), y, fmt, dtype, (top + 31) // 16 * 16, lengths, garbage=gen(2))
    q = torch.randn(b, h * group, n, 128, generator=gen(3)).to(dtype)
    got = c.attend(q.cuda(), window=window, sinks=sinks, counts=i32(*[min(n, m) for m in lengths])).cpu().double()
    value = each.one_hot(top, torch.float64)
    total = torch.cat((torch.zeros(1, 128, dtype=torch.float64), value.cumsum(0)))
    for i, length in enumerate(lengths):
        for r in range(min(n, length)):
            pos = length - min(n, length) + r
            low = max(0, pos + 1 - window) if window else 0
            first = min(sinks, low)
            want = (total[pos + 1] - total[low] + total[first]) / (pos + 1 - low + first)
            err = (got[i, :, r] - want).abs()
            assert (err <= each.one_hot_bound(want, dtype, length)).all(), \
                f"sequence {i}, row {r}: channels {(err > each.one_hot_bound(want, dtype, length)).any(0).nonzero().flatten().tolist()[:8]}"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,h,group,n", [([40000, 20011], 2, 16, 1), ([131000], 8, 4, 1), ([33001] * 8, 8, 4, 1), ([20001], 2, 4, 32), ([700] * 64, 2, 4, 32)])
def test_a_loud_token_is_found(fmt, dtype, lengths, h, group, n):
    """Each row favours one token above all others, the first or the last of a
    block, block after block: its output is that token's value."""
    if dtype == torch.float32 and n > 1:
        pytest.skip("fp32 has one kernel: its other cases take it")
    b, top, per = len(lengths), max(lengths), n * group
    g = gen(8)
    small = torch.randn(b, 1, top, 128, generator=g).to(dtype)
    zeros = torch.zeros(b, h, top, 128, dtype=dtype)
    v = ref.held(small.expand(b, h, top, 128), fmt, dtype, (top + 15) // 16 * 16, lengths)
    vv = [ref.values(v[0][i, :1], v[1][i, :1], v[2][i, :1], m)[0] for i, m in enumerate(lengths)]
    for turn in range(3):
        x, q = zeros.clone(), torch.zeros(b, h * group, n, 128, dtype=dtype)
        hot = torch.zeros(b, h, per, dtype=torch.long)
        for i, m in enumerate(lengths):
            last = m - n  # every row sees it
            blocks = torch.randperm(max(last // 16, 1), generator=g)
            for j in range(h):
                for r in range(per):
                    z = ((j * per + r) + turn * h * per) % len(blocks)
                    hot[i, j, r] = min(int(blocks[z]) * 16 + (15 if (r + turn) % 2 else 0), last) if r else last - turn
                    x[i, j, hot[i, j, r], r % 128] = 64.0
                    q[i, j * group + r % group, r // group, r % 128] = 64.0
        k = ref.held(x, fmt, dtype, (top + 15) // 16 * 16, lengths)
        c = lkv.Cache8.from_tensors(*(t.cuda() for pair in zip(k, v) for t in pair), i32(*lengths))
        got = c.attend(q.cuda()).cpu().double()
        for i in range(b):
            for j in range(h):
                for r in range(per):
                    same = [s for s in range(r % 128, per, 128)]  # rows that share the channel share their tokens
                    if len({int(hot[i, j, s]) for s in same}) > 1:
                        continue
                    want = vv[i][hot[i, j, r]]
                    err = (got[i, j * group + r % group, r // group] - want).abs()
                    # the weight of the token is 2^(y - reference): in fp16 off by 2^-11; the others' are below 2^-500
                    lim = want.abs() * (2.0 ** -11 + 2.0 ** -16 + ref.half_step(dtype) * 1.01) + 2.0 ** -24 * vv[i].abs().max()
                    assert (err <= lim).all(), f"sequence {i}, KV head {j}, row {r}: token {int(hot[i, j, r])}"


@pytest.mark.parametrize("dtype", DTYPES)
def test_lengths_that_change_between_streamed_calls(dtype):
    """Writes that take tokens back and add others, each followed at once by a
    call whose split over CTAs follows from the lengths: the same bits as with
    a pause after every call."""
    b, h, cap = 3, 2, 40960
    g = gen(17)
    x, y = (torch.randn(b, h, cap, 128, generator=g).to(dtype).cuda() for _ in range(2))
    c = lkv.Cache8(batch=b, n_kv_heads=h, capacity=cap, dtype=dtype)
    c.write(x, y)
    assert _lib.lkv_cache8_attend_workspace(c._at, 4, 1, 0, 0, 0) > 0, "not a streamed call"
    q = torch.randn(b, 8, 1, 128, generator=g).to(dtype).cuda()
    k1, v1 = x[:, :, :1].contiguous(), y[:, :, :1].contiguous()
    # the last full block of each prefix holds what follows; the starts are multiples of 16, falling
    starts = [i32(*(16 * max(0, 2500 - 60 * i - 700 * s) for s in range(b))) for i in range(30)]

    def run(pause):
        c.lengths.fill_(cap)
        got = []
        for s in starts:
            c.write(k1, v1, start=s)
            pause()
            got.append(c.attend(q))
            pause()
            c.write(k1, v1)
            pause()
            got.append(c.attend(q))
            pause()
        return got

    one = run(torch.cuda.synchronize)
    for _ in range(3):
        for m, n in zip(one, run(lambda: None)):
            assert torch.equal(m, n)
    c.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,h,group,n", [(1, 4, 8, 1), (2, 1, 32, 1), (64, 2, 32, 8)])
def test_every_code(fmt, dtype, b, h, group, n):
    """Rows that favour one token each get that token's values: every code, in every type."""
    code = (torch.arange(48 * 128) * 37 % 256).to(torch.uint8).view(48, 128)
    if fmt == "e4m3":
        code[code & 0x7f == 0x7f] = 0  # not a NaN
    assert len(code[:32].unique()) >= 254
    code = code.view(ref.CODE[fmt])
    one = torch.zeros(48, 128)
    one[torch.arange(32), torch.arange(32)] = 1.0
    every = lambda x: x.expand(b, h, *x.shape).contiguous().cuda()  # noqa: E731
    scale = torch.tensor([0.75, 0.125, 96.0])
    c = lkv.Cache8.from_tensors(every(one.to(ref.CODE[fmt]).view(torch.int8)).view(ref.CODE[fmt]), every(code.view(torch.int8)).view(ref.CODE[fmt]),
                                every(torch.full((3,), 64.0)), every(scale), every(torch.zeros(16, 128, dtype=dtype)),
                                every(torch.zeros(16, 128, dtype=dtype)), i32(*[48] * b))
    row = torch.arange(h * group) % 32
    q = torch.zeros(b, h * group, n, 128, dtype=dtype)
    q[:, torch.arange(h * group), :, row] = 64.0
    want = (code.float().double() * scale.repeat_interleave(16)[:, None].double())[row][None, :, None]
    err = (c.attend(q.cuda()).cpu().double() - want).abs()
    # a weight in fp16 is off by 2^-11, exp2 and the logarithm of a scale by 2^-18; the others' weights are below 2^-500
    assert (err <= want.abs() * (2.0 ** -11 + 2.0 ** -18 + ref.half_step(dtype) * 1.01)).all()


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_read_is_the_product_in_fp32_rounded_to_the_type(fmt, dtype):
    """Bit for bit."""
    x = rows(gen(14), 2, 3, 333, dtype)
    c = lkv.Cache8(batch=2, n_kv_heads=3, capacity=336, dtype=dtype, fmt=fmt)
    c.write(x.cuda(), x.cuda())
    want = (c.k_codes.float() * c.k_scale.repeat_interleave(16, 2)[..., None]).to(dtype)
    for got in c.read(333):
        assert torch.equal(got[:, :, :320], want[:, :, :320])
        assert torch.equal(got[:, :, 320:], x[:, :, 320:].cuda())


# ---------------------------------------------------------------- NaN

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,h,group,n", [([300, 17], 2, 4, 1), ([9000], 1, 4, 1), ([20011, 20000], 1, 4, 3), ([700] * 64, 2, 4, 64),
                                               ([20001], 2, 4, 128)])
def test_a_query_that_is_not_a_number(dtype, lengths, h, group, n):
    """Its row of the output is NaN, however the call is split, and no other row is."""
    b, top = len(lengths), max(lengths)
    g = gen(n)
    x, y = (torch.randn(b, h, top, 128, generator=g).to(dtype) for _ in range(2))
    c, k, v = make(x, y, "int8", dtype, (top + 15) // 16 * 16, lengths)
    q = torch.randn(b, h * group, n, 128, generator=g).to(dtype)
    bad = torch.rand(b, h * group, n, generator=g) < 0.1
    bad[0, 1, n - 1], bad[0, 0, n - 1] = True, False
    q2 = q.clone()
    q2[..., 77][bad] = float("nan")
    got = c.attend(q2.cuda()).cpu()
    assert got[bad].isnan().all()
    for i, length in enumerate(lengths):
        kk, vv = (ref.values(a[0][i], a[1][i], a[2][i], length) for a in (k, v))
        want, lim = each.attend(q[i].double(), kk, vv, each.units(v[1][i], v[2][i], length), n, 128 ** -0.5, 0, 0, dtype)
        assert ((got[i].double() - want).abs() <= lim)[~bad[i]].all()
    c.check()
