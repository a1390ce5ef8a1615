"""The Python calls of rotary positions and the 8-bit cache: what they refuse
and what they keep."""
import math

import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _cache8_each as each
from tests import _cache8_ref as ref
from tests.test_gpu_rope import check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def small():
    c = lkv.Cache8(batch=2, n_kv_heads=2, capacity=64, dtype=BF16)
    k, v = (torch.randn(2, 2, 40, 128, device="cuda").to(BF16) for _ in range(2))
    c.write(k, v)
    return c, k, torch.randn(2, 8, 3, 128, device="cuda").to(BF16)


def test_sizes_below_minus_2_31_are_refused():
    """-2^32 is not 0: it does not come out as attention over everything."""
    c, k, q = small()
    for kw in (dict(window=-2 ** 32), dict(window=3, sinks=-2 ** 32), dict(max_len=-2 ** 33), dict(window=-2 ** 31 - 5)):
        with pytest.raises(ValueError):
            c.attend(q, **kw)
    for n in (-1, -2 ** 32, 2 ** 31):
        with pytest.raises(ValueError):
            c.read(n)
    with pytest.raises(_lib.LKVError):
        c.attend(q, window=-1)
    c.check()


def test_a_bound_that_grows_asks_for_few_workspaces(monkeypatch):
    """max_len one larger each step, as a server passes it: right outputs, and a
    size of workspace asked for now and then only."""
    c = lkv.Cache8(batch=1, n_kv_heads=2, capacity=40960, dtype=BF16)
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(1, 2, 8000, 128, generator=g).to(BF16) for _ in range(2))
    c.write(k.cuda(), v.cuda())
    q = torch.randn(1, 8, 1, 128, generator=g).to(BF16)
    kk, vv = (ref.held(x, "int8", BF16, 8000, [8000]) for x in (k, v))
    want, lim = each.attend(q[0].double(), *(ref.values(*(t[0] for t in x), 8000) for x in (kk, vv)), each.units(vv[1][0], vv[2][0], 8000), 1,
                            128 ** -0.5, 0, 0, BF16)
    q = q.cuda()
    asked = []
    ask = _lib.lkv_cache8_attend_workspace
    monkeypatch.setattr(_lib, "lkv_cache8_attend_workspace", lambda *a: asked.append(a[1:]) or ask(*a))
    for m in range(8000, 9000):
        got = c.attend(q, max_len=m)
        if m % 100 == 0:
            assert ((got[0].cpu().double() - want).abs() <= lim).all()  # whatever the split
    assert len(asked) <= 1000 // 64 + 2
    # a bound is never made smaller, and one past the capacity is none
    for m in (1, 15, 16, 17, 127, 128, 129, 8191, 8192, 8193, 40959, 40960, 40961, 2 ** 31 - 1):
        c._ws_bytes.clear()
        c.attend(q, max_len=m)
        bound = asked[-1][-1]
        assert bound == 0 if m >= 40960 else bound == 0 or m <= bound <= m + max(15, m // 64)
    c.check()


def test_tensors_that_require_gradients():
    """No call has a backward pass: where gradients are recorded it says so
    rather than cut the graph; under no_grad, and detached, it runs."""
    c, k, q = small()
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    r = lkv.Rope()
    leaf, kl, free = q.clone().requires_grad_(), k[:, :, :3].contiguous().requires_grad_(), k[:, :, :3].contiguous()
    calls = [lambda: c.attend(leaf), lambda: c.attend(leaf * 2), lambda: r.apply(leaf, pos), lambda: r.apply(q, pos, kl), lambda: c.write(kl, free),
             lambda: c.write(free, kl), lambda: r.apply(q, pos, q_out=leaf), lambda: c.attend(q, out=leaf),
             lambda: c.read(3, k_out=kl, v_out=free.clone())]
    before = c.lengths.tolist()
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    assert c.lengths.tolist() == before and leaf.grad is None
    want = c.attend(q)
    with torch.no_grad():
        assert torch.equal(c.attend(leaf), want)
        r.apply(leaf, pos, kl)
        c.write(kl, free)
    with torch.inference_mode():
        assert c.attend(leaf).shape == want.shape
    assert c.attend(leaf.detach()).shape == want.shape
    c.check()


def test_check_reports_an_attention_that_gave_up():
    """The word that a kernel's bounded wait sets is set here by the host: it
    comes before what writes recorded, once, and the cache goes on."""
    c, k, q = small()
    want = c.attend(q)
    timeout, rest = 8, 1 | 2 | 4
    for bits, status in ((timeout, _lib.LKV_ETIMEOUT), (timeout | rest, _lib.LKV_ETIMEOUT), (rest, _lib.LKV_ECAPACITY), (2 | 4, _lib.LKV_ECAPACITY),
                         (1 | 4, _lib.LKV_EINVAL), (4, _lib.LKV_EINVAL)):
        c._ticket[-1] = bits
        with pytest.raises(_lib.LKVError) as e:
            c.check()
        assert e.value.status == status
        c.check()
        assert torch.equal(c.attend(q), want)
        c.check()
    assert c._ticket.tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_frequencies_of_ones_own(dtype, layout):
    """A table filled by the program: YaRN's ramp over pair indexes, which no scaling of Rope's gives."""
    base, factor, orig, fast, slow = 1e6, 4.0, 32768, 32.0, 1.0

    def pair(turns):
        return 128 * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = math.floor(pair(fast)), math.ceil(pair(slow))
    f = [base ** (-2 * i / 128) for i in range(64)]
    keep = [1 - min(1.0, max(0.0, (i - low) / (high - low))) for i in range(64)]
    f = [x * (g + (1 - g) / factor) for x, g in zip(f, keep)]
    gain = 0.1 * math.log(factor) + 1
    r = lkv.Rope(base=base, layout=layout)
    for i, x in enumerate(f):
        r.table.turn[i] = round(x / (2 * math.pi) * 2 ** 64)
    r.table.gain = gain
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(2, h, 40, 128, generator=g).to(dtype).cuda() for h in (8, 2))
    pos = torch.randint(0, 1 << 17, (2, 40), generator=g, dtype=torch.int32).cuda()
    q2, k2 = r.apply(q, pos, k)
    rates = torch.tensor(f, dtype=torch.float64)
    check(q2, q, pos, rates, gain, layout)
    check(k2, k, pos, rates, gain, layout)
    paper, _ = ref.rope_rates(128, base=base, scaling="yarn", factor=factor, orig_len=orig)
    assert (rates / paper).max() > 1.3  # another ramp than scaling="yarn"
