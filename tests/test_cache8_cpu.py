"""Host side of the rotary positions and the 8-bit cache (no GPU): the rotary
table against its formulas, and the refusal of every kind of bad argument
before anything is launched."""
import ctypes as C
import math

import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests import _cache8_ref as ref


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


@pytest.mark.parametrize("rd", [2, 6, 34, 64, 128])
@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=4.0, orig_len=4096), dict(scaling="yarn", factor=1.0, orig_len=1, beta_slow=0.0),
    dict(scaling="yarn", factor=16.0, orig_len=32768, beta_fast=8.0, beta_slow=2.0)])
def test_rope_table(rd, kw):
    if kw.get("scaling") == "ntk" and rd == 2:
        pytest.skip("no pair to stretch")
    r = lkv.Rope(rotary_dim=rd, layout="interleaved", **kw)
    rates, gain = ref.rope_rates(rd, **kw)
    assert r.table.rotary_dim == rd and r.table.layout == _lib.LKV_ROPE_INTERLEAVED
    # one fp64 rounding for each of pow, the products and the division by 2 pi,
    # and half of the table's unit, 2^-64 turns: an entry is a whole number of units
    for i, f in enumerate(rates.tolist()):
        assert abs(r.table.turn[i] / 2.0 ** 64 - f / (2 * math.pi)) <= 8 * 2.0 ** -53 * f + 2.0 ** -65, i
    assert all(r.table.turn[i] == 0 for i in range(rd // 2, 64))
    assert abs(r.table.gain - gain) <= gain * 2.0 ** -24


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130), dict(base=0.5), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
    dict(scaling="ntk", factor=2.0, rotary_dim=2), dict(scaling="ntk", factor=1e308, base=1e300),
    dict(scaling="yarn", factor=2.0, orig_len=0), dict(scaling="yarn", factor=2.0, orig_len=8, beta_fast=1.0),
    dict(scaling="yarn", factor=2.0, orig_len=8, beta_slow=-1.0)])
def test_rope_table_refuses(kw):
    with pytest.raises(_lib.LKVError) as e:
        lkv.Rope(**kw)
    assert e.value.status == _lib.LKV_EINVAL and "lkv_rope_init" in str(e.value)


def test_rope_init_null_and_unknown():
    L = _lib.load()
    good = _lib.lkv_rope_params(128, 0, 0, 0, 1e4, 1.0, 32.0, 1.0)
    t = _lib.lkv_rope()
    assert L.lkv_rope_init(None, C.byref(t)) == _lib.LKV_EINVAL
    assert L.lkv_rope_init(C.byref(good), None) == _lib.LKV_EINVAL
    for field, value in (("layout", 2), ("layout", -1), ("scaling", 4), ("scaling", -1)):
        bad = _lib.lkv_rope_params(128, 0, 0, 0, 1e4, 1.0, 32.0, 1.0)
        setattr(bad, field, value)
        assert L.lkv_rope_init(C.byref(bad), C.byref(t)) == _lib.LKV_EINVAL


A = 1 << 20  # an aligned address that nothing dereferences: every call below is refused


def test_rope_apply_refuses():
    L = _lib.load()
    t = lkv.Rope().table
    at = C.addressof(t)
    far = [A * (i + 1) for i in range(5)]

    def call(table=at, dtype=1, batch=1, heads=2, kv=1, n=4, q=far[0], k=far[1], pos=far[2], qo=far[3], ko=far[4]):
        return L.lkv_rope_apply(table, dtype, batch, heads, kv, n, q, k, pos, qo, ko, None)

    E = _lib.LKV_EINVAL
    assert call(table=None) == E and call(dtype=2) == E and call(batch=-1) == E and call(heads=-1) == E
    assert call(kv=-2) == E and call(n=-1) == E and call(heads=40000) == E
    for name in ("q", "k", "pos", "qo", "ko"):
        assert call(**{name: None}) == E
        assert call(**{name: far[0] + A // 2 + 2}) == E, name
    assert call(qo=far[0] + 256) == E          # partly over its own input
    assert call(qo=far[1]) == E and call(ko=far[0]) == E and call(ko=far[3]) == E
    assert call(qo=far[2]) == E
    empty = _lib.lkv_rope()
    assert call(table=C.addressof(empty)) == E
    assert call(batch=0) == _lib.LKV_OK and call(n=0) == _lib.LKV_OK and call(heads=0, kv=0) == _lib.LKV_OK


def _view(**kw):
    f = dict(batch=2, n_kv_heads=2, capacity=64, dtype=1, code=0, reserved=0, k_codes=A, v_codes=2 * A,
             k_scale=3 * A, v_scale=4 * A, k_tail=5 * A, v_tail=6 * A, lengths=7 * A, ticket=8 * A)
    f.update(kw)
    return _lib.lkv_cache8(**f)


BAD_VIEWS = [dict(batch=0), dict(batch=(1 << 20) + 1), dict(n_kv_heads=0), dict(n_kv_heads=5000), dict(capacity=0), dict(capacity=24),
             dict(capacity=-16), dict(dtype=2), dict(code=2), dict(code=-1), dict(k_codes=None), dict(v_codes=None),
             dict(k_scale=None), dict(v_scale=None), dict(k_tail=None), dict(v_tail=None), dict(lengths=None),
             dict(ticket=None), dict(k_codes=A + 8), dict(v_tail=6 * A + 4), dict(k_scale=3 * A + 2),
             dict(lengths=7 * A + 1)]


@pytest.mark.parametrize("bad", BAD_VIEWS)
def test_cache_calls_refuse_a_bad_view(bad):
    L = _lib.load()
    v = C.addressof(c := _view(**bad))
    out = C.c_int64()
    assert L.lkv_cache8_write(v, 20 * A, 21 * A, 1, None, None, None) == _lib.LKV_EINVAL
    assert L.lkv_cache8_read(v, None, 1, 20 * A, 21 * A, None) == _lib.LKV_EINVAL
    assert L.lkv_cache8_attend(v, 20 * A, 4, 1, None, 1.0, 0, 0, 0, 21 * A, None, 0, None) == _lib.LKV_EINVAL
    assert L.lkv_cache8_attend_workspace(v, 4, 1, 0, 0, 0, C.byref(out)) == _lib.LKV_EINVAL
    assert L.lkv_cache8_status(v, None) == _lib.LKV_EINVAL
    assert _lib.lkv_last_error(None)
    del c


def test_cache_calls_refuse_bad_arguments():
    L = _lib.load()
    c = _view()
    v, E = C.addressof(c), _lib.LKV_EINVAL
    for fn, args in ((L.lkv_cache8_write, (20 * A, 21 * A, 1, None, None)), (L.lkv_cache8_read, (None, 1, 20 * A, 21 * A))):
        assert fn(None, *args, None) == E
    q, o = 20 * A, 21 * A
    assert L.lkv_cache8_write(v, None, o, 1, None, None, None) == E
    assert L.lkv_cache8_write(v, q, None, 1, None, None, None) == E
    assert L.lkv_cache8_write(v, q, o, -1, None, None, None) == E
    assert L.lkv_cache8_write(v, q + 8, o, 1, None, None, None) == E
    assert L.lkv_cache8_write(v, q, o, 1, A + 1, None, None) == E
    assert L.lkv_cache8_write(v, 5 * A, o, 1, None, None, None) == E          # keys in the tail
    assert L.lkv_cache8_write(v, q, o, 1, 7 * A, None, None) == E             # start is the lengths
    assert L.lkv_cache8_write(v, q, o, 1, None, 8 * A, None) == E
    assert L.lkv_cache8_read(v, None, -1, q, o, None) == E
    assert L.lkv_cache8_read(v, None, 1, None, o, None) == E
    assert L.lkv_cache8_read(v, None, 1, q, q, None) == E
    assert L.lkv_cache8_read(v, None, 1, A, o, None) == E
    assert L.lkv_cache8_read(v, q, 1, q, o, None) == E

    def attend(q=q, group=4, n=1, counts=None, scale=1.0, window=0, sinks=0, max_len=0, out=o):
        return L.lkv_cache8_attend(v, q, group, n, counts, scale, window, sinks, max_len, out, None, 0, None)

    assert attend(q=None) == E and attend(out=None) == E and attend(q=q + 4) == E and attend(out=o + 8) == E
    assert attend(group=0) == E and attend(group=129) == E and attend(n=-1) == E and attend(n=(1 << 24) + 1) == E
    assert attend(scale=float("nan")) == E and attend(scale=float("inf")) == E and attend(scale=3e38) == E
    assert attend(window=-1) == E and attend(sinks=-1) == E and attend(max_len=-1) == E
    assert attend(counts=A + 2) == E and attend(out=q) == E and attend(out=A) == E and attend(out=5 * A) == E
    assert attend(counts=o) == E
    assert L.lkv_cache8_attend_workspace(v, 4, 1, 0, 0, 0, None) == E
    # nothing to do: no launch
    assert attend(n=0) == _lib.LKV_OK
    assert L.lkv_cache8_write(v, None, None, 0, None, None, None) == _lib.LKV_OK
    assert L.lkv_cache8_read(v, None, 0, None, None, None) == _lib.LKV_OK


def test_rope_refuses_sizes_past_32_bits():
    for kw in (dict(rotary_dim=2 ** 32 + 64), dict(scaling="yarn", factor=2.0, orig_len=2 ** 32 + 8)):
        with pytest.raises(ValueError):
            lkv.Rope(**kw)


def test_python_wrappers_refuse_host_tensors():
    with pytest.raises(ValueError):
        lkv.Rope().apply(torch.zeros(1, 1, 1, 128), torch.zeros(1, 1, dtype=torch.int32))
    z = torch.zeros(1, 1, 16, 128, dtype=torch.int8)
    with pytest.raises(ValueError):
        lkv.Cache8.from_tensors(z, z, torch.zeros(1, 1, 1), torch.zeros(1, 1, 1), torch.zeros(1, 1, 16, 128),
                                torch.zeros(1, 1, 16, 128), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        lkv.Cache8(batch=1, n_kv_heads=1, capacity=24, dtype=torch.float32, device="cpu")
    with pytest.raises(ValueError):
        lkv.Cache8(batch=1, n_kv_heads=1, capacity=16, dtype=torch.float32, fmt="int4", device="cpu")


def test_reference_e4m3_is_torchs_cast():
    """The tests' own e4m3 rounding, on every fp16 value in range, is the cast's."""
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.float16)
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    assert torch.equal(ref.e4m3(x.double()).float(), x.float().to(torch.float8_e4m3fn).float())
