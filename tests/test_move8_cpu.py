"""Host side of taking and keeping tokens of the 8-bit cache, of attention behind
shared prefixes and of rotary positions on several axes (no GPU): refusals before anything is launched."""
import ctypes as C

import pytest

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib
from tests.test_cache8_arrays_cpu import ARRAYS
from tests.test_cache8_cpu import A, BAD_VIEWS, _view

E = _lib.LKV_EINVAL


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


def other(**kw):
    at = {name: (100 + i) * A for i, name in enumerate(ARRAYS)}
    return _view(**(at | kw))


@pytest.mark.parametrize("bad", BAD_VIEWS)
def test_bad_views(bad):
    L, out = _lib.load(), C.c_int64()
    good, wrong = _view(), _view(**bad)
    g, w = C.addressof(good), C.addressof(wrong)
    for to, source in ((w, None), (w, w), (g, w)):
        assert L.lkv_cache8_take(to, source, None, None, 20 * A, 1 << 20, None) == E
        assert L.lkv_cache8_take_workspace(to, source, C.byref(out)) == E
        assert L.lkv_cache8_keep(to, source, 20 * A, 1, 21 * A, None) == E


def test_take_and_keep_refuse():
    L, out = _lib.load(), C.c_int64()
    c, s = _view(), other()
    v, f = C.addressof(c), C.addressof(s)

    def take(to=v, source=f, sequences=20 * A, lengths=21 * A, ws=22 * A, bytes=1 << 20):
        return L.lkv_cache8_take(to, source, sequences, lengths, ws, bytes, None)

    def keep(to=v, source=f, blocks=20 * A, m=2, counts=21 * A):
        return L.lkv_cache8_keep(to, source, blocks, m, counts, None)

    assert take(to=None) == E and keep(to=None) == E and L.lkv_cache8_take_workspace(None, None, C.byref(out)) == E
    assert L.lkv_cache8_take_workspace(v, f, None) == E
    # within the cache: a snapshot of two tails of [2][2][16][128] bf16 and of two lengths
    assert L.lkv_cache8_take_workspace(v, None, C.byref(out)) == 0 and out.value == 2 * 2 * 2 * 16 * 128 * 2 + 16
    assert L.lkv_cache8_take_workspace(v, f, C.byref(out)) == 0 and out.value == 0
    assert take(source=None, ws=None) == E and take(source=None, bytes=100) == E and take(source=v, bytes=2 * 2 * 2 * 16 * 128 * 2) == E
    assert take(source=None, ws=22 * A + 8) == E
    for at in (A, 3 * A, 5 * A, 7 * A, 8 * A):
        assert take(source=None, ws=at) == E and take(sequences=at) == E and take(lengths=at) == E
        assert keep(blocks=at) == E and keep(counts=at) == E
    assert take(source=None, sequences=22 * A + 16) == E and take(source=None, lengths=22 * A) == E
    assert take(sequences=20 * A + 2) == E and take(lengths=20 * A + 1) == E
    assert keep(blocks=20 * A + 2) == E and keep(counts=20 * A + 2) == E and keep(m=-1) == E
    assert keep(counts=None) == E and keep(blocks=None) == E
    for kw in (dict(n_kv_heads=3), dict(dtype=0), dict(code=1)):
        x = other(**kw)
        assert take(source=C.addressof(x)) == E and keep(source=C.addressof(x)) == E
    x = other(batch=3)
    assert keep(source=C.addressof(x)) == E
    big = _view(batch=1025, lengths=7 * A, ticket=8 * A, k_codes=50 * A, v_codes=70 * A, k_scale=90 * A, v_scale=91 * A, k_tail=92 * A, v_tail=112 * A)
    assert take(to=C.addressof(big), source=None, bytes=1 << 40) == E
    assert "1024" in _lib.lkv_last_error(None)
    # one array shared with another cache, or the same cache with one array of its own
    for i, name in enumerate(ARRAYS):
        x, y = other(**{name: getattr(c, name)}), _view(**{name: (100 + i) * A})
        assert take(source=C.addressof(x)) == E and keep(source=C.addressof(x)) == E
        assert take(source=C.addressof(y)) == E and keep(source=C.addressof(y)) == E
    y = _view(v_codes=A)
    assert take(to=C.addressof(y), source=None) == E and keep(to=C.addressof(y), source=None) == E


@pytest.mark.parametrize("bad", BAD_VIEWS)
def test_shared_attention_bad_views(bad):
    L, out = _lib.load(), C.c_int64()
    good, wrong = other(), _view(**bad)
    g, w = C.addressof(good), C.addressof(wrong)
    for c, p in ((w, g), (g, w), (w, w), (None, g), (g, None)):
        assert L.lkv_cache8_attend_shared(c, p, 20 * A, 21 * A, 4, 1, None, 1.0, 0, 22 * A, 23 * A, 1 << 20, None) == E
        assert L.lkv_cache8_attend_shared_workspace(c, p, 4, 1, 0, C.byref(out)) == E


def test_shared_attention_refuses():
    L, out = _lib.load(), C.c_int64()
    c, p = _view(), other()
    v, f = C.addressof(c), C.addressof(p)

    def call(c=v, p=f, of=20 * A, q=21 * A, group=4, n=1, counts=None, scale=1.0, max_len=0, o=22 * A, ws=23 * A, bytes=1 << 20):
        return L.lkv_cache8_attend_shared(c, p, of, q, group, n, counts, scale, max_len, o, ws, bytes, None)

    assert L.lkv_cache8_attend_shared_workspace(v, f, 4, 1, 0, None) == E
    for kw in (dict(group=0), dict(group=129), dict(n=-1), dict(n=(1 << 24) + 1), dict(max_len=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(scale=3e38), dict(q=None), dict(o=None), dict(q=21 * A + 8), dict(o=22 * A + 8), dict(ws=23 * A + 8), dict(counts=24 * A + 2),
               dict(of=20 * A + 1), dict(o=21 * A + 256), dict(o=20 * A), dict(counts=22 * A, o=22 * A)):
        assert call(**kw) == E, kw
    for x in (c, p):  # the output in a cache
        for name in ARRAYS:
            assert call(o=getattr(x, name)) == E, name
    for kw in (dict(n_kv_heads=3), dict(dtype=0), dict(code=1), dict(batch=1025)):
        x = other(**kw)
        assert call(p=C.addressof(x)) == E and L.lkv_cache8_attend_shared_workspace(v, C.addressof(x), 4, 1, 0, C.byref(out)) == E
    big = _view(batch=1025)
    assert call(c=C.addressof(big)) == E
    assert call(n=0) == _lib.LKV_OK
    assert L.lkv_cache8_attend_shared_workspace(v, f, 4, 0, 0, C.byref(out)) == _lib.LKV_OK and out.value == 0


def test_rope_axes_refuse():
    L = _lib.load()
    t = lkv.Rope().table
    at = C.addressof(t)
    far = [A * (i + 1) for i in range(5)]
    good = (C.c_uint8 * 64)(*[i % 3 for i in range(64)])

    def call(table=at, axis=good, axes=3, dtype=1, batch=1, heads=2, kv=1, n=4, q=far[0], k=far[1], pos=far[2], qo=far[3], ko=far[4]):
        return L.lkv_rope_apply_axes(table, axis, axes, dtype, batch, heads, kv, n, q, k, pos, qo, ko, None)

    assert call(table=None) == E and call(axis=None) == E and call(axes=0) == E and call(axes=5) == E and call(axes=2) == E and call(axes=-1) == E
    assert "axis" in _lib.lkv_last_error(None) or "axes" in _lib.lkv_last_error(None)
    assert call(dtype=2) == E and call(batch=-1) == E and call(heads=40000) == E and call(kv=-2) == E and call(n=-1) == E
    for name in ("q", "k", "pos", "qo", "ko"):
        assert call(**{name: None}) == E
        assert call(**{name: far[0] + A // 2 + 2}) == E, name
    assert call(qo=far[0] + 256) == E and call(qo=far[1]) == E and call(ko=far[0]) == E and call(ko=far[3]) == E
    assert call(qo=far[2] + 32) == E  # the third axis's positions: [3][1][4] int32
    assert call(batch=0) == _lib.LKV_OK and call(n=0) == _lib.LKV_OK and call(heads=0, kv=0) == _lib.LKV_OK


def test_rope_sections_tables():
    """Sections of their own begin their frequencies anew; sections of one rotation do not."""
    whole, apart, one = lkv.Rope(base=1e6, sections=(16, 24, 24)), lkv.Rope(base=1e6, sections=(16, 24, 24), own_base=True), lkv.Rope(base=1e6)
    assert list(whole.table.turn) == list(one.table.turn) and whole.n_axes == 3 and one.n_axes == 0
    assert list(whole._axis) == [0] * 16 + [1] * 24 + [2] * 24
    for at, s in ((0, 16), (16, 24), (40, 24)):
        assert list(apart.table.turn)[at:at + s] == list(lkv.Rope(base=1e6, rotary_dim=2 * s).table.turn)[:s]
