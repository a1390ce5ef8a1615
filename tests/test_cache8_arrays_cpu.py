"""A cache whose own arrays share memory is not written (no GPU: refused before a launch)."""
import ctypes as C
import itertools

import pytest

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib

A = 1 << 20  # an aligned address that nothing dereferences: every call below is refused
ARRAYS = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "lengths", "ticket")


@pytest.fixture(scope="module", autouse=True)
def _built():
    lkv.build()


@pytest.mark.parametrize("one,two", list(itertools.combinations(ARRAYS, 2)))
def test_write_refuses_arrays_that_share_memory(one, two):
    """The last bytes of one array are the first of another, either way round."""
    b, h, cap = 5, 2, 64
    size = dict(k_codes=b * h * cap * 128, v_codes=b * h * cap * 128, k_scale=b * h * cap // 4, v_scale=b * h * cap // 4,
                k_tail=b * h * 16 * 256, v_tail=b * h * 16 * 256, lengths=4 * b, ticket=4 * (b + 1))
    for first, second in ((one, two), (two, one)):
        at = {name: A * (i + 1) for i, name in enumerate(ARRAYS)}
        at[second] = at[first] + (size[first] - 1) // 16 * 16
        view = _lib.lkv_cache8(b, h, cap, 1, 0, 0, *(at[name] for name in ARRAYS))
        assert _lib.load().lkv_cache8_write(C.addressof(view), 20 * A, 21 * A, 1, None, None, None) == _lib.LKV_EINVAL
        assert "arrays overlap" in _lib.lkv_last_error(None)
