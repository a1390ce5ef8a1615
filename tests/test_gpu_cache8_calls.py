"""The Python calls of rotary positions and the 8-bit cache: what they refuse
and what they keep."""
import pytest
import torch

import cluster_indexed_kv_gb300 as lkv
from cluster_indexed_kv_gb300 import _lib

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
