"""The visible range of a block's tokens (no GPU): the kernels' own function,
compiled for the host with overflow checks, against 64-bit arithmetic."""
import itertools
import os
import subprocess

import pytest

from cluster_indexed_kv_gb300 import builder

SRC = r"""
#include <cstdio>
#include "attend8.cuh"
int main() {
  long long tok, pos, window, sinks;
  while (std::scanf("%lld %lld %lld %lld", &tok, &pos, &window, &sinks) == 4) {
    int see[3];
    lkv::token_range((int)(tok < 0 ? lkv::kNoToken : tok), (int)pos, (int)window, (int)sinks, see);
    for (int i = 0; i < 16; ++i) std::printf("%d", (int)lkv::sees(see, i));
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("ranges")
    (d / "ranges.cu").write_text(SRC)
    exe = str(d / "ranges")
    flags = ["-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I" + builder.INCLUDE, "-I" + builder.CSRC]
    check = ["-Xcompiler", "-fsanitize=signed-integer-overflow", "-Xcompiler", "-fno-sanitize-recover=all"]
    r = subprocess.run([builder.nvcc(), *builder.ARCH, *flags, *check, str(d / "ranges.cu"), "-o", exe, "-lubsan"], capture_output=True, text=True)
    if r.returncode != 0 and "cannot find -lubsan" in r.stderr:
        pytest.skip("no overflow checks in this compiler")
    assert r.returncode == 0, r.stderr
    assert os.path.exists(exe)
    return exe


def test_token_range(program):
    """Blocks from the first to the last of the largest cache, and one that is
    not there (-1); positions from -1 on, windows and sinks of any size."""
    top = 1 << 30
    tok = [-1, 0, 16, 4096, top // 2, top - 32, top - 16]
    pos = [-1, 0, 1, 15, 16, 31, 4100, top // 2 + 3, top - 17, top - 16, top - 1]
    window = [0, 1, 15, 16, 17, 5000, top - 1]
    sinks = [0, 1, 20, 4105, top]
    cases = list(itertools.product(tok, pos, window, sinks))
    r = subprocess.run([program], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    for (t, p, w, s), got in zip(cases, r.stdout.split(), strict=True):
        want = "".join(str(int(t >= 0 and t + i <= p and (w == 0 or t + i > p - w or t + i < s))) for i in range(16))
        assert got == want, (t, p, w, s)
