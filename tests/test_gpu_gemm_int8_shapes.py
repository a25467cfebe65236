"""Every tile shape of moe_grouped_gemm_int8: each is reached, by the launch log
(MOE_ROUTE_LOG=1, read in a child process), and gives the reference's result with
every epilogue, with tails in every direction and with segments longer than a tile."""
import os
import re
import subprocess
import sys

import pytest

from parity_util import log
from test_gpu_gemm_int8 import case, check

pytestmark = pytest.mark.gpu

# counts, K, N, gated -> (rows of a tile, threads, LDS)
SHAPES = [
    (([20, 3], 256, 128, False), ("32", "256", "32768")),         # narrow, whole lines
    (([20, 3], 272, 128, False), ("32", "256", "32768")),         # narrow, shared lines
    (([20, 3], 256, 128, True), ("32", "256", "65536")),
    (([3] * 40, 256, 4104, False), ("32", "256", "65536")),       # whole lines
    (([5] * 40, 272, 4104, False), ("32", "256", "65536")),
    (([97, 90, 80], 8336, 744, False), ("32", "256", "32768")),   # few tiles, deep
    (([97, 90, 80], 8336, 1504, True), ("32", "256", "65536")),
    (([120] * 12, 2032, 1032, False), ("128", "256", "81920")),
    (([2048], 4096, 4096, False), ("128", "512", "147456")),
    (([1000] * 8, 4096, 4096, True), ("256", "256", "163840")),
]


def test_rule_reaches_every_shape():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.path.insert(0, 'tests')\n"
            "from test_gpu_gemm_int8 import case, check\n"
            f"for c, K, N, g in {[c for c, _ in SHAPES]!r}:\n"
            "    check(case(c, K, N, gated=g), 'silu')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=110, env=dict(os.environ, MOE_ROUTE_LOG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = re.findall(r"grouped_gemm_int8 grid=\d+ block=(\d+) lds=(\d+) param=(\d+)", r.stderr)
    assert [(p, b, l) for b, l, p in got] == [want for _, want in SHAPES]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("counts,K,N", [
    ([20, 33, 1], 400, 200), ([2, 0, 40, 5], 128, 56),            # narrow, a segment past a tile
    ([7] * 30, 144, 2088), ([40, 1, 2, 3] * 8, 256, 2056),        # 64 wide
    ([97, 90], 4112, 1000),
])
@pytest.mark.parametrize("gated", [False, True])
def test_skinny_epilogues(act, counts, K, N, gated):
    N = (N + 15) // 16 * 16 if gated else N
    log(f"int8 skinny {act} {len(counts)} K={K} N={N} gated={gated}")
    check(case(counts, K, N, seed=N, bias=True, residual=True, gated=gated, R=sum(counts) + 9), act)


@pytest.mark.parametrize("counts,K,N", [([120] * 12, 2032, 1032), ([2048], 2032, 4088),
                                        ([1030] * 8, 1040, 2072), ([300, 5, 0, 777] * 4, 1104, 2056)])
@pytest.mark.parametrize("gated", [False, True])
def test_wide_epilogues(counts, K, N, gated):
    N = (N + 15) // 16 * 16 if gated else N
    log(f"int8 wide {counts[:4]} K={K} N={N} gated={gated}")
    check(case(counts, K, N, seed=N, bias=True, residual=True, gated=gated, align=8), "gelu")
