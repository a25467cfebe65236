"""Which skinny launches of moe_grouped_gemm_int8 stream their weights past the caches
(non-temporal loads): those of up to 20 rows an expert whose weight rows are whole
128-byte lines. Read from the launch log (MOE_ROUTE_LOG=1) in a child process; each
result is the reference's."""
import os
import re
import subprocess
import sys

import pytest

from parity_util import log

pytestmark = pytest.mark.gpu

# counts, K, N, gated -> (streamed, LDS: 32768 for tiles of 32 weight rows, 65536 for 64)
CASES = [
    (([20, 3], 256, 128, False), (True, 32768)),
    (([20, 3], 272, 128, False), (False, 32768)),
    (([20, 3], 256, 128, True), (True, 65536)),
    (([20, 3], 272, 128, True), (False, 65536)),
    (([20, 20], 384, 128, False), (True, 32768)),
    (([20, 20], 320, 128, False), (False, 32768)),                # half a line over
    (([3] * 40, 256, 4104, False), (True, 65536)),
    (([5] * 40, 272, 4104, False), (False, 65536)),
    (([5] * 40, 128, 4112, True), (True, 65536)),
    (([5] * 40, 144, 4112, True), (False, 65536)),
    (([97, 90, 80], 8320, 744, False), (False, 32768)),           # more rows: read again
    (([97, 90, 80], 8320, 1504, True), (False, 65536)),
]


def test_streamed_where_rows_are_whole_lines():
    log("int8 streamed")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.path.insert(0, 'tests')\n"
            "from test_gpu_gemm_int8 import case, check\n"
            f"for c, K, N, g in {[c for c, _ in CASES]!r}:\n"
            "    check(case(c, K, N, gated=g), 'silu')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=110, env=dict(os.environ, MOE_ROUTE_LOG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = re.findall(r"\[moe_route\] (streamed_)?grouped_gemm_int8 grid=\d+ block=256 lds=(\d+) "
                     r"param=32\b", r.stderr)
    assert [(bool(s), int(lds)) for s, lds in got] == [want for _, want in CASES]
