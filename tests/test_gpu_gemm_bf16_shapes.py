"""moe_grouped_gemm_bf16 on every tile shape.

The shape goes by the capacity (rows of a over the experts), N and K, so small
ragged segments in a large buffer reach each of them; the tolerance is that of
test_gpu_gemm_bf16.py.
"""
import os
import re
import subprocess
import sys

import pytest
import torch

from parity_util import log
from test_gpu_gemm_bf16 import case, run

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (rows of a tile, threads) of a shape in the launch log
LOGGED = {"large": (256, 256), "medium": (128, 512), "small": (128, 256), "skinny": (32, 256)}

# shape: (experts, capacity, N, inner sizes: one k-block to several turns of the
# ring with every remainder, and odd tails). The last column tile holds 16 columns,
# 8 in the gated form.
SHAPES = {
    "large": (3, 12000, 1040, (8, 64, 72, 200, 264, 328, 392, 584)),
    "medium": (6, 6000, 1040, (1544, 1600, 1608, 1672)),
    "small": (6, 6000, 400, (8, 64, 72, 200, 264, 328, 392, 584)),
    "skinny": (8, 240, 1040, (8, 64, 72, 256, 264, 584)),
}
# rows of the segments: ends inside a tile, a tile whose second half is empty,
# whole tiles, one row, none
COUNTS = {"large": (257, 130, 391), "medium": (129, 1, 0, 128, 300, 60),
          "small": (129, 1, 0, 128, 300, 60), "skinny": (33, 1, 0, 32, 70, 5, 31, 64)}


def shape_case(shape, K, gated, bias=False, residual=False, seed=None):
    E, R, N, _ = SHAPES[shape]
    counts = COUNTS[shape]
    assert len(counts) == E
    # the rows before the first segment and behind the last are no one's
    return case(counts, K, N, R=R, seed=K if seed is None else seed, bias=bias, residual=residual,
                gated=gated, first=0 if shape == "skinny" else 5)


ALL = [(s, K, g) for s in SHAPES for K in SHAPES[s][3] for g in (False, True)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_infinite_sums(shape, gated, act):
    """z = +inf, from an infinite input or a sum past fp32, is +inf after every
    activation: relu z, z sigmoid(z) and z/2 erfc(-z/sqrt 2) all grow with z. Large
    finite z are themselves (one rounding, 2^-8), times the up half when gated."""
    log(f"shape infinite {shape} gated={gated} {act}")
    c = shape_case(shape, 264 if shape != "medium" else 1544, gated)
    c["w"] = c["w"].abs() + 0.01
    r = c["off"][0]
    c["a"][r] = c["a"][r].abs()
    c["a"][r, 7] = float("inf")
    c["a"][r + 1] = 3.3e38                               # K terms of at least 3e36
    c["a"][r + 2] = 1e15                                 # z and z^2 are finite
    y = run(c, act)
    assert (y[r:r + 2] == float("inf")).all()
    z = c["a"][r + 2].double() @ c["w"][0].double().T
    N = z.shape[0]
    want = z[:N // 2] * z[N // 2:] if gated else z
    # the sum of positive terms is off by K 2^-23 of itself, squared when gated
    tol = 2.0 ** -8 + 3 * c["a"].shape[1] * 2.0 ** -23
    assert ((y[r + 2].double() - want).abs() <= tol * want).all()


def test_shapes_reached():
    """From the launch log, read in a child process: each case above runs on the
    shape it is listed under, and rows of whole 128-byte lines are streamed by
    the skinny tiles of small capacities, others not."""
    cases = [(s, K, g) for s, K, g in ALL]
    code = ("import sys; sys.path.insert(0, 'tests')\n"
            "from test_gpu_gemm_bf16_shapes import shape_case\n"
            "from test_gpu_gemm_bf16 import run\n"
            f"for s, K, g in {cases!r}:\n"
            "    run(shape_case(s, K, g), 'none')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=110, env=dict(os.environ, MOE_ROUTE_LOG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = re.findall(r"(\w*)grouped_gemm_bf16 grid=\d+ block=(\d+) lds=\d+ param=(\d+)", r.stderr)
    assert len(got) == len(cases)
    for (shape, K, _), (prefix, block, rows) in zip(cases, got):
        assert (int(rows), int(block)) == LOGGED[shape], (shape, K)
        assert (prefix == "streamed_") == (shape == "skinny" and K % 64 == 0), (shape, K, prefix)
