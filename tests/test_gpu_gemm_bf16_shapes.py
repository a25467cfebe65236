"""moe_grouped_gemm_bf16 on every tile shape: epilogues, tails of the inner
dimension and of the columns, segments that end inside a tile, in-place
residuals, non-finite rows, and rows behind 2^32 bytes.

The shape goes by the capacity (rows of a over the experts), N and K, so small
ragged segments in a large buffer reach each of them; the tolerance is that of
test_gpu_gemm_bf16.py. test_shapes_reached reads from the launch log that every
case runs on the shape it is listed under.
"""
import os
import re
import subprocess
import sys

import pytest
import torch

from parity_util import log
from test_gpu_gemm_bf16 import SENTINEL, case, check, run

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


@pytest.mark.parametrize("shape,K,gated", ALL)
def test_inner_sizes(shape, K, gated):
    log(f"shapes {shape} K={K} gated={gated}")
    check(shape_case(shape, K, gated), "none")
    check(shape_case(shape, K, gated, bias=True, residual=True), "gelu")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_epilogues_of_each_shape(shape, gated, act):
    log(f"shape epilogues {shape} gated={gated} {act}")
    K = SHAPES[shape][3][-2]
    for bias, residual in ((False, False), (True, False), (False, True), (True, True)):
        check(shape_case(shape, K, gated, bias=bias, residual=residual), act)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_residual_in_place(shape, gated):
    """residual = y gives the same bits as a residual of its own, repeatedly."""
    from combine_moe_route_amd import moe_grouped_gemm_bf16
    log(f"shape in place {shape} gated={gated}")
    c = shape_case(shape, SHAPES[shape][3][-1], gated, bias=True, residual=True)
    want = run(c, "silu")
    off = torch.tensor(c["off"], dtype=torch.int32, device=DEV)
    first, end = c["off"][0], c["off"][-1]
    for _ in range(3):
        y = c["residual"].clone()
        moe_grouped_gemm_bf16(c["a"], off, c["w"], bias=c["bias"], act="silu", gated=gated,
                              residual=y, y=y)
        assert torch.equal(y[first:end], want[first:end])
        assert torch.equal(y[:first], c["residual"][:first])
        assert torch.equal(y[end:], c["residual"][end:])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_non_finite_rows(shape, gated):
    """NaN and inf in a row reach that row only; NaN outside the segments
    reaches nothing."""
    log(f"shape non-finite {shape} gated={gated}")
    c = shape_case(shape, SHAPES[shape][3][-1], gated, residual=True)
    first, end = c["off"][0], c["off"][-1]
    clean = run(c, "silu")
    c["a"][:first] = float("nan")
    c["a"][end:] = float("nan")
    c["residual"][end:] = float("nan")
    hit = [first, first + 31, c["off"][1], end - 1]      # two rows of one tile, a first, the last
    c["a"][hit[0], -1] = float("nan")
    c["a"][hit[1], 0] = float("inf")
    c["a"][hit[2], 3] = float("-inf")
    c["a"][hit[3], :] = float("nan")
    y = run(c, "silu")
    assert torch.isnan(y[hit[0]]).all() and torch.isnan(y[hit[3]]).all()
    keep = torch.ones(y.shape[0], dtype=torch.bool, device=DEV)
    keep[hit] = False
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))


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


# ------------------------------------------------------------------ far rows

# Rows of a, or of y and residual, that start beyond 2^32 bytes. All values are
# small integers, so every sum is exact in fp32 and y is its one rounding to bf16.
# shape: (experts, capacity, K, N, gated)
FAR = {
    "skinny, a": (1024, 32768, 65592, 16, False),
    "skinny streamed, a, gated": (1024, 32768, 65600, 16, True),
    "skinny, y": (1024, 32768, 8, 65592, False),
    "skinny, y, gated": (1024, 32768, 8, 131184, True),
    "small, a": (1, 2_090_000, 1032, 128, False),
    "small, y": (1, 16_800_000, 8, 128, False),
    "small, y, gated": (1, 11_300_000, 8, 384, True),
    "medium, a": (1024, 102_400, 21_000, 256, False),
    "large, a and y": (2, 600_000, 4096, 4096, False),
    "large, y, gated": (2, 600_000, 64, 8192, True),
}


def far_call(E, R, K, N, gated, rows, offsets):
    """(y, integers wanted for the last `rows` rows): the last expert has them."""
    from combine_moe_route_amd import moe_grouped_gemm_bf16
    gen = torch.Generator(DEV).manual_seed(R + K)
    ints = lambda *s: torch.randint(-1, 2, s, device=DEV, generator=gen).to(torch.bfloat16)  # noqa: E731
    n_out = N // 2 if gated else N
    a = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
    res = torch.zeros((R, n_out), dtype=torch.bfloat16, device=DEV)
    y = torch.full((R, n_out), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    a[R - rows:], w[E - 1], res[R - rows:] = ints(rows, K), ints(N, K), ints(rows, n_out)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    moe_grouped_gemm_bf16(a, off, w, gated=gated, residual=res, y=y)
    torch.cuda.synchronize()
    z = a[R - rows:].double() @ w[E - 1].double().T
    if gated:
        z = z[:, :n_out] * z[:, n_out:]
    want = z + res[R - rows:].double()
    assert float(want.abs().max()) < 2.0 ** 24           # exact in fp32
    return y, want


@pytest.mark.parametrize("name", list(FAR))
def test_far_rows(name):
    E, R, K, N, gated = FAR[name]
    n_out = N // 2 if gated else N
    assert R * max(K, n_out) * 2 - 20 * max(K, n_out) * 2 > 2 ** 32
    log(f"far rows {name}")
    rows = 20
    y, want = far_call(E, R, K, N, gated, rows, [R - rows] * E + [R])
    assert torch.equal(y[R - rows:].double(), want.to(torch.bfloat16).double())
    assert (y[:R - rows].view(torch.int16) == SENTINEL).all()


def test_far_shapes_reached():
    """The far cases run on the shapes they are named by (launch log, child
    process; no expert has rows there, so nothing is computed)."""
    code = ("import sys; sys.path.insert(0, 'tests')\n"
            "import torch\n"
            "from test_gpu_gemm_bf16_shapes import DEV, FAR\n"
            "from combine_moe_route_amd import moe_grouped_gemm_bf16\n"
            "for E, R, K, N, g in FAR.values():\n"
            "    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)\n"
            "    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)\n"
            "    moe_grouped_gemm_bf16(e(R, K), off, e(E, N, K), gated=g)\n"
            "    torch.cuda.synchronize()\n"
            "    torch.cuda.empty_cache()\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=110, env=dict(os.environ, MOE_ROUTE_LOG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = re.findall(r"(\w*)grouped_gemm_bf16 grid=\d+ block=(\d+) lds=\d+ param=(\d+)", r.stderr)
    assert len(got) == len(FAR)
    for name, (prefix, block, rows) in zip(FAR, got):
        assert (int(rows), int(block)) == LOGGED[name.split(",")[0].split()[0]], name
        assert (prefix == "streamed_") == ("streamed" in name), name
