"""moe_grouped_gemm_bf16 against a plain implementation in 64 bits.

Tolerance, from the arithmetic. bf16 products are exact in fp32; the fp32 sum
over K terms, in any order, is off by at most (K - 1) 2^-24 of the sum of
their magnitudes M, and a matrix core that truncates while it aligns the
terms of one step by at most twice that: dz = K 2^-23 M, with the bias as one
more term. The activations are Lipschitz (relu 1, silu 1.1, gelu 1.13) and
their own fp32 evaluation is within 2^-20 of |z| (exp, erfc, a reciprocal and
two products of a few units of 2^-24 each, amplified by at most |z| 2^-24 in
the exponent, where z > 16 has already saturated: 16 units). Products and the
residual round once each (2^-24), the result once to bf16 (2^-8 relative,
half a step):
  plain  da = L dz + 2^-20 |z|,                 y = a + r
  gated  dv = da (|u| + du) + |a| du + 2^-24 |a u|
  |gpu - y| <= 2^-8 (|y| + d) + d + 2^-133 with d = da or dv, + 2^-24 |y|.
"""
import math

import numpy as np
import pytest
import torch

from parity_util import log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SENTINEL = 0x7FC1
LIP = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13}


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    return z


def reference(a, off, w, bias, act, gated, residual):
    """(y64, tolerance) of the rows of the segments, on the CPU, by row number."""
    E, N, K = w.shape
    a, w = a.double().cpu(), w.double().cpu()
    out = {}
    for e in range(E):
        r0, r1 = off[e], off[e + 1]
        if r1 <= r0:
            continue
        x = a[r0:r1]
        z, m = x @ w[e].T, x.abs() @ w[e].abs().T
        if bias is not None:
            b = bias[e].double().cpu()
            z, m = z + b, m + b.abs()
        dz = (K + 1) * 2.0 ** -23 * m
        if gated:
            g, u, du = z[:, :N // 2], z[:, N // 2:], dz[:, N // 2:]
            v = act64(act, g)
            da = LIP[act] * dz[:, :N // 2] + (2.0 ** -20 * g.abs() if act in ("silu", "gelu") else 0)
            d = da * (u.abs() + du) + v.abs() * du + 2.0 ** -24 * (v * u).abs()
            y = v * u
        else:
            y = act64(act, z)
            d = LIP[act] * dz + (2.0 ** -20 * z.abs() if act in ("silu", "gelu") else 0)
        if residual is not None:
            y = y + residual[r0:r1].double().cpu()
        d = d + 2.0 ** -24 * y.abs()
        out[(r0, r1)] = (y, 2.0 ** -8 * (y.abs() + d) + d + 2.0 ** -133)
    return out


def case(counts, K, N, R=None, seed=0, bias=False, residual=False, gated=False, align=1, first=0):
    rng = torch.Generator(DEV).manual_seed(seed)
    off = [first]
    for c in counts:
        off.append(off[-1] + (c + align - 1) // align * align)
    R = off[-1] if R is None else R
    E, n_out = len(counts), N // 2 if gated else N
    mk = lambda *s: torch.randn(s, device=DEV, generator=rng).to(torch.bfloat16)  # noqa: E731
    return dict(a=mk(R, K), off=off, w=(torch.randn((E, N, K), device=DEV, generator=rng)
                                        / math.sqrt(K)).to(torch.bfloat16),
                bias=mk(E, N) if bias else None, residual=mk(R, n_out) if residual else None,
                gated=gated)


def run(c, act):
    from combine_moe_route_amd import moe_grouped_gemm_bf16
    R, N = c["a"].shape[0], c["w"].shape[1]
    n_out = N // 2 if c["gated"] else N
    y = torch.full((R, n_out), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    off = torch.tensor(c["off"], dtype=torch.int32, device=DEV)
    got = moe_grouped_gemm_bf16(c["a"], off, c["w"], bias=c["bias"], act=act, gated=c["gated"],
                                residual=c["residual"], y=y)
    assert got is y
    torch.cuda.synchronize()
    return y


def check(c, act, off=None):
    y = run(c, act)
    R = y.shape[0]
    off = c["off"] if off is None else off
    ref = reference(c["a"], off, c["w"], c["bias"], act, c["gated"], c["residual"])
    covered = torch.zeros(R, dtype=torch.bool)
    for (r0, r1), (want, tol) in ref.items():
        covered[r0:r1] = True
        err = (y[r0:r1].double().cpu() - want).abs()
        bad = ~(err <= tol)
        if bad.any():
            i = bad.nonzero()[0].tolist()
            raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off in rows {r0}..{r1}, first "
                                 f"{i}: {float(y[r0 + i[0], i[1]])} for {float(want[i[0], i[1]])}, "
                                 f"tolerance {float(tol[i[0], i[1]])}")
    rest = y.view(torch.int16).cpu()[~covered]
    assert (rest == SENTINEL).all(), "rows of no segment were written"
    return y


@pytest.mark.parametrize("counts,K,N", [
    ([1], 8, 8), ([1], 64, 256), ([3], 72, 264), ([17], 128, 16), ([5, 0, 9, 1], 200, 520),
    ([0, 0, 3], 1016, 64), ([16, 17, 31, 32, 33], 256, 304), ([64, 65, 127, 128], 192, 256),
    ([129, 1, 255], 320, 512), ([300, 700], 136, 768), ([1000], 512, 1032), ([2] * 40, 264, 128),
    ([257, 0, 0, 513], 64, 272), ([4096], 128, 256), ([1] * 600, 64, 32),
])
@pytest.mark.parametrize("gated", [False, True])
def test_segments_and_sizes(counts, K, N, gated):
    if gated:
        N = (N + 15) // 16 * 16
    log(f"gemm_bf16 {counts if len(counts) < 9 else len(counts)} K={K} N={N} gated={gated}")
    check(case(counts, K, N, seed=K + N, gated=gated), "none")
    check(case(counts, K, N, seed=K + N + 1, gated=gated, bias=True, residual=True), "silu")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("counts", [[5, 3], [90, 140], [700, 600]])
def test_epilogues(act, gated, bias, residual, counts):
    log(f"epilogue {act} gated={gated} bias={bias} residual={residual} {counts}")
    check(case(counts, 152, 336, seed=7, bias=bias, residual=residual, gated=gated), act)


def test_capacity_gaps_and_bad_offsets():
    """Rows before the first segment, between padded ones and behind the last
    stay as they were; offsets past the capacity are clamped; a decreasing
    pair is an empty segment."""
    log("capacity")
    check(case([3, 40, 0, 7], 64, 64, R=200, first=5), "relu")
    check(case([30, 1, 130], 96, 72, R=600, align=128, residual=True), "gelu")
    c = case([10, 20], 64, 64, R=25)
    check(c, "none", off=[0, 10, 25])
    c = case([10, 20], 64, 64, R=30)
    c["off"] = [0, 20, 10]
    check(c, "none")
    c["off"] = [-5, 6, 2 ** 31 - 1]
    check(c, "none", off=[0, 6, 30])


def test_nan_in_rows_of_no_segment_and_inf_inside():
    """What lies outside the segments does not reach any output; inf and NaN
    inside reach their own row only."""
    log("non-finite")
    c = case([20, 33], 80, 96, R=128, bias=True, residual=True)
    for t in (c["a"], c["residual"]):
        t[53:] = float("nan")
    check(c, "silu")
    clean = run(c, "none").float()
    c["a"][7, 79] = float("nan")
    c["a"][9, 0] = float("inf")
    y = run(c, "none").float()
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[9]).any()
    keep = [r for r in range(53) if r not in (7, 9)]
    assert torch.equal(y[keep], clean[keep])


def test_residual_in_place_and_repeatable():
    log("in place")
    from combine_moe_route_amd import moe_grouped_gemm_bf16
    for counts in ([3, 9], [200, 311]):
        c = case(counts, 128, 256, residual=True)
        want = run(c, "none")
        assert torch.equal(run(c, "none"), want)
        y = c["residual"].clone()
        off = torch.tensor(c["off"], dtype=torch.int32, device=DEV)
        moe_grouped_gemm_bf16(c["a"], off, c["w"], residual=y, y=y)
        assert torch.equal(y, want)


def test_no_rows():
    from combine_moe_route_amd import moe_grouped_gemm_bf16
    log("no rows")
    w = torch.zeros((2, 16, 16), dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert moe_grouped_gemm_bf16(w.new_zeros((0, 16)), off, w).shape == (0, 16)
    y = w.new_full((5, 16), 3.0)
    moe_grouped_gemm_bf16(w.new_zeros((5, 16)), off, w, y=y)
    torch.cuda.synchronize()
    assert (y == 3.0).all()


def test_weights_past_32_bit_offsets():
    """An expert whose weights start beyond 2^32 bytes."""
    log("large weights")
    E, N, K = 5, 16384, 32768       # 1 GiB an expert
    c = dict(a=torch.randn((20, K), device=DEV).to(torch.bfloat16), off=[0, 0, 0, 0, 0, 20],
             w=torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV).normal_(0, 1 / 181.0),
             bias=None, residual=None, gated=True)
    y = run(c, "silu")
    cols = torch.tensor([0, 1, 127, 128, 4000, 8190, 8191])
    z = c["a"].double() @ c["w"][4][torch.cat([cols, cols + N // 2]).to(DEV)].double().T
    m = c["a"].double().abs() @ c["w"][4][torch.cat([cols, cols + N // 2]).to(DEV)].double().abs().T
    g, u = z[:, :7], z[:, 7:]
    dz = (K + 1) * 2.0 ** -23 * m
    v = act64("silu", g)
    da = 1.1 * dz[:, :7] + 2.0 ** -20 * g.abs()
    d = da * (u.abs() + dz[:, 7:]) + v.abs() * dz[:, 7:] + 2.0 ** -23 * (v * u).abs()
    err = (y[:, cols.to(DEV)].double() - v * u).abs()
    assert (err <= 2.0 ** -8 * ((v * u).abs() + d) + d).all()


def test_python_refusals():
    from combine_moe_route_amd import MoeRouteError, moe_grouped_gemm_bf16
    c = case([4, 4], 64, 64)
    off = torch.tensor(c["off"], dtype=torch.int32, device=DEV)
    a, w = c["a"], c["w"]
    with pytest.raises(ValueError):
        moe_grouped_gemm_bf16(a, off, w, act="tanh")
    with pytest.raises(ValueError):
        moe_grouped_gemm_bf16(a, off, w[:, :, :32].contiguous())
    with pytest.raises(ValueError):
        moe_grouped_gemm_bf16(a, off[:2], w)
    with pytest.raises(ValueError):
        moe_grouped_gemm_bf16(a, off, w, residual=a[:, :32].contiguous())
    with pytest.raises(ValueError):
        moe_grouped_gemm_bf16(a.t(), off, w)
    with pytest.raises(TypeError):
        moe_grouped_gemm_bf16(a.float(), off, w)
    with pytest.raises(TypeError):
        moe_grouped_gemm_bf16(a, off, w, bias=torch.zeros((2, 64), device=DEV))
    with pytest.raises(MoeRouteError):
        moe_grouped_gemm_bf16(a[:, :60].contiguous(), off, w[:, :, :60].contiguous())
    with pytest.raises(MoeRouteError):
        moe_grouped_gemm_bf16(a, off, w[:, :24].contiguous(), gated=True)


def test_rows_past_32_bit_offsets():
    """A segment whose rows of a, residual and y start beyond 2^32 bytes."""
    log("large rows")
    R, K, N = 600_000, 4096, 4096
    a = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV)
    y = torch.full((R, N), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    first, gen = R - 300, torch.Generator(DEV).manual_seed(3)
    a[first:] = torch.randn((300, K), device=DEV, generator=gen).to(torch.bfloat16)
    w = (torch.randn((2, N, K), device=DEV, generator=gen) / 64).to(torch.bfloat16)
    from combine_moe_route_amd import moe_grouped_gemm_bf16
    for segs in ([first, first + 20, R], [first, R, R], [R - 9, R, R]):
        y.view(torch.int16).fill_(SENTINEL)
        moe_grouped_gemm_bf16(a, torch.tensor(segs, dtype=torch.int32, device=DEV), w, y=y)
        torch.cuda.synchronize()
        base = segs[0]
        ref = reference(a[base:], [s - base for s in segs], w[:, :64].contiguous(), None, "none",
                        False, None)
        for (r0, r1), (want, tol) in ref.items():
            assert ((y[base + r0:base + r1, :64].double().cpu() - want).abs() <= tol).all()
        assert (y[base - 1].view(torch.int16) == SENTINEL).all()
        assert (y[0].view(torch.int16) == SENTINEL).all()


def test_tile_shapes_of_the_rule():
    """Each tile shape is reached, by the launch log (MOE_ROUTE_LOG=1), and gives
    the reference's result; read in a child process."""
    import os
    import re
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cases = [  # counts, K, N, gated -> (rows of a tile, threads)
        (([20, 3], 128, 128, False), ("32", "256")),          # streamed weights
        (([20, 3], 136, 128, True), ("32", "256")),           # not whole lines
        (([97, 90, 80], 4168, 744, False), ("32", "256")),    # few tiles, deep
        (([120] * 12, 1016, 1032, False), ("128", "256")),
        (([2048], 2048, 4096, False), ("128", "512")),
        (([1000] * 8, 2048, 4096, True), ("256", "256")),
    ]
    code = ("import sys; sys.path.insert(0, 'tests')\n"
            "from test_gpu_gemm_bf16 import case, check\n"
            f"for c, K, N, g in {[c for c, _ in cases]!r}:\n"
            "    check(case(c, K, N, gated=g), 'silu')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=110, env=dict(os.environ, MOE_ROUTE_LOG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = re.findall(r"grouped_gemm_bf16 grid=\d+ block=(\d+) lds=\d+ param=(\d+)", r.stderr)
    assert [(p, b) for b, p in got] == [want for _, want in cases]
