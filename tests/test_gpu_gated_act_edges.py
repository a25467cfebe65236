"""moe_gated_act_quant_fp8 where fp32 ends: products past its range, gates whose
exponential leaves it, a NaN among finite values, and that calls repeat.

Tolerances as in test_gpu_gated_act.py (scale, half an E4M3 step, division),
with the activation's own error per test.
"""
import math

import numpy as np
import pytest
import torch

from parity_util import log
from test_gpu_gated_act import act64, run

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FMAX = float(np.finfo(np.float32).max)
ACTS = ["none", "relu", "silu", "gelu"]


def compare(h, act, dv):
    """Codes and scales of every row against v = act(g) u, clamped to fp32's
    range, which is off by at most dv(g, u, v) + 2^-24 |v|."""
    R, I = h.shape[0], h.shape[1] // 2
    out, sc = run(h, [0, R], act)
    x = h.double()
    g, u = x[:, :I], x[:, I:]
    v = act64(act, g) * u
    dv = dv(g, u, v) + 2.0 ** -24 * v.abs()
    v = v.clamp(-FMAX, FMAX)
    blk = lambda t: t.reshape(R, I // 128, 128).amax(dim=2)  # noqa: E731
    s = sc.double()
    assert torch.isfinite(s).all()
    assert ((s - blk(v.abs()) / 448).abs() <= (blk(dv) + 2.0 ** -24 * blk(v.abs())) / 448
            + 2.0 ** -150).all()
    srep = s.repeat_interleave(128, dim=1)
    val = out.view(torch.float8_e4m3fn).double() * srep
    assert torch.isfinite(val).all()
    half = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * srep)
    tol = torch.where(srep > 0, half + 2 * dv + 2.0 ** -23 * v.abs(), v.abs())
    bad = ~((val - v).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(val[bad][0]), float(v[bad][0]), float(tol[bad][0]))
    return out, sc


def normal(R, I, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    return torch.randn((R, 2 * I), device=DEV, generator=gen).to(torch.bfloat16)


@pytest.mark.parametrize("act", ACTS)
def test_products_past_fp32(act):
    """Finite h whose g u passes 3.4e38: where act(g) u does not, it is as any
    other value; where it does, it counts as the largest finite value of its
    sign, and the rest of the block keeps finite scale and codes."""
    log(f"gated_act past fp32 {act}")
    I = 256
    h = normal(10, I, 5)
    h[0] *= 1e20                                         # most products pass, of both signs
    h[1, 3], h[1, I + 3] = 2e20, 3e20                    # one that does
    h[2, 3], h[2, I + 3] = -2e20, 3e20                   # a gate that closes (relu, silu, gelu)
    h[3, 130], h[3, I + 130] = 1.2, 3.1e38               # g u past it, silu and gelu of g not
    h[4, 130], h[4, I + 130] = -1.2, 3.1e38
    h[5, :I], h[5, I:] = 3.3e38, -3.3e38
    h[6, :I], h[6, I:] = -3.3e38, 3.3e38
    h[7, :128], h[7, I:I + 128] = -2e20, 3e20            # a whole block closed, one as it was
    h[8, 0], h[8, I] = 3.3e38, 1.0                       # near the range's end
    h[9, 0], h[9, I] = -1.0, 3.3e38
    # the activation is within 2^-20 of |g| where it is not exact
    soft = act in ("silu", "gelu")
    out, sc = compare(h, act, lambda g, u, v: 2.0 ** -20 * (g * u).abs().clamp(max=4 * FMAX)
                      if soft else 0 * v)
    top = np.float32(FMAX) / np.float32(448)
    assert (sc[5] == float(top)).all()
    assert (out[5].view(torch.float8_e4m3fn).float() == -448).all()
    if act != "none":
        assert (sc[6] == 0).all() and (out[6] & 0x7F == 0).all() and sc[7, 0] == 0 and sc[7, 1] > 0
    # a row without such a product has the codes it has alone
    plain = normal(10, I, 5)
    o2, s2 = run(plain, [0, 10], act)
    assert torch.equal(out[1, 128:], o2[1, 128:]) and torch.equal(sc[1, 1], s2[1, 1])
    assert torch.equal(out[7, 128:], o2[7, 128:]) and torch.equal(sc[7, 1], s2[7, 1])


def test_silu_gates_far_below_zero():
    """silu(g) u with g = -60 .. -120 and u up to 2^120: relative 2^-20, but
    exponentials below 2^-126 (g below -87.3) may count as 0."""
    log("gated_act silu far gates")
    I, rows = 128, 61
    h = torch.empty((rows, 2 * I), dtype=torch.bfloat16, device=DEV)
    for r in range(rows):
        h[r, :I] = -60.0 - r
        h[r, I:] = 2.0 ** 119 * (1 + torch.arange(I, device=DEV) / I)
    compare(h, "silu", lambda g, u, v: 2.0 ** -20 * v.abs() + torch.where(
        g < -87.3, 2.0 ** -126 * (g * u).abs(), 0.0))


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_nan_stays_nan(act):
    """A NaN in either half has the code of NaN; the block's other values are
    those of the block with a zero in its place."""
    log(f"gated_act NaN {act}")
    I = 256
    h = normal(4, I, 6)
    zero = h.clone()
    for r, c in ((0, 5), (1, I + 5), (2, 200), (3, I + 255)):
        h[r, c] = float("nan")
        zero[r, c] = 0
    out, sc = run(h, [0, 4], act)
    o0, s0 = run(zero, [0, 4], act)
    hit = torch.isnan(h[:, :I]) | torch.isnan(h[:, I:])
    assert hit.sum() == 4
    assert (out[hit] & 0x7F == 0x7F).all()
    assert torch.equal(out[~hit], o0[~hit]) and torch.equal(sc, s0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("R,I", [(1, 128), (700, 1408), (5000, 2048)])
def test_calls_repeat(act, R, I):
    """The same call gives the same bits (no order of blocks or lanes enters)."""
    log(f"gated_act repeats {act} R={R} I={I}")
    h = normal(R, I, 7)
    out, sc = run(h, [0, R], act)
    for _ in range(3):
        o2, s2 = run(h, [0, R], act)
        assert torch.equal(out, o2) and torch.equal(sc, s2)
