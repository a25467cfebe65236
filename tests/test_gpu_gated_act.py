"""moe_gated_act_quant_fp8 against a plain implementation in 64 bits.

Tolerance, from the arithmetic. v = act(g) u in fp32: the activation is
within 2^-20 of |g| (see the bf16 grouped GEMM's tests; relu and none are
exact), the product rounds once. With V the block's largest |v| and dV the
largest error in the block, the scale V / 448 is within (dV + 2^-24 V) / 448
(one correctly rounded division) plus half the subnormal spacing, 2^-150.
A code times the GPU's scale has to be within half an E4M3 step of the GPU's
own v: steps are 2^-3 of the value's binade, so at most 2^-4 |v| in the
normal range (|v| / s >= 2^-6), and half of 2^-9 s below it; plus dv, plus
the division's rounding, 2^-23 |v|. Saturated codes are within the same bound
because |v| <= 448 s (1 + 2^-23).
"""
import math

import numpy as np
import pytest
import torch

from parity_util import log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    return z


def run(h, off, act, R=None):
    from combine_moe_route_amd import moe_gated_act_quant_fp8
    R, I = h.shape[0], h.shape[1] // 2
    out = torch.full((R, I), 0x7F, dtype=torch.uint8, device=DEV)
    sc = torch.full((R, I // 128), -3.0, device=DEV)
    got = moe_gated_act_quant_fp8(h, torch.tensor(off, dtype=torch.int32, device=DEV), act=act,
                                  out=out, out_scales=sc)
    assert got[0] is out and got[1] is sc
    torch.cuda.synchronize()
    return out, sc


def check(h, off, act):
    out, sc = run(h, off, act)
    R, I = out.shape
    used = max(0, min(R, off[-1]))
    assert (out[used:] == 0x7F).all() and (sc[used:] == -3.0).all(), "rows behind the last segment"
    x = h[:used].double()
    g, u = x[:, :I], x[:, I:]
    v = act64(act, g) * u
    dv = 2.0 ** -24 * v.abs()
    if act in ("silu", "gelu"):
        dv = dv + 2.0 ** -20 * g.abs() * u.abs()
    blk = lambda t: t.reshape(used, I // 128, 128)  # noqa: E731
    V, dV = blk(v.abs()).amax(dim=2), blk(dv).amax(dim=2)
    s = sc[:used].double()
    tol_s = (dV + 2.0 ** -24 * V) / 448 + 2.0 ** -150
    assert ((s - V / 448).abs() <= tol_s).all()
    val = out[:used].view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, dim=1)
    assert torch.isfinite(val).all()
    srep = s.repeat_interleave(128, dim=1)
    half = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * srep)
    err = (val - v).abs()
    # blocks whose scale rounds to zero hold zeros
    tol = torch.where(srep > 0, half + 2 * dv + 2.0 ** -23 * v.abs(), v.abs())
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float(err[bad][0]), float(tol[bad][0]))
    return out, sc


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("R,I,off", [
    (1, 128, [0, 1]), (7, 256, [0, 2, 7]), (40, 1408, [0, 3, 3, 33]), (513, 384, [0, 500, 513]),
    (64, 2048, [0, 0]), (9, 128, [0, 4, 100]), (3000, 640, [0, 1, 2999]),
])
def test_sizes(act, R, I, off):
    log(f"gated_act {act} R={R} I={I}")
    gen = torch.Generator(DEV).manual_seed(R + I)
    h = torch.randn((R, 2 * I), device=DEV, generator=gen).to(torch.bfloat16)
    check(h, off, act)


def test_values():
    """Zero rows, one large value in a block, subnormal results, large gates
    of either sign, rows behind the end that hold NaN."""
    log("gated_act values")
    R, I = 24, 256
    gen = torch.Generator(DEV).manual_seed(3)
    h = torch.randn((R, 2 * I), device=DEV, generator=gen).to(torch.bfloat16)
    h[0] = 0
    h[1, :I] = 0
    h[2, 5] = 3e4
    h[3] *= 1e-18
    h[4] *= 1e-19
    h[5] *= 1e-22
    h[6, :I] = -200.0
    h[7, :I] = 200.0
    h[8, :I] = -30.0
    h[9] *= 1e18
    h[20:] = float("nan")
    for act in ("none", "relu", "silu", "gelu"):
        check(h, [0, 20], act)
    out, sc = run(h, [0, 20], "silu")
    assert (out[0] == 0).all() and (sc[0] == 0).all() and (sc[1] == 0).all()


def test_large_rows():
    """Rows whose byte offsets pass 2^32; the last ones are compared."""
    log("gated_act large")
    R, I = 300_000, 4096
    h = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=DEV).normal_()
    out, sc = run(h, [0, R - 1], "silu")
    assert (out[R - 1] == 0x7F).all()
    tail = h[R - 50:R - 1].clone()
    o2, s2 = check(tail, [0, 49], "silu")
    assert torch.equal(out[R - 50:R - 1], o2) and torch.equal(sc[R - 50:R - 1], s2)


def test_python_refusals():
    from combine_moe_route_amd import MoeRouteError, moe_gated_act_quant_fp8
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    h = torch.zeros((4, 512), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        moe_gated_act_quant_fp8(h, off, act="tanh")
    with pytest.raises(TypeError):
        moe_gated_act_quant_fp8(h.float(), off)
    with pytest.raises(ValueError):
        moe_gated_act_quant_fp8(h[:, :511].contiguous(), off)
    with pytest.raises(ValueError):
        moe_gated_act_quant_fp8(h, off, out=torch.zeros((4, 128), dtype=torch.uint8, device=DEV))
    with pytest.raises(MoeRouteError):
        moe_gated_act_quant_fp8(h[:, :400].contiguous(), off)
    with pytest.raises(MoeRouteError):
        moe_gated_act_quant_fp8(h, off[:1])
