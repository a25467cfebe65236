"""moe_gated_act_quant_int8 against a plain implementation in 64 bits.

Tolerance, from the arithmetic; u = 2^-24. v = act(g) u_ in fp32 is within
dv = u |v| + 2^-20 |g u_| (silu, gelu; relu and none round the product only).
With V the row's largest |v| and dV the largest error of the row, the scale is
within (dV + u V) / 127 + 2^-150. A code is the nearest whole number to the GPU's
127 v / V, which is within 127 (dv + |v| dV / V) / (V - dV) of the exact one, plus
4 u |q| for the factor in two parts and the product; then half a step.
"""
import math

import pytest
import torch

from parity_util import log
from test_gpu_gated_act import act64

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


def run(h, off, act):
    from combine_moe_route_amd import moe_gated_act_quant_int8
    R, I = h.shape[0], h.shape[1] // 2
    out = torch.full((R, I), 0x55, dtype=torch.int8, device=DEV)
    sc = torch.full((R,), -3.0, device=DEV)
    got = moe_gated_act_quant_int8(h, torch.tensor(off, dtype=torch.int32, device=DEV), act=act,
                                   out=out, out_scales=sc)
    assert got[0] is out and got[1] is sc
    torch.cuda.synchronize()
    return out, sc


def check(h, off, act):
    out, sc = run(h, off, act)
    R, I = out.shape
    used = max(0, min(R, off[-1]))
    assert (out[used:] == 0x55).all() and (sc[used:] == -3.0).all(), "rows behind the last segment"
    x = h[:used].double()
    g, w = x[:, :I], x[:, I:]
    v = act64(act, g) * w
    dv = U * v.abs() + 2.0 ** -150
    if act in ("silu", "gelu"):
        dv = dv + 2.0 ** -20 * (g * w).abs()
    V, dV = v.abs().amax(1, keepdim=True), dv.amax(1, keepdim=True)
    s = sc[:used].double()[:, None]
    assert ((s - V / 127).abs() <= (dV + U * V) / 127 + 2.0 ** -150).all()
    live = s > 0
    q = torch.where(live, 127 * v / V.clamp_min(1e-300), 0.0)
    tol = 0.5 + 127 * (dv + v.abs() * dV / V.clamp_min(1e-300)) / (V - dV).clamp_min(2.0 ** -149) \
        + 4 * U * q.abs()
    bad = ~((out[:used].double() - q).abs() <= torch.where(live, tol, 0.0))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
    return out, sc


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("R,I,off", [
    (1, 16, [0, 1]), (50, 64, [0, 2, 7]), (19, 256, [0, 19]), (40, 272, [0, 3, 3, 33]),
    (9, 512, [0, 8]), (513, 528, [0, 500, 513]), (70, 1040, [0, 70]), (64, 2048, [0, 0]),
    (21, 2048, [0, 4, 100]), (6, 2064, [0, 6]), (33, 4096, [0, 31]), (5, 4112, [0, 5]),
    (4, 8192, [0, 4]), (3, 8208, [0, 3]), (3, 18432, [0, 2]), (2, 32768, [0, 2]),
    (3000, 640, [0, 1, 2999]), (1100, 2048, [0, 1099]), (1500, 1040, [0, 700, 1500]),
    (1023, 1536, [0, 1023]), (1024, 1536, [0, 1024]), (1200, 2064, [0, 1200]),
])
def test_sizes(act, R, I, off):
    log(f"gated_act_int8 {act} R={R} I={I}")
    gen = torch.Generator(DEV).manual_seed(R + I)
    check(torch.randn((R, 2 * I), device=DEV, generator=gen).to(torch.bfloat16), off, act)


@pytest.mark.parametrize("I,R", [(64, 24), (512, 24), (2048, 24), (2048, 1100), (4096, 24), (16384, 24)])
def test_values(I, R):
    """Zero rows, one large value in a row, tiny and huge rows, large gates of
    either sign, products past fp32's range, rows behind the end that hold NaN."""
    log(f"gated_act_int8 values I={I} R={R}")
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
    h[10, :I] *= 1e-5
    h[11, I:] *= 1e25
    h[20:] = float("nan")
    for act in ("none", "relu", "silu", "gelu"):
        out, sc = check(h, [0, 20], act)
        assert (out[:2] == 0).all() and (sc[:2] == 0).all()
    # a product past the range counts as the largest finite value
    h[12, 3], h[12, I + 3] = 3e38, -3e38
    for act in ("none", "silu", "gelu"):
        out, sc = run(h, [0, 20], act)
        assert float(sc[12]) == pytest.approx(torch.finfo(torch.float32).max / 127, rel=1e-6)
        assert int(out[12, 3]) == -127 and (out[12, :3] == 0).all()


def test_nan_rows():
    """A NaN gives its row the scale NaN and zero codes, and no other row."""
    log("gated_act_int8 nan")
    for I in (64, 2048, 4096):
        h = torch.randn((8, 2 * I), device=DEV).to(torch.bfloat16)
        clean = run(h, [0, 8], "silu")
        for act in ("none", "silu", "gelu"):
            bad = h.clone()
            bad[2, I - 1] = float("nan")
            bad[5, I] = float("nan")
            out, sc = run(bad, [0, 8], act)
            assert torch.isnan(sc[[2, 5]]).all() and (out[[2, 5]] == 0).all()
            if act == "silu":
                keep = [0, 1, 3, 4, 6, 7]
                assert torch.equal(out[keep], clean[0][keep]) and torch.equal(sc[keep], clean[1][keep])


def test_large_rows():
    """Rows whose byte offsets pass 2^32; the last ones are compared."""
    log("gated_act_int8 large")
    R, I = 300_000, 4096
    h = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=DEV).normal_()
    out, sc = run(h, [0, R - 1], "silu")
    assert (out[R - 1] == 0x55).all()
    tail = h[R - 50:R - 1].clone()
    o2, s2 = check(tail, [0, 49], "silu")
    assert torch.equal(out[R - 50:R - 1], o2) and torch.equal(sc[R - 50:R - 1], s2)


def test_bad_row_counts_and_refusals():
    from combine_moe_route_amd import MoeRouteError, moe_gated_act_quant_int8
    h = torch.randn((4, 512), device=DEV).to(torch.bfloat16)
    out, sc = run(h, [0, -7], "silu")
    assert (out == 0x55).all() and (sc == -3.0).all()
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        moe_gated_act_quant_int8(h, off, act="tanh")
    with pytest.raises(TypeError):
        moe_gated_act_quant_int8(h.float(), off)
    with pytest.raises(ValueError):
        moe_gated_act_quant_int8(h[:, :511].contiguous(), off)
    with pytest.raises(TypeError):
        moe_gated_act_quant_int8(h, off, out=torch.zeros((4, 256), dtype=torch.uint8, device=DEV))
    with pytest.raises(MoeRouteError):
        moe_gated_act_quant_int8(h[:, :400].contiguous(), off)
    with pytest.raises(MoeRouteError):
        moe_gated_act_quant_int8(h, off[:1])
