"""A NaN in v = act(g) u of moe_gated_act_quant_int8: the row gets the scale NaN and
zero codes whatever the gate, also where act(g) is 0 (0 times NaN is NaN), and no
other row changes by a bit."""
import pytest
import torch

from parity_util import log
from test_gpu_gated_act_int8 import DEV, run

pytestmark = pytest.mark.gpu

# the gate next to a NaN in the up half: act(g) is 0, or tiny, or ordinary
GATES = [-1.0, -0.0, 0.0, 2.0, -30.0, -87.5, -88.0, -89.0, -100.0, -3e4, -1e38]
SIZES = [16, 64, 256, 272, 1040, 2048, 4096, 8208, 32768]   # every width of a row's lanes


@pytest.mark.parametrize("I", SIZES)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_nan_behind_any_gate(act, I):
    log(f"gated_act_int8 nan {act} I={I}")
    gen = torch.Generator(DEV).manual_seed(I)
    R = 2 * len(GATES) + 3
    h = torch.randn((R, 2 * I), device=DEV, generator=gen).to(torch.bfloat16)
    for i, g in enumerate(GATES):
        h[2 * i + 1, (5 * i) % I] = g
    clean, cs = run(h, [0, R], act)
    assert torch.isfinite(cs).all()
    bad = h.clone()
    for i in range(len(GATES)):
        bad[2 * i + 1, I + (5 * i) % I] = float("nan")
    out, sc = run(bad, [0, R], act)
    hit = torch.zeros(R, dtype=torch.bool, device=DEV)
    hit[1:2 * len(GATES):2] = True
    assert torch.isnan(sc[hit]).all(), [g for g, s in zip(GATES, sc[hit].tolist()) if s == s]
    assert (out[hit] == 0).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(sc[~hit], cs[~hit])


@pytest.mark.parametrize("I", SIZES)
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_nan_in_the_gate_and_rows_of_nan(act, I):
    """A NaN gate next to any up value, zero among them; a row of nothing else."""
    h = torch.randn((6, 2 * I), device=DEV).to(torch.bfloat16)
    h[1, I - 1], h[1, 2 * I - 1] = float("nan"), 0.0
    h[3, 0], h[3, I] = float("nan"), -2.0
    h[4] = float("nan")
    out, sc = run(h, [0, 6], act)
    assert torch.isnan(sc[[1, 3, 4]]).all() and (out[[1, 3, 4]] == 0).all()
    assert torch.isfinite(sc[[0, 2, 5]]).all()


@pytest.mark.parametrize("I", [64, 2048, 4096])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_far_gate_next_to_a_huge_up(act, I):
    """act(g) is 0 in fp32 at g = -100, so g u past fp32 counts as 0 and the row is that
    of u = 0. Both are within 2^-20 |g u| + 2^-24 |v| of act(g) u elsewhere."""
    gen = torch.Generator(DEV).manual_seed(I)
    h = torch.randn((8, 2 * I), device=DEV, generator=gen).to(torch.bfloat16)
    h[2, 7], h[2, I + 7] = -100.0, 0.0
    want, ws = run(h, [0, 8], act)
    h[2, I + 7] = 3e38
    out, sc = run(h, [0, 8], act)
    far = (h[2, :I].float() * h[2, I:].float()).abs()
    far[7] = 0.0
    dv = 2 * (2.0 ** -20 + 2.0 ** -24) * float(far.max())
    V = 127 * float(ws[2])
    assert abs(float(sc[2] - ws[2])) <= (dv + 2.0 ** -23 * V) / 127
    assert 127 * 2 * dv < 0.5 * V                     # less than one code
    assert int((out[2].int() - want[2].int()).abs().max()) <= 1 and out[2, 7] == 0
    keep = [0, 1, 3, 4, 5, 6, 7]
    assert torch.equal(out[keep], want[keep]) and torch.equal(sc[keep], ws[keep])
