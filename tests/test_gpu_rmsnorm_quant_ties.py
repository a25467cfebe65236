"""Codes of moe_rmsnorm_quant whose quotient lies exactly between two codes: nearest, even
at ties, as exact arithmetic has it. The values are bf16 numbers with few bits, so that the
products with the weight and the quotients are exact, whatever the token's factor is; an
implementation that rounds v and its scale on the way breaks such ties by its errors."""
from fractions import Fraction

import pytest
import torch

from parity_util import log

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def e4m3(q):
    """The E4M3 value nearest to the fraction q, even at ties."""
    a, e = abs(q), -6
    while a >= Fraction(2) ** (e + 1):
        e += 1
    step = Fraction(2) ** (e - 3)
    return float(round(a / step) * step) * (-1 if q < 0 else 1)   # round: ties to even


def run(x, w, residual, quant):
    from combine_moe_route_amd import moe_rmsnorm_quant
    t = lambda a: None if a is None else torch.tensor(a, device=DEV).to(torch.bfloat16)  # noqa: E731
    out, _, _, _ = moe_rmsnorm_quant(t(x), t(w), residual=t(residual), quant=quant)
    return (out.view(torch.float8_e4m3fn) if quant == "fp8" else out).double().tolist()


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -9, 2.0 ** 20, 2.0 ** 63])
@pytest.mark.parametrize("split", [False, True])
def test_int8_ties(scale, split):
    """Halves of whole numbers up to 127, the row's largest |v| 127."""
    log(f"norm int8 ties scale={scale} split={split}")
    v = [127.0] + [k + 0.5 for k in range(127)] + [-k - 0.5 for k in range(127)] + [0.0]
    for w in (1.0, -3.0, 0.75):
        x = [a * scale for a in v]
        res = None
        if split:                                    # h = x + residual, exactly v
            res = [a / 2 for a in x]
            x = res
        got = run([x], [w] * len(v), None if res is None else [res], "int8")[0]
        assert got == [float(round(Fraction(a) * (1 if w > 0 else -1))) for a in v]


@pytest.mark.parametrize("H", [128, 1152, 8192])
@pytest.mark.parametrize("top", [448.0, 224.0, 3.5])
def test_fp8_ties(top, H):
    """Midpoints of neighbouring codes in every binade, subnormal codes among them."""
    log(f"norm fp8 ties top={top} H={H}")
    mids = [Fraction(2 * m + 1) * Fraction(2) ** (e - 4) for e in range(-6, 9) for m in range(8, 16)]
    mids += [Fraction(2 * m + 1, 2 ** 10) for m in range(8)]
    mids = [q for q in mids if q < 448]
    unit = Fraction(top) / 448
    row, want = [], []
    for b in range(H // 128):
        part = [Fraction(448)] + [m * (-1) ** i for i, m in enumerate(mids[b % 2::2][:120])]
        part += [Fraction(0)] * (128 - len(part))
        row += [float(q * unit) for q in part]
        want += [e4m3(q) for q in part]
    got = run([row, row], [0.5] * H, None, "fp8")
    assert got[0] == want and got[1] == want
