"""moe_rmsnorm_quant against a plain implementation in 64 bits.

Tolerances, from the arithmetic; u = 2^-24 is half a step of fp32.
  h      one addition: dh = u |h| (none without a residual)
  sum    one more rounding, to bf16: 2^-8 |h|, half a subnormal step 2^-134
  r      the sum of H squares: each is off by 2 u through h, and passes through at
         most 64 + 6 + 16 additions (a lane's, a wave's, the waves'); mean, eps,
         root (one unit) and reciprocal: half of 89 u, and 4 u: below 2^-18 r
  v      h w rounds once (2^-150 if it is subnormal), times r once: with dh
         dv = (2^-18 + 4 u) |v| + 2^-149 r + 2^-149
  s      (dv of the largest + 2 u V) / top, half a subnormal step 2^-150
  codes  q = top v / V has no r in it: h w of the value and of the largest are off
         by 2 u each, the factor (two parts) and the product by 2 u: 6 u |q|, or
         top 2^-149 / max |h w| where h w is subnormal. Then half a step: 1/2 for
         int8, max(2^-4 |q|, 2^-10) for E4M3.
"""
import math

import pytest
import torch

from parity_util import log

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


def make(T, H, residual, seed, loud=True, pad=0):
    gen = torch.Generator(DEV).manual_seed(seed)
    mk = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    amp = 1.0 + 20.0 * (torch.rand(H + pad, device=DEV, generator=gen) < 0.01) if loud else 1.0
    x = (mk(T, H + pad) * amp).to(torch.bfloat16)[:, :H]
    res = mk(T, H).to(torch.bfloat16) if residual else None
    return x, res, (1.0 + 0.3 * mk(H)).to(torch.bfloat16)


def run(x, res, w, quant, eps=1e-6, in_place=False):
    from combine_moe_route_amd import moe_rmsnorm_quant
    T, H = x.shape
    fp8 = quant == "fp8"
    sum_out = None
    if res is not None:
        res = res.clone()
        sum_out = res if in_place else torch.full_like(res, 7.0)
    out = torch.full((T, H), 0x55, dtype=torch.uint8, device=DEV)
    out = out if fp8 else out.view(torch.int8)
    sc = torch.full((T, H // 128) if fp8 else (T,), -3.0, device=DEV)
    y = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV)
    got = moe_rmsnorm_quant(x, w, residual=res, eps=eps, quant=quant, sum_out=sum_out, y=y, out=out,
                            out_scales=sc)
    assert got[0] is out and got[1] is sc and got[2] is y and got[3] is sum_out
    torch.cuda.synchronize()
    return out, sc, y, sum_out


def inside(name, got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first {i}: "
                             f"{float(got[i])} for {float(want[i])}, tolerance {float(tol[i])}")


def check(x, res, w, quant, eps=1e-6, in_place=False):
    out, sc, y, total = run(x, res, w, quant, eps, in_place)
    T, H = x.shape
    h = x.double()
    dh = torch.zeros_like(h)
    if res is not None:
        h = h + res.double()
        dh = U * h.abs()
        inside("sum", total, h, 2.0 ** -8 * (h.abs() + dh) + dh + 2.0 ** -134)
    r = 1.0 / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps)
    hw = h * w.double()
    v = hw * r
    dv = (2.0 ** -18 + 4 * U) * v.abs() + 2.0 ** -149 * r + 2.0 ** -149
    inside("y", y, v, 2.0 ** -8 * (v.abs() + dv) + dv + 2.0 ** -134)
    B, top = (128, 448.0) if quant == "fp8" else (H, 127.0)
    blk = lambda t: t.reshape(T, H // B, B)  # noqa: E731
    V, dV, A = blk(v.abs()).amax(2), blk(dv).amax(2), blk(hw.abs()).amax(2)
    s = sc.double().reshape(T, H // B)
    inside("scale", s, V / top, (dV + 2 * U * V) / top + 2.0 ** -150)
    rep = lambda t: t.repeat_interleave(B, dim=1)  # noqa: E731
    live = rep(s) > 0
    q = torch.where(live, top * v / rep(V).clamp_min(1e-300), 0.0)
    half = torch.maximum(2.0 ** -4 * q.abs(), torch.full_like(q, 2.0 ** -10)) if quant == "fp8" else 0.5
    tol = half + 6 * U * q.abs() + top * 2.0 ** -149 / rep(A).clamp_min(2.0 ** -149)
    codes = out.view(torch.float8_e4m3fn) if quant == "fp8" else out
    inside("code", codes, q, torch.where(live, tol, 0.0))
    return out, sc, y, total


@pytest.mark.parametrize("quant", ["int8", "fp8"])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 256), (5, 512), (4, 640), (7, 1024), (9, 1152),
                                 (2, 4096), (130, 7168), (3, 8192), (2, 8320), (2, 16384),
                                 (3, 32768), (2, 65536)])
def test_sizes(T, H, quant):
    log(f"rmsnorm {quant} T={T} H={H}")
    for residual in (False, True):
        check(*make(T, H, residual, T + H), quant, in_place=residual and T % 2 == 1)


@pytest.mark.parametrize("T,H", [(1, 8), (6, 16), (65, 72), (4, 504), (5, 520), (3, 1032), (33, 4104),
                                 (2, 8200), (1, 65528)])
def test_odd_widths(T, H):
    log(f"rmsnorm int8 T={T} H={H}")
    check(*make(T, H, True, H), "int8")
    check(*make(T, H, False, H + 1, pad=24), "int8")


def test_strided_rows_and_optional_outputs():
    from combine_moe_route_amd import moe_rmsnorm_quant
    log("rmsnorm strides")
    x, res, w = make(37, 1024, True, 5, pad=64)
    assert not x.is_contiguous()
    for quant in ("int8", "fp8"):
        out, sc, y, total = check(x, res, w, quant)
        o2, s2, y2, t2 = moe_rmsnorm_quant(x, w, residual=res, quant=quant)
        assert y2 is None and torch.equal(o2, out) and torch.equal(s2, sc) and torch.equal(t2, total)
        o3, s3, y3, t3 = moe_rmsnorm_quant(x, w, quant=quant, with_y=True)
        assert t3 is None
        ref = check(x, None, w, quant)
        assert torch.equal(o3, ref[0]) and torch.equal(y3, ref[2])


def test_values():
    """Zero rows, one channel far above the others, tiny and huge rows (squares
    past fp32's range), zero weights; then the same with other eps."""
    log("rmsnorm values")
    x, res, w = make(16, 1280, True, 9, loud=False)
    x[0] = 0
    res[0] = 0
    res[1] = -x[1]                                   # cancels to zero
    x[2, 77] = 30000.0
    x[3] *= 1e-18
    res[3] *= 1e-18
    x[4] *= 1e-37
    res[4] *= 1e-37
    x[5] *= 1e18
    x[6] *= 1e30
    x[7] *= 3e37
    res[7] *= 3e37
    x[8, 1279] = 3.3e38
    x[9, 128:256] = 0
    res[9, 128:256] = 0
    w[300:310] = 0
    w[311] = 1000.0
    for quant in ("int8", "fp8"):
        for eps in (1e-6, 1e-30, 1.0):
            out, sc, y, total = check(x, res, w, quant, eps=eps)
            assert (out[:2] == 0).all() and (sc[:2] == 0).all() and (y[:2] == 0).all()
        check(x, None, w, quant)
    # weights so small that h w is subnormal
    check(x, res, (w.float() * 1e-36).to(torch.bfloat16), "int8")
    check(x, res, (w.float() * 1e-36).to(torch.bfloat16), "fp8")


def test_largest_weights_and_x_as_its_own_residual():
    log("rmsnorm large weights")
    x, _, w = make(10, 2048, False, 4, loud=False)
    x[3:] *= 2.0 ** 58
    x[6:] *= 2.0 ** 60
    w = (w.float() * 2.0 ** 58).to(torch.bfloat16)
    w[7] = 2.0 ** 60
    for quant in ("int8", "fp8"):
        check(x, None, w, quant)
        check(x, x, w, quant)


def test_least_alignment():
    """Codes at a multiple of 8 bytes, scales at one of 4, the rest at 16."""
    from combine_moe_route_amd import moe_rmsnorm_quant
    log("rmsnorm alignment")
    x, res, w = make(21, 1032, True, 8)
    ref = run(x, res, w, "int8")
    out = torch.zeros(21 * 1032 + 8, dtype=torch.int8, device=DEV)[8:].view(21, 1032)
    sc = torch.zeros(22, device=DEV)[1:]
    sums = torch.zeros(21 * 1032 + 8, dtype=torch.bfloat16, device=DEV)[8:].view(21, 1032)
    assert out.data_ptr() % 16 == 8 and sc.data_ptr() % 8 == 4
    moe_rmsnorm_quant(x, w, residual=res, sum_out=sums, out=out, out_scales=sc)
    assert torch.equal(out, ref[0]) and torch.equal(sc, ref[1]) and torch.equal(sums, ref[3])


def test_many_short_rows():
    log("rmsnorm many rows")
    check(*make(300_001, 8, True, 4), "int8")
    check(*make(70_003, 128, True, 5), "fp8", in_place=True)


def test_non_finite_tokens():
    """A token with an infinity or NaN gets NaN scales and zero codes; the others
    are as without it."""
    log("rmsnorm non-finite")
    for H in (256, 4096):
        x, res, w = make(12, H, True, 2)
        for quant in ("int8", "fp8"):
            clean = run(x, res, w, quant)
            bx, br = x.clone(), res.clone()
            bx[1, 3] = float("nan")
            br[4, H - 1] = float("inf")
            bx[6] = float("-inf")
            bx[7, 5], br[7, 5] = 3.3e38, 3.3e38      # the addition overflows
            bx[9, 0], br[9, 0] = float("inf"), float("-inf")
            out, sc, y, total = run(bx, br, w, quant)
            bad = torch.zeros(12, dtype=torch.bool, device=DEV)
            bad[[1, 4, 6, 7, 9]] = True
            assert torch.isnan(sc[bad]).all() and torch.isnan(y[bad]).all() and (out[bad] == 0).all()
            for a, b in zip((out, sc, y, total), clean):
                assert torch.equal(a[~bad], b[~bad])
            assert torch.isinf(total[7, 5]) and torch.isnan(total[9, 0]) and torch.isnan(total[1, 3])


def test_no_tokens_and_guards():
    from combine_moe_route_amd import moe_rmsnorm_quant
    log("rmsnorm guards")
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    out, sc, y, total = moe_rmsnorm_quant(w.new_zeros((0, 256)), w, with_y=True)
    assert out.shape == (0, 256) and sc.shape == (0,) and y.shape == (0, 256) and total is None
    # nothing but the tokens' rows is written
    for T, H in ((1, 264), (5, 2048), (6, 72)):
        x, res, w = make(T, H, True, 1)
        big = lambda dt, n: torch.full((n + 128,), 77, dtype=dt, device=DEV)  # noqa: E731
        bo, bs, by, bt = big(torch.int8, T * H), big(torch.float32, T), big(torch.bfloat16, T * H), \
            big(torch.bfloat16, T * H)
        cut = lambda t, n: t[64:64 + n]  # noqa: E731
        moe_rmsnorm_quant(x, w, residual=res, sum_out=cut(bt, T * H).view(T, H),
                          y=cut(by, T * H).view(T, H), out=cut(bo, T * H).view(T, H),
                          out_scales=cut(bs, T))
        torch.cuda.synchronize()
        for b in (bo, bs, by, bt):
            assert (b[:64] == 77).all() and (b[-64:] == 77).all()


def test_rows_past_32_bit_offsets():
    log("rmsnorm large")
    from combine_moe_route_amd import moe_rmsnorm_quant
    T, H = 600_000, 8192
    x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV).normal_()
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    out, sc, y, _ = moe_rmsnorm_quant(x, w, with_y=True)
    tail = x[-9:].clone()
    o2, s2, y2, _ = check(tail, None, w, "int8")
    assert torch.equal(out[-9:], o2) and torch.equal(sc[-9:], s2) and torch.equal(y[-9:], y2)


def test_python_refusals():
    from combine_moe_route_amd import MoeRouteError, moe_rmsnorm_quant
    x, res, w = make(4, 256, True, 1)
    with pytest.raises(ValueError):
        moe_rmsnorm_quant(x, w, quant="int4")
    with pytest.raises(TypeError):
        moe_rmsnorm_quant(x.float(), w)
    with pytest.raises(ValueError):
        moe_rmsnorm_quant(x[0], w)
    with pytest.raises(ValueError):
        moe_rmsnorm_quant(x, w[:128].contiguous())
    with pytest.raises(TypeError):
        moe_rmsnorm_quant(x, w.float())
    with pytest.raises(ValueError):
        moe_rmsnorm_quant(x, w, residual=res[:2])
    with pytest.raises(ValueError):
        moe_rmsnorm_quant(x.t().contiguous().t(), w)
    with pytest.raises(TypeError):
        moe_rmsnorm_quant(x, w, out=torch.empty((4, 256), dtype=torch.uint8, device=DEV))
    with pytest.raises(MoeRouteError):
        moe_rmsnorm_quant(x, w, eps=0.0)
    with pytest.raises(MoeRouteError):
        moe_rmsnorm_quant(x, w, sum_out=torch.empty_like(res))
    with pytest.raises(MoeRouteError):
        moe_rmsnorm_quant(x, w, y=x)
    with pytest.raises(MoeRouteError):
        moe_rmsnorm_quant(x[:, :136], w[:136].contiguous(), quant="fp8",
                          out_scales=torch.empty((4, 1), device=DEV))
