"""moe_grouped_gemm_int8 against a plain implementation in 64 bits.

Tolerance, from the arithmetic; u = 2^-24. The sum t of the products is a whole
number below 2^31, exact on both sides. z = fp32(t) a_s w_s + b rounds three times
and once more at the bias: dz = 4 u (|t a_s w_s| + |b|) + 2^-149. The rest is the
bf16 product's epilogue: activations are Lipschitz (relu 1, silu 1.1, gelu 1.13)
and within 2^-20 |z| themselves, products and the residual round once each, the
result once to bf16:
  plain  d = L dz + 2^-20 |z|
  gated  d = da (|z2| + dz2) + |a| dz2 + u |a z2|
  |gpu - y| <= 2^-8 (|y| + d) + d + 2^-133, with u |y| added to d.
"""
import math

import pytest
import torch

from parity_util import log
from test_gpu_gemm_bf16 import LIP, SENTINEL, act64

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


def reference(c, act, off=None):
    """(y64, tolerance) of the rows of the segments, by row range."""
    a, w = c["a"].double().cpu(), c["w"].double().cpu()
    a_s, w_s = c["a_scales"].double().cpu(), c["w_scales"].double().cpu()
    off = c["off"] if off is None else off
    N, gated, out = w.shape[1], c["gated"], {}
    for e in range(w.shape[0]):
        r0, r1 = off[e], off[e + 1]
        if r1 <= r0:
            continue
        z = (a[r0:r1] @ w[e].T) * torch.outer(a_s[r0:r1], w_s[e])
        m = z.abs()
        if c["bias"] is not None:
            b = c["bias"][e].double().cpu()
            z, m = z + b, m + b.abs()
        dz = 4 * U * m + 2.0 ** -149
        rough = 2.0 ** -20 if act in ("silu", "gelu") else 0.0
        if gated:
            g, z2, d2 = z[:, :N // 2], z[:, N // 2:], dz[:, N // 2:]
            v = act64(act, g)
            da = LIP[act] * dz[:, :N // 2] + rough * g.abs()
            y, d = v * z2, da * (z2.abs() + d2) + v.abs() * d2 + U * (v * z2).abs()
        else:
            y, d = act64(act, z), LIP[act] * dz + rough * z.abs()
        if c["residual"] is not None:
            y = y + c["residual"][r0:r1].double().cpu()
        d = d + U * y.abs()
        out[(r0, r1)] = (y, 2.0 ** -8 * (y.abs() + d) + d + 2.0 ** -133)
    return out


def case(counts, K, N, R=None, seed=0, bias=False, residual=False, gated=False, align=1, first=0):
    gen = torch.Generator(DEV).manual_seed(seed)
    off = [first]
    for c in counts:
        off.append(off[-1] + (c + align - 1) // align * align)
    R = off[-1] if R is None else R
    E, n_out = len(counts), N // 2 if gated else N
    codes = lambda *s: torch.randint(-127, 128, s, device=DEV, generator=gen, dtype=torch.int8)  # noqa: E731
    sc = lambda *s: 0.5 + torch.rand(s, device=DEV, generator=gen)  # noqa: E731
    mk = lambda *s: torch.randn(s, device=DEV, generator=gen).to(torch.bfloat16)  # noqa: E731
    return dict(a=codes(R, K), a_scales=sc(R) / 73.0, off=off, w=codes(E, N, K),
                w_scales=sc(E, N) / 73.0 / math.sqrt(K), bias=mk(E, N) if bias else None,
                residual=mk(R, n_out) if residual else None, gated=gated)


def run(c, act="none"):
    from combine_moe_route_amd import moe_grouped_gemm_int8
    R, N = c["a"].shape[0], c["w"].shape[1]
    n_out = N // 2 if c["gated"] else N
    y = torch.full((R, n_out), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    off = torch.tensor(c["off"], dtype=torch.int32, device=DEV)
    got = moe_grouped_gemm_int8(c["a"], c["a_scales"], off, c["w"], c["w_scales"], bias=c["bias"],
                                act=act, gated=c["gated"], residual=c["residual"], y=y)
    assert got is y
    torch.cuda.synchronize()
    return y


def check(c, act, off=None):
    y = run(c, act)
    covered = torch.zeros(y.shape[0], dtype=torch.bool)
    for (r0, r1), (want, tol) in reference(c, act, off).items():
        covered[r0:r1] = True
        bad = ~((y[r0:r1].double().cpu() - want).abs() <= tol)
        if bad.any():
            i = bad.nonzero()[0].tolist()
            raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off in rows {r0}..{r1}, first "
                                 f"{i}: {float(y[r0 + i[0], i[1]])} for {float(want[i[0], i[1]])}, "
                                 f"tolerance {float(tol[i[0], i[1]])}")
    assert (y.view(torch.int16).cpu()[~covered] == SENTINEL).all(), "rows of no segment were written"
    return y


@pytest.mark.parametrize("counts,K,N", [
    ([1], 16, 8), ([1], 128, 256), ([3], 144, 264), ([17], 256, 16), ([5, 0, 9, 1], 400, 520),
    ([0, 0, 3], 2032, 64), ([16, 17, 31, 32, 33], 512, 304), ([64, 65, 127, 128], 384, 256),
    ([129, 1, 255], 640, 512), ([300, 700], 272, 768), ([1000], 1024, 1032), ([2] * 40, 528, 128),
    ([257, 0, 0, 513], 128, 272), ([4096], 256, 256), ([1] * 600, 128, 32), ([40], 112, 24),
    ([1] * 1024, 16, 8), ([0] * 1023 + [70], 32, 16),
])
@pytest.mark.parametrize("gated", [False, True])
def test_segments_and_sizes(counts, K, N, gated):
    if gated:
        N = (N + 15) // 16 * 16
    log(f"gemm_int8 {counts if len(counts) < 9 else len(counts)} K={K} N={N} gated={gated}")
    check(case(counts, K, N, seed=K + N, gated=gated), "none")
    check(case(counts, K, N, seed=K + N + 1, gated=gated, bias=True, residual=True), "silu")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("counts", [[5, 3], [90, 140], [700, 600]])
def test_epilogues(act, gated, bias, residual, counts):
    log(f"int8 epilogue {act} gated={gated} bias={bias} residual={residual} {counts}")
    check(case(counts, 304, 336, seed=7, bias=bias, residual=residual, gated=gated), act)


SHAPES = [   # counts, K, N -> rows of a tile, threads
    ([20, 3], 256, 128), ([20, 3], 272, 128), ([97, 90, 80], 8336, 744), ([120] * 12, 2032, 1032),
    ([2048], 4096, 4096), ([1000] * 8, 4096, 2048),
]


@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_whole_numbers(counts, K, N):
    """With scales of 1 the result is the exact sum, rounded to fp32 and to bf16:
    bit for bit. Extreme codes give the largest sums."""
    log(f"int8 whole numbers {len(counts)} K={K} N={N}")
    c = case(counts, K, N, seed=3)
    c["a_scales"].fill_(1.0)
    c["w_scales"].fill_(1.0)
    c["a"][0] = -128
    c["w"][0, 0] = -128
    c["w"][0, 1] = 127
    y = run(c)
    for e, (r0, r1) in enumerate(zip(c["off"], c["off"][1:])):
        t = c["a"][r0:r1].double() @ c["w"][e].double().T
        assert torch.equal(y[r0:r1], t.float().to(torch.bfloat16))


def test_largest_inner_dimension():
    log("int8 K 131056")
    K = 2 ** 17 - 16
    for rows, N in ((3, 8), (300, 264)):
        c = case([rows], K, N, seed=1)
        c["a_scales"].fill_(1.0)
        c["w_scales"].fill_(1.0)
        c["a"][1] = -128
        c["w"][0, 5] = -128                          # sum 2^31 - 2^18
        y = run(c)
        t = c["a"].double() @ c["w"][0].double().T
        assert float(t[1, 5]) == 2.0 ** 31 - 2.0 ** 18
        assert torch.equal(y, t.float().to(torch.bfloat16))


def test_capacity_gaps_and_bad_offsets():
    """Rows before the first segment, between padded ones and behind the last
    stay as they were; offsets past the capacity are clamped; a decreasing
    pair is an empty segment."""
    log("int8 capacity")
    check(case([3, 40, 0, 7], 64, 64, R=200, first=5), "relu")
    check(case([30, 1, 130], 96, 72, R=600, align=128, residual=True), "gelu")
    c = case([10, 20], 64, 64, R=25)
    check(c, "none", off=[0, 10, 25])
    c = case([10, 20], 64, 64, R=30)
    c["off"] = [0, 20, 10]
    check(c, "none")
    c["off"] = [-5, 6, 2 ** 31 - 1]
    check(c, "none", off=[0, 6, 30])


def test_scales_of_all_sizes():
    """Scales whose product leaves fp32's range while the result does not, zero
    scales, and NaN or inf ones, which reach their own row or column only."""
    log("int8 scales")
    for counts in ([9, 20], [150, 200]):
        c = case(counts, 160, 96, R=sum(counts) + 8, residual=True, bias=True)
        c["a_scales"][2] = 1e-30
        c["w_scales"][0, 4] = 1e-30                  # row 2: product 1e-60
        c["a_scales"][3] = 1e30
        c["w_scales"][0, 5] = 1e-28
        c["a_scales"][4] = 0.0
        c["a_scales"][sum(counts):] = float("nan")   # rows of no segment
        c["w_scales"][0, 6] = 0.0
        check(c, "none")
        clean = run(c).float()
        c["a_scales"][1] = float("nan")
        c["a_scales"][7] = float("inf")
        y = run(c).float()
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[7]).any()
        keep = [r for r in range(sum(counts)) if r not in (1, 7)]
        assert torch.equal(y[keep], clean[keep])


def test_residual_in_place_and_repeatable():
    log("int8 in place")
    from combine_moe_route_amd import moe_grouped_gemm_int8
    for counts in ([3, 9], [200, 311]):
        c = case(counts, 256, 256, residual=True)
        want = run(c)
        assert torch.equal(run(c), want)
        y = c["residual"].clone()
        off = torch.tensor(c["off"], dtype=torch.int32, device=DEV)
        moe_grouped_gemm_int8(c["a"], c["a_scales"], off, c["w"], c["w_scales"], residual=y, y=y)
        assert torch.equal(y, want)


def test_no_rows():
    from combine_moe_route_amd import moe_grouped_gemm_int8
    log("int8 no rows")
    w, ws = torch.zeros((2, 16, 16), dtype=torch.int8, device=DEV), torch.ones((2, 16), device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert moe_grouped_gemm_int8(w.new_zeros((0, 16)), ws.new_zeros(0), off, w, ws).shape == (0, 16)
    y = torch.full((5, 16), 3.0, dtype=torch.bfloat16, device=DEV)
    moe_grouped_gemm_int8(w.new_zeros((5, 16)), ws.new_ones(5), off, w, ws, y=y)
    torch.cuda.synchronize()
    assert (y == 3.0).all()


def test_weights_and_rows_past_32_bit_offsets():
    """An expert whose weights, and a segment whose rows, start beyond 2^32
    bytes."""
    log("int8 large")
    from combine_moe_route_amd import moe_grouped_gemm_int8
    E, N, K = 5, 16384, 65536                        # 1 GiB an expert
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV)
    w.view(torch.int32).random_()
    c = case([0, 0, 0, 0, 20], K, 16)
    ws = torch.rand((E, N), device=DEV) / 73 / 256
    y = moe_grouped_gemm_int8(c["a"], c["a_scales"], torch.tensor(c["off"], dtype=torch.int32, device=DEV),
                              w, ws)
    cols = torch.tensor([0, 1, 127, 128, 4000, 16382, 16383], device=DEV)
    c["w"], c["w_scales"] = w[:, cols].contiguous(), ws[:, cols].contiguous()
    (want, tol), = reference(c, "none").values()
    assert ((y[:, cols].double().cpu() - want).abs() <= tol).all()
    del w, y
    R, K, N = 1_100_000, 4096, 4096
    a = torch.zeros((R, K), dtype=torch.int8, device=DEV)
    a_s = torch.ones(R, device=DEV) / 73
    y = torch.full((R, N), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    first = R - 300
    c = case([20, 280], K, N)
    a[first:], a_s[first:] = c["a"], c["a_scales"]
    for segs in ([first, first + 20, R], [first, R, R], [R - 9, R, R]):
        y.view(torch.int16).fill_(SENTINEL)
        moe_grouped_gemm_int8(a, a_s, torch.tensor(segs, dtype=torch.int32, device=DEV), c["w"],
                              c["w_scales"], y=y)
        torch.cuda.synchronize()
        base = segs[0]
        part = dict(c, a=a[base:], a_scales=a_s[base:], w=c["w"][:, :64].contiguous(),
                    w_scales=c["w_scales"][:, :64].contiguous())
        for (r0, r1), (want, tol) in reference(part, "none", [s - base for s in segs]).items():
            assert ((y[base + r0:base + r1, :64].double().cpu() - want).abs() <= tol).all()
        assert (y[base - 1].view(torch.int16) == SENTINEL).all()
        assert (y[0].view(torch.int16) == SENTINEL).all()


def test_python_refusals():
    from combine_moe_route_amd import MoeRouteError, moe_grouped_gemm_int8
    c = case([4, 4], 64, 64)
    off = torch.tensor(c["off"], dtype=torch.int32, device=DEV)
    a, sa, w, sw = c["a"], c["a_scales"], c["w"], c["w_scales"]
    with pytest.raises(ValueError):
        moe_grouped_gemm_int8(a, sa, off, w, sw, act="tanh")
    with pytest.raises(ValueError):
        moe_grouped_gemm_int8(a, sa, off, w[:, :, :32].contiguous(), sw)
    with pytest.raises(ValueError):
        moe_grouped_gemm_int8(a, sa, off[:2], w, sw)
    with pytest.raises(ValueError):
        moe_grouped_gemm_int8(a, sa[:4], off, w, sw)
    with pytest.raises(ValueError):
        moe_grouped_gemm_int8(a, sa, off, w, sw[:, :32].contiguous())
    with pytest.raises(TypeError):
        moe_grouped_gemm_int8(a.view(torch.uint8), sa, off, w, sw)
    with pytest.raises(TypeError):
        moe_grouped_gemm_int8(a, sa.double(), off, w, sw)
    with pytest.raises(ValueError):
        moe_grouped_gemm_int8(a.t(), sa, off, w, sw)
    with pytest.raises(MoeRouteError):
        moe_grouped_gemm_int8(a[:, :40].contiguous(), sa, off, w[:, :, :40].contiguous(), sw)
    with pytest.raises(MoeRouteError):
        moe_grouped_gemm_int8(a, sa, off, w[:, :24].contiguous(), sw[:, :24].contiguous(), gated=True)
