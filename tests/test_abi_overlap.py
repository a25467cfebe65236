"""Operands that lie on top of a call's outputs: every call here is refused on
the host before any HIP call. No test launches a kernel."""
from test_abi_layer import A, B, EINVAL, gact, gemm, scored


def test_gemm_bf16_offsets():
    y = A + 2 ** 26                                  # 1000 x 512 bf16
    end = y + 1000 * 512 * 2
    for at in (y, y + 16, end - 4, y - 9 * 4 + 4):   # 9 offsets
        assert gemm(off=at) == EINVAL


def test_gated_act_offsets():
    out, sc = A + 2 ** 24, B + 2 ** 20               # 1000 x 256 codes, 1000 x 2 scales
    for at in (out, out + 4, out + 1000 * 256 - 4, out - 9 * 4 + 4,
               sc, sc + 8, sc + 1000 * 2 * 4 - 4, sc - 9 * 4 + 4):
        assert gact(off=at) == EINVAL


def test_scored_outputs():
    """16 tokens of 64 fp32 logits at A, bias [64], outputs 16 x 4."""
    logits, bias, n = A + 16 * 64 * 4, B + 8192, 16 * 4 * 4
    for out in ("idx", "w"):
        for at in (A, A + 4, logits - 4, A - n + 4, bias, bias + 64 * 4 - 4, bias - n + 4):
            assert scored(**{out: at}) == EINVAL, (out, hex(at))
    for d in (0, 4, n - 4, 4 - n):
        assert scored(w=B + d) == EINVAL
    # rows far apart: an output on the last row, or across the next row's start
    for out in ("idx", "w"):
        for at in (A + 15 * 4000 + 4, A + 15 * 4000 + 252, A + 2 * 4000 - n + 4, A + 14 * 4000):
            assert scored(ld=1000, **{out: at}) == EINVAL, (out, hex(at))
    # shared slots count, bf16 logits are half as long
    assert scored(dt=1, ns=60, idx=A + 16 * 64 * 2 - 4) == EINVAL
    assert scored(ns=60, idx=A - 16 * 64 * 4 + 4) == EINVAL
    assert scored(ns=60, w=B + 16 * 64 * 4 - 4) == EINVAL
