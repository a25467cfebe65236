"""Operands that lie on top of a call's outputs: every call here is refused on
the host before any HIP call. No test launches a kernel."""
from test_abi_layer import A, B, EINVAL, gact, gemm


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
