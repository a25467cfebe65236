"""Argument checks of moe_route_scored, moe_grouped_gemm_bf16 and
moe_gated_act_quant_fp8: every call here is rejected on the host before any
HIP call, or does nothing. No test launches a kernel."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

binding = pytest.importorskip("combine_moe_route_amd.binding")
lib = binding.lib

OK, EINVAL, EALIGN, ENULL = 0, -1, -3, -5
A, B = 0x100000, 0x200000      # fake device addresses, never dereferenced


def test_enumerations_match_header():
    text = open(os.path.join(ROOT, "include", "moe_route.h")).read()
    for prefix, table in (("MOE_SCORE_", binding.MOE_SCORES), ("MOE_ACT_", binding.MOE_ACTS)):
        for name, val in table.items():
            assert re.search(rf"\b{prefix}{name.upper()}\s*=\s*{val}\b", text), name
    assert re.search(r"\bMOE_LOGITS_F32\s*=\s*0\b", text)
    assert re.search(r"\bMOE_LOGITS_BF16\s*=\s*1\b", text)


def scored(**kw):
    a = dict(l=A, dt=0, ld=64, T=16, E=64, k=4, score=1, bias=B + 8192, G=8, KG=4, top=2, renorm=1,
             scale=1.0, ns=0, sw=1.0, idx=B, w=B + 4096)
    a.update(kw)
    return lib.moe_route_scored(a["l"], a["dt"], a["ld"], a["T"], a["E"], a["k"], a["score"],
                                a["bias"], a["G"], a["KG"], a["top"], a["renorm"], a["scale"],
                                a["ns"], a["sw"], a["idx"], a["w"], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=2 ** 31), dict(k=0), dict(k=65), dict(E=0), dict(E=1025, ld=1025, G=1, KG=1),
    dict(ns=-1), dict(ns=961), dict(ns=2 ** 31 - 1), dict(dt=2), dict(dt=-1), dict(score=2),
    dict(score=-1), dict(G=0), dict(G=7), dict(G=128), dict(KG=0), dict(KG=9), dict(k=33),
    dict(top=0), dict(top=3), dict(ld=63), dict(ld=-64), dict(ld=2 ** 40),
    dict(T=2 ** 30, ld=2 ** 20), dict(T=2 ** 29, ns=1), dict(T=2 ** 28, k=1, E=1024, ld=1024),
])
def test_scored_limits(kw):
    assert scored(**kw) == EINVAL


def test_scored_pointers():
    assert scored(l=None) == ENULL
    assert scored(idx=None) == ENULL
    assert scored(w=None) == ENULL
    assert scored(l=A + 2) == EALIGN                 # fp32 logits
    assert scored(l=A + 1, dt=1) == EALIGN           # bf16 logits
    assert scored(bias=B + 2) == EALIGN
    assert scored(idx=B + 1) == EALIGN
    assert scored(w=B + 2) == EALIGN
    assert scored(T=0, l=None, idx=None, w=None, bias=None) == OK
    assert scored(T=0, k=0) == EINVAL                # limits come first


def gemm(**kw):
    a = dict(a=A, off=B, w=A + 2 ** 24, bias=None, res=None, E=8, N=512, K=256, R=1000, act=0,
             gated=0, y=A + 2 ** 26)
    a.update(kw)
    return lib.moe_grouped_gemm_bf16(a["a"], a["off"], a["w"], a["bias"], a["res"], a["E"], a["N"],
                                     a["K"], a["R"], a["act"], a["gated"], a["y"], None)


@pytest.mark.parametrize("kw", [
    dict(E=0), dict(E=1025), dict(N=0), dict(N=12), dict(N=2 ** 20 + 8), dict(N=24, gated=1),
    dict(K=0), dict(K=4), dict(K=12), dict(K=2 ** 20 + 8), dict(R=-1), dict(R=2 ** 31),
    dict(act=-1), dict(act=4), dict(R=2 ** 31 - 1, N=2 ** 20),
])
def test_gemm_bf16_limits(kw):
    assert gemm(**kw) == EINVAL


def test_gemm_bf16_pointers():
    for p in ("a", "off", "w", "y"):
        assert gemm(**{p: None}) == ENULL
    assert gemm(a=A + 8) == EALIGN
    assert gemm(w=A + 2 ** 24 + 8) == EALIGN
    assert gemm(y=A + 2 ** 26 + 8) == EALIGN
    assert gemm(bias=B + 8) == EALIGN
    assert gemm(res=B + 2) == EALIGN
    assert gemm(off=B + 2) == EALIGN
    assert gemm(R=0, a=None, off=None, w=None, y=None) == OK


def test_gemm_bf16_overlaps():
    """y on top of an operand is refused (every call here overlaps, so nothing
    is launched); the residual may be y itself only."""
    y = A + 2 ** 26                                  # 1000 x 512 bf16
    end = y + 1000 * 512 * 2
    for p in ("a", "w", "bias", "res"):
        for at in (y + 16, end - 16):
            assert gemm(**{p: at}) == EINVAL, p
    for p in ("a", "w", "bias"):
        assert gemm(**{p: y}) == EINVAL, p
    assert gemm(a=y - 1000 * 256 * 2 + 16) == EINVAL
    assert gemm(w=y - 8 * 512 * 256 * 2 + 16) == EINVAL
    assert gemm(res=y - 1000 * 512 * 2 + 16) == EINVAL
    assert gemm(gated=1, res=y + 1000 * 256 * 2 - 16) == EINVAL


def gact(**kw):
    a = dict(h=A, off=B, E=8, R=1000, I=256, act=2, out=A + 2 ** 24, sc=B + 2 ** 20)
    a.update(kw)
    return lib.moe_gated_act_quant_fp8(a["h"], a["off"], a["E"], a["R"], a["I"], a["act"], a["out"],
                                       a["sc"], None)


def test_gated_act_refusals():
    for kw in (dict(E=0), dict(E=1025), dict(R=-1), dict(R=2 ** 31), dict(I=0), dict(I=64),
               dict(I=200), dict(I=2 ** 20 + 128), dict(act=4), dict(act=-1)):
        assert gact(**kw) == EINVAL, kw
    for p in ("h", "off", "out", "sc"):
        assert gact(**{p: None}) == ENULL
    assert gact(h=A + 8) == EALIGN
    assert gact(out=A + 2 ** 24 + 8) == EALIGN
    assert gact(sc=B + 2) == EALIGN
    assert gact(off=B + 1) == EALIGN
    out = A + 2 ** 24                                # 1000 x 256 codes
    assert gact(h=out) == EINVAL
    assert gact(h=out - 1000 * 512 * 2 + 16) == EINVAL
    assert gact(h=out + 1000 * 256 - 64) == EINVAL
    assert gact(sc=out + 64) == EINVAL
    assert gact(sc=A + 64) == EINVAL
    assert gact(R=0, h=None, off=None, out=None, sc=None) == OK
