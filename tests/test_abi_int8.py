"""Argument checks of moe_rmsnorm_quant, moe_dispatch_quantized,
moe_grouped_gemm_int8 and moe_gated_act_quant_int8: every call here is rejected
on the host before any HIP call, or does nothing. No test launches a kernel."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

binding = pytest.importorskip("combine_moe_route_amd.binding")
lib = binding.lib

OK, EINVAL, ENOSPC, EALIGN, ENULL = 0, -1, -2, -3, -5
MB = 1 << 20                   # fake device addresses, never dereferenced


def test_enumeration_matches_header():
    text = open(os.path.join(ROOT, "include", "moe_route.h")).read()
    assert re.search(r"\bMOE_QUANT_INT8\s*=\s*0\b", text) and binding.MOE_QUANTS["int8"] == 0
    assert re.search(r"\bMOE_QUANT_FP8_E4M3\s*=\s*1\b", text) and binding.MOE_QUANTS["fp8"] == 1


# ------------------------------------------------------------------ norm

def norm(**kw):
    a = dict(x=1 * MB, ld=512, res=2 * MB, w=3 * MB, T=100, H=512, eps=1e-6, q=0, sum=4 * MB,
             y=5 * MB, out=6 * MB, sc=7 * MB)
    a.update(kw)
    return lib.moe_rmsnorm_quant(a["x"], a["ld"], a["res"], a["w"], a["T"], a["H"], a["eps"], a["q"],
                                 a["sum"], a["y"], a["out"], a["sc"], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=2 ** 31), dict(T=2 ** 24, H=8192, ld=8192), dict(H=0), dict(H=4),
    dict(H=516), dict(H=65544, ld=65544), dict(H=136, q=1), dict(H=64, q=1), dict(q=2), dict(q=-1),
    dict(ld=504), dict(ld=516), dict(ld=-512), dict(ld=2 ** 31 + 8), dict(T=2 ** 20, ld=2 ** 21),
    dict(eps=0.0), dict(eps=1e-31), dict(eps=-1.0), dict(eps=2.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(res=None),
])
def test_norm_limits(kw):
    assert norm(**kw) == EINVAL


def test_norm_pointers():
    for p in ("x", "w", "out", "sc"):
        assert norm(**{p: None}) == ENULL, p
    for p in ("x", "res", "w", "sum", "y"):
        assert norm(**{p: 8 * MB + 8}) == EALIGN, p
    assert norm(out=6 * MB + 4) == EALIGN
    assert norm(out=6 * MB + 8, q=1) == EALIGN
    assert norm(sc=7 * MB + 2) == EALIGN
    assert norm(T=0, x=None, w=None, out=None, sc=None) == OK
    assert norm(T=0, H=4) == EINVAL                  # limits come first


def test_norm_overlaps():
    rows = 100 * 512 * 2
    ends = dict(sum=rows, y=rows, out=100 * 512, sc=400)
    for o, n in ends.items():
        at = dict(sum=4, y=5, out=6, sc=7)[o] * MB
        for i, m in (("x", rows), ("res", rows), ("w", 1024)):
            for addr in (at + 16, at + n - 16, at - m + 16):
                assert norm(**{i: addr}) == EINVAL, (o, i, addr)
            if (o, i) != ("sum", "res"):
                assert norm(**{i: at}) == EINVAL, (o, i)
        for p, m in ends.items():
            if p != o:
                assert norm(**{p: at}) == EINVAL and norm(**{p: at + n - 16}) == EINVAL, (o, p)
    # in place: the weight, x and the other outputs still may not lie on it
    for p in ("x", "w", "y", "out", "sc"):
        assert norm(sum=2 * MB, **{p: 2 * MB + 512}) == EINVAL, p
    # an output on a later row of strided x
    assert norm(ld=4096, out=1 * MB + 50 * 8192) == EINVAL
    assert norm(ld=4096, sc=1 * MB + 50 * 8192 + 1008) == EINVAL


# ------------------------------------------------------------------ dispatch

def disp(**kw):
    a = dict(x=1 * MB, xs=2 * MB, idx=3 * MB, T=64, H=256, S=2, E=16, k=4, G=1, A=8, out=4 * MB,
             sc=5 * MB, cnt=6 * MB, off=7 * MB, goff=8 * MB, src=9 * MB, dst=10 * MB, ws=11 * MB,
             n=1 << 20)
    a.update(kw)
    return lib.moe_dispatch_quantized(a["x"], a["xs"], a["idx"], a["T"], a["H"], a["S"], a["E"],
                                      a["k"], a["G"], a["A"], a["out"], a["sc"], a["cnt"], a["off"],
                                      a["goff"], a["src"], a["dst"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw", [
    dict(H=0), dict(H=8), dict(H=24), dict(H=65552), dict(H=-16), dict(S=0), dict(S=-1),
    dict(S=257), dict(T=-1), dict(T=2 ** 31), dict(k=0), dict(k=17), dict(E=1025), dict(E=0),
    dict(G=0), dict(G=3), dict(A=0), dict(A=1025), dict(T=2 ** 29, k=4), dict(T=2 ** 26, H=2048, k=1),
])
def test_dispatch_limits(kw):
    assert disp(**kw) == EINVAL


def test_dispatch_pointers():
    for p in ("x", "xs", "idx", "out", "sc", "cnt", "off", "src", "dst", "ws"):
        assert disp(**{p: None}) == ENULL, p
    for p in ("x", "out"):
        assert disp(**{p: 12 * MB + 8}) == EALIGN, p
    for p in ("xs", "idx", "sc", "cnt", "off", "goff", "src", "dst", "ws"):
        assert disp(**{p: 12 * MB + 2}) == EALIGN, p
    assert disp(n=16) == ENOSPC


def test_dispatch_overlaps():
    rows = 64 * 4 + 16 * 7
    sizes = dict(x=64 * 256, xs=64 * 8, idx=64 * 16, out=rows * 256, sc=rows * 8, cnt=64, off=68,
                 goff=8, src=rows * 4, dst=64 * 16)
    at = dict(x=1, xs=2, idx=3, out=4, sc=5, cnt=6, off=7, goff=8, src=9, dst=10, ws=11)
    inputs = ("x", "xs", "idx")
    for o in at:
        if o in inputs:
            continue
        for p in sizes:
            if p != o:
                assert disp(**{p: at[o] * MB}) == EINVAL, (o, p)
    assert disp(x=4 * MB + rows * 256 - 16) == EINVAL
    assert disp(x=4 * MB - 64 * 256 + 16) == EINVAL


# ------------------------------------------------------------------ product

def gemm(**kw):
    a = dict(a=1 * MB, sa=2 * MB, off=3 * MB, w=32 * MB, sw=4 * MB, bias=None, res=None, E=8, N=512,
             K=256, R=1000, act=0, gated=0, y=64 * MB)
    a.update(kw)
    return lib.moe_grouped_gemm_int8(a["a"], a["sa"], a["off"], a["w"], a["sw"], a["bias"], a["res"],
                                     a["E"], a["N"], a["K"], a["R"], a["act"], a["gated"], a["y"],
                                     None)


@pytest.mark.parametrize("kw", [
    dict(E=0), dict(E=1025), dict(N=0), dict(N=12), dict(N=2 ** 20 + 8), dict(N=24, gated=1),
    dict(K=0), dict(K=8), dict(K=24), dict(K=2 ** 17), dict(K=-16), dict(R=-1), dict(R=2 ** 31),
    dict(act=-1), dict(act=4), dict(R=2 ** 31 - 1, N=2 ** 20),
])
def test_gemm_limits(kw):
    assert gemm(**kw) == EINVAL


def test_gemm_pointers():
    for p in ("a", "sa", "off", "w", "sw", "y"):
        assert gemm(**{p: None}) == ENULL, p
    for p in ("a", "w", "sw", "bias", "res", "y"):
        assert gemm(**{p: 96 * MB + 8}) == EALIGN, p
    for p in ("sa", "off"):
        assert gemm(**{p: 96 * MB + 2}) == EALIGN, p
    assert gemm(R=0, a=None, sa=None, off=None, w=None, sw=None, y=None) == OK


def test_gemm_overlaps():
    y, n = 64 * MB, 1000 * 512 * 2
    sizes = dict(a=1000 * 256, sa=4000, off=36, w=8 * 512 * 256, sw=8 * 512 * 4, bias=8 * 512 * 2,
                 res=n)
    for p, m in sizes.items():
        for at in (y + 16, y + n - 16, y - m // 16 * 16 + 16):
            assert gemm(**{p: at}) == EINVAL, (p, at - y)
        if p != "res":
            assert gemm(**{p: y}) == EINVAL, p
    assert gemm(gated=1, res=y + n // 2 - 16) == EINVAL


# ------------------------------------------------------------------ activation

def gact(**kw):
    a = dict(h=16 * MB, off=1 * MB, E=8, R=1000, I=272, act=2, out=32 * MB, sc=2 * MB)
    a.update(kw)
    return lib.moe_gated_act_quant_int8(a["h"], a["off"], a["E"], a["R"], a["I"], a["act"], a["out"],
                                        a["sc"], None)


def test_act_refusals():
    for kw in (dict(E=0), dict(E=1025), dict(R=-1), dict(R=2 ** 31), dict(I=0), dict(I=8), dict(I=24),
               dict(I=32784), dict(act=4), dict(act=-1), dict(R=2 ** 23, I=16384)):
        assert gact(**kw) == EINVAL, kw
    for p in ("h", "off", "out", "sc"):
        assert gact(**{p: None}) == ENULL
    assert gact(h=16 * MB + 8) == EALIGN
    assert gact(out=32 * MB + 8) == EALIGN
    assert gact(sc=2 * MB + 2) == EALIGN
    assert gact(off=1 * MB + 1) == EALIGN
    out, n = 32 * MB, 1000 * 272
    for p, m in (("h", 4 * n), ("off", 36), ("sc", 4000)):
        for at in (out, out + n - 16, out - m // 16 * 16 + 16):
            assert gact(**{p: at}) == EINVAL, p
    for at in (2 * MB, 2 * MB + 3984, 2 * MB - 4 * n + 16):
        assert gact(h=at) == EINVAL
    for at in (2 * MB, 2 * MB + 3996, 2 * MB - 32):
        assert gact(off=at) == EINVAL
    assert gact(R=0, h=None, off=None, out=None, sc=None) == OK
