"""The INT8 expert layer's operators together, as a layer uses them: the norm,
the gate, the dispatch of its codes, the two products with the gated activation
between them, combine, and the shared expert on top; each step checked on what the
step before it gave. The same recorded in HIP graphs, replayed with new inputs,
side by side and on other streams; and the FP8 codes of the norm through the FP8
products."""
import math

import numpy as np
import pytest
import torch

import oracle
from moe_synth import bf16_bits_to_f32, gen_fp8_weight_codes, gen_weight_scales
from parity_util import bf16_to_np, combine_within_tolerance, log
from test_gpu_gated_act_int8 import check as check_act
from test_gpu_gemm_int8 import reference
from test_gpu_rmsnorm_quant import check as check_norm, make as make_norm
from test_gpu_route_scored import check as check_route

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def weights(E, N, K, gen):
    w = torch.randn((E, N, K), device=DEV, generator=gen) / math.sqrt(K)
    s = w.abs().amax(dim=2) / 127
    return torch.round(w / s[:, :, None]).to(torch.int8), s


def within(y, c, act="none"):
    for (r0, r1), (want, tol) in reference(c, act).items():
        assert ((y[r0:r1].double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("T,H,I,E,k,align", [(150, 256, 192, 16, 4, 1), (40, 512, 144, 64, 6, 16),
                                             (1, 256, 64, 8, 2, 1), (900, 128, 320, 4, 2, 128)])
def test_int8_layer(T, H, I, E, k, align):
    from combine_moe_route_amd import moe_combine, moe_dispatch_quantized, moe_grouped_gemm_int8
    log(f"int8 layer T={T} H={H} I={I} E={E} k={k} align={align}")
    gen = torch.Generator(DEV).manual_seed(4)
    x, res, nw = make_norm(T, H, True, 3)
    q, qs, y0, _ = check_norm(x, res, nw, "int8")
    gate = torch.randn((E, H), device=DEV, generator=gen) / math.sqrt(H)
    idx, wt = check_route(y0.float() @ gate.T, k)
    d = moe_dispatch_quantized(q, qs, idx, E, 1, align)
    ref = oracle.dispatch(q.cpu().numpy().view(np.uint16), idx.cpu().numpy(), E, 1, align, False)
    off = d.expert_offsets.tolist()
    R = off[-1]
    assert off == ref.expert_offsets.tolist() and np.array_equal(d.dst_row.cpu().numpy(), ref.dst_row)
    assert np.array_equal(d.out[:R].cpu().numpy().view(np.uint16), ref.out)
    (w1, s1), (w2, s2) = weights(E, 2 * I, H, gen), weights(E, H, I, gen)
    h = moe_grouped_gemm_int8(d.out, d.out_scales, d.expert_offsets, w1, s1)
    base = dict(bias=None, residual=None, gated=False, off=off)
    within(h, dict(base, a=d.out, a_scales=d.out_scales, w=w1, w_scales=s1))
    a2, a2s = check_act(h, off, "silu")
    pad = d.row_src[:R] < 0
    assert (a2[:R][pad] == 0).all() and (a2s[:R][pad] == 0).all()
    eo = moe_grouped_gemm_int8(a2, a2s, d.expert_offsets, w2, s2)
    within(eo, dict(base, a=a2, a_scales=a2s, w=w2, w_scales=s2))
    y = moe_combine(eo, d.dst_row, wt)
    want = oracle.combine(bf16_to_np(eo), d.dst_row.cpu().numpy(), wt.cpu().numpy())
    ok, ulp, _ = combine_within_tolerance(bf16_to_np(y), want)
    assert ok.all() and ulp.all()
    # the shared expert on the tokens themselves, added to the routed experts' sum in place
    whole = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    (v1, t1), (v2, t2) = weights(1, 2 * I, H, gen), weights(1, H, I, gen)
    hs = moe_grouped_gemm_int8(q, qs, whole, v1, t1)
    a3, a3s = check_act(hs, [0, T], "silu")
    routed = y.clone()
    out = moe_grouped_gemm_int8(a3, a3s, whole, v2, t2, residual=y, y=y)
    assert out is y
    within(out, dict(base, a=a3, a_scales=a3s, w=v2, w_scales=t2, residual=routed, off=[0, T]))


def test_nan_token_stays_alone():
    """A token with a NaN ends as NaN and changes no other token."""
    from combine_moe_route_amd import (moe_combine, moe_dispatch_quantized, moe_gated_act_quant_int8,
                                       moe_grouped_gemm_int8, moe_rmsnorm_quant)
    log("int8 layer nan")
    T, H, I, E, k = 50, 256, 128, 8, 2
    gen = torch.Generator(DEV).manual_seed(4)
    x, res, nw = make_norm(T, H, True, 3)
    (w1, s1), (w2, s2) = weights(E, 2 * I, H, gen), weights(E, H, I, gen)
    idx = torch.stack([torch.arange(T) % E, (torch.arange(T) + 3) % E], 1).to(torch.int32).to(DEV)
    wt = torch.full((T, k), 0.5, device=DEV)

    def layer(x):
        q, qs, _, _ = moe_rmsnorm_quant(x, nw, residual=res)
        d = moe_dispatch_quantized(q, qs, idx, E)
        h = moe_grouped_gemm_int8(d.out, d.out_scales, d.expert_offsets, w1, s1)
        a, s = moe_gated_act_quant_int8(h, d.expert_offsets)
        return moe_combine(moe_grouped_gemm_int8(a, s, d.expert_offsets, w2, s2), d.dst_row, wt)

    clean = layer(x)
    bad = x.clone()
    bad[17, 200] = float("nan")
    y = layer(bad)
    assert torch.isnan(y[17]).all()
    keep = torch.arange(T, device=DEV) != 17
    assert torch.equal(y[keep], clean[keep])


def test_norm_codes_through_the_fp8_layer():
    """The norm's FP8 codes and 1x128 scales are the operands of the FP8 product."""
    from combine_moe_route_amd import moe_dispatch_quantized, moe_grouped_gemm_fp8
    log("norm -> fp8 product")
    T, H, N, E, k = 90, 512, 256, 8, 2
    x, res, nw = make_norm(T, H, True, 6)
    q, qs, _, _ = check_norm(x, res, nw, "fp8")
    idx = torch.stack([torch.arange(T) % E, (torch.arange(T) + 3) % E], 1).to(torch.int32).to(DEV)
    d = moe_dispatch_quantized(q, qs, idx, E, 1, 16)
    w, ws = gen_fp8_weight_codes(E, N, H, 1), gen_weight_scales(E, N, H, 1)
    y = moe_grouped_gemm_fp8(d.out, d.out_scales, d.expert_offsets, torch.from_numpy(w).to(DEV),
                             torch.from_numpy(ws).to(DEV))
    off = d.expert_offsets.cpu().numpy()
    R = int(off[-1])
    ref = oracle.grouped_gemm_fp8(d.out.cpu().numpy(), d.out_scales.cpu().numpy(), off, w, ws)
    e = ((H // 128 + 2) * 2.0 ** -24 + 2.0 ** -12) * ref.mag[:R]
    err = np.abs(bf16_bits_to_f32(bf16_to_np(y[:R])).astype(np.float64) - ref.y64[:R])
    assert (err <= 2.0 ** -8 * (np.abs(ref.y64[:R]) + e) + e + 2.0 ** -133).all()


class Layer:
    """One INT8 layer over fixed buffers, as a captured step needs."""

    def __init__(self, T, H, I, E, k, seed, align=1):
        from combine_moe_route_amd import alloc_dispatch_quantized
        self.T, self.H, self.E, self.k, self.align = T, H, E, k, align
        gen = torch.Generator(DEV).manual_seed(seed)
        z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        self.x, self.res, self.logits = z(T, H), z(T, H), z(T, E, dt=torch.float32)
        self.nw = (1 + 0.2 * torch.randn(H, device=DEV, generator=gen)).to(torch.bfloat16)
        self.w1, self.s1 = weights(E, 2 * I, H, gen)
        self.w2, self.s2 = weights(E, H, I, gen)
        self.v1, self.t1 = weights(1, 2 * I, H, gen)
        self.v2, self.t2 = weights(1, H, I, gen)
        self.q, self.qs, self.n = z(T, H, dt=torch.int8), z(T, dt=torch.float32), z(T, H)
        self.idx, self.wt = z(T, k, dt=torch.int32), z(T, k, dt=torch.float32)
        self.d = alloc_dispatch_quantized(T, H, E, k, row_align=align, device=DEV)
        R = self.d.out.shape[0]
        self.h, self.eo, self.y = z(R, 2 * I), z(R, H), z(T, H)
        self.a, self.s = z(R, I, dt=torch.int8), z(R, dt=torch.float32)
        self.hs, self.b, self.bs = z(T, 2 * I), z(T, I, dt=torch.int8), z(T, dt=torch.float32)
        self.whole = torch.tensor([0, T], dtype=torch.int32, device=DEV)

    def load(self, seed):
        gen = torch.Generator(DEV).manual_seed(1000 + seed)
        self.x.copy_(torch.randn((self.T, self.H), device=DEV, generator=gen))
        self.res.copy_(torch.randn((self.T, self.H), device=DEV, generator=gen))
        self.logits.copy_(torch.randn((self.T, self.E), device=DEV, generator=gen))
        self.logits[seed % self.T] = -math.inf

    def step(self):
        import combine_moe_route_amd as m
        m.moe_rmsnorm_quant(self.x, self.nw, residual=self.res, sum_out=self.res, y=self.n,
                            out=self.q, out_scales=self.qs)
        m.moe_route_scored(self.logits, self.k, topk_idx=self.idx, topk_w=self.wt)
        m.moe_dispatch_quantized(self.q, self.qs, self.idx, self.E, row_align=self.align, bufs=self.d)
        off = self.d.expert_offsets
        m.moe_grouped_gemm_int8(self.d.out, self.d.out_scales, off, self.w1, self.s1, y=self.h)
        m.moe_gated_act_quant_int8(self.h, off, out=self.a, out_scales=self.s)
        m.moe_grouped_gemm_int8(self.a, self.s, off, self.w2, self.s2, y=self.eo)
        m.moe_combine(self.eo, self.d.dst_row, self.wt, self.y)
        m.moe_grouped_gemm_int8(self.q, self.qs, self.whole, self.v1, self.t1, y=self.hs)
        m.moe_gated_act_quant_int8(self.hs, self.whole, out=self.b, out_scales=self.bs)
        m.moe_grouped_gemm_int8(self.b, self.bs, self.whole, self.v2, self.t2, residual=self.y, y=self.y)

    def got(self):
        return [t.clone() for t in (self.res, self.n, self.q, self.qs, self.idx, self.wt, self.y)]


def capture(layer):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.step()
    torch.cuda.synchronize()
    return g


@pytest.mark.parametrize("T,align", [(1, 1), (60, 16), (700, 128)])
def test_graph_replays_match_eager(T, align):
    log(f"int8 layer graph T={T}")
    layer = Layer(T, 256, 192, 16, 4, 1, align)
    layer.load(0)
    g = capture(layer)
    for seed in (1, 2, 3, 1):
        layer.load(seed)                             # the step updates the residual in place
        g.replay()
        torch.cuda.synchronize()
        got = layer.got()
        torch.randn(1 << 20, device=DEV).sum().item()     # eager work between the replays
        layer.load(seed)
        layer.step()
        torch.cuda.synchronize()
        for a, b in zip(got, layer.got()):
            assert torch.equal(a, b)


def test_two_graphs_side_by_side():
    """Two layers' graphs replayed at once on two streams: nothing is shared."""
    log("two int8 graphs")
    layers = [Layer(300, 256, 256, 16, 4, 1), Layer(90, 512, 128, 16, 2, 2, 8)]
    for i, l in enumerate(layers):
        l.load(i)
    graphs = [capture(l) for l in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for seed in range(3):
        want = []
        for i, l in enumerate(layers):
            l.load(10 * seed + i)
            l.step()
            torch.cuda.synchronize()
            want.append(l.got())
            l.load(10 * seed + i)
            l.y.zero_()
            l.idx.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for l, w in zip(layers, want):
            for a, b in zip(l.got(), w):
                assert torch.equal(a, b)


def test_on_another_stream():
    """Calls go to torch's current stream: a step behind a long piece of work on a
    side stream sees what that work wrote."""
    log("int8 side stream")
    layer = Layer(64, 256, 128, 8, 2, 5)
    layer.load(3)
    layer.step()
    torch.cuda.synchronize()
    want = layer.got()
    layer.load(4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn((6000, 6000), device=DEV)
        for _ in range(4):
            big = big @ big * 1e-4
        layer.load(3)
        layer.step()
    s.synchronize()
    for a, b in zip(layer.got(), want):
        assert torch.equal(a, b)
