"""The expert layer's operators together, as a layer uses them: scored
routing, dispatch, the experts' products and combine, in bf16 and in FP8,
each step checked on what the step before it gave; the same recorded in HIP
graphs, replayed with new inputs, on other streams and side by side."""
import math

import numpy as np
import pytest
import torch

import oracle
from moe_synth import bf16_bits_to_f32, gen_fp8_weight_codes, gen_weight_scales, gen_x_bf16
from parity_util import bf16_to_np, combine_within_tolerance, log, to_dev_bf16
from test_gpu_gated_act import check as check_gated_act
from test_gpu_gemm_bf16 import reference
from test_gpu_route_scored import bias_of, check as check_route, logits_of

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def within(y, want):
    for (r0, r1), (ref, tol) in want.items():
        assert ((y[r0:r1].double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,H,I,E,k,align", [(150, 256, 192, 16, 4, 1), (40, 512, 128, 64, 6, 16),
                                             (1, 256, 64, 8, 2, 1), (900, 128, 320, 4, 2, 128)])
def test_bf16_layer(T, H, I, E, k, align):
    from combine_moe_route_amd import moe_combine, moe_dispatch, moe_grouped_gemm_bf16
    log(f"bf16 layer T={T} H={H} I={I} E={E} k={k} align={align}")
    logits = logits_of(T, E, 1, masked=0.05 if T > 1 else 0.0)
    idx, wt = check_route(logits, k, bias=bias_of(E, 2), n_group=4, topk_group=3, scale=2.5)
    x_np = gen_x_bf16(T, H, 3)
    x = to_dev_bf16(x_np, DEV)
    ref = oracle.dispatch(x_np, idx.cpu().numpy(), E, 1, align, False)
    d = moe_dispatch(x, idx, E, 1, align)
    off = d.expert_offsets.tolist()
    assert off == ref.expert_offsets.tolist()
    R = off[-1]
    assert np.array_equal(bf16_to_np(d.out[:R]), ref.out)
    assert np.array_equal(d.dst_row.cpu().numpy(), ref.dst_row)
    gen = torch.Generator(DEV).manual_seed(4)
    mk = lambda *s: (torch.randn(s, device=DEV, generator=gen) / math.sqrt(s[-1])).to(torch.bfloat16)  # noqa: E731
    w1, w2, b1 = mk(E, 2 * I, H), mk(E, H, I), mk(E, 2 * I)
    h = moe_grouped_gemm_bf16(d.out, d.expert_offsets, w1, bias=b1, act="silu", gated=True)
    within(h, reference(d.out, off, w1, b1, "silu", True, None))
    eo = moe_grouped_gemm_bf16(h, d.expert_offsets, w2)
    within(eo, reference(h, off, w2, None, "none", False, None))
    y = moe_combine(eo, d.dst_row, wt)
    want = oracle.combine(bf16_to_np(eo), d.dst_row.cpu().numpy(), wt.cpu().numpy())
    ok, ulp, _ = combine_within_tolerance(bf16_to_np(y), want)
    assert ok.all() and ulp.all()
    assert (y[(idx < 0).all(dim=1)] == 0).all()
    # the shared expert, added to the routed experts' sum in place
    whole = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    s1, s2 = mk(1, 2 * I, H), mk(1, H, I)
    hs = moe_grouped_gemm_bf16(x, whole, s1, act="silu", gated=True)
    routed = y.clone()
    out = moe_grouped_gemm_bf16(hs, whole, s2, residual=y, y=y)
    assert out is y
    within(out, reference(hs, [0, T], s2, None, "none", False, routed))


def test_fp8_layer():
    from combine_moe_route_amd import (moe_combine, moe_dispatch, moe_gated_act_quant_fp8,
                                       moe_grouped_gemm_fp8)
    T, H, I, E, k, align = 200, 256, 256, 8, 2, 16
    log("fp8 layer")
    idx, wt = check_route(logits_of(T, E, 5), k, bias=bias_of(E, 5), n_group=4, topk_group=2)
    x_np = gen_x_bf16(T, H, 6)
    d = moe_dispatch(to_dev_bf16(x_np, DEV), idx, E, 1, align, fp8=True)
    w1, s1 = gen_fp8_weight_codes(E, 2 * I, H, 1), gen_weight_scales(E, 2 * I, H, 1)
    w2, s2 = gen_fp8_weight_codes(E, H, I, 2), gen_weight_scales(E, H, I, 2)
    g = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    h = moe_grouped_gemm_fp8(d.out, d.out_scales, d.expert_offsets, g(w1), g(s1))
    off = d.expert_offsets.cpu().numpy()
    R = int(off[-1])
    codes, scales = check_gated_act(h, off.tolist(), "silu")
    q, qs = moe_gated_act_quant_fp8(h, d.expert_offsets)
    assert torch.equal(q[:R], codes[:R]) and torch.equal(qs[:R], scales[:R])
    pad = d.row_src[:R] < 0
    assert (q[:R][pad] == 0).all() and (qs[:R][pad] == 0).all()
    eo = moe_grouped_gemm_fp8(q, qs, d.expert_offsets, g(w2), g(s2))
    ref = oracle.grouped_gemm_fp8(q.cpu().numpy(), qs.cpu().numpy(), off, w2, s2)
    e = ((I // 128 + 2) * 2.0 ** -24 + 2.0 ** -12) * ref.mag[:R]
    err = np.abs(bf16_bits_to_f32(bf16_to_np(eo[:R])).astype(np.float64) - ref.y64[:R])
    assert (err <= 2.0 ** -8 * (np.abs(ref.y64[:R]) + e) + e + 2.0 ** -133).all()
    y = moe_combine(eo, d.dst_row, wt)
    want = oracle.combine(bf16_to_np(eo), d.dst_row.cpu().numpy(), wt.cpu().numpy())
    ok, ulp, _ = combine_within_tolerance(bf16_to_np(y), want)
    assert ok.all() and ulp.all()


class Layer:
    """One bf16 and one FP8 layer over fixed buffers, as a captured step needs."""

    def __init__(self, T, H, I, E, k, seed):
        from combine_moe_route_amd import alloc_dispatch
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        gen = torch.Generator(DEV).manual_seed(seed)
        bf = lambda *s: (torch.randn(s, device=DEV, generator=gen) / math.sqrt(s[-1])).to(torch.bfloat16)  # noqa: E731
        self.x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        self.logits = torch.empty((T, E), device=DEV)
        self.bias = 0.05 * torch.randn(E, device=DEV, generator=gen)
        self.w1, self.w2 = bf(E, 2 * I, H), bf(E, H, I)
        c = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        self.q1, self.t1 = c(gen_fp8_weight_codes(E, 2 * I, H, seed)), c(gen_weight_scales(E, 2 * I, H, seed))
        self.q2, self.t2 = c(gen_fp8_weight_codes(E, H, I, seed)), c(gen_weight_scales(E, H, I, seed))
        self.idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
        self.wt = torch.empty((T, k), device=DEV)
        self.d = alloc_dispatch(T, H, E, k, device=DEV)
        self.d8 = alloc_dispatch(T, H, E, k, row_align=16, fp8=True, device=DEV)
        R, R8 = self.d.out.shape[0], self.d8.out.shape[0]
        z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        self.h, self.eo, self.y = z(R, I), z(R, H), z(T, H)
        self.h8, self.eo8, self.y8 = z(R8, 2 * I), z(R8, H), z(T, H)
        self.a8, self.s8 = z(R8, I, dt=torch.uint8), z(R8, I // 128, dt=torch.float32)
        from combine_moe_route_amd import moe_grouped_gemm_workspace_bytes
        self.ws = z(moe_grouped_gemm_workspace_bytes(R8, E), dt=torch.uint8)

    def load(self, seed):
        gen = torch.Generator(DEV).manual_seed(1000 + seed)
        self.x.copy_(torch.randn((self.T, self.H), device=DEV, generator=gen))
        self.logits.copy_(torch.randn((self.T, self.E), device=DEV, generator=gen))
        self.logits[seed % self.T] = -math.inf

    def step(self):
        import combine_moe_route_amd as m
        m.moe_route_scored(self.logits, self.k, bias=self.bias, n_group=4, topk_group=2,
                           topk_idx=self.idx, topk_w=self.wt)
        m.moe_dispatch(self.x, self.idx, self.E, bufs=self.d)
        off = self.d.expert_offsets
        m.moe_grouped_gemm_bf16(self.d.out, off, self.w1, act="silu", gated=True, y=self.h)
        m.moe_grouped_gemm_bf16(self.h, off, self.w2, y=self.eo)
        m.moe_combine(self.eo, self.d.dst_row, self.wt, self.y)
        m.moe_dispatch(self.x, self.idx, self.E, row_align=16, fp8=True, bufs=self.d8)
        off8 = self.d8.expert_offsets
        m.moe_grouped_gemm_fp8(self.d8.out, self.d8.out_scales, off8, self.q1, self.t1, self.h8, self.ws)
        m.moe_gated_act_quant_fp8(self.h8, off8, out=self.a8, out_scales=self.s8)
        m.moe_grouped_gemm_fp8(self.a8, self.s8, off8, self.q2, self.t2, self.eo8, self.ws)
        m.moe_combine(self.eo8, self.d8.dst_row, self.wt, self.y8)

    def got(self):
        return [t.clone() for t in (self.idx, self.wt, self.y, self.y8)]


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


@pytest.mark.parametrize("T", [1, 60, 700])
def test_graph_replays_match_eager(T):
    log(f"layer graph T={T}")
    layer = Layer(T, 256, 256, 16, 4, 1)
    layer.load(0)
    g = capture(layer)
    for seed in (1, 2, 3, 1):
        layer.load(seed)
        g.replay()
        torch.cuda.synchronize()
        got = layer.got()
        torch.randn(1 << 20, device=DEV).sum().item()     # eager work between the replays
        layer.step()
        torch.cuda.synchronize()
        for a, b in zip(got, layer.got()):
            assert torch.equal(a, b)


def test_two_graphs_side_by_side():
    """Two layers' graphs replayed at once on two streams: nothing is shared."""
    log("two graphs")
    layers = [Layer(300, 256, 256, 16, 4, 1), Layer(90, 512, 128, 16, 2, 2)]
    for i, l in enumerate(layers):
        l.load(i)
    graphs = [capture(l) for l in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for seed in range(3):
        for i, l in enumerate(layers):
            l.load(10 * seed + i)
            l.step()
        torch.cuda.synchronize()
        want = [l.got() for l in layers]
        for l in layers:
            l.y.zero_()
            l.y8.zero_()
            l.idx.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for l, w in zip(layers, want):
            for a, b in zip(l.got(), w):
                assert torch.equal(a, b)
