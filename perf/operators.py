"""Cases and plain forms of the expert-layer operators: scored routing, the
bf16 grouped GEMM with its epilogue, and the gated activation that quantises
between the two FP8 grouped GEMMs.

run(state) is one pass through one operator: the plain form in elementary
torch operations, or, where ``own`` is true, the framework's call.
"""
import math

import numpy as np
import torch

own = False

INF = float("inf")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a sequence being generated, 256 experts in 8 groups
        dict(name="route_one_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_top=2, dtype="float32", pad=0, masked=0.0),
        # a decode batch, 384 experts without groups, scores with a balance bias
        dict(name="route_decode", op="route", T=128, E=384, k=8, score="sigmoid", bias=True,
             n_group=1, topk_group=1, group_top=2, dtype="bfloat16", pad=0, masked=0.0),
        # odd batch, softmax, three of eight groups of 20 by their best expert; some experts
        # masked, a few tokens wholly (padding), logits a slice of a wider projection
        dict(name="route_odd_masked", op="route", T=5003, E=160, k=6, score="softmax", bias=False,
             n_group=8, topk_group=3, group_top=1, dtype="float32", pad=5, masked=0.1),
        # a prefill batch
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_top=2, dtype="float32", pad=0, masked=0.0),
        # one token through two of eight experts: gate and up projections, bound by the weights
        dict(name="experts_one_token", op="gemm", T=1, E=8, k=2, K=4096, N=16384, align=1,
             act="silu", gated=True, bias=False, residual=False),
        # a decode batch over 256 experts, about four rows each
        dict(name="experts_decode", op="gemm", T=128, E=256, k=8, K=7168, N=4096, align=1,
             act="silu", gated=True, bias=False, residual=False),
        # ragged segments, odd widths, every part of the ungated epilogue
        dict(name="experts_odd", op="gemm", T=777, E=12, k=3, K=1016, N=1032, align=1,
             act="gelu", gated=False, bias=True, residual=True),
        # a shared expert's down projection added to what the routed experts gave
        dict(name="shared_down", op="gemm", T=4096, E=1, k=1, K=2048, N=7168, align=1,
             act="none", gated=False, bias=False, residual=True),
        # gate and up projections of a prefill batch, segments padded to 128 rows
        dict(name="experts_prefill", op="gemm", T=16384, E=256, k=8, K=7168, N=4096, align=128,
             act="silu", gated=True, bias=False, residual=False),
        # one token between the FP8 products
        dict(name="act_one_token", op="act", T=1, E=256, k=8, I=2048, align=1, act="silu"),
        # odd batch, widths of 11 blocks
        dict(name="act_odd", op="act", T=1237, E=61, k=5, I=1408, align=8, act="gelu"),
        # a prefill batch between the FP8 products
        dict(name="act_prefill", op="act", T=16384, E=256, k=8, I=2048, align=128, act="silu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route", "gemm", "gemm", "act"))
    if op == "route":
        n_group = rng.choice((1, 1, 2, 4, 5, 8, 16))
        per = max(1, _log_int(rng, 8, 1024) // n_group)
        E = n_group * per
        topk_group = rng.randint((n_group + 1) // 2, n_group)
        k = min(rng.randint(1, 12), topk_group * per)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k,
                    score=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.5,
                    n_group=n_group, topk_group=topk_group, group_top=rng.choice((1, 2)),
                    dtype=rng.choice(("float32", "bfloat16")), pad=rng.choice((0, 0, 1, 8)),
                    masked=rng.choice((0.0, 0.0, 0.2)))
    E = _log_int(rng, 1, 64)
    k = min(E, rng.randint(1, 8))
    if op == "gemm":
        gated = rng.random() < 0.5
        return dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=k, K=8 * _log_int(rng, 8, 600),
                    N=(16 if gated else 8) * _log_int(rng, 8, 300 if gated else 600),
                    align=rng.choice((1, 1, 8, 128)), act=rng.choice(("none", "relu", "silu", "gelu")),
                    gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k, I=128 * rng.randint(1, 24),
                align=rng.choice((1, 8, 128)), act=rng.choice(("relu", "silu", "gelu")))


# ------------------------------------------------------------------ inputs

def _segments(case, gen):
    """Segment offsets as routing gives them: a popularity prior over the
    experts, k distinct ones for each token, segments padded to `align`."""
    T, E, k, A = case["T"], case["E"], case["k"], case["align"]
    prior = 0.5 * torch.randn(E, device="cuda", generator=gen)
    noise = torch.rand((T, E), device="cuda", generator=gen).clamp_(1e-20, 1 - 1e-7)
    idx = (prior - torch.log(-torch.log(noise))).topk(k, dim=1).indices
    counts = np.bincount(idx.flatten().cpu().numpy(), minlength=E)
    off = np.zeros(E + 1, np.int64)
    off[1:] = np.cumsum((counts + A - 1) // A * A)
    return counts, off


def _rows(counts, off, width, gen, rows):
    """bf16 rows, normal; the pad rows at the segments' ends are zero."""
    x = torch.randn((rows, width), device="cuda", generator=gen, dtype=torch.bfloat16)
    r = np.arange(rows)
    e = np.minimum(np.searchsorted(off[1:], r, side="right"), len(counts) - 1)
    x[torch.from_numpy(np.nonzero(r - off[e] >= counts[e])[0]).cuda()] = 0
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        dt = getattr(torch, case["dtype"])
        wide = torch.randn((T, E + case["pad"]), device="cuda", generator=gen)
        if case["masked"]:
            wide[torch.rand(wide.shape, device="cuda", generator=gen) < case["masked"]] = -INF
            wide[torch.rand(T, device="cuda", generator=gen) < case["masked"] / 4] = -INF
        wide = wide.to(dt)
        bias = 0.05 * torch.randn(E, device="cuda", generator=gen) if case["bias"] else None
        return dict(case=case, logits=wide[:, :E], bias=bias,
                    idx=torch.empty((T, case["k"]), dtype=torch.int32, device="cuda"),
                    w=torch.empty((T, case["k"]), dtype=torch.float32, device="cuda"))
    counts, off = _segments(case, gen)
    used = int(off[-1])
    # buffers hold what the dispatch may need for any routing; rows behind the
    # last segment stay as they were, zero here
    R = case["T"] * case["k"] + case["E"] * (case["align"] - 1)
    s = dict(case=case, used=used, cap=int((off[1:] - off[:-1]).max()),
             off=torch.from_numpy(off.astype(np.int32)).cuda())
    if case["op"] == "act":
        I = case["I"]
        s["h"] = _rows(counts, off, 2 * I, gen, R)
        s["out"] = torch.zeros((R, I), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros((R, I // 128), dtype=torch.float32, device="cuda")
        return s
    E, K, N = case["E"], case["K"], case["N"]
    n_out = N // 2 if case["gated"] else N
    s["a"] = _rows(counts, off, K, gen, R)
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
    s["w"] = w.normal_(0.0, 1.0 / math.sqrt(K), generator=gen)
    s["bias"] = torch.randn((E, N), device="cuda", generator=gen, dtype=torch.bfloat16) \
        if case["bias"] else None
    s["residual"] = torch.randn((R, n_out), device="cuda", generator=gen, dtype=torch.bfloat16) \
        if case["residual"] else None
    s["y"] = torch.zeros((R, n_out), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "route":
        return _plain_route(s, case)
    if case["op"] == "gemm":
        return _plain_gemm(s, case)
    return _plain_act(s, case)


def _own(s, case):
    import combine_moe_route_amd as moe
    if case["op"] == "route":
        idx, w = moe.moe_route_scored(
            s["logits"], case["k"], score=case["score"], bias=s["bias"], n_group=case["n_group"],
            topk_group=case["topk_group"], group_top=case["group_top"], renorm=True, scale=2.5,
            topk_idx=s["idx"], topk_w=s["w"])
        return {"idx": idx, "w": w}
    if case["op"] == "gemm":
        return {"y": moe.moe_grouped_gemm_bf16(
            s["a"], s["off"], s["w"], bias=s["bias"], act=case["act"], gated=case["gated"],
            residual=s["residual"], y=s["y"])}
    out, scales = moe.moe_gated_act_quant_fp8(s["h"], s["off"], act=case["act"], out=s["out"],
                                              out_scales=s["scales"])
    return {"codes": out.view(torch.float8_e4m3fn), "scales": scales}


def _plain_route(s, case):
    """Scores rounded once from 64 bits (neighbours at the border of the
    choice are closer than 32-bit errors); the choice on their 32-bit values."""
    T, E = s["logits"].shape
    k, G = case["k"], case["n_group"]
    logits = s["logits"].double()
    live = logits > -INF
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        top = logits.amax(dim=1, keepdim=True)
        e = torch.where(live, torch.exp(logits - torch.where(top > -INF, top, 0.0)), 0.0)
        score = e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)
    score = score.float()
    key = score if s["bias"] is None else score + s["bias"]
    key = torch.where(live, key, -INF)
    if G > 1:
        best = key.view(T, G, E // G).topk(min(case["group_top"], E // G), dim=2).values
        group = torch.where(best[:, :, 0] > -INF, torch.where(best > -INF, best, 0.0).sum(dim=2), -INF)
        first = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter_(1, first, True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1, output_size=E), key, -INF)
    key, idx = torch.sort(key, dim=1, descending=True, stable=True)
    key, idx = key[:, :k], idx[:, :k]
    w = torch.where(key > -INF, score.gather(1, idx), 0.0)
    total = w.sum(dim=1, keepdim=True)
    w = w / torch.where(total > 0, total, 1.0) * 2.5
    return {"idx": torch.where(key > -INF, idx, -1).to(torch.int32), "w": w}


def _act(name, z):
    if name == "relu":
        return torch.clamp_min(z, 0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _plain_gemm(s, case):
    a, w, off = s["a"], s["w"], s["off"].long()
    E, N = case["E"], case["N"]
    rows = torch.arange(s["used"], device=a.device)
    # segments side by side, each as long as the longest, zero behind its end
    at = off[:-1, None] + torch.arange(s["cap"], device=a.device)
    seg = torch.where((at < off[1:, None])[:, :, None],
                      a[at.clamp(max=a.shape[0] - 1)].float(), 0.0)
    z = torch.matmul(seg, w.float().transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None, :]
    e = torch.searchsorted(off[1:].contiguous(), rows, right=True)
    z = z[e, rows - off[e]]
    y = _act(case["act"], z[:, :N // 2]) * z[:, N // 2:] if case["gated"] else _act(case["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"][:s["used"]].float()
    s["y"][:s["used"]] = y
    return {"y": s["y"]}


def _plain_act(s, case):
    I = case["I"]
    h = s["h"][:s["used"]].float()
    v = (_act(case["act"], h[:, :I]) * h[:, I:]).view(-1, I // 128, 128)
    scales = v.abs().amax(dim=2) / 448.0
    q = v / torch.where(scales > 0, scales, 1.0)[:, :, None]
    codes = s["out"].view(torch.float8_e4m3fn)
    codes[:s["used"]] = q.to(torch.float8_e4m3fn).view(-1, I)
    s["scales"][:s["used"]] = scales
    return {"codes": codes, "scales": s["scales"]}


# ------------------------------------------------------------------ needed work

def work(case):
    T, k = case["T"], case["k"]
    if case["op"] == "route":
        E = case["E"]
        size = 4 if case["dtype"] == "float32" else 2
        return dict(bytes=T * E * size + 4 * E * case["bias"] + 8 * T * k, flops=0)
    if case["op"] == "act":
        return dict(bytes=T * k * case["I"] * (4 + 1 + 4 / 128), flops=0)
    E, K, N = case["E"], case["K"], case["N"]
    n_out = N // 2 if case["gated"] else N
    hit = E * (1.0 - (1.0 - k / E) ** T)      # experts that have rows
    return dict(bytes=2 * (T * k * K + hit * N * K + hit * N * case["bias"]
                           + T * k * n_out * (2 if case["residual"] else 1)),
                flops=2 * T * k * N * K)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return {"idx": None, "w": _exact_weights(s, case)}
    off = s["off"].tolist()
    if case["op"] == "act":
        I = case["I"]
        codes = torch.zeros((len(s["h"]), I), dtype=torch.float64)
        scales = torch.zeros((len(s["h"]), I // 128), dtype=torch.float64)
        for r in range(0, s["used"], 8192):
            h = s["h"][r:min(r + 8192, s["used"])].double()
            v = _exact_act(case["act"], h[:, :I]) * h[:, I:]
            v = v.reshape(len(h), I // 128, 128)
            sc = v.abs().max(dim=2).values / 448
            q = torch.nan_to_num(v / sc[:, :, None])
            codes[r:r + len(h)] = q.to(torch.float8_e4m3fn).double().reshape(len(h), I).cpu()
            scales[r:r + len(h)] = sc.cpu()
        return {"codes": codes, "scales": scales}
    if 2.0 * s["used"] * case["K"] * case["N"] > 2e14:
        return None
    N, parts = case["N"], []
    for e in range(case["E"]):
        if off[e + 1] > off[e]:
            z = s["a"][off[e]:off[e + 1]].double() @ s["w"][e].double().T
            if s["bias"] is not None:
                z += s["bias"][e].double()
            parts.append(_exact_act(case["act"], z[:, :N // 2]) * z[:, N // 2:] if case["gated"]
                         else _exact_act(case["act"], z))
    y = torch.cat(parts)
    if s["residual"] is not None:
        y = y + s["residual"][:s["used"]].double()
    return {"y": torch.cat([y, y.new_zeros((len(s["a"]) - s["used"], y.shape[1]))])}


def _exact_act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    return z.clamp(min=0.0) if name == "relu" else z


def _exact_weights(s, case):
    """Weights of the chosen experts, ranked by (key, lower index) row by row
    over numpy's 64-bit scores."""
    l = s["logits"].double().cpu().numpy()
    T, E = l.shape
    k, G = case["k"], case["n_group"]
    with np.errstate(all="ignore"):
        if case["score"] == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-l))
        else:
            p = np.exp(l - l.max(axis=1, keepdims=True))
            p = np.nan_to_num(p / p.sum(axis=1, keepdims=True))
    key = p.astype(np.float32)
    if s["bias"] is not None:
        key = key + s["bias"].cpu().numpy()
    key[np.isneginf(l)] = -np.inf
    if G > 1:
        per = np.sort(key.reshape(T, G, E // G), axis=2)[:, :, ::-1][:, :, :case["group_top"]]
        rank = np.where(np.isneginf(per), np.float32(0), per).sum(axis=2, dtype=np.float32)
        rank[np.isneginf(per[:, :, 0])] = -np.inf
        late = np.argsort(-rank, axis=1, kind="stable")[:, case["topk_group"]:]
        key.reshape(T, G, E // G)[np.arange(T)[:, None], late] = -np.inf
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, idx, 1)
    w[np.isneginf(np.take_along_axis(key, idx, 1))] = 0.0
    total = w.sum(axis=1, keepdims=True)
    return torch.from_numpy(2.5 * w / np.where(total > 0, total, 1.0))
