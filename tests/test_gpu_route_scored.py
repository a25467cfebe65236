"""moe_route_scored against a plain implementation in 64 bits (numpy): the
choice exactly, the weights within their derived tolerance.

The scores are fp32 roundings of the 64-bit scores; the choice is then exact
fp32 arithmetic on both sides (one addition of the bias, one addition of the
two best keys of a group), so the indices have to be equal, ties included.

Weights: w = scale * s / sum. s is within half a unit (2^-24 relative) of the
64-bit score, the fp32 sum of k terms adds at most (k - 1) 2^-24 relative
(all terms are positive), its terms half a unit, the division and the product
with scale half a unit each: relative (k + 4) 2^-24. Scores below the normal
range (2^-126) are off by up to half the spacing there, 2^-150 absolute,
before the division: 2^-150 k scale / sum more.
"""
import numpy as np
import pytest
import torch

from parity_util import log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def plain(logits, k, score="sigmoid", bias=None, n_group=1, topk_group=1, group_top=2,
          renorm=True, scale=1.0, n_shared=0, shared_w=1.0):
    """(idx [T, k+n_shared], w64, the sum of the chosen scores) for float64 logits."""
    l = np.array(logits, np.float64)
    T, E = l.shape
    l[np.isnan(l)] = -np.inf
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s64 = 1.0 / (1.0 + np.exp(-l))
        else:
            l = np.minimum(l, np.finfo(np.float32).max)
            p = np.exp(l - l.max(axis=1, keepdims=True))
            p[np.isneginf(l)] = 0.0
            tot = p.sum(axis=1, keepdims=True)
            s64 = np.where(tot > 0, p / np.where(tot > 0, tot, 1.0), 0.0)
        key = s64.astype(np.float32)
        if bias is not None:
            key = key + np.asarray(bias, np.float32)
        key[np.isneginf(l) | np.isnan(key)] = -np.inf
        per = E // n_group
        out = np.full((T, k + n_shared), -1, np.int32)
        w = np.zeros((T, k + n_shared))
        total = np.zeros(T)
        for t in range(T):
            groups = key[t].reshape(n_group, per)
            rank = []
            for g in range(n_group):
                best = np.sort(groups[g])[::-1][:group_top]
                live = best[~np.isneginf(best)]
                if len(live):
                    rank.append((-np.sum(live, dtype=np.float32), g))
            kept = {g for _, g in sorted(rank)[:topk_group]}
            cand = [(-key[t, e], e) for e in range(E)
                    if e // per in kept and not np.isneginf(key[t, e])]
            pick = [e for _, e in sorted(cand)[:k]]
            out[t, :len(pick)] = pick
            sc = s64[t, pick]
            total[t] = sc.sum()
            if renorm:
                sc = sc / total[t] if np.float32(total[t]) > 0 else 0.0 * sc
            w[t, :len(pick)] = sc * scale
            out[t, k:] = E + np.arange(n_shared)
            w[t, k:] = shared_w
    return out, w, total


def check(logits, k, **kw):
    """logits: a GPU tensor (any row stride)."""
    from combine_moe_route_amd import moe_route_scored
    bias = kw.pop("bias", None)
    idx, w = moe_route_scored(logits, k, bias=None if bias is None else torch.tensor(bias).to(DEV),
                              **kw)
    torch.cuda.synchronize()
    ri, rw, total = plain(logits.double().cpu().numpy(), k, bias=bias, **kw)
    gi, gw = idx.cpu().numpy(), w.double().cpu().numpy()
    bad = np.argwhere(gi != ri)
    assert not len(bad), f"{len(bad)} indices differ, first {bad[0]}: {gi[bad[0][0]]} {ri[bad[0][0]]}"
    scale = kw.get("scale", 1.0)
    div = np.maximum(total, 1e-300) if kw.get("renorm", True) else np.ones_like(total)
    tol = (k + 4) * 2.0 ** -24 * np.abs(rw) + \
        ((k + 1) * abs(scale) * 2.0 ** -150 / div)[:, None] + 2.0 ** -149
    tol = np.where(total[:, None] < 2.0 ** -140, np.maximum(tol, abs(scale)), tol)
    err = np.abs(gw - rw)
    assert np.all(err <= tol), f"weights off: {np.max(err / tol)} of the tolerance"
    return idx, w


def logits_of(T, E, seed, dtype=torch.float32, spread=1.0, masked=0.0, pad=0):
    rng = np.random.default_rng([77, seed])
    x = (spread * rng.standard_normal((T, E + pad))).astype(np.float32)
    if masked:
        x[rng.random(x.shape) < masked] = -np.inf
        x[rng.random(T) < masked] = -np.inf
    return torch.from_numpy(x).to(DEV, dtype)[:, :E]


def bias_of(E, seed, spread=0.05):
    return (spread * np.random.default_rng([78, seed]).standard_normal(E)).astype(np.float32)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,G,KG,top", [
    (1, 256, 8, 8, 4, 2), (3, 1, 1, 1, 1, 1), (70, 8, 2, 1, 1, 2), (33, 64, 6, 8, 3, 1),
    (129, 160, 6, 8, 3, 1), (65, 384, 8, 1, 1, 2), (17, 1024, 8, 16, 5, 2), (9, 1024, 64, 4, 3, 2),
    (5, 300, 100, 3, 2, 1), (31, 30, 5, 5, 2, 2), (31, 30, 4, 30, 7, 2), (2, 1024, 1024, 1, 1, 1),
    (40, 12, 3, 4, 2, 2), (64, 128, 8, 4, 2, 2), (200, 96, 7, 6, 3, 2), (257, 256, 8, 2, 1, 2),
    (50, 1000, 3, 8, 2, 2), (11, 768, 8, 16, 16, 2), (37, 256, 16, 32, 8, 2), (90, 512, 10, 1, 1, 2),
])
def test_shapes(score, T, E, k, G, KG, top):
    log(f"route_scored {score} T={T} E={E} k={k} G={G}/{KG} top={top}")
    for dtype, pad, seed in ((torch.float32, 0, 1), (torch.bfloat16, 0, 2), (torch.float32, 3, 3),
                             (torch.bfloat16, 1, 4)):
        l = logits_of(T, E, seed, dtype, pad=pad)
        check(l, k, score=score, bias=bias_of(E, seed), n_group=G, topk_group=KG, group_top=top,
              scale=2.5)
        check(l, k, score=score, n_group=G, topk_group=KG, group_top=top, renorm=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,KG", [(256, 8, 8, 4), (384, 8, 1, 1), (60, 9, 5, 2), (1024, 12, 1, 1)])
def test_masked_experts_and_rows(score, E, k, G, KG):
    """Masks of -inf that leave few experts, or none; NaN counts as masked."""
    log(f"masked {score} E={E}")
    T = 80
    for masked in (0.3, 0.97):
        l = logits_of(T, E, 5, masked=masked)
        l[3, :] = float("nan")
        l[4, 1::2] = float("nan")
        l[5, :] = -float("inf")
        l[5, E - 1] = 0.25
        idx, w = check(l, k, score=score, n_group=G, topk_group=KG, bias=bias_of(E, 6))
        assert (idx[3] == -1).all() and (w[3] == 0).all()
        assert idx[5, 0] == E - 1 and w[5, 0] == 1.0 and (idx[5, 1:] == -1).all()
    # a bias of -inf takes an expert out for every token
    b = bias_of(E, 7)
    b[::3] = -np.inf
    b[1] = np.nan
    idx, _ = check(logits_of(T, E, 8), k, score=score, n_group=G, topk_group=KG, bias=b)
    idx = idx.cpu().numpy()
    assert not ((idx % 3 == 0) & (idx >= 0)).any() and not (idx == 1).any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,KG", [(64, 8, 8, 4), (48, 4, 1, 1), (40, 9, 4, 2)])
def test_ties_and_extremes(score, E, k, G, KG):
    """Equal keys and groups go to the lower index; saturated scores, the
    type's lowest value, +inf, subnormal scores."""
    log(f"ties {score} E={E}")
    T = 40
    rng = np.random.default_rng(9)
    x = rng.integers(-1, 2, (T, E)).astype(np.float32)      # many ties
    x[1] = 0.0
    x[2, ::2] = -0.0
    x[3] = np.finfo(np.float32).min
    x[4] = 40.0 + np.arange(E)                              # sigmoid rounds to 1
    x[5] = -80.0 - 0.5 * np.arange(E)                       # scores down to subnormal
    x[6, 7] = np.inf
    x[7, :] = np.inf
    x[8] = np.finfo(np.float32).max
    for dtype in (torch.float32, torch.bfloat16):
        l = torch.from_numpy(x).to(DEV, dtype)
        for bias in (None, np.zeros(E, np.float32), -np.ones(E, np.float32)):
            check(l, k, score=score, n_group=G, topk_group=KG, bias=bias)


def test_close_scores():
    """Neighbours a few fp32 units apart: a score one unit off would change
    the choice."""
    log("close scores")
    T, E, k = 2000, 256, 8
    rng = np.random.default_rng(10)
    x = (0.5 + 1e-5 * rng.standard_normal((T, E))).astype(np.float32)
    l = torch.from_numpy(x).to(DEV)
    check(l, k, n_group=8, topk_group=4, bias=bias_of(E, 11, 1e-6))
    check(l, k, score="softmax", n_group=8, topk_group=4)


def test_shared_slots_and_given_outputs():
    log("shared slots")
    T, E, k = 50, 64, 6
    l = logits_of(T, E, 12)
    check(l, k, n_shared=2, shared_w=0.75, n_group=4, topk_group=2)
    from combine_moe_route_amd import moe_route_scored
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -7.0, device=DEV)
    got = moe_route_scored(l, k, topk_idx=idx, topk_w=w)
    assert got[0] is idx and got[1] is w
    ref = moe_route_scored(l, k)
    assert torch.equal(idx, ref[0]) and torch.equal(w, ref[1])
    e = moe_route_scored(l[:0], k)
    assert e[0].shape == (0, k)


@pytest.mark.parametrize("T,E,k,G,KG,top", [
    (9, 1024, 8, 1024, 100, 1), (7, 1000, 5, 500, 50, 2), (6, 1023, 9, 3, 2, 2), (4, 1024, 70, 2, 1, 2),
    (2100, 512, 8, 2, 1, 2), (2100, 1024, 4, 2, 1, 2), (2050, 40, 20, 5, 4, 1), (2048, 250, 8, 1, 1, 2),
    (3, 1024, 64, 1, 1, 2), (5, 1021, 33, 1, 1, 2), (2100, 12, 9, 2, 1, 2), (2060, 257, 12, 1, 1, 1),
    # the sorted kernel with 8, 16, 32 and 64 lanes per token, with groups and without
    (16400, 100, 5, 5, 3, 2), (8200, 256, 8, 8, 4, 2), (8300, 240, 8, 10, 4, 1), (4100, 512, 7, 2, 1, 2),
    (2100, 1024, 8, 16, 5, 2), (2200, 1000, 3, 1, 1, 1), (8200, 70, 8, 1, 1, 1), (2050, 510, 1, 1, 1, 1),
])
def test_many_groups_wide_groups_and_both_kernels(T, E, k, G, KG, top):
    """Groups of one expert, groups wider than the lanes, odd widths, k past the
    lanes; batches on either side of the switch to fewer lanes per token."""
    if k > KG * (E // G):
        k = KG * (E // G)
    log(f"groups T={T} E={E} k={k} G={G}/{KG}")
    rows = min(T, 40)
    from combine_moe_route_amd import moe_route_scored
    for score, dtype in (("sigmoid", torch.float32), ("softmax", torch.bfloat16)):
        l = logits_of(T, E, 20, dtype, masked=0.1)
        kw = dict(score=score, n_group=G, topk_group=KG, group_top=top)
        idx, w = moe_route_scored(l, k, bias=torch.tensor(bias_of(E, 21), device=DEV), **kw)
        pick = torch.linspace(0, T - 1, rows).long()
        ri, rw, total = plain(l[pick.to(DEV)].double().cpu().numpy(), k, bias=bias_of(E, 21), **kw)
        assert np.array_equal(idx.cpu().numpy()[pick], ri)
        err = np.abs(w.double().cpu().numpy()[pick] - rw)
        assert np.all(err <= (k + 4) * 2.0 ** -24 * np.abs(rw) + 2.0 ** -149)


def test_large_batch_strided_and_row_sample():
    """A prefill batch whose row offsets pass 2^31 bytes; rows sampled."""
    log("large strided")
    from combine_moe_route_amd import moe_route_scored
    T, E, k, ld = 16384, 256, 8, 40000
    base = torch.empty((T, ld), device=DEV)
    base[:, 100:100 + E] = torch.randn((T, E), device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    l = base[:, 100:100 + E]
    idx, w = moe_route_scored(l, k, bias=torch.tensor(bias_of(E, 13), device=DEV), n_group=8,
                              topk_group=4)
    for t in (0, 1, 8191, 13421, 13422, T - 1):
        ri, rw, _ = plain(l[t:t + 1].double().cpu().numpy(), k, bias=bias_of(E, 13), n_group=8,
                          topk_group=4)
        assert np.array_equal(idx[t:t + 1].cpu().numpy(), ri)
        assert np.allclose(w[t:t + 1].double().cpu().numpy(), rw, rtol=(k + 4) * 2.0 ** -24, atol=0)


def test_python_refusals():
    from combine_moe_route_amd import MoeRouteError, moe_route_scored
    l = logits_of(4, 64, 0)
    with pytest.raises(TypeError):
        moe_route_scored(l.half(), 4)
    with pytest.raises(TypeError):
        moe_route_scored(l.cpu(), 4)
    with pytest.raises(ValueError):
        moe_route_scored(l, 4, score="tanh")
    with pytest.raises(ValueError):
        moe_route_scored(l.t(), 2)
    with pytest.raises(ValueError):
        moe_route_scored(l[0].expand(4, 64), 2)          # rows on top of each other
    with pytest.raises(TypeError):
        moe_route_scored(l, 4, bias=torch.zeros(64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        moe_route_scored(l, 4, bias=torch.zeros(63, device=DEV))
    for kw in (dict(k=0), dict(k=65), dict(k=4, n_group=7), dict(k=33, n_group=4, topk_group=2),
               dict(k=4, n_group=4, topk_group=5), dict(k=4, group_top=3),
               dict(k=4, n_shared=961)):
        with pytest.raises((MoeRouteError, RuntimeError)):
            moe_route_scored(l, **kw)
