"""moe_route_scored on the shapes that one wave works through row by row: wide
groups that the chunk layout has no room for, at large batches too, and rows
far apart; and bits that repeat. Choice and tolerance as in
test_gpu_route_scored.py."""
import numpy as np
import pytest
import torch

from parity_util import log
from test_gpu_route_scored import DEV, bias_of, check, logits_of, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,G,KG,top", [
    (3, 64, 6, 1, 1, 2), (1, 8, 2, 1, 1, 1), (2, 64, 4, 8, 3, 2), (4, 40, 40, 1, 1, 2),
    (2, 200, 8, 8, 4, 2), (3, 1000, 9, 8, 2, 1),
])
def test_rows_far_apart(score, dtype, T, E, k, G, KG, top):
    """Rows more than 2^20 elements apart, from 8 to 1000 experts."""
    log(f"route far apart {score} {dtype} T={T} E={E} k={k} G={G}/{KG}")
    ld = 2 ** 20 + 8
    base = torch.full((T, ld), float("nan"), device=DEV, dtype=dtype)
    base[:, 3:3 + E] = logits_of(T, E, E + T, dtype, masked=0.1 if T > 2 else 0.0)
    check(base[:, 3:3 + E], k, score=score, bias=bias_of(E, 1), n_group=G, topk_group=KG,
          group_top=top, scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,G,KG,top", [
    (1, 1000, 8, 5, 3, 2), (2100, 1000, 8, 5, 3, 2), (5000, 645, 6, 5, 2, 1), (2048, 1020, 12, 5, 4, 2),
    (300, 1023, 3, 11, 4, 2), (2100, 700, 70, 4, 2, 2), (3000, 130, 65, 1, 1, 2),
])
def test_wide_groups(score, T, E, k, G, KG, top):
    """Five groups of 129 to 204 experts and k above 64, small and large batches."""
    log(f"route wide groups {score} T={T} E={E} k={k} G={G}/{KG}")
    from combine_moe_route_amd import moe_route_scored
    l = logits_of(T, E, 30, masked=0.05)
    kw = dict(score=score, n_group=G, topk_group=KG, group_top=top)
    b = bias_of(E, 31)
    idx, w = moe_route_scored(l, k, bias=torch.tensor(b, device=DEV), **kw)
    pick = torch.unique(torch.linspace(0, T - 1, min(T, 40)).long())
    ri, rw, _ = plain(l[pick.to(DEV)].double().cpu().numpy(), k, bias=b, **kw)
    assert np.array_equal(idx.cpu().numpy()[pick.numpy()], ri)
    err = np.abs(w.double().cpu().numpy()[pick.numpy()] - rw)
    assert np.all(err <= (k + 4) * 2.0 ** -24 * np.abs(rw) + 2.0 ** -149)
    for _ in range(2):
        i2, w2 = moe_route_scored(l, k, bias=torch.tensor(b, device=DEV), **kw)
        assert torch.equal(idx, i2) and torch.equal(w, w2)


def test_outputs_between_the_rows():
    """Outputs in the gaps between the rows of logits overlap none of them."""
    log("route outputs in gaps")
    from combine_moe_route_amd import MoeRouteError, moe_route_scored
    T, E, k, ld = 50, 64, 6, 1000
    base = torch.zeros((T, ld), device=DEV)
    base[:, :E] = logits_of(T, E, 40)
    want = moe_route_scored(base[:, :E], k)
    flat = base.view(-1)
    idx = flat[E:E + T * k].view(torch.int32).view(T, k)                     # behind row 0
    w = flat[2 * ld - T * k:2 * ld].view(T, k)                               # before row 2
    moe_route_scored(base[:, :E], k, topk_idx=idx, topk_w=w)
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    for at in (E - 1, 2 * ld - T * k + 1, T * ld - ld, 3 * ld + 5):
        with pytest.raises(MoeRouteError):
            moe_route_scored(base[:, :E], k, topk_w=flat[at:at + T * k].view(T, k))
