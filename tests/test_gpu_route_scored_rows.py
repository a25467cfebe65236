"""moe_route_scored: outputs between strided rows."""
import pytest
import torch

from parity_util import log
from test_gpu_route_scored import DEV, logits_of

pytestmark = pytest.mark.gpu


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
