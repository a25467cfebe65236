"""Which launches moe_dispatch_quantized makes, by the launch log (MOE_ROUTE_LOG=1, read
in a child process), on both sides of the border between one launch and several; each
call's tables and rows are the oracle's."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from parity_util import log
from test_gpu_dispatch_quantized import DEV

pytestmark = pytest.mark.gpu

ONE, TWO, THREE = ["count+scan+scatter"], ["count", "scan+scatter"], ["count", "scan", "scatter"]

# T, H, S, E, k, groups, align -> launches
PLANS = [
    ((4096, 16, 0, 1, 1, 1, 1), ONE),                # 4096 slots an expert, one choice a token
    ((4097, 16, 0, 1, 1, 1, 1), THREE),
    ((32768, 16, 0, 8, 1, 1, 1), ONE),
    ((32768, 16, 0, 7, 1, 1, 4), THREE),
    ((32769, 16, 0, 9, 1, 1, 1), THREE),             # more than 32768 slots
    ((2048, 32, 2, 2, 2, 1, 8), ONE),                # 2048 an expert, more choices
    ((2049, 32, 2, 2, 2, 1, 8), THREE),             # 65 tiles of 32 tokens
    ((16384, 32, 2, 16, 2, 4, 8), ONE),
    ((16384, 32, 2, 15, 2, 3, 8), THREE),
    ((4096, 48, 0, 16, 8, 1, 5), ONE),
    ((4096, 48, 0, 8, 8, 1, 5), THREE),
    ((2000, 1040, 3, 40, 16, 1, 100), ONE),
    ((2000, 64, 3, 40, 17, 1, 100), TWO),            # at most 64 tiles
    ((32, 16, 0, 1024, 1024, 1, 1), ONE),
    ((1, 7168, 0, 1, 1, 1, 1), ONE),
]


def test_launches_on_both_sides_of_the_border():
    log("dispatch_quantized plan")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.path.insert(0, 'tests')\n"
            "from test_gpu_dispatch_quantized import check\n"
            f"for case in {[c for c, _ in PLANS]!r}:\n"
            "    print('@', file=sys.stderr, flush=True)\n"
            "    check(*case)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=110, env=dict(os.environ, MOE_ROUTE_LOG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = [re.findall(r"\[moe_route\] (\S+)", part) for part in r.stderr.split("@\n")[1:]]
    assert got == [want for _, want in PLANS]


@pytest.mark.parametrize("T,E,k", [(32768, 8, 1), (30000, 300, 1), (8000, 31, 4)])
def test_every_slot_to_one_expert(T, E, k):
    """One launch, and one counter that takes every token."""
    from combine_moe_route_amd import moe_dispatch_quantized
    log(f"dispatch_quantized one expert T={T}")
    idx = np.full((T, k), -1, np.int32)
    idx[:, k - 1] = E - 1
    codes = np.random.default_rng(T).integers(0, 256, (T, 16), dtype=np.uint8)
    b = moe_dispatch_quantized(torch.from_numpy(codes).to(DEV), torch.ones(T, device=DEV),
                               torch.from_numpy(idx).to(DEV), E, 1, 3)
    ref = oracle.dispatch(codes.view(np.uint16), idx, E, 1, 3, False)
    R = ref.num_rows
    assert np.array_equal(b.dst_row.cpu().numpy(), ref.dst_row)
    assert np.array_equal(b.row_src[:R].cpu().numpy(), ref.row_src)
    assert np.array_equal(b.expert_counts.cpu().numpy(), ref.expert_counts)
    assert np.array_equal(b.expert_offsets.cpu().numpy(), ref.expert_offsets)
    assert np.array_equal(b.out[:R].cpu().numpy().view(np.uint16), ref.out)
