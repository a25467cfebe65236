"""moe_dispatch_quantized against the CPU oracle: the layout of the oracle's
bf16 dispatch of the same bytes, codes and scales copied bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from parity_util import log

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def routing(T, E, k, seed, dropped=0.0):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)) + 0.3 * rng.random(E), axis=1)[:, :k].astype(np.int32)
    if dropped:
        idx[rng.random((T, k)) < dropped] = -1
    return idx


def check(T, H, S, E, k, groups=1, align=1, seed=0, dropped=0.0, dtype=torch.int8):
    from combine_moe_route_amd import alloc_dispatch_quantized, moe_dispatch_quantized
    log(f"dispatch_quantized T={T} H={H} S={S} E={E} k={k} groups={groups} align={align}")
    rng = np.random.default_rng([seed, T, H])
    codes = rng.integers(0, 256, (T, H), dtype=np.uint8)
    scales = rng.random((T, max(S, 1)), dtype=np.float32) + 0.01
    if T > 2:
        scales[2] = np.nan                           # carried as it is
    idx = routing(T, E, k, seed, dropped)
    x = torch.from_numpy(codes).to(DEV).view(dtype)
    xs = torch.from_numpy(scales).to(DEV)
    if S == 0:                                       # one scale a token, as a vector
        xs = xs[:, 0].contiguous()
    b = alloc_dispatch_quantized(T, H, E, k, groups, align, dtype, None if S == 0 else S, DEV)
    b.out.view(torch.uint8).fill_(0x77)
    b.out_scales.fill_(-5.0)
    b.row_src.fill_(-9)
    got = moe_dispatch_quantized(x, xs, torch.from_numpy(idx).to(DEV), E, groups, align, bufs=b)
    assert got is b
    torch.cuda.synchronize()
    ref = oracle.dispatch(codes.view(np.uint16), idx, E, groups, align, False)
    R = ref.num_rows
    c = lambda t: t.cpu().numpy()  # noqa: E731
    assert np.array_equal(c(b.expert_counts), ref.expert_counts)
    assert np.array_equal(c(b.expert_offsets), ref.expert_offsets)
    assert np.array_equal(c(b.group_offsets), ref.group_offsets)
    assert np.array_equal(c(b.dst_row), ref.dst_row)
    assert np.array_equal(c(b.row_src[:R]), ref.row_src)
    assert np.array_equal(c(b.out[:R].view(torch.uint8)).view(np.uint16), ref.out)
    src = ref.row_src
    want = np.where((src >= 0)[:, None], scales[np.maximum(src, 0) // k], np.float32(0))
    assert np.array_equal(c(b.out_scales[:R]).reshape(want.shape), want, equal_nan=True)
    # rows behind the last segment stay as they were
    assert (b.out[R:].view(torch.uint8) == 0x77).all() and (b.out_scales[R:] == -5.0).all()
    assert (b.row_src[R:] == -9).all()
    return b


@pytest.mark.parametrize("T,H,S,E,k,groups,align", [
    (1, 16, 0, 1, 1, 1, 1), (1, 7168, 0, 256, 8, 1, 1), (3, 32, 1, 8, 2, 2, 4),
    (128, 7168, 0, 256, 8, 32, 1), (128, 1408, 11, 60, 6, 1, 16), (77, 1040, 0, 5, 3, 5, 7),
    (200, 128, 128, 4, 4, 1, 1), (300, 9216, 72, 16, 2, 1, 128), (1000, 48, 3, 1024, 4, 1, 1),
    (4097, 512, 4, 64, 8, 8, 1), (5000, 256, 0, 300, 12, 1, 3), (2, 65536, 512, 8, 2, 1, 1),
    (20000, 64, 0, 256, 8, 1, 128), (65, 2048, 0, 1, 1, 1, 1024),
])
def test_layout(T, H, S, E, k, groups, align):
    check(T, H, S, E, k, groups, align)


@pytest.mark.parametrize("T,H,S,E,k,groups,align", [
    (32, 16, 0, 1024, 1024, 1, 1), (33, 16, 1, 1000, 1000, 4, 2), (32768, 16, 0, 1, 1, 1, 1),
    (32769, 16, 0, 1, 1, 1, 1), (16384, 32, 2, 3, 2, 3, 8), (16385, 32, 2, 3, 2, 3, 8),
    (4096, 48, 0, 8, 8, 1, 5), (1500, 1040, 3, 2, 2, 1, 100), (1024, 64, 0, 64, 64, 1, 1),
    (7, 16, 0, 1024, 3, 1, 1024),
])
def test_around_the_limit_of_one_launch(T, H, S, E, k, groups, align):
    """32768 slots and a few more; many slots a token; experts that every token
    chooses."""
    check(T, H, S, E, k, groups, align)


@pytest.mark.parametrize("T", [90, 5000])
def test_one_hot_expert_and_unaligned_table(T):
    """Every token's first choice is the same expert; the table starts at an odd
    element, and ids out of range of either sign are dropped."""
    from combine_moe_route_amd import moe_dispatch_quantized
    log(f"dispatch_quantized hot T={T}")
    idx = routing(T, 30, 3, 5) + 1
    idx[:, 0] = 0
    idx[5, 1], idx[6, 2], idx[7, 0] = 31, -2 ** 31, 2 ** 31 - 1
    flat = torch.zeros(3 * T + 1, dtype=torch.int32, device=DEV)
    flat[1:] = torch.from_numpy(idx.reshape(-1)).to(DEV)
    codes = np.random.default_rng(1).integers(0, 256, (T, 32), dtype=np.uint8)
    b = moe_dispatch_quantized(torch.from_numpy(codes).to(DEV), torch.ones(T, device=DEV),
                               flat[1:].view(T, 3), 31, 1, 4)
    ref = oracle.dispatch(codes.view(np.uint16), idx, 31, 1, 4, False)
    R = ref.num_rows
    assert np.array_equal(b.dst_row.cpu().numpy(), ref.dst_row)
    assert np.array_equal(b.row_src[:R].cpu().numpy(), ref.row_src)
    assert np.array_equal(b.out[:R].cpu().numpy().view(np.uint16), ref.out)
    assert np.array_equal(b.expert_counts.cpu().numpy(), ref.expert_counts)


def test_dropped_slots_and_bytes():
    check(500, 96, 3, 12, 4, align=8, seed=1, dropped=0.3)
    check(40, 96, 0, 12, 4, align=1, seed=2, dropped=1.0)
    check(600, 128, 1, 8, 2, seed=3, dtype=torch.uint8)


def test_same_as_the_copying_dispatch_and_no_tokens():
    """The tables are those of moe_dispatch; an empty batch writes zero counts."""
    from combine_moe_route_amd import moe_dispatch, moe_dispatch_quantized
    log("dispatch_quantized tables")
    T, H, E, k = 700, 256, 40, 5
    idx = torch.from_numpy(routing(T, E, k, 7, 0.1)).to(DEV)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    d = moe_dispatch(x, idx, E, 4, 16)
    bytes_ = x.view(torch.uint8)                     # [T, 2 H]
    q = moe_dispatch_quantized(bytes_, torch.ones(T, device=DEV), idx, E, 4, 16)
    R = int(d.expert_offsets[-1])
    assert torch.equal(q.out[:R].view(torch.bfloat16).view(torch.int16), d.out[:R].view(torch.int16))
    for a, b in ((q.dst_row, d.dst_row), (q.expert_offsets, d.expert_offsets),
                 (q.expert_counts, d.expert_counts), (q.row_src[:R], d.row_src[:R])):
        assert torch.equal(a, b)
    assert torch.equal(q.out_scales[:R] == 1, q.row_src[:R] >= 0)
    e = moe_dispatch_quantized(bytes_[:0], torch.ones(0, device=DEV), idx[:0], E, 1, 16)
    assert (e.expert_counts == 0).all() and (e.expert_offsets == 0).all()


def test_rows_past_32_bit_offsets():
    """Rows that start beyond 2^32 bytes, on the sending and the receiving side."""
    from combine_moe_route_amd import moe_dispatch_quantized
    log("dispatch_quantized large")
    T, H = 700_000, 7168
    x = torch.empty((T, H), dtype=torch.int8, device=DEV)
    x.view(torch.int32).random_()
    xs = torch.rand(T, device=DEV)
    idx = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    idx[::2] = 1
    b = moe_dispatch_quantized(x, xs, idx, 2)
    odd = torch.arange(T - 2001, T, 2, device=DEV)   # expert 0: odd tokens, in order
    even = odd[1:] - 1
    n0 = T // 2
    assert torch.equal(b.out[n0 - len(odd):n0], x[odd]) and torch.equal(b.out_scales[n0 - len(odd):n0], xs[odd])
    assert torch.equal(b.out[T - len(even):], x[even]) and torch.equal(b.out_scales[T - len(even):], xs[even])


def test_python_refusals():
    from combine_moe_route_amd import MoeRouteError, alloc_dispatch_quantized, moe_dispatch_quantized
    x = torch.zeros((4, 64), dtype=torch.int8, device=DEV)
    xs = torch.zeros(4, device=DEV)
    idx = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        moe_dispatch_quantized(x.float(), xs, idx, 2)
    with pytest.raises(ValueError):
        moe_dispatch_quantized(x[0], xs, idx, 2)
    with pytest.raises(ValueError):
        moe_dispatch_quantized(x, xs[:3].contiguous(), idx, 2)
    with pytest.raises(TypeError):
        moe_dispatch_quantized(x, xs.double(), idx, 2)
    with pytest.raises(TypeError):
        moe_dispatch_quantized(x, xs, idx.long(), 2)
    with pytest.raises(ValueError):
        moe_dispatch_quantized(x, xs, idx[:3].contiguous(), 2)
    with pytest.raises(ValueError):                  # scales of another form
        moe_dispatch_quantized(x, xs, idx, 2,
                               bufs=alloc_dispatch_quantized(4, 64, 2, 2, scales=1, device=DEV))
    with pytest.raises(TypeError):                   # codes of another type
        moe_dispatch_quantized(x, xs, idx, 2,
                               bufs=alloc_dispatch_quantized(4, 64, 2, 2, dtype=torch.uint8, device=DEV))
    with pytest.raises(MoeRouteError):
        moe_dispatch_quantized(x[:, :40].contiguous(), xs, idx, 2)
    b = alloc_dispatch_quantized(4, 64, 2, 2, device=DEV)
    with pytest.raises(MoeRouteError):
        moe_dispatch_quantized(b.out[:4], xs, idx, 2, bufs=b)
