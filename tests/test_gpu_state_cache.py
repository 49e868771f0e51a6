"""The 8-bit state cache against its definition in float64 on the CPU: every
code is the nearest one (ties to even), the scale is max|v| / q to one float32
rounding, values read back as code * scale exactly."""

import pytest
import torch

from selective_state_space_amd import ssd

from _gpu import log

pytestmark = pytest.mark.gpu

Q = {"int8": 127.0, "fp8": 448.0}
DT = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
U = 2.0 ** -24


def pool_of(num, size, fmt, fill=3):
    codes = torch.full((num, size), fill, dtype=torch.int8).view(DT[fmt]).cuda()
    scales = torch.full((num, -(-size // 64)), 0.5).cuda()
    return codes, scales


def nearest(v, amax, fmt):
    """The code's value nearest to v q / amax in float64, ties to even."""
    u = v.double() * Q[fmt] / amax.double()
    if fmt == "int8":
        return u.round()
    shift = 4 - torch.frexp(u)[1].clamp(min=-5)
    return torch.ldexp(torch.ldexp(u, shift).round(), -shift)


def blocks(state):
    n, size = state.shape
    pad = -size % 64
    return torch.nn.functional.pad(state, (0, pad)).view(n, -1, 64)


def check_rows(state, codes, scales, fmt):
    """Stored rows of `state` (CPU, finite), already gathered from the pool."""
    b = blocks(state)
    amax = b.abs().amax(-1)
    live = amax >= 2.0 ** -100
    ref_scale = torch.where(live, amax.double() / Q[fmt], torch.zeros_like(amax).double())
    assert ((scales.double() - ref_scale).abs() <= U * ref_scale).all()
    safe = torch.where(live, amax, torch.ones_like(amax))
    want = torch.where(live[..., None], nearest(b, safe[..., None], fmt), torch.zeros(()).double())
    got = blocks(codes.float()).double()
    assert torch.equal(got, want)


def values(codes, scales, size):
    """code * scale in float32: the one rounding that reading makes."""
    return (blocks(codes.float()) * scales[..., None]).view(codes.shape[0], -1)[:, :size]


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("n,num,size", [(1, 1, 8), (2, 3, 64), (3, 9, 72), (5, 8, 4096 + 8),
                                        (4, 6, 40960), (2, 2, 515 * 16)])
def test_round_trip(fmt, n, num, size):
    log("state cache", fmt, n, num, size)
    g = torch.Generator().manual_seed(size)
    nblk = -(-size // 64)
    state = torch.randn(n, size, generator=g)
    state *= torch.exp(3 * torch.randn(n, nblk, generator=g)).repeat_interleave(64, 1)[:, :size]
    slots = torch.randperm(num, generator=g)[:n].to(torch.int32)
    codes, scales = pool_of(num, size, fmt)
    c0, s0 = codes.view(torch.int8).cpu().clone(), scales.cpu().clone()
    ssd.ssd_cache_write(state.cuda(), codes, scales, slots.cuda())
    idx = slots.long()
    hc, hs = codes.cpu(), scales.cpu()
    check_rows(state, hc.view(torch.int8)[idx].view(DT[fmt]), hs[idx], fmt)
    rest = torch.ones(num, dtype=torch.bool)
    rest[idx] = False
    assert torch.equal(hc.view(torch.int8)[rest], c0[rest]) and torch.equal(hs[rest], s0[rest])
    # read: every slot twice, a slot below and one past the pool
    order = torch.cat([slots, slots.flip(0), torch.tensor([-1, num], dtype=torch.int32)])
    back = ssd.ssd_cache_read(codes, scales, order.cuda()).cpu()
    row = values(hc.view(torch.int8)[idx].view(DT[fmt]), hs[idx], size)
    assert torch.equal(back[:n], row) and torch.equal(back[n:2 * n], row.flip(0))
    assert not back[2 * n:].any()


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_values_at_the_borders(fmt):
    """Ties and their float32 neighbours: v = (k + 1/2) amax / q for every code border."""
    if fmt == "int8":
        mids = torch.arange(0, 127).double() + 0.5
        amax = torch.tensor([127.0, 1.0, 0.37, 3e20])
    else:
        codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        mids = (codes[1:] + codes[:-1]) / 2
        mids = torch.cat([mids, mids[-1:]])
        amax = torch.tensor([448.0, 1.0, 0.37, 3e20])
    rows = []
    for a in amax:
        v = (mids * a.double() / Q[fmt]).float()
        inf = torch.tensor(float("inf"))
        for w in (v, torch.nextafter(v, inf), torch.nextafter(v, -inf), -v):
            for half in (w[:63], w[63:126]):
                rows.append(torch.cat([half, a[None]]))
    state = torch.stack(rows)
    codes, scales = pool_of(state.shape[0], 64, fmt)
    ssd.ssd_cache_write(state.cuda(), codes, scales)
    check_rows(state, codes.cpu(), scales.cpu(), fmt)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_empty_tiny_and_not_finite_blocks(fmt):
    size = 6 * 64
    state = torch.randn(2, size, generator=torch.Generator().manual_seed(1))
    state[0, 0:64] = 0.0
    state[0, 64:128] = 2.0 ** -101       # below the smallest block kept
    state[0, 128:192] *= 2.0 ** -90
    state[0, 200] = float("inf")
    state[0, 300] = float("nan")
    state[0, 383] = -float("inf")
    state[1, 5] = 3e38                   # q / max underflows no code
    codes, scales = pool_of(2, size, fmt)
    ssd.ssd_cache_write(state.cuda(), codes, scales)
    back = ssd.ssd_cache_read(codes, scales, shape=(6, 64)).cpu()
    assert back.shape == (2, 6, 64)
    assert not back[0, :2].any()
    assert back[0, 3:].isnan().all()
    assert back[0, 2].isfinite().all() and back[1].isfinite().all()
    keep = torch.cat([state[0, 128:192], state[1]]).view(7, 64)
    check_rows(keep, torch.cat([codes.cpu().view(torch.int8)[0, 128:192],
                                codes.cpu().view(torch.int8)[1]]).view(DT[fmt]).view(7, 64),
               torch.cat([scales.cpu()[0, 2:3], scales.cpu()[1]]).view(7, 1), fmt)


def test_padded_rows_and_no_states():
    codes, scales = pool_of(3, 128, "int8")
    c0, s0 = codes.clone(), scales.clone()
    state = torch.randn(3, 128).cuda()
    slots = torch.tensor([-1, 3, 2 ** 31 - 1], dtype=torch.int32).cuda()
    ssd.ssd_cache_write(state, codes, scales, slots)
    assert torch.equal(codes, c0) and torch.equal(scales, s0)
    ssd.ssd_cache_write(state[:0], codes, scales, slots[:0])
    assert ssd.ssd_cache_read(codes, scales, slots[:0]).shape == (0, 128)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements: its last slots are written and read."""
    size, num = 80 * 64 * 128, 6600
    assert size * num > 2 ** 32
    codes = torch.zeros(num, size, dtype=torch.int8, device="cuda")
    scales = torch.zeros(num, size // 64, device="cuda")
    state = torch.randn(2, size, device="cuda")
    slots = torch.tensor([num - 1, 1], dtype=torch.int32).cuda()
    ssd.ssd_cache_write(state, codes, scales, slots)
    idx = slots.long().cpu()
    rows = torch.stack([codes[i] for i in idx])
    check_rows(state.cpu(), rows.cpu(), torch.stack([scales[i] for i in idx]).cpu(), "int8")
    back = ssd.ssd_cache_read(codes, scales, slots)
    assert torch.equal(back.cpu(), values(rows.cpu(), scales[slots.long()].cpu(), size))
    assert not codes[2].any() and not codes[num - 2].any()


def test_graph_replays_and_another_stream():
    codes, scales = pool_of(4, 640, "fp8")
    state = torch.randn(2, 640).cuda()
    slots = torch.tensor([3, 0], dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssd.ssd_cache_write(state, codes, scales, slots)
        ssd.ssd_cache_read(codes, scales, slots)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_cache_write(state, codes, scales, slots)
        back = ssd.ssd_cache_read(codes, scales, slots)
    for r in range(3):
        state.copy_(torch.randn(2, 640))
        c2, s2 = pool_of(4, 640, "fp8")
        ssd.ssd_cache_write(state, c2, s2, slots)
        ref = ssd.ssd_cache_read(c2, s2, slots)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back, ref)
