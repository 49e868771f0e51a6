"""The ends of the range: steps and decay rates at the top of float32, against the
recurrence in float64 on the CPU with the bounds of its float32 error that
test_gpu_selective_scan.py derives."""

import pytest
import torch

from selective_state_space_amd import ssd

from _gpu import log
from test_gpu_selective_scan import IO, check, forward, gradients, make, run_bwd, run_fwd, up

pytestmark = pytest.mark.gpu

INF = float("inf")
# one segment of one tile and of several, and several segments; the forms of few rows
SIZES = [(1, 8, 20, 16), (2, 70, 37, 8), (1, 300, 64, 16), (1, 1030, 20, 64), (1, 200, 33, 32)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,Dm,N", SIZES)
def test_softplus_of_the_largest_steps(io, Bt, T, Dm, N):
    """softplus(r) is r far above 20, up to the largest finite r (x is small there, so that
    d x stays finite, and no subnormal)."""
    log("softplus, large steps", io, Bt, T, Dm, N)
    m = make(Bt, T, Dm, N, io, seed=31)
    for t, v in ((T - 1, 3e38), (T // 2, 2.5e38), (3, 1e30), (1, 120.0)):
        m["dt"][:, t] = v
        m["x"][:, t] = m["x"][:, t] * min(1.0, 1e4 / v)
    m["A"][:2] = 0.0
    m["dt"][:, T // 3, ::2] = -3e38
    m["dt"][:, T // 3, 1::2] = -INF
    y, ey, h, E, _ = forward(m)
    got, fin = run_fwd(m)
    check(got, y, ey, "y")
    check(fin, h, E, "final")
    # the last token once more, as a step from the state before it
    before = {k: (v[:, :T - 1].contiguous() if k in ("x", "dt", "B", "C", "z") else v)
              for k, v in m.items()}
    _, state = run_fwd(before)
    c = lambda k: up(m[k][:, T - 1].contiguous())
    yt = ssd.ssd_selective_scan_step(state, c("x"), c("dt"), up(m["A"]), c("B"), c("C"),
                                     up(m["D"]), dt_bias=up(m["dt_bias"]), dt_softplus=True,
                                     z_t=c("z"))
    check(yt, y[:, T - 1], ey[:, T - 1], "y step")
    check(state, h, E, "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,Dm,N", SIZES)
def test_softplus_of_infinity(io, Bt, T, Dm, N):
    """softplus(inf) = inf: the state before is forgotten and d x B is infinite, with its
    sign.  In the last token, as a later one would decay an infinite state."""
    m = make(Bt, T, Dm, N, io, seed=32, gate=False)
    for k in ("x", "B"):
        m[k][:, T - 1] = torch.where(m[k][:, T - 1].abs() < 0.1, m[k].new_ones(()), m[k][:, T - 1])
    m["dt"][:, T - 1] = INF
    want = (m["x"][:, T - 1, :, None].double() * m["B"][:, T - 1, None, :].double()).sign() * INF
    _, fin = run_fwd(m)
    assert torch.equal(fin.double().cpu(), want)
    c = lambda k: up(m[k][:, T - 1].contiguous())
    state = torch.ones(Bt, Dm, N, device="cuda")
    ssd.ssd_selective_scan_step(state, c("x"), c("dt"), up(m["A"]), c("B"), c("C"), up(m["D"]),
                                dt_bias=up(m["dt_bias"]), dt_softplus=True)
    assert torch.equal(state.double().cpu(), want)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,Dm,N", SIZES)
def test_gradients_of_the_largest_steps(io, Bt, T, Dm, N):
    """The last token takes a step of 3e38: its gradients carry d (dy is small there), and
    nothing passes to the tokens before it."""
    log("gradients, large steps", io, Bt, T, Dm, N)
    m = make(Bt, T, Dm, N, io, seed=33)
    m["dt"][:, T - 1] = 3e38
    m["x"][:, T - 1] *= 1e4 / 3e38
    m["dy"][:, T - 1] *= 1e-10
    out = run_bwd(m, dfinal=False)
    for k, (ref, bound) in gradients(m, dfinal=False).items():
        check(out[k], ref, bound, k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,Dm,N", SIZES)
@pytest.mark.parametrize("gate", [True, False])
def test_decay_rates_at_the_lowest_value(io, Bt, T, Dm, N, gate):
    """A rate of the type's lowest value forgets the state at any step, and keeps it where
    d = 0 (an input at -inf); the tokens past the end of a sequence's last tile too."""
    log("lowest decay rates", io, Bt, T, Dm, N)
    m = make(Bt, T, Dm, N, io, seed=34, gate=gate)
    m["A"][1::3] = torch.finfo(torch.float32).min
    m["A"][2, ::2] = torch.finfo(torch.float32).min
    m["dt"][:, T // 2] = -INF
    m["dt"][:, T - 1, 1::2] = -INF
    y, ey, h, E, _ = forward(m)
    got, fin = run_fwd(m)
    check(got, y, ey, "y")
    check(fin, h, E, "final")
    # d A is 0 or below -1e30 here, so decay and its bound are exact: 1 or 0
    out = run_bwd(m)
    ref = gradients(m)
    for k in ("dx", "dB", "dC", "dD", "dinit") + (("dz",) if gate else ()):
        check(out[k], *ref[k], k)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_largest_states_read_back_finite(fmt):
    """Blocks whose largest magnitude is next to the top of float32: scale and codes as
    defined (the scale to an ulp), every value finite and within half a code's step."""
    q = 127.0 if fmt == torch.int8 else 448.0
    bits = torch.arange(0x7f7fffff - 127, 0x7f7fffff + 1, dtype=torch.int32)
    amax = bits.view(torch.float32)
    state = amax[:, None] * torch.linspace(-1, 1, 64)
    state[:, 0] = amax
    state[:, 63] = -amax
    codes = torch.zeros(128, 64, dtype=torch.int8).view(fmt).cuda()
    scales = torch.zeros(128, 1).cuda()
    ssd.ssd_cache_write(state.cuda(), codes, scales)
    back = ssd.ssd_cache_read(codes, scales).cpu().double()
    want = amax.double()[:, None] / q
    assert ((scales.cpu().double() - want).abs() <= 2.0 ** -23 * want).all()
    assert back.isfinite().all()
    # half a step (int8: of the scale; e4m3: 2^-4 of the value, or 2^-10 of the scale), an ulp
    # of the scale and the rounding of the product
    v = state.double()
    step = want * 0.5 if fmt == torch.int8 else torch.maximum(2.0 ** -4 * v.abs(), want * 2.0 ** -10)
    assert ((back - v).abs() <= step + 2.0 ** -22 * v.abs()).all()
