"""Every form of the kernels that the convolution and the selective scan choose by size
(layer_forms.py), against the formulas in float64 on the CPU, with the references and
tolerances of test_gpu_conv1d.py and test_gpu_selective_scan.py."""

import pytest
import torch

from selective_state_space_amd import ssd

import test_gpu_conv1d as conv
import test_gpu_selective_scan as scan
from _gpu import log
from layer_forms import CONV_BWD, CONV_FWD, CONV_STEP, SCAN_BWD, SCAN_FWD, SCAN_STEP
from test_gpu_selective_scan import IO, U, up

pytestmark = pytest.mark.gpu

NAN = float("nan")


def ids(cases):
    return [("-".join(str(v) for v in c)).replace(" ", "") for c in cases]


# ---------------------------------------------------------------------------
# the selective scan

PAIRS = [("f32", True, True), ("bf16", True, False), ("bf16", False, True),
         ("f32", False, False)]
# (type, gate, lengths); a cut scan of 4 states takes the kernels of a whole one and the pass
# before it, which knows no gate
PROMPTS = [c + p for c in SCAN_FWD for p in PAIRS[:2 if c[1] == 4 and c[2] else 4]]


@pytest.mark.parametrize("sizes,states,cut,io,gate,lens", PROMPTS, ids=ids(PROMPTS))
def test_scan_prompt(sizes, states, cut, io, gate, lens):
    Bt, T, Dm, N = sizes
    log("selective scan fwd", io, sizes, states, cut, gate, lens)
    m = scan.make(Bt, T, Dm, N, io, seed=Bt + T, gate=gate)
    eff = kw = None
    if lens:
        g = torch.Generator().manual_seed(T)
        eff = torch.randint(0, T + 1, (Bt,), generator=g)
        eff[0], eff[Bt - 1] = T, 0
        if Bt > 2:
            eff[1] = 17
        kw = dict(seq_lens=eff.to(torch.int32).cuda())
        eff = eff.tolist()
    y, ey, h, E, _ = scan.forward(m, eff)
    if lens:
        for k in ("x", "dt", "B", "C", "z"):
            if m[k] is not None:
                for b, n in enumerate(eff):
                    m[k][b, n:] = NAN
    got, fin = scan.run_fwd(m, **(kw or {}))
    scan.check(got, y, ey, "y")
    scan.check(fin, h, E, "final")
    if lens:
        dead = torch.arange(T)[None, :] >= torch.tensor(eff)[:, None]
        assert not got.cpu()[dead].any()
    yio, _ = scan.run_fwd(m, y_io_dtype=True, **(kw or {}))
    assert yio.dtype == IO[io] and torch.equal(yio, got.to(IO[io]))


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,states,cut", SCAN_BWD, ids=ids(SCAN_BWD))
def test_scan_gradients(sizes, states, cut, io, gate):
    Bt, T, Dm, N = sizes
    log("selective scan bwd", io, sizes, states, cut, gate)
    m = scan.make(Bt, T, Dm, N, io, seed=Bt + T + 1, gate=gate)
    out = scan.run_bwd(m)
    for k, (ref, bound) in scan.gradients(m).items():
        scan.check(out[k], ref, bound, k)
    again = scan.run_bwd(m)
    for k in out:
        assert (out[k] is None and again[k] is None) or torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,channels", SCAN_STEP, ids=ids(SCAN_STEP))
def test_scan_step(sizes, channels, io, gate):
    """One step over a shuffled pool; padded rows at both ends and among the others."""
    Bt, Dm, N = sizes
    log("selective scan step", io, sizes, channels, gate)
    m = scan.make(Bt, 1, Dm, N, io, seed=Bt + N, gate=gate)
    g = torch.Generator().manual_seed(2)
    pool = Bt + 3
    state = torch.randn(pool, Dm, N, generator=g) * 0.3
    slots = torch.randperm(pool, generator=g)[:Bt].to(torch.int32)
    m["init"] = state[slots.long()].clone()
    dead = [0, 3, Bt - 1]
    for i, v in zip(dead, (-1, pool, 2 ** 31 - 1)):
        slots[i] = v
    live = [i for i in range(Bt) if i not in dead]
    y, ey, h, E, _ = scan.forward(m)
    one = lambda k: None if m[k] is None else up(m[k])[:, 0]
    args = (one("x"), one("dt"), up(m["A"]), one("B"), one("C"), up(m["D"]))
    kw = dict(slots=slots.cuda(), dt_bias=up(m["dt_bias"]), dt_softplus=True, z_t=one("z"))
    st, keep = state.cuda(), state.cuda()
    got = ssd.ssd_selective_scan_step(st, *args, **kw)
    scan.check(got[live], y[live, 0], ey[live, 0], "y")
    assert not got[dead].any()
    idx = slots.long()[live]
    scan.check(st.cpu()[idx], h[live], E[live], "state")
    rest = torch.ones(pool, dtype=torch.bool)
    rest[idx] = False
    assert torch.equal(st.cpu()[rest], state[rest])
    yio = ssd.ssd_selective_scan_step(keep, *args, y_io_dtype=True, **kw)
    assert yio.dtype == IO[io] and torch.equal(yio, got.to(IO[io])) and torch.equal(keep, st)


# ---------------------------------------------------------------------------
# the convolution

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("sizes,run", CONV_FWD, ids=ids(CONV_FWD))
def test_conv_prompt(sizes, run, W, io):
    """Whole prompts, then right-padded ones that end inside a run and at its borders."""
    Bt, T, splits = sizes
    C = sum(splits)
    log("conv1d fwd", io, sizes, run, W)
    m = conv.make(Bt, T, C, W, io, seed=run + W, slack=3, lead=5)
    args = (up(m["weight"]), up(m["bias"]))
    init = up(m["init"])
    ys, fin = ssd.ssd_conv1d_fwd(conv.xslice(m, "cuda"), *args, splits=splits, init_state=init)
    y, pre, S, xp = conv.formula(m, True)
    tol = conv.bound(y, pre, S, W, True, IO[io])
    for got, ref, tl in zip(ys, y.split(splits, 2), tol.split(splits, 2)):
        conv.check(got, ref, tl, "y")
    assert torch.equal(fin.double().cpu(), xp[:, T:])
    g = torch.Generator().manual_seed(W)
    lens = torch.randint(0, T + 1, (Bt,), generator=g)
    ends = [0, 1, run - 1, run, run + 1, 2 * run, T]
    lens[:min(Bt, len(ends))] = torch.tensor(ends[:Bt])
    dead = torch.arange(T)[None, :] >= lens[:, None]
    m["rows"][dead] = NAN
    y[dead], tol[dead] = 0.0, 1e-30
    ys, fin = ssd.ssd_conv1d_fwd(conv.xslice(m, "cuda"), *args, splits=splits, init_state=init,
                                 final_state=init, seq_lens=lens.to(torch.int32).cuda())
    for got, ref, tl in zip(ys, y.split(splits, 2), tol.split(splits, 2)):
        conv.check(got, ref, tl, "y, lengths")
        assert not got.cpu()[dead].any()
    rows = lens[:, None] + torch.arange(W - 1)
    want = torch.gather(xp, 1, rows[:, :, None].expand(-1, -1, C))
    assert fin is init and torch.equal(fin.double().cpu(), want)


def conv_gradients(m, splits, dy, dfinal, run, silu):
    """The formula's gradients, with the sums' bounds by the run of tokens that a lane takes:
    run products added in turn, two joins of the workgroup's runs, the sum over workgroups in
    double, one last rounding."""
    ref = conv.grads(m, splits, silu, dy, dfinal)
    _, pre, S, xp = conv.formula(m, silu)
    W, T = m["weight"].shape[1], pre.shape[1]
    d = torch.cat([v.double() for v in dy], 2)
    s = torch.sigmoid(pre)
    dp = d * (s * (1 + pre * (1 - s)) if silu else 1.0)
    edp = U * dp.abs()
    if silu:   # as in conv.grads: the errors of pre and of silu'
        edp = edp + d.abs() * (0.5 * U * (W + 2) * S
                               + U * (8 + 2 * pre.abs()) * (1 + pre.abs()))
    each = edp + U * (min(T, run) + 4) * dp.abs()
    bw = torch.stack([(each * xp[:, k:k + T].abs()).sum((0, 1)) for k in range(W)], 1)
    return dict(ref, dweight=(ref["dweight"][0], bw), dbias=(ref["dbias"][0], each.sum((0, 1))))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W,silu", [(2, True), (3, True), (4, True), (4, False)])
@pytest.mark.parametrize("sizes,run", CONV_BWD, ids=ids(CONV_BWD))
def test_conv_gradients(sizes, run, W, silu, io):
    Bt, T, splits = sizes
    C = sum(splits)
    log("conv1d bwd", io, sizes, run, W, silu)
    m = conv.make(Bt, T, C, W, io, seed=run + W + 1, slack=2, lead=3)
    g = torch.Generator().manual_seed(run)
    dy = [torch.randn(Bt, T, c, generator=g) for c in splits]
    dfinal = torch.randn(Bt, W - 1, C, generator=g)
    args = (conv.xslice(m, "cuda"), up(m["weight"]), [up(v) for v in dy], up(m["bias"]))
    kw = dict(silu=silu, init_state=up(m["init"]), dfinal=up(dfinal))
    out = ssd.ssd_conv1d_bwd(*args, **kw)
    for k, (ref, bound) in conv_gradients(m, splits, dy, dfinal, run, silu).items():
        conv.check(out[k], ref, bound + 1e-30, k)
    again = ssd.ssd_conv1d_bwd(*args, **kw)
    for k in out:
        assert torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("sizes,rows", CONV_STEP, ids=ids(CONV_STEP))
def test_conv_step(sizes, rows, W, io):
    """Two steps over a shuffled pool.  Padded rows at every place of a group of four, a group
    of nothing else, and one in the last, short group."""
    Bt, splits = sizes
    C = sum(splits)
    log("conv1d step", io, sizes, rows, W)
    m = conv.make(Bt, 2, C, W, io, seed=W, slack=3, lead=1)
    g = torch.Generator().manual_seed(9)
    pool = Bt + 5
    slots = torch.randperm(pool, generator=g)[:Bt].to(torch.int32)
    state = torch.randn(pool, W - 1, C, generator=g).to(IO[io])
    m["init"] = state[slots.long()].clone()
    dead = [0, 5, 10, 15, 20, 21, 22, 23, 40, 43, 257]
    for j, i in enumerate(dead):
        slots[i] = (-1, pool, 2 ** 31 - 1)[j % 3]
    live = [i for i in range(Bt) if i not in dead]
    y, pre, S, xp = conv.formula(m, True)
    tol = conv.bound(y, pre, S, W, True, IO[io])
    y[dead] = 0.0
    x, st = conv.xslice(m, "cuda"), state.cuda()
    for t in range(2):
        ys = ssd.ssd_conv1d_step(st, x[:, t], up(m["weight"]), up(m["bias"]), splits=splits,
                                 slots=slots.cuda())
        for got, ref, tl in zip(ys, y[:, t].split(splits, 1), tol[:, t].split(splits, 1)):
            conv.check(got, ref, tl, "y step %d" % t)
            assert not got[dead].any()
    got = st.cpu()
    idx = slots.long()[live]
    assert torch.equal(got[idx].double(), xp[live, 2:])
    rest = torch.ones(pool, dtype=torch.bool)
    rest[idx] = False
    assert torch.equal(got[rest], state[rest])
