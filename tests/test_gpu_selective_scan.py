"""The per-channel selective scan (prompt, single token, gradients) against the
recurrence in float64 on the CPU.

Tolerances come from the arithmetic: next to every value the reference carries
a first-order bound of its float32 error, grown step by step along the
recurrence.  U is half a unit in the last place (2^-24).  Elementary steps: a
rounded sum or product U; the hardware exponential, logarithm and reciprocal 2
U each; an exponential's argument v adds U |v| per rounding of it.  Outputs in
the io dtype add finfo.eps / 2 of the value.  The bounds are worst cases; the
errors met stay well below them.
"""

import pytest
import torch

from selective_state_space_amd import ssd

from _gpu import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(Bt, T, Dm, N, io, seed=0, bias=True, softplus=True, gate=True, init=True):
    g = torch.Generator().manual_seed(seed)
    dt = IO[io]
    r = lambda *s: torch.randn(*s, generator=g)
    m = dict(x=r(Bt, T, Dm).to(dt), B=(r(Bt, T, N) * N ** -0.5).to(dt),
             C=(r(Bt, T, N) * N ** -0.5).to(dt), D=r(Dm),
             A=-torch.arange(1, N + 1).float() * torch.exp(0.2 * r(Dm, N)),
             z=r(Bt, T, Dm).to(dt) if gate else None,
             init=r(Bt, Dm, N) * 0.3 if init else None, softplus=softplus,
             dt_bias=None, dy=r(Bt, T, Dm), dfinal=r(Bt, Dm, N))
    if softplus:
        m["dt"] = r(Bt, T, Dm).to(dt)
        if bias:
            dt0 = 1e-3 * torch.exp(torch.rand(Dm, generator=g) * 4.6)
            m["dt_bias"] = torch.log(torch.expm1(dt0))
        else:
            m["dt"] = m["dt"] - 3
    else:
        m["dt"] = (1e-3 * torch.exp(torch.rand(Bt, T, Dm, generator=g) * 4.6)).to(dt)
        if bias:
            m["dt_bias"] = torch.full((Dm,), 0.01)
    return m


def up(t):
    return None if t is None else t.cuda()


def steps(m):
    """d and the error bound of d, and dt + bias."""
    raw = m["dt"].double()
    if m["dt_bias"] is not None:
        raw = raw + m["dt_bias"].double()
    if not m["softplus"]:
        return raw, U * raw.abs(), raw
    d = torch.where(raw > 20, raw, torch.nn.functional.softplus(raw))
    # the rounding of dt + bias passes through softplus' = sigmoid (0 at -inf)
    return d, U * (raw.abs() * torch.sigmoid(raw)).nan_to_num() + 12 * U * d, raw


def silu(z):
    """silu(z), its derivative, and their error bounds."""
    s = torch.sigmoid(z)
    f, df = z * s, s * (1 + z * (1 - s))
    return f, df, f.abs() * (5 + 2 * z.abs()) * U, s * (1 + z.abs()) * (8 + 2 * z.abs()) * U


def forward(m, lens=None):
    """(y, bound, final, bound, history) in float64."""
    x, B, C, A, D = (m[k].double() for k in ("x", "B", "C", "A", "D"))
    Bt, T, Dm = x.shape
    d, ed, _ = steps(m)
    if lens is not None:
        dead = torch.arange(T)[None, :, None] >= torch.tensor(lens)[:, None, None]
        zero = lambda t: torch.where(dead.expand_as(t), torch.zeros_like(t), t)
        d, ed, x, B, C = zero(d), zero(ed), zero(x), zero(B), zero(C)
    h = torch.zeros(Bt, Dm, A.shape[1], dtype=torch.float64) if m["init"] is None \
        else m["init"].double()
    E = torch.zeros_like(h)
    hist = [(h, E)]
    y, ey = torch.empty_like(x), torch.empty_like(x)
    for t in range(T):
        dt = d[:, t, :, None]
        a = torch.exp(dt * A)
        ra = A.abs() * ed[:, t, :, None] + 4 * U * (dt * A).abs() + 3 * U
        u = dt * x[:, t, :, None]
        uB = u * B[:, t, None]
        eu = ed[:, t, :, None] * x[:, t, :, None].abs() + U * u.abs()
        # (2 U |h|: the sums of d and the joins of segments)
        E = a * (E + (ra + 2 * U) * h.abs()) + eu * B[:, t, None].abs() + U * uB.abs()
        h = a * h + uB
        E = E + U * h.abs()
        hist.append((h, E))
        hC = h * C[:, t, None]
        y[:, t] = hC.sum(-1) + D * x[:, t]
        ey[:, t] = ((E * C[:, t, None].abs()).sum(-1) + 10 * U * hC.abs().sum(-1)
                    + 2 * U * ((D * x[:, t]).abs() + y[:, t].abs()))
    pre, epre = y, ey
    if m["z"] is not None:
        f, _, ef, _ = silu(m["z"].double())
        if lens is not None:
            f, ef = zero(f), zero(ef)
        y, ey = pre * f, epre * f.abs() + pre.abs() * ef + U * (pre * f).abs()
    return y, ey, h, E, (hist, pre, epre)


def gradients(m, dfinal=True):
    _, _, _, _, (hist, pre, epre) = forward(m)
    x, B, C, A, D = (m[k].double() for k in ("x", "B", "C", "A", "D"))
    Bt, T, Dm = x.shape
    d, ed, raw = steps(m)
    dy = m["dy"].double()
    out = {}
    p, ep = dy, torch.zeros_like(dy)
    if m["z"] is not None:
        f, df, ef, edf = silu(m["z"].double())
        dz = dy * pre * df
        out["dz"] = (dz, dy.abs() * (epre * df.abs() + pre.abs() * edf) + 4 * U * dz.abs())
        p, ep = dy * f, dy.abs() * ef + U * (dy * f).abs()
    car = m["dfinal"].double() if dfinal else torch.zeros_like(hist[0][0])
    Ec = torch.zeros_like(car)
    dx, dd = torch.empty_like(x), torch.empty_like(x)
    edx, edd = torch.empty_like(x), torch.empty_like(x)
    dB, dC, eB, eC = (torch.empty_like(B) for _ in range(4))
    dA, eA = torch.zeros_like(A), torch.zeros_like(A)
    many = T / 8 + 60          # the longest run of float32 additions into a sum over tokens
    for t in reversed(range(T)):
        h, Eh = hist[t + 1]
        hp, Ehp = hist[t]
        dt, xt = d[:, t, :, None], x[:, t, :, None]
        a = torch.exp(dt * A)
        ra = A.abs() * ed[:, t, :, None] + 4 * U * (dt * A).abs() + 3 * U
        u, eu = dt * xt, ed[:, t, :, None] * xt.abs() + U * (dt * xt).abs()
        Bv, Cv = B[:, t, None], C[:, t, None]
        pt, ept = p[:, t, :, None], ep[:, t, :, None]
        g = pt * Cv + car
        Eg = ept * Cv.abs() + Ec + U * g.abs()
        dB[:, t], dC[:, t] = (g * u).sum(1), (pt * h).sum(1)
        eB[:, t] = (Eg * u.abs() + g.abs() * eu + 14 * U * (g * u).abs()).sum(1)
        eC[:, t] = (ept * h.abs() + pt.abs() * Eh + 14 * U * (pt * h).abs()).sum(1)
        gB = (g * Bv).sum(-1)
        egB = (Eg * Bv.abs() + 10 * U * (g * Bv).abs()).sum(-1)
        car = g * a
        Ec = a * (Eg + (ra + 2 * U) * g.abs()) + U * car.abs()
        q = car * hp
        eq = Ec * hp.abs() + car.abs() * Ehp + U * q.abs()
        qA = (q * A).sum(-1)
        eqA = (eq * A.abs() + 12 * U * (q * A).abs()).sum(-1)
        dA += (q * dt).sum(0)
        eA += (eq * dt + q.abs() * ed[:, t, :, None] + many * U * (q * dt).abs()).sum(0)
        dx[:, t] = d[:, t] * gB + D * p[:, t]
        edx[:, t] = (ed[:, t] * gB.abs() + d[:, t] * egB + D.abs() * ep[:, t]
                     + 2 * U * ((d[:, t] * gB).abs() + (D * p[:, t]).abs()))
        dd[:, t] = x[:, t] * gB + qA
        edd[:, t] = (x[:, t].abs() * egB + eqA + 2 * U * ((x[:, t] * gB).abs() + qA.abs()))
    ddt, eddt = dd, edd
    if m["softplus"]:
        sg = torch.where(raw > 20, torch.ones_like(raw), torch.sigmoid(raw))
        ddt, eddt = dd * sg, edd * sg + dd.abs() * sg * (6 + 3 * raw.abs()) * U
    px = p * x
    out.update(dx=(dx, edx), ddt=(ddt, eddt), dA=(dA, eA), dB=(dB, eB), dC=(dC, eC),
               dD=(px.sum((0, 1)), (ep * x.abs() + many * U * px.abs()).sum((0, 1))),
               ddt_bias=(ddt.sum((0, 1)), (eddt + many * U * ddt.abs()).sum((0, 1))),
               dinit=(car, Ec))
    return out


def check(got, ref, bound, what):
    assert got.isfinite().all(), what
    d = (got.double().cpu() - ref).abs()
    r = float((d / (1.02 * bound + 1e-30)).max()) if d.numel() else 0.0
    log("  %-10s err/tol = %.3f" % (what, r))
    assert r <= 1.0, "%s: %.3fx the tolerance" % (what, r)


def run_fwd(m, **kw):
    return ssd.ssd_selective_scan_fwd(
        up(m["x"]), up(m["dt"]), up(m["A"]), up(m["B"]), up(m["C"]), up(m["D"]),
        init_state=up(m["init"]), dt_bias=up(m["dt_bias"]), dt_softplus=m["softplus"],
        z=up(m["z"]), **kw)


def run_bwd(m, dfinal=True, **kw):
    return ssd.ssd_selective_scan_bwd(
        up(m["x"]), up(m["dt"]), up(m["A"]), up(m["B"]), up(m["C"]), up(m["D"]), up(m["dy"]),
        init_state=up(m["init"]), dfinal=up(m["dfinal"]) if dfinal else None,
        dt_bias=up(m["dt_bias"]), dt_softplus=m["softplus"], z=up(m["z"]), **kw)


SHAPES = [(1, 1, 64, 16), (2, 3, 5, 16), (1, 37, 64, 8), (2, 16, 130, 16), (3, 17, 33, 32),
          (1, 70, 18, 64), (1, 300, 257, 16), (2, 130, 64, 64), (1, 129, 515, 8)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,Dm,N", SHAPES)
def test_prompt(io, Bt, T, Dm, N):
    log("selective scan fwd", io, Bt, T, Dm, N)
    m = make(Bt, T, Dm, N, io, seed=T)
    y, ey, h, E, _ = forward(m)
    got, fin = run_fwd(m)
    assert got.dtype == torch.float32
    check(got, y, ey, "y")
    check(fin, h, E, "final")
    yio, _ = run_fwd(m, y_io_dtype=True)
    assert yio.dtype == IO[io] and torch.equal(yio, got.to(IO[io]))
    # plain: no bias, softplus, gate or initial state
    m = make(Bt, T, Dm, N, io, seed=T + 1, bias=False, softplus=False, gate=False, init=False)
    y, ey, h, E, _ = forward(m)
    got, fin = run_fwd(m)
    check(got, y, ey, "y plain")
    check(fin, h, E, "final")


@pytest.mark.parametrize("Bt,T,Dm,N", [(1, 4133, 64, 16), (2, 1000, 40, 8), (1, 2049, 20, 64),
                                       (1, 777, 130, 32)])
def test_split_over_time(Bt, T, Dm, N):
    """Long sequences with few channels run in segments."""
    dims = ssd.ScanDims(Bt, T, Dm, N, ssd.SSD_F32)
    assert ssd.ssd_selective_scan_workspace_size(dims) > 0
    log("selective scan split", Bt, T, Dm, N)
    m = make(Bt, T, Dm, N, "f32", seed=3)
    y, ey, h, E, _ = forward(m)
    got, fin = run_fwd(m)
    check(got, y, ey, "y")
    check(fin, h, E, "final")
    again, fin2 = run_fwd(m)
    assert torch.equal(got, again) and torch.equal(fin, fin2)


@pytest.mark.parametrize("T", [45, 500])
def test_lengths(T):
    """Right-padded prompts, NaN in the padding, final states in place of initial ones."""
    lens = [0, 1, 16, 17, T - 1, T, T + 5, -2]
    eff = [min(max(n, 0), T) for n in lens]
    m = make(len(lens), T, 37, 16, "bf16", seed=5)
    y, ey, h, E, _ = forward(m, eff)
    for b, n in enumerate(eff):
        for k in ("x", "dt", "z", "B", "C"):
            m[k][b, n:] = float("nan")
    state = up(m["init"]).clone()
    m2 = dict(m, init=None)
    got, fin = ssd.ssd_selective_scan_fwd(
        up(m["x"]), up(m["dt"]), up(m["A"]), up(m["B"]), up(m["C"]), up(m["D"]),
        init_state=state, final_state=state, seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(),
        dt_bias=up(m["dt_bias"]), dt_softplus=True, z=up(m["z"]))
    assert fin is state
    check(fin, h, E, "final")
    check(got, y, ey, "y")
    for b, n in enumerate(eff):
        assert not got[b, n:].any()
    assert torch.equal(fin[0], up(m["init"])[0])


def test_no_tokens_and_no_sequences():
    m = make(2, 0, 40, 16, "f32")
    y, fin = run_fwd(m)
    assert y.shape == (2, 0, 40) and torch.equal(fin.cpu(), m["init"])
    out = run_bwd(m)
    assert torch.equal(out["dinit"].cpu(), m["dfinal"])
    assert not out["dA"].any() and not out["dD"].any() and not out["ddt_bias"].any()
    m = make(0, 5, 40, 16, "f32")
    y, fin = run_fwd(m)
    assert y.shape == (0, 5, 40)
    out = run_bwd(m)
    assert not out["dA"].any() and not out["dD"].any()


def test_extreme_steps():
    """No decay, full decay, d = 0, steps far above the softplus threshold and far below."""
    m = make(1, 40, 64, 16, "f32", seed=8, bias=False)
    m["dt"][0, 3] = 25.0
    m["dt"][0, 5] = -200.0
    m["dt"][0, 6] = -float("inf")
    m["dt"][0, 7] = 20.0
    m["A"][:8] = 0.0
    m["A"][8:16] = -1e6
    y, ey, h, E, _ = forward(m)
    got, fin = run_fwd(m)
    check(got, y, ey, "y")
    check(fin, h, E, "final")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,Dm,N", [(1, 5, 16), (3, 64, 8), (9, 33, 64), (40, 130, 32),
                                     (600, 64, 16), (530, 270, 16)])
def test_step(io, Bt, Dm, N):
    """Two steps over a shuffled pool with padded rows against the prompt form."""
    log("selective scan step", io, Bt, Dm, N)
    m = make(Bt, 2, Dm, N, io, seed=Bt)
    g = torch.Generator().manual_seed(2)
    pool = Bt + 3
    state = torch.randn(pool, Dm, N, generator=g) * 0.3
    slots = torch.randperm(pool, generator=g)[:Bt].to(torch.int32)
    m["init"] = state[slots.long()].clone()
    dead = [i for i in (1, 5) if i < Bt]
    for j, i in enumerate(dead):
        slots[i] = (-1, pool + 7)[j]
    y, ey, h, E, _ = forward(m)
    st, sl = state.cuda(), slots.cuda()
    live = [i for i in range(Bt) if i not in dead]
    for t in range(2):
        args = (st, up(m["x"])[:, t], up(m["dt"])[:, t], up(m["A"]), up(m["B"])[:, t],
                up(m["C"])[:, t], up(m["D"]))
        kw = dict(slots=sl, dt_bias=up(m["dt_bias"]), dt_softplus=True, z_t=up(m["z"])[:, t])
        keep = st.clone()
        got = ssd.ssd_selective_scan_step(*args, **kw)
        check(got[live], y[live, t], ey[live, t], "y step %d" % t)
        assert not got[dead].any()
        yio = ssd.ssd_selective_scan_step(keep, *args[1:], y_io_dtype=True, **kw)
        assert yio.dtype == IO[io] and torch.equal(yio, got.to(IO[io])) and torch.equal(keep, st)
    idx = slots.long()[live]
    check(st[idx.cuda()], h[live], E[live], "state")
    rest = torch.ones(pool, dtype=torch.bool)
    rest[idx] = False
    assert torch.equal(st.cpu()[rest], state[rest])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,Dm,N", SHAPES)
def test_gradients(io, Bt, T, Dm, N):
    log("selective scan bwd", io, Bt, T, Dm, N)
    m = make(Bt, T, Dm, N, io, seed=T)
    out = run_bwd(m)
    for k, (ref, bound) in gradients(m).items():
        check(out[k], ref, bound, k)
    again = run_bwd(m)
    for k in out:
        assert torch.equal(out[k], again[k]), k
    m = make(Bt, T, Dm, N, io, seed=T + 1, bias=False, softplus=False, gate=False, init=False)
    out = run_bwd(m, dfinal=False, want_dinit=False)
    assert out["dz"] is None and out["dinit"] is None and out["ddt_bias"] is None
    ref = gradients(m, dfinal=False)
    for k in ("dx", "ddt", "dA", "dB", "dC", "dD"):
        check(out[k], *ref[k], k + " plain")


@pytest.mark.parametrize("Bt,T,Dm,N", [(1, 2133, 64, 16), (2, 700, 40, 8), (1, 1025, 20, 64),
                                       (1, 500, 130, 32)])
def test_gradients_split_over_time(Bt, T, Dm, N):
    log("selective scan bwd split", Bt, T, Dm, N)
    m = make(Bt, T, Dm, N, "f32", seed=4)
    out = run_bwd(m)
    for k, (ref, bound) in gradients(m).items():
        check(out[k], ref, bound, k)


def test_gradient_differences():
    """Central differences of the float64 recurrence along random directions."""
    m = make(2, 21, 6, 8, "f32", seed=6)
    out = run_bwd(m)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", dt_bias="ddt_bias", z="dz",
                 init="dinit")

    def loss(mm):
        y, _, h, _, _ = forward(mm)
        return float((y * m["dy"].double()).sum() + (h * m["dfinal"].double()).sum())

    g = torch.Generator().manual_seed(1)
    for key, name in names.items():
        v = torch.randn(m[key].shape, generator=g, dtype=torch.float64)
        eps = 1e-5
        num = (loss(dict(m, **{key: m[key].double() + eps * v}))
               - loss(dict(m, **{key: m[key].double() - eps * v}))) / (2 * eps)
        terms = out[name].double().cpu() * v
        # differences: eps^2 / 6 of third derivatives (|A|^3 up to 1e3) and 1e-13 / eps of
        # the loss; the gradient: float32 along at most 21 tokens of 8 states
        tol = float(terms.abs().sum()) * 400 * U + 1e-5
        assert abs(float(terms.sum()) - num) <= tol, (name, float(terms.sum()), num, tol)


def test_offsets_past_32_bits():
    """A prompt of more than 2^32 elements, and a state pool of as many: the last tokens
    continue the state of the tokens before them."""
    Dm, N = 4160, 16
    T = 2 ** 32 // Dm + 130
    x = torch.randn(1, 4099, Dm, device="cuda").to(torch.bfloat16).repeat(1, -(-T // 4099), 1)[:, :T]
    assert x.numel() > 2 ** 32
    dt = (x.flip(2) - 3).contiguous()
    B = torch.randn(1, T, N, device="cuda").to(torch.bfloat16)
    C = torch.randn(1, T, N, device="cuda").to(torch.bfloat16)
    A = -torch.arange(1, N + 1, device="cuda").float().repeat(Dm, 1)
    D = torch.randn(Dm, device="cuda")
    cut = T - 100
    part = lambda t, a, b: t[:, a:b].contiguous()
    run = lambda a, b, h: ssd.ssd_selective_scan_fwd(
        part(x, a, b), part(dt, a, b), A, part(B, a, b), part(C, a, b), D, init_state=h,
        dt_softplus=True, y_io_dtype=True)
    y, fin = run(0, T, None)
    last, fin = y[:, cut:].float().clone(), fin.clone()
    del y
    # (tokens 2000 back reach the end through exp(-sum of d) below 1e-9, so two starts agree)
    _, h = run(cut - 2000, cut, None)
    yt, ft = run(cut, T, h)
    # bf16 outputs, off by half a step each, and float32 sums of 16 states and their decay
    tol = 2.0 ** -8 * torch.maximum(last.abs(), yt.float().abs()) * 2 + 1e-4 * last.abs().max()
    assert ((last - yt.float()).abs() <= tol).all()
    assert float((fin - ft).abs().max()) <= 1e-4 * float(ft.abs().max())
    del x, dt
    num = 2 ** 32 // (Dm * N) + 3
    pool = torch.zeros(num, Dm, N, device="cuda")
    assert pool.numel() > 2 ** 32
    pool[num - 1], pool[1] = fin[0], ft[0]
    small = torch.cat([fin, ft])
    xt = torch.randn(2, Dm, device="cuda").to(torch.bfloat16)
    args = (xt, xt.flip(1), A, B[0, :2], C[0, :2], D)
    yp = ssd.ssd_selective_scan_step(pool, *args, dt_softplus=True,
                                     slots=torch.tensor([num - 1, 1], dtype=torch.int32).cuda())
    ys = ssd.ssd_selective_scan_step(small, *args, dt_softplus=True)
    assert torch.equal(yp, ys)
    assert torch.equal(pool[num - 1], small[0]) and torch.equal(pool[1], small[1])
    assert not pool[num - 2].any() and not pool[0].any()


def test_graph_replays_follow_the_inputs():
    """Forward (split over time), step and gradients in one graph: every replay equals the
    eager calls on that replay's inputs, with eager work between."""
    m = make(1, 400, 40, 16, "bf16", seed=9)
    t = {k: up(v) for k, v in m.items() if isinstance(v, torch.Tensor)}
    pool = torch.zeros(1, 40, 16, device="cuda")

    def work(pool):
        kw = dict(dt_bias=t["dt_bias"], dt_softplus=True)
        y, fin = ssd.ssd_selective_scan_fwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"],
                                            init_state=t["init"], z=t["z"], **kw)
        s = ssd.ssd_selective_scan_step(pool, t["x"][:, 0], t["dt"][:, 0], t["A"], t["B"][:, 0],
                                        t["C"][:, 0], t["D"], z_t=t["z"][:, 0], **kw)
        gr = ssd.ssd_selective_scan_bwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["dy"],
                                        init_state=t["init"], dfinal=t["dfinal"], z=t["z"], **kw)
        return [y, fin, s] + [gr[k] for k in sorted(gr)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(pool)
    for r in range(3):
        t["x"].copy_(torch.randn(t["x"].shape, device="cuda"))
        t["dy"].copy_(torch.randn(t["dy"].shape, device="cuda"))
        eager_pool = pool.clone()
        ref = [v.clone() for v in work(eager_pool)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, ref):
            assert torch.equal(o, v)
        assert torch.equal(pool, eager_pool)
