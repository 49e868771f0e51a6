"""The short causal convolution (prompt, single token, gradients) against the
formula in float64 on the CPU.

Tolerances, from the arithmetic: pre is a float32 sum of W + 1 terms, so it is
off by at most (W + 2) half-ulps of S = |bias| + sum |w x|, and silu adds 4
half-ulps of the result and the rounding of its exponent's argument, 2 |pre|
half-ulps; |silu'| <= 1.1.  An output in the io dtype adds its own rounding,
finfo.eps / 2 of the value.  Copied states are equal bit for bit.
"""

import pytest
import torch

from selective_state_space_amd import ssd

from _gpu import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(Bt, T, C, W, io, seed=0, bias=True, init=True, slack=0, lead=0):
    """Seeded inputs on the CPU; x is a slice of rows of C + slack + lead channels."""
    g = torch.Generator().manual_seed(seed)
    dt = IO[io]
    rows = torch.randn(Bt, T, lead + C + slack, generator=g).to(dt)
    return dict(rows=rows, lead=lead, C=C,
                weight=torch.randn(C, W, generator=g) * W ** -0.5,
                bias=torch.randn(C, generator=g) * 0.1 if bias else None,
                init=torch.randn(Bt, W - 1, C, generator=g).to(dt) if init else None)


def xslice(m, device=None):
    rows = m["rows"] if device is None else m["rows"].to(device)
    return rows[..., m["lead"]:m["lead"] + m["C"]]


def up(t):
    return None if t is None else t.cuda()


def padded(m):
    x = xslice(m).double()
    W = m["weight"].shape[1]
    head = (torch.zeros(x.shape[0], W - 1, x.shape[2], dtype=torch.float64) if m["init"] is None
            else m["init"].double())
    return torch.cat([head, x], 1)


def formula(m, silu):
    """(y, pre, S, the padded inputs) in float64."""
    xp = padded(m)
    w = m["weight"].double()
    W, T = w.shape[1], xp.shape[1] - w.shape[1] + 1
    b = 0.0 if m["bias"] is None else m["bias"].double()
    pre = b + sum(xp[:, k:k + T] * w[:, k] for k in range(W))
    S = (torch.as_tensor(b).abs() + sum((xp[:, k:k + T] * w[:, k]).abs() for k in range(W)))
    return (pre * torch.sigmoid(pre) if silu else pre), pre, S, xp


def bound(y, pre, S, W, silu, dtype):
    b = U * (W + 2) * S * (1.1 if silu else 1.0)
    if silu:
        b = b + U * (4 + 2 * pre.abs()) * y.abs()
    return b + (torch.finfo(dtype).eps / 2 * y.abs() if dtype != torch.float32 else 0.0) + 1e-30


def check(got, ref, tol, what):
    d = (got.double().cpu() - ref).abs()
    r = float((d / tol).max()) if d.numel() else 0.0
    log("  %-24s err/tol = %.3f" % (what, r))
    assert got.isfinite().all() and r <= 1.0, "%s: %.3fx the tolerance" % (what, r)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,splits,W", [
    (1, 1, (64,), 4), (2, 2, (8, 8, 8), 4), (1, 3, (1,), 2), (3, 37, (33, 5, 64), 3),
    (2, 129, (512, 128, 128), 4), (1, 1000, (7, 64, 0), 4), (4, 65, (1031,), 2)])
@pytest.mark.parametrize("silu,bias,init", [(True, True, True), (False, False, False)])
def test_prompt(io, Bt, T, splits, W, silu, bias, init):
    C = sum(splits)
    log("conv1d fwd", io, Bt, T, splits, W, silu, bias, init)
    m = make(Bt, T, C, W, io, 1, bias, init, slack=3, lead=5)
    ys, fin = ssd.ssd_conv1d_fwd(xslice(m, "cuda"), up(m["weight"]), up(m["bias"]), silu=silu,
                                 splits=splits, init_state=up(m["init"]))
    y, pre, S, xp = formula(m, silu)
    tol = bound(y, pre, S, W, silu, IO[io])
    for got, ref, tl in zip(ys, y.split(splits, 2), tol.split(splits, 2)):
        assert got.dtype == IO[io] and got.is_contiguous()
        check(got, ref, tl, "y")
    assert torch.equal(fin.double().cpu(), xp[:, T:])


def test_strides_alignment_and_order():
    """A transposed batch, a broadcast sequence and a [Bt,C,T] tensor whose channels are
    not consecutive (made dense by the binding) give the same outputs as a dense copy."""
    m = make(3, 50, 72, 4, "bf16", 2)
    w, b = up(m["weight"]), up(m["bias"])
    x = xslice(m, "cuda")
    (y0,), f0 = ssd.ssd_conv1d_fwd(x.contiguous(), w, b)
    tb = x.transpose(0, 1).contiguous().transpose(0, 1)
    ct = x.transpose(1, 2).contiguous().transpose(1, 2)
    for v in (tb, ct):
        (y1,), f1 = ssd.ssd_conv1d_fwd(v, w, b)
        assert torch.equal(y0, y1) and torch.equal(f0, f1)
    (y1,), _ = ssd.ssd_conv1d_fwd(x[:1].expand(3, -1, -1), w, b)
    for i in range(3):
        assert torch.equal(y1[i], y0[0])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_lengths_and_continuation(io):
    """Right-padded batch: lengths 0, 1, inside the taps, whole and past T (clamped); NaN in
    the padding never reaches an output; final states continue the sequences, in place."""
    T, W, C = 41, 4, 40
    lens = [0, 1, 2, 17, T, T + 9, -3]
    Bt = len(lens)
    m = make(Bt, T, C, W, io, 3)
    eff = [min(max(n, 0), T) for n in lens]
    for b, n in enumerate(eff):
        m["rows"][b, n:] = float("nan")
    state = up(m["init"]).clone()
    (y,), fin = ssd.ssd_conv1d_fwd(xslice(m, "cuda"), up(m["weight"]), up(m["bias"]),
                                   init_state=state, final_state=state,
                                   seq_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    assert fin is state
    for b, n in enumerate(eff):
        one = dict(m, rows=m["rows"][b:b + 1, :n], init=m["init"][b:b + 1])
        ref, pre, S, xp = formula(one, True)
        check(y[b:b + 1, :n], ref, bound(ref, pre, S, W, True, IO[io]), "len %d" % n)
        assert not y[b, n:].any()
        assert torch.equal(fin[b].double().cpu(), xp[0, n:])


def test_two_halves_equal_one_call():
    m = make(2, 100, 64, 4, "bf16", 4)
    x, w, b, s = xslice(m, "cuda"), up(m["weight"]), up(m["bias"]), up(m["init"])
    (y,), fin = ssd.ssd_conv1d_fwd(x, w, b, init_state=s)
    (ya,), s1 = ssd.ssd_conv1d_fwd(x[:, :33], w, b, init_state=s)
    (yb,), s2 = ssd.ssd_conv1d_fwd(x[:, 33:], w, b, init_state=s1)
    assert torch.equal(torch.cat([ya, yb], 1), y) and torch.equal(s2, fin)


@pytest.mark.parametrize("C", [4096, 4101])
def test_large_outputs_equal_their_parts(C):
    """Outputs past 256 MB are stored nontemporally: the same values as two shorter calls."""
    T = 33000
    assert T * C * 2 > 256 << 20 and T * C < 256 << 20
    x = torch.randn(1, T, C, device="cuda").to(torch.bfloat16)
    w, b = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    (y,), fin = ssd.ssd_conv1d_fwd(x, w, b)
    (ya,), s1 = ssd.ssd_conv1d_fwd(x[:, :17000], w, b)
    (yb,), s2 = ssd.ssd_conv1d_fwd(x[:, 17000:], w, b, init_state=s1)
    assert torch.equal(y[:, :17000], ya) and torch.equal(y[:, 17000:], yb)
    assert torch.equal(fin, s2)


def test_step_pool_past_32_bit_offsets():
    C, W = 4096, 4
    num = 2 ** 32 // (C * (W - 1)) + 3
    pool = torch.zeros(num, W - 1, C, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 2 ** 32
    small = torch.randn(2, W - 1, C, device="cuda").to(torch.bfloat16)
    pool[num - 1], pool[1] = small[0], small[1]
    x = torch.randn(2, C, device="cuda").to(torch.bfloat16)
    w = torch.randn(C, W, device="cuda")
    (y,) = ssd.ssd_conv1d_step(pool, x, w, slots=torch.tensor([num - 1, 1], dtype=torch.int32).cuda())
    (ref,) = ssd.ssd_conv1d_step(small, x, w)
    assert torch.equal(y, ref)
    assert torch.equal(pool[num - 1], small[0]) and torch.equal(pool[1], small[1])
    assert not pool[num - 2].any() and not pool[0].any()


@pytest.mark.parametrize("T", [0, 1, 2])
def test_shorter_than_the_taps(T):
    m = make(2, T, 24, 4, "f32", 5)
    (y,), fin = ssd.ssd_conv1d_fwd(xslice(m, "cuda"), up(m["weight"]), init_state=up(m["init"]))
    assert torch.equal(fin.double().cpu(), padded(m)[:, T:])
    (y,), fin = ssd.ssd_conv1d_fwd(xslice(m, "cuda"), up(m["weight"]))
    m["init"] = None
    assert torch.equal(fin.double().cpu(), padded(m)[:, T:]) and y.shape == (2, T, 24)


def test_no_sequences():
    m = make(0, 9, 24, 4, "f32", 5)
    (y,), fin = ssd.ssd_conv1d_fwd(xslice(m, "cuda"), up(m["weight"]))
    assert y.shape == (0, 9, 24) and fin.shape == (0, 3, 24)
    out = ssd.ssd_conv1d_bwd(xslice(m, "cuda"), up(m["weight"]), y, bias=torch.zeros(24).cuda())
    assert not out["dweight"].any() and not out["dbias"].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,splits,W,silu", [(1, (64,), 4, True), (5, (33, 5, 7), 3, True),
                                              (300, (1024, 64, 64), 4, True),
                                              (7, (40,), 2, False)])
def test_step(io, Bt, splits, W, silu):
    """Steps over a shuffled pool against the prompt form, with padded rows."""
    C = sum(splits)
    log("conv1d step", io, Bt, splits, W)
    m = make(Bt, 3, C, W, io, 6, slack=2, lead=1)
    g = torch.Generator().manual_seed(9)
    pool = Bt + 5
    slots = torch.randperm(pool, generator=g)[:Bt].to(torch.int32)
    state = torch.randn(pool, W - 1, C, generator=g).to(IO[io])
    m["init"] = state[slots.long()].clone()
    dead = [i for i in (2, 4) if i < Bt]
    for j, i in enumerate(dead):
        slots[i] = (-1, pool)[j]
    before = state.clone()
    st, sl = state.cuda(), slots.cuda()
    y, pre, S, xp = formula(m, silu)
    tol = bound(y, pre, S, W, silu, IO[io])
    x = xslice(m, "cuda")
    for t in range(3):
        ys = ssd.ssd_conv1d_step(st, x[:, t], up(m["weight"]), up(m["bias"]), silu=silu,
                                 splits=splits, slots=sl)
        for got, ref, tl in zip(ys, y[:, t].split(splits, 1), tol[:, t].split(splits, 1)):
            ref = ref.clone()
            ref[dead] = 0.0
            check(got, ref, tl, "y step %d" % t)
            assert not got[dead].any()
    got = st.cpu()
    live = [i for i in range(Bt) if i not in dead]
    idx = slots.long()[live]
    assert torch.equal(got[idx].double(), xp[live, 3:])
    rest = torch.ones(pool, dtype=torch.bool)
    rest[idx] = False
    assert torch.equal(got[rest], before[rest])   # slots not named are left as they were


def test_step_without_slots_on_another_stream():
    m = make(6, 1, 48, 4, "bf16", 7)
    w, b = up(m["weight"]), up(m["bias"])
    x = xslice(m, "cuda")[:, 0]
    s1, s2 = up(m["init"]).clone(), up(m["init"]).clone()
    (y1,) = ssd.ssd_conv1d_step(s1, x, w, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        (y2,) = ssd.ssd_conv1d_step(s2, x, w, b)
    side.synchronize()
    assert torch.equal(y1, y2) and torch.equal(s1, s2)


def grads(m, splits, silu, dy, dfinal):
    """The formula's gradients in float64, with bounds: each is a sum of products, off by
    at most its number of float32 roundings times the sum of its terms' magnitudes."""
    _, pre, S, xp = formula(m, silu)
    w = m["weight"].double()
    W = w.shape[1]
    T = pre.shape[1]
    d = torch.cat([v.double() for v in dy], 2)
    s = torch.sigmoid(pre)
    act = s * (1 + pre * (1 - s)) if silu else torch.ones_like(pre)
    dp = d * act
    # error of dp: of act (|act''| <= 0.5 times the error of pre; 8 + 2|pre| half-ulps of
    # its own arithmetic, whose terms stay below 1 + |pre|) and one product
    edp = d.abs() * (0.5 * U * (W + 2) * S + U * (8 + 2 * pre.abs()) * (1 + pre.abs())) if silu \
        else torch.zeros_like(d)
    edp = edp + U * dp.abs()
    dxp, bx = torch.zeros_like(xp), torch.zeros_like(xp)
    if dfinal is not None:
        dxp[:, T:] += dfinal.double()
    dw, bw = torch.empty_like(w), torch.empty_like(w)
    n = d.shape[0] * T
    terms = min(n, 32) + 8          # a run's serial sum, then the joins
    for k in range(W):
        dxp[:, k:k + T] += dp * w[:, k]
        bx[:, k:k + T] += (edp + U * (W + 2) * dp.abs()) * w[:, k].abs()
        dw[:, k] = (dp * xp[:, k:k + T]).sum((0, 1))
        bw[:, k] = ((edp + U * terms * dp.abs()) * xp[:, k:k + T].abs()).sum((0, 1))
    if dfinal is not None:
        bx[:, T:] += 2 * U * dfinal.double().abs()
    db = dp.sum((0, 1))
    bb = (edp + U * terms * dp.abs()).sum((0, 1))
    return dict(dx=(dxp[:, W - 1:], bx[:, W - 1:]), dinit=(dxp[:, :W - 1], bx[:, :W - 1]),
                dweight=(dw, bw), dbias=(db, bb))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,T,splits,W,silu", [
    (1, 1, (64,), 4, True), (2, 2, (5,), 4, True), (3, 37, (33, 5, 64), 3, True),
    (2, 300, (128, 64, 64), 4, True), (1, 700, (1030,), 4, False), (4, 70, (36,), 2, True),
    (2, 0, (36,), 4, True)])
def test_gradients(io, Bt, T, splits, W, silu):
    C = sum(splits)
    log("conv1d bwd", io, Bt, T, splits, W, silu)
    m = make(Bt, T, C, W, io, 8, lead=3)
    g = torch.Generator().manual_seed(4)
    dy = [torch.randn(Bt, T, c, generator=g) for c in splits]
    dfinal = torch.randn(Bt, W - 1, C, generator=g)
    args = (xslice(m, "cuda"), up(m["weight"]), [up(v) for v in dy], up(m["bias"]))
    out = ssd.ssd_conv1d_bwd(*args, silu=silu, init_state=up(m["init"]), dfinal=up(dfinal))
    ref = grads(m, splits, silu, dy, dfinal)
    for k, (r, b) in ref.items():
        check(out[k], r, b + 1e-30, k)
    again = ssd.ssd_conv1d_bwd(*args, silu=silu, init_state=up(m["init"]), dfinal=up(dfinal))
    for k in out:
        assert torch.equal(out[k], again[k])
    # without the optional ones
    out = ssd.ssd_conv1d_bwd(args[0], args[1], args[2], silu=silu, want_dinit=False)
    m["init"] = m["bias"] = None
    ref = grads(m, splits, silu, dy, None)
    assert out["dinit"] is None and out["dbias"] is None
    for k in ("dx", "dweight"):
        check(out[k], ref[k][0], ref[k][1] + 1e-30, k)


def test_gradient_differences():
    """Central differences of the float64 formula along random directions: the loss changes
    by the gradients' product with the direction."""
    m = make(2, 19, 12, 4, "f32", 10)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(2, 19, 12, generator=g)
    dfinal = torch.randn(2, 3, 12, generator=g)
    out = ssd.ssd_conv1d_bwd(xslice(m, "cuda"), up(m["weight"]), up(dy), up(m["bias"]),
                             init_state=up(m["init"]), dfinal=up(dfinal))

    def loss(mm):
        y, _, _, xp = formula(mm, True)
        return float((y * dy.double()).sum() + (xp[:, 19:] * dfinal.double()).sum())

    for key, name in (("rows", "dx"), ("weight", "dweight"), ("bias", "dbias"),
                      ("init", "dinit")):
        v = torch.randn(m[key].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        num = (loss(dict(m, **{key: m[key].double() + h * v}))
               - loss(dict(m, **{key: m[key].double() - h * v}))) / (2 * h)
        terms = out[name].double().cpu() * v
        # differences: h^2 / 6 of a third derivative below 10 per term, and 1e-16 / h of the
        # loss; the gradient: float32 sums of a few dozen terms
        tol = float(terms.abs().sum()) * 100 * U + 1e-6
        assert abs(float(terms.sum()) - num) <= tol, (name, float(terms.sum()), num, tol)


def test_graph_replays_follow_the_inputs():
    """Forward, step and gradients captured in one graph; each replay equals the eager calls
    on the inputs of that replay, with eager work between."""
    m = make(2, 64, 40, 4, "bf16", 11)
    x, w, b = xslice(m, "cuda").contiguous(), up(m["weight"]), up(m["bias"])
    pool = torch.zeros(2, 3, 40, dtype=torch.bfloat16, device="cuda")
    dy = torch.randn(2, 64, 40, device="cuda")

    def work(pool):
        (y,), fin = ssd.ssd_conv1d_fwd(x, w, b)
        (t,) = ssd.ssd_conv1d_step(pool, x[:, 0], w, b)
        gr = ssd.ssd_conv1d_bwd(x, w, dy, b)
        return [y, fin, t, gr["dx"], gr["dweight"], gr["dbias"], gr["dinit"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(pool)
    for r in range(3):
        x.copy_(torch.randn(x.shape, device="cuda"))
        dy.copy_(torch.randn(dy.shape, device="cuda"))
        eager_pool = pool.clone()
        ref = [v.clone() for v in work(eager_pool)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, ref):
            assert torch.equal(o, v)
        assert torch.equal(pool, eager_pool)
