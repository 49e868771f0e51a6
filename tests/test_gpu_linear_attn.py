"""Linear attention with a decay for each head against its float64 recurrence: prompts,
single tokens, gradients; every type, padded and shared dimension, ragged lengths, cut
sequences, states, strides, decays at both ends."""

import pytest
import torch

from selective_state_space_amd import ssd
from _block import TYPES, U, assert_near, attn_bar, attn_inputs, attn_ref, gen, randn

pytestmark = pytest.mark.gpu


def terms(T, K, V):
    """Roundings that one output passes through: the dot products over K (or V), the sums over
    tokens (decayed: not more than T), a few for each decay."""
    return T + 2 * max(K, V) + 64


def ref_args(c, kw):
    return (c["q"], c["k"], c["v"], c["log_decay"], kw["scale"], kw.get("init_state"),
            kw.get("seq_lens"))


def check_fwd(c, kw, **more):
    y, fin = ssd.ssd_linear_attn_fwd(**c, **kw, **more)
    yr, fr = attn_ref(*ref_args(c, kw))
    T, K, V = c["q"].shape[1], c["q"].shape[3], c["v"].shape[3]
    assert y.dtype == c["q"].dtype and fin.dtype == torch.float32
    assert_near(y, yr, attn_bar(y.dtype, terms(T, K, V)), "y")
    assert_near(fin, fr, attn_bar(torch.float32, terms(T, K, V)), "final")
    return y, fin


def check_bwd(c, kw):
    got = ssd.ssd_linear_attn_bwd(**c, **kw)
    ref = attn_ref(*ref_args(c, kw), dy=c["dy"], dfinal=kw.get("dfinal"))
    T, K, V = c["q"].shape[1], c["q"].shape[3], c["v"].shape[3]
    for n in ("dq", "dk", "dv", "dinit"):
        io = torch.float32 if n == "dinit" else c["q"].dtype
        assert got[n].dtype == io
        assert_near(got[n], ref[n], attn_bar(io, terms(T, K, V)), n)
    return got


# around the chunk's lengths (32 and 64 tokens) and a tile's (16)
LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 129, 200]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(T, io):
    c, kw = attn_inputs(T, 2, T, 3, 3, 64, 64, TYPES[io], init=T % 2 == 0, grads=True)
    dy, df = c.pop("dy"), kw.pop("dfinal", None)
    check_fwd(c, kw)
    check_bwd(dict(c, dy=dy), dict(kw, **({} if df is None else dict(dfinal=df))))


DIMS = [(8, 8), (16, 48), (48, 16), (64, 128), (128, 64), (128, 128), (80, 136), (136, 72),
        (256, 64), (64, 256), (256, 256), (200, 248), (120, 128)]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("K,V", DIMS)
def test_dims(K, V, io):
    c, kw = attn_inputs(K + V, 2, 150, 2, 2, K, V, TYPES[io], init=True, grads=True)
    dy, df = c.pop("dy"), kw.pop("dfinal")
    check_fwd(c, kw)
    check_bwd(dict(c, dy=dy), dict(kw, dfinal=df))


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("H,G", [(4, 1), (6, 2), (6, 3), (5, 5)])
def test_shared_heads(H, G, io):
    c, kw = attn_inputs(H * G, 2, 70, H, G, 64, 72, TYPES[io], init=True, lens=[70, 33],
                        grads=True)
    dy, df = c.pop("dy"), kw.pop("dfinal")
    check_fwd(c, kw)
    check_bwd(dict(c, dy=dy), dict(kw, dfinal=df))


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("init", [False, True])
def test_padded_batch(io, init):
    """Lengths of 0, 1, past the end and negative; what lies behind a length is not read, and
    its outputs are zeros."""
    lens = [0, 1, 64, 65, 100, 130, -3]
    c, kw = attn_inputs(5, 7, 100, 2, 2, 64, 64, TYPES[io], init=init, lens=lens, grads=True)
    for b, n in enumerate(lens):
        for t in ("q", "k", "v", "dy"):
            c[t][b, max(n, 0):] = float("nan")
    plain = {n: t.nan_to_num(0.0) for n, t in c.items()}
    dy, df = c.pop("dy"), kw.pop("dfinal", None)
    y, fin = ssd.ssd_linear_attn_fwd(**c, **kw)
    yr, fr = attn_ref(*ref_args(plain, kw))
    assert_near(y, yr, attn_bar(y.dtype, terms(100, 64, 64)), "y")
    assert_near(fin, fr, attn_bar(torch.float32, terms(100, 64, 64)), "final")
    got = ssd.ssd_linear_attn_bwd(**c, dy=dy, dfinal=df, **kw)
    ref = attn_ref(*ref_args(plain, kw), dy=plain["dy"], dfinal=df)
    for n, t in got.items():
        assert_near(t, ref[n], attn_bar(t.dtype, terms(100, 64, 64)), n)
    for b, n in enumerate(lens):
        n = min(max(n, 0), 100)
        assert not y[b, n:].any()
        for t in ("dq", "dk", "dv"):
            assert not got[t][b, n:].any()
        if n == 0 and init:
            assert torch.equal(fin[b], kw["init_state"][b])
            assert torch.equal(got["dinit"][b], df[b])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("T,lens", [(1500, None), (3000, [3000, 1300]), (4096, [0, 4095])])
def test_cut_over_time(T, lens, io):
    """Few heads: sequences are cut, lengths that end in the first, a middle and the last
    part."""
    Bt = 2 if lens else 1
    c, kw = attn_inputs(T, Bt, T, 2, 2, 64, 64, TYPES[io], init=True, lens=lens, grads=True)
    c["log_decay"] = torch.tensor([-0.5, -0.0004], device="cuda")
    dims = ssd.AttnDims(Bt, T, 2, 2, 64, 64, 0, 0, 0, 0, 0, 0, 1 if io == "bf16" else 0, 1.0)
    layout = ssd.linear_attn_layout(dims)
    assert layout.fwd_segments > 1 and layout.bwd_segments > 1
    dy, df = c.pop("dy"), kw.pop("dfinal")
    check_fwd(c, kw)
    check_bwd(dict(c, dy=dy), dict(kw, dfinal=df))


@pytest.mark.parametrize("T", [40, 2000])
def test_state_in_place(T):
    """init_state and final_state in one tensor, in one pass and cut over time; a prompt in
    two calls is the prompt in one."""
    c, kw = attn_inputs(3, 1, T, 2, 2, 64, 64, torch.float32, init=True)
    init = kw.pop("init_state")
    y, fin = ssd.ssd_linear_attn_fwd(**c, init_state=init, **kw)
    own = init.clone()
    y2, fin2 = ssd.ssd_linear_attn_fwd(**c, init_state=own, final_state=own, **kw)
    assert fin2 is own and torch.equal(fin, own) and torch.equal(y, y2)
    cut = T // 3
    part = lambda s: {n: (t[:, s] if t.dim() == 4 else t) for n, t in c.items()}
    own = init.clone()
    ya, _ = ssd.ssd_linear_attn_fwd(**part(slice(0, cut)), init_state=own, final_state=own, **kw)
    yb, _ = ssd.ssd_linear_attn_fwd(**part(slice(cut, T)), init_state=own, final_state=own, **kw)
    bar = attn_bar(torch.float32, terms(T, 64, 64))
    assert_near(torch.cat([ya, yb], 1), y, 2 * bar, "y")
    assert_near(own, fin, 2 * bar, "final")


@pytest.mark.parametrize("io", TYPES)
def test_decays(io):
    """From none to forgetting at once: exp(0) = 1, a long memory, one token's, exp(-1000),
    the lowest float32 and -infinity."""
    rates = [0.0, -1e-6, -0.3, -30.0, -1000.0, torch.finfo(torch.float32).min, -float("inf")]
    c, kw = attn_inputs(11, 1, 140, len(rates), len(rates), 64, 64, TYPES[io], init=True,
                        grads=True)
    c["log_decay"] = torch.tensor(rates, device="cuda")
    dy, df = c.pop("dy"), kw.pop("dfinal")
    y, fin = ssd.ssd_linear_attn_fwd(**c, **kw)
    yr, fr = attn_ref(*ref_args(c, kw))
    got = ssd.ssd_linear_attn_bwd(**c, dy=dy, dfinal=df, **kw)
    ref = attn_ref(*ref_args(c, kw), dy=dy, dfinal=df)
    for h in range(len(rates)):   # each head on its own: they differ in size
        n = terms(140, 64, 64)
        assert_near(y[:, :, h], yr[:, :, h], attn_bar(y.dtype, n), "y %d" % h)
        assert_near(fin[:, h], fr[:, h], attn_bar(torch.float32, n), "final %d" % h)
        for t in ("dq", "dk", "dv"):
            assert_near(got[t][:, :, h], ref[t][:, :, h], attn_bar(y.dtype, n), "%s %d" % (t, h))
        assert_near(got["dinit"][:, h], ref["dinit"][:, h], attn_bar(torch.float32, n),
                    "dinit %d" % h)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strided(io, off):
    """Slices of one projection's rows, in place (off 0 and 8) or, where rows start off 16
    bytes, copied: the same bits as dense tensors."""
    H, G, K, V, Bt, T = 4, 2, 64, 32, 2, 70
    g = gen(2)
    row = H * K + G * K + G * V
    proj = randn(g, Bt, T, row + 16, dtype=TYPES[io])[:, :, off:off + row]
    q, k, v = (t.unflatten(2, (n, -1)) for t, n in zip(proj.split((H * K, G * K, G * V), 2),
                                                       (H, G, G)))
    decay = -torch.rand(H, generator=g, device="cuda")
    y, fin = ssd.ssd_linear_attn_fwd(q, k, v, decay)
    yd, fd = ssd.ssd_linear_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), decay)
    assert torch.equal(y, yd) and torch.equal(fin, fd)
    dy = randn(g, Bt, T, H, V, dtype=TYPES[io])
    a = ssd.ssd_linear_attn_bwd(q, k, v, decay, dy)
    b = ssd.ssd_linear_attn_bwd(q.contiguous(), k.contiguous(), v.contiguous(), decay, dy)
    assert all(torch.equal(a[n], b[n]) for n in a)
    # time first, and one token's keys for every token (stride 0)
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    kt = k[:, :1].expand(-1, T, -1, -1)
    y, _ = ssd.ssd_linear_attn_fwd(qt, kt, v, decay)
    yd, _ = ssd.ssd_linear_attn_fwd(q.contiguous(), kt.contiguous(), v.contiguous(), decay)
    assert torch.equal(y, yd)


def test_empty():
    z = lambda *s: torch.zeros(*s, device="cuda")
    init = torch.randn(2, 3, 64, 64, device="cuda")
    decay = -torch.ones(3, device="cuda")
    y, fin = ssd.ssd_linear_attn_fwd(z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3, 64), decay,
                                     init_state=init)
    assert y.shape == (2, 0, 3, 64) and torch.equal(fin, init)
    _, fin = ssd.ssd_linear_attn_fwd(z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3, 64), decay)
    assert not fin.any()
    got = ssd.ssd_linear_attn_bwd(z(2, 0, 3, 64), z(2, 0, 1, 64), z(2, 0, 1, 64), decay,
                                  z(2, 0, 3, 64), dfinal=init)
    assert torch.equal(got["dinit"], init)
    y, fin = ssd.ssd_linear_attn_fwd(z(0, 5, 3, 64), z(0, 5, 3, 64), z(0, 5, 3, 64), decay)
    assert y.shape == (0, 5, 3, 64) and fin.shape == (0, 3, 64, 64)


@pytest.mark.parametrize("io", TYPES)
def test_reruns_and_outputs(io):
    """Reruns give the same bits, outputs passed in too; no final state where none is asked."""
    c, kw = attn_inputs(9, 1, 1700, 2, 1, 64, 64, TYPES[io], init=True, grads=True)
    dy, df = c.pop("dy"), kw.pop("dfinal")
    y, fin = ssd.ssd_linear_attn_fwd(**c, **kw)
    y2, none = ssd.ssd_linear_attn_fwd(**c, y=torch.empty_like(y), want_final=False, **kw)
    assert none is None and torch.equal(y, y2)
    a = ssd.ssd_linear_attn_bwd(**c, dy=dy, dfinal=df, **kw)
    b = ssd.ssd_linear_attn_bwd(**c, dy=dy, dfinal=df, want_dinit=False, **kw)
    assert b["dinit"] is None
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dv"))


def test_gradients_against_differences():
    """The loss sum(w y) + sum(u final) along random directions, float32 kernels: central
    differences of the float64 recurrence, whose own error is of order step^2."""
    c, kw = attn_inputs(21, 2, 75, 4, 2, 16, 24, torch.float32, init=True, lens=[75, 40],
                        grads=True)
    dy, df = c.pop("dy"), kw.pop("dfinal")
    got = ssd.ssd_linear_attn_bwd(**c, dy=dy, dfinal=df, **kw)
    g = gen(22)

    def loss(x):
        y, fin = attn_ref(x["q"], x["k"], x["v"], c["log_decay"], kw["scale"], x["init_state"],
                          kw["seq_lens"])
        return float((y * dy.double()).sum() + (fin * df.double()).sum())

    base = {n: t.double() for n, t in dict(c, init_state=kw["init_state"]).items()}
    for n in ("q", "k", "v", "init_state"):
        way = torch.randn(base[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        diff = (loss(dict(base, **{n: base[n] + h * way}))
                - loss(dict(base, **{n: base[n] - h * way}))) / (2 * h)
        grad = got["dinit" if n == "init_state" else "d" + n].double()
        along = float((grad * way).sum())
        size = float(grad.norm())   # a random direction's slope is of this size
        assert abs(along - diff) <= 1e-5 * size * way.numel() ** 0.5, (n, along, diff)


# ---------------------------------------------------------------------------
# single tokens

@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("K,V", [(8, 8), (16, 40), (64, 64), (72, 128), (128, 80), (128, 128),
                                 (256, 256), (24, 136)])
def test_step(K, V, io):
    H, G, Bt, pool = 4, 2, 5, 9
    g = gen(K * V)
    q, k, v = (randn(g, Bt, n, d, dtype=TYPES[io]) for n, d in ((H, K), (G, K), (G, V)))
    decay = -torch.rand(H, generator=g, device="cuda")
    state = randn(g, pool, H, K, V)
    slots = torch.tensor([7, 0, -1, 3, 9], dtype=torch.int32, device="cuda")   # two are padding
    before = state.clone()
    y = ssd.ssd_linear_attn_step(state, q, k, v, decay, slots=slots)
    live = [0, 1, 3]
    at = [7, 0, 3]
    yr, sr = attn_ref(q[live][:, None], k[live][:, None], v[live][:, None], decay, K ** -0.5,
                      before[at])
    assert_near(state[at], sr, attn_bar(torch.float32, 16), "state")
    # one sum over K in float32 and the output's rounding
    assert_near(y[live], yr[:, 0], 2.0 ** -24 * (2 * K) ** 0.5 + (io == "bf16") * U[y.dtype], "y")
    assert not y[[2, 4]].any()
    rest = [i for i in range(pool) if i not in at]
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("io", TYPES)
def test_steps_are_the_prompt(io):
    c, kw = attn_inputs(31, 3, 20, 4, 2, 64, 128, TYPES[io], init=True)
    y, fin = ssd.ssd_linear_attn_fwd(**c, **kw)
    state = kw["init_state"].clone()
    ys = [ssd.ssd_linear_attn_step(state, c["q"][:, t], c["k"][:, t], c["v"][:, t],
                                   c["log_decay"], scale=kw["scale"]) for t in range(20)]
    bar = attn_bar(TYPES[io], terms(20, 64, 128))
    assert_near(torch.stack(ys, 1), y.double(), 2 * bar, "y")
    assert_near(state, fin.double(), 2 * attn_bar(torch.float32, terms(20, 64, 128)), "state")


def test_step_empty_and_decays():
    z = lambda *s: torch.zeros(*s, device="cuda")
    y = ssd.ssd_linear_attn_step(z(0, 2, 64, 64), z(0, 2, 64), z(0, 2, 64), z(0, 2, 64), z(2))
    assert y.shape == (0, 2, 64)
    state = torch.randn(1, 2, 64, 64, device="cuda")
    before = state.clone()
    v = torch.randn(1, 2, 64, device="cuda")
    decay = torch.tensor([0.0, -float("inf")], device="cuda")
    ssd.ssd_linear_attn_step(state, z(1, 2, 64), torch.ones(1, 2, 64, device="cuda"), v, decay)
    assert torch.equal(state[0, 0], before[0, 0] + v[0, 0])
    assert torch.equal(state[0, 1], v[0, 1].expand(64, 64))


BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("K,V", [(64, 64), (128, 72), (136, 64), (64, 256)])
@pytest.mark.parametrize("at", [0, 1, 15, 16, 17, 31, 32, 50, 69])
def test_what_is_not_finite_stays_behind_its_token(at, K, V, io):
    """An infinity or a NaN in token `at` of a key, a value or a query leaves the tokens before
    it, other sequences and other heads as they are; in a value, the other columns too."""
    T, H, G = 70, 4, 2
    c, kw = attn_inputs(9, 2, T, H, G, K, V, TYPES[io], init=True, grads=True)
    dy, df = c.pop("dy"), kw.pop("dfinal")
    y, _ = ssd.ssd_linear_attn_fwd(**c, **kw)
    bar = attn_bar(y.dtype, terms(T, K, V))
    for i, name in enumerate("kvq"):
        d = {n: t.clone() for n, t in c.items()}
        d[name][1, at, 1, 3] = BAD[(i + at) % 3]
        got, fin = ssd.ssd_linear_attn_fwd(**d, **kw)
        heads = slice(1, 2) if name == "q" else slice(2, 4)     # that read it
        others = [h for h in range(H) if not (heads.start <= h < heads.stop)]
        assert torch.equal(got[0], y[0]) and torch.equal(got[1][:, others], y[1][:, others])
        assert_near(got[1, :at, heads], y[1, :at, heads], 2 * bar, "%s before" % name)
        if name == "v":
            keep = [j for j in range(V) if j != 3]
            assert_near(got[1][:, heads][..., keep], y[1][:, heads][..., keep], 2 * bar, "columns")
            assert not torch.isfinite(got[1, at:, heads, 3]).any()
        else:
            assert not torch.isfinite(got[1, at, heads]).any()
        if name == "q":
            assert_near(got[1, at + 1:, heads], y[1, at + 1:, heads], 2 * bar, "after")
            assert torch.isfinite(fin).all()
    # backwards, a bad dy reaches dk and dv of the tokens up to it, and dq of its own alone
    want = ssd.ssd_linear_attn_bwd(**c, dy=dy, dfinal=df, **kw)
    bad = dy.clone()
    bad[1, at, 1, 3] = float("nan")
    got = ssd.ssd_linear_attn_bwd(**c, dy=bad, dfinal=df, **kw)
    for n in ("dk", "dv"):
        assert torch.equal(got[n][0], want[n][0])
        assert torch.equal(got[n][1, :, 1:], want[n][1, :, 1:])
        assert_near(got[n][1, at + 1:], want[n][1, at + 1:], 2 * bar, n + " behind")
        assert not torch.isfinite(got[n][1, at, 0]).all()
    assert_near(got["dq"][1, :at], want["dq"][1, :at], 2 * bar, "dq before")
    assert_near(got["dq"][1, at + 1:], want["dq"][1, at + 1:], 2 * bar, "dq behind")
