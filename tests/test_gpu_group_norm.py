"""The group norm behind a mixer against its float64 form: every form, type and way that a
row lies on lanes; strides, lengths, large means, gradients."""

import pytest
import torch

from selective_state_space_amd import ssd
from _block import TYPES, U, assert_near, gen, norm_ref, randn

pytestmark = pytest.mark.gpu

FORMS = ["plain", "silu", "gate", "gated_input"]


def bar(io, S):
    """Relative 2-norm: sums over S channels, and some 32 roundings of a lane's own arithmetic
    (2 of the transcendental unit's, off by a whole step, count four), of independent signs;
    a bf16 output rounds once more, half a step at most."""
    f = 2.0 ** -24 * (S + 32) ** 0.5
    return f if io == torch.float32 else U[io] + f


def inputs(seed, Bt, T, C, io, form, affine=True, dy=True):
    g = gen(seed)
    x = (randn(g, Bt, T, C) + 0.5) * torch.exp(randn(g, C, scale=0.3))
    c = dict(x=x.to(io))
    kw = dict(form=form)
    if form.startswith("gate"):
        kw["z"] = randn(g, Bt, T, C, dtype=io)
    if affine:
        kw["weight"], kw["bias"] = 1.0 + randn(g, C, scale=0.2), randn(g, C, scale=0.2)
    return c["x"], kw, randn(g, Bt, T, C, dtype=io) if dy else None


def check(x, groups, kw, dy, seq_lens=None):
    S = x.shape[-1] // groups
    y = ssd.ssd_group_norm_fwd(x, groups, seq_lens=seq_lens, **kw)
    assert y.dtype == x.dtype and y.is_contiguous()
    assert_near(y, norm_ref(x, groups, lens=seq_lens, **kw), bar(x.dtype, S), "y")
    if dy is None:
        return y, None
    got = ssd.ssd_group_norm_bwd(x, groups, dy, seq_lens=seq_lens, **kw)
    ref = norm_ref(x, groups, lens=seq_lens, dy=dy, **kw)
    tokens = x.shape[0] * x.shape[1]
    for n, r in ref.items():
        io = x.dtype if n in ("dx", "dz") else torch.float32
        assert got[n].dtype == io
        # weight and bias gradients: sums over the tokens too
        assert_near(got[n], r, bar(io, 3 * S + (0 if n in ("dx", "dz") else tokens)), n)
    assert {n for n, t in got.items() if t is not None} == set(ref)
    return y, got


# one to 16 accesses of single or 16-byte vectors on 16, 64, 256 and 1024 lanes
SIZES = [(1, 1), (3, 5), (7, 16), (2, 64), (4, 128), (1, 100), (5, 160), (2, 512), (1, 1000),
         (3, 260), (1, 2048), (2, 1536), (1, 5120), (1, 4098), (1, 8192), (1, 16384), (1, 16383),
         (1, 9000)]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("groups,size", SIZES)
def test_sizes(groups, size, io):
    form = FORMS[(groups + size) % 4]
    x, kw, dy = inputs(size, 2, 5, groups * size, TYPES[io], form)
    if size == 1:   # one channel: nothing is left of it but the bias
        y = ssd.ssd_group_norm_fwd(x, groups, **kw)
        assert torch.isfinite(y).all()
        return
    check(x, groups, dict(kw, rms=size % 3 == 0), dy)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("affine", [False, True])
def test_forms(form, rms, affine, io):
    for groups, size in ((4, 128), (2, 50), (1, 640)):
        x, kw, dy = inputs(groups, 3, 7, groups * size, TYPES[io], form, affine)
        check(x, groups, dict(kw, rms=rms), dy)


@pytest.mark.parametrize("io", TYPES)
def test_many_tokens(io):
    """Runs of several tokens per lane, the last shorter; sums over all of them."""
    for Bt, T, groups, size in ((2, 4099, 2, 64), (1, 6001, 1, 512), (3, 1111, 1, 2048)):
        x, kw, dy = inputs(T, Bt, T, groups * size, TYPES[io], "gate")
        check(x, groups, kw, dy)


def test_weight_or_bias_alone():
    x, kw, dy = inputs(1, 2, 9, 256, torch.float32, "silu")
    for n in ("weight", "bias"):
        one = {k: v for k, v in kw.items() if k != n}
        _, got = check(x, 2, one, dy)
        assert got["d" + n] is None


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form", ["plain", "gate"])
def test_strided(form, io):
    """Slices of wider rows, off 16 bytes too, time first, and one row for all tokens: read in
    place."""
    g = gen(4)
    for off, pad in ((0, 16), (1, 3), (8, 40)):
        wide = randn(g, 2, 6, 256 + pad + off, dtype=TYPES[io])
        x = wide[:, :, off:off + 256]
        z = wide.flip(2)[:, :, pad:pad + 256] if form == "gate" else None
        check(x, 2, dict(form=form, z=z), randn(g, 2, 6, 256, dtype=TYPES[io]))
    x = randn(g, 6, 2, 256, dtype=TYPES[io]).transpose(0, 1)
    z = randn(g, 2, 1, 256, dtype=TYPES[io]).expand(-1, 6, -1) if form == "gate" else None
    check(x, 2, dict(form=form, z=z), randn(g, 2, 6, 256, dtype=TYPES[io]))


@pytest.mark.parametrize("io", TYPES)
def test_tokens_alone(io):
    """[Bt,C] is one token of each sequence."""
    x, kw, dy = inputs(8, 4, 1, 384, TYPES[io], "gate")
    y, got = check(x, 3, kw, dy)
    one = {n: t[:, 0] if n == "z" else t for n, t in kw.items()}
    assert torch.equal(ssd.ssd_group_norm_fwd(x[:, 0], 3, **one), y[:, 0])
    flat = ssd.ssd_group_norm_bwd(x[:, 0], 3, dy[:, 0], **one)
    assert flat["dx"].shape == (4, 384) and torch.equal(flat["dx"], got["dx"][:, 0])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form", FORMS)
def test_padded_batch(form, io):
    lens = [0, 7, 3, 100, -2]
    x, kw, dy = inputs(6, 5, 7, 192, TYPES[io], form)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref_y = norm_ref(x, 3, lens=seq_lens, **kw)
    ref = norm_ref(x, 3, lens=seq_lens, dy=dy, **kw)
    for b, n in enumerate(lens):
        for t in (x, dy, kw.get("z")):
            if t is not None:
                t[b, max(n, 0):] = float("nan")
    y = ssd.ssd_group_norm_fwd(x, 3, seq_lens=seq_lens, **kw)
    got = ssd.ssd_group_norm_bwd(x, 3, dy, seq_lens=seq_lens, **kw)
    assert_near(y, ref_y, bar(x.dtype, 64), "y")
    for n, r in ref.items():
        assert_near(got[n], r, bar(got[n].dtype, 3 * 64 + 35), n)
    for b, n in enumerate(lens):
        assert not y[b, max(n, 0):].any() and not got["dx"][b, max(n, 0):].any()


def test_large_mean():
    """A mean of 2^10 deviations: each channel less the mean is known to 2^-24 2^10 of a
    deviation, and so the output."""
    g = gen(3)
    x = randn(g, 2, 3, 1024) + 1024.0
    y = ssd.ssd_group_norm_fwd(x, 1)
    assert_near(y, norm_ref(x, 1), 2.0 ** -24 * 2.0 ** 10, "y")


def test_constant_and_small_rows():
    """No deviation: eps alone, so zeros (then the bias); and rows far below eps."""
    b = torch.arange(64.0, device="cuda")
    for rms in (False, True):
        y = ssd.ssd_group_norm_fwd(torch.zeros(2, 3, 64, device="cuda"), 2, bias=b, rms=rms)
        assert torch.equal(y, b.expand(2, 3, 64))
    x = torch.full((1, 1, 64), 3.0, device="cuda")
    assert not ssd.ssd_group_norm_fwd(x, 2).any()
    g = gen(9)
    x = randn(g, 1, 4, 64, scale=1e-18)
    check(x, 2, dict(eps=1e-5), None)


def test_extreme_gates():
    """silu at gates of +-200 and +-3e4: 0 and z, slopes 0 and 1."""
    g = gen(12)
    x = randn(g, 1, 2, 64)
    z = torch.tensor([-3e4, -200.0, 200.0, 3e4], device="cuda").repeat(16).expand(1, 2, 64)
    for form in ("gate", "gated_input"):
        check(x, 1, dict(form=form, z=z.contiguous(), eps=1e-5), randn(g, 1, 2, 64))


def test_empty():
    z = lambda *s: torch.zeros(*s, device="cuda")
    for shape in ((0, 4, 64), (3, 0, 64)):
        assert ssd.ssd_group_norm_fwd(z(*shape), 2).shape == shape
        got = ssd.ssd_group_norm_bwd(z(*shape), 2, z(*shape), weight=z(64) + 1, bias=z(64))
        assert got["dx"].shape == shape
        assert not got["dweight"].any() and not got["dbias"].any()


@pytest.mark.parametrize("form", FORMS)
def test_gradients_against_differences(form):
    """Central differences of the float64 form along random directions."""
    x, kw, dy = inputs(17, 2, 3, 96, torch.float32, form)
    got = ssd.ssd_group_norm_bwd(x, 3, dy, **kw)
    base = dict(x=x.double(), **{n: t.double() for n, t in kw.items() if n != "form"})
    g = gen(18)
    for n in base:
        way = torch.randn(base[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        at = [float((norm_ref(groups=3, form=form, **dict(base, **{n: base[n] + s * way}))
                     * dy.double()).sum()) for s in (h, -h)]
        along = float((got["d" + n].double() * way).sum())
        size = float(got["d" + n].double().norm()) * way.numel() ** 0.5
        assert abs(along - (at[0] - at[1]) / (2 * h)) <= 1e-5 * size, n


def test_reruns_and_outputs():
    x, kw, dy = inputs(5, 2, 700, 1024, torch.bfloat16, "gate")
    y = ssd.ssd_group_norm_fwd(x, 8, **kw)
    out = torch.empty_like(y)
    assert ssd.ssd_group_norm_fwd(x, 8, y=out, **kw) is out and torch.equal(out, y)
    a, b = (ssd.ssd_group_norm_bwd(x, 8, dy, **kw) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
