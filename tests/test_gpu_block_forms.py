"""Every form that sizes choose of linear attention and of the 4-bit products, against float64."""

import pytest
import torch

from selective_state_space_amd import ssd

from _block import TYPES, attn_inputs, gen, randn
from block_forms import ATTN_BWD, ATTN_FWD
from test_gpu_group_norm import FORMS, check as check_norm, inputs as norm_inputs
from test_gpu_linear_attn import check_bwd, check_fwd
from test_gpu_w4 import check, packed

pytestmark = pytest.mark.gpu


def lengths(Bt, T):
    """Whole sequences, empty ones, and all between."""
    return [T if b % 3 == 0 else (7 * b * b) % (T + 1) for b in range(Bt)]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("sizes", [s for s, *_ in ATTN_FWD])
def test_linear_attn_fwd(sizes, io):
    Bt, T, H, G, K, V = sizes
    c, kw = attn_inputs(Bt + T, Bt, T, H, G, K, V, TYPES[io], init=True, lens=lengths(Bt, T))
    check_fwd(c, kw)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("sizes", [s for s, *_ in ATTN_BWD])
def test_linear_attn_bwd(sizes, io):
    Bt, T, H, G, K, V = sizes
    c, kw = attn_inputs(Bt + T, Bt, T, H, G, K, V, TYPES[io], init=True, lens=lengths(Bt, T),
                        grads=True)
    check_bwd(c, kw)


# one and two tiles of outputs for every number of row tiles, and two and four outputs a
# wavefront for one and two rows
@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("rows,outputs", [(1, 8191), (1, 8193), (2, 8191), (2, 8195),
                                          (9, 8100), (9, 12400), (9, 8300), (25, 2000), (25, 4000),
                                          (25, 8300), (40, 4000), (40, 4200), (60, 900),
                                          (60, 4000), (60, 4200), (100, 500), (100, 2100)])
def test_w4_linear(rows, outputs, io):
    g = gen(rows + outputs)
    codes, scales = packed(g, outputs, 192, 64)
    check(randn(g, rows, 192, dtype=TYPES[io]), codes, scales, randn(g, outputs))


# groups on 4, 8, 16, 32 and 64 lanes, 2 accesses on 64, workgroups of 256 and 1024 lanes; of
# channels in 16-byte accesses of either type, and of single ones
@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("groups,size", [
    (9, 7), (11, 8), (7, 13), (9, 16), (5, 27), (7, 32), (3, 50), (5, 64), (3, 101),
    (3, 128), (3, 200), (3, 256), (2, 301), (2, 512), (2, 1024), (2, 1200), (1, 1501), (1, 2501),
    (1, 2600), (1, 6000), (1, 12000)])
def test_group_norm(groups, size, io):
    for form in FORMS:
        x, kw, dy = norm_inputs(size, 3, 41, groups * size, TYPES[io], form)
        lens = torch.tensor([41, 0, 17], dtype=torch.int32, device="cuda")
        check_norm(x, groups, kw, dy, lens)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("groups,size", [(37, 2), (21, 4)])
def test_group_norm_of_a_few_channels(groups, size, io):
    """Two or four channels may lie as near to each other as they like, and then u - mean, and
    the terms of dx, cancel: a bar relative to the result holds for no arithmetic of 32 bits.
    Errors are held to the terms instead.  With m the mean, x - m is off by some half steps of
    |x| + |m|, so the normalised c by those of C = (|x| + |m|) rstd, and y = c w + b by those
    of C |w| + |b|; rstd by a few relative half steps, since sum(x - m) = 0 takes the mean's
    error out of the variance to first order.  dx = rstd (d - mean d - c mean(d c)) has the
    terms |d|, mean |d|, C mean |d c| and |c| mean(|d| C), and the weights' gradients |dy| C and
    |dy| summed.  Each passes through S + 32 roundings of independent signs, the sums over
    tokens through as many more."""
    io = TYPES[io]
    x, kw, dy = norm_inputs(size, 3, 41, groups * size, io, "plain")
    w, b = kw["weight"].double(), kw["bias"].double()
    split = lambda t: t.unflatten(-1, (groups, size))
    X = split(x.double())
    m = X.mean(-1, keepdim=True)
    rstd = ((X - m).square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    c, C, d = (X - m) * rstd, (X.abs() + m.abs()) * rstd, split(dy.double() * w)
    mean = lambda t: t.mean(-1, keepdim=True)
    tokens = lambda t: t.flatten(2).sum((0, 1))
    D = split(dy.double())
    y = ssd.ssd_group_norm_fwd(x, groups, **kw)
    got = dict(ssd.ssd_group_norm_bwd(x, groups, dy, **kw), y=y)
    n, f = x.shape[0] * x.shape[1], torch.float32
    for name, ref, terms, count, out in (
            ("y", c.flatten(2) * w + b, C.flatten(2) * w.abs() + b.abs(), size, io),
            ("dx", (rstd * (d - mean(d) - c * mean(d * c))).flatten(2),
             (rstd * (d.abs() + mean(d.abs()) + C * mean((d * c).abs())
                      + c.abs() * mean(d.abs() * C))).flatten(2), size, io),
            ("dweight", tokens(D * c), tokens(D.abs() * C), size + n, f),
            ("dbias", tokens(D), tokens(D.abs()), size + n, f)):
        bar = 2.0 ** -24 * (count + 32) ** 0.5 * float(terms.norm())
        if out == torch.bfloat16:
            bar += 2.0 ** -8 * float(ref.norm())
        off = float((got[name].double() - ref).norm())
        print("  %-8s off %.3g of %.3g" % (name, off, bar), flush=True)
        assert off <= bar, name


@pytest.mark.parametrize("io", TYPES)
def test_batches_of_padding_alone(io):
    """Every length zero: outputs and gradients are zeros, states pass through."""
    for Bt, T, H, G, K, V in ((3, 40, 4, 2, 64, 72), (1, 1100, 2, 2, 64, 64)):
        c, kw = attn_inputs(1, Bt, T, H, G, K, V, TYPES[io], init=True, lens=[0] * Bt, grads=True)
        dy, df = c.pop("dy"), kw.pop("dfinal")
        nan = {n: torch.full_like(t, float("nan")) if t.dim() > 1 else t for n, t in c.items()}
        y, fin = ssd.ssd_linear_attn_fwd(**nan, **kw)
        assert not y.any() and torch.equal(fin, kw["init_state"])
        got = ssd.ssd_linear_attn_bwd(**nan, dy=torch.full_like(dy, float("nan")), dfinal=df, **kw)
        assert not any(got[n].any() for n in ("dq", "dk", "dv")) and torch.equal(got["dinit"], df)
    x = torch.full((3, 9, 70), float("nan"), device="cuda").to(TYPES[io])
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    w = torch.ones(70, device="cuda")
    assert not ssd.ssd_group_norm_fwd(x, 7, w, w, seq_lens=lens).any()
    got = ssd.ssd_group_norm_bwd(x, 7, x, w, w, seq_lens=lens)
    assert not any(got[n].any() for n in ("dx", "dweight", "dbias"))
    state = torch.randn(4, 2, 64, 64, device="cuda")
    keep = state.clone()
    q = torch.randn(3, 2, 64, device="cuda").to(TYPES[io])
    y = ssd.ssd_linear_attn_step(state, q, q, q, -torch.ones(2, device="cuda"),
                                 slots=torch.tensor([-1, 4, 1 << 30], dtype=torch.int32).cuda())
    assert not y.any() and torch.equal(state, keep)


@pytest.mark.parametrize("op", ["linear_attn", "linear_attn_bwd", "step", "norm", "w4"])
def test_offsets_past_32_bits(op):
    """Rows, states and weights whose byte (and element) offsets pass 2^32: a batch row, a pool
    slot or an output there reads and writes its own."""
    far = (1 << 31) + (1 << 20)          # elements
    g, bf = gen(7), torch.bfloat16
    if op.startswith("linear_attn"):
        H, T, d = 2, 40, 64
        flat = torch.empty(far * 2 + 4096 * T, dtype=bf, device="cuda")
        take = lambda: torch.as_strided(flat, (2, T, H, d), (far * 2, 3 * H * d, d, 1))
        q = take()
        k, v = (torch.as_strided(flat, q.shape, q.stride(), i * H * d) for i in (1, 2))
        for t in (q, k, v):
            t.copy_(randn(g, *t.shape, dtype=bf))
        r = torch.tensor([-0.3, -0.01], device="cuda")
        dense = [t.contiguous() for t in (q, k, v)]
        if op == "linear_attn":
            got, want = ssd.ssd_linear_attn_fwd(q, k, v, r), ssd.ssd_linear_attn_fwd(*dense, r)
        else:
            dy = randn(g, 2, T, H, d, dtype=bf)
            got = tuple(ssd.ssd_linear_attn_bwd(q, k, v, r, dy).values())
            want = tuple(ssd.ssd_linear_attn_bwd(*dense, r, dy).values())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    elif op == "step":
        H, K, V = 4, 128, 128
        n = far // (H * K * V) + 2                              # slots; 8 GiB of states
        state = torch.empty(n, H, K, V, device="cuda")
        slots = torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda")
        start = randn(g, 2, H, K, V)
        state[slots.long()] = start
        q, k, v = (randn(g, 2, H, K) for _ in range(3))
        r = -torch.rand(H, generator=g, device="cuda")
        y = ssd.ssd_linear_attn_step(state, q, k, v, r, slots=slots)
        assert torch.equal(y, ssd.ssd_linear_attn_step(start, q, k, v, r))
        assert torch.equal(state[slots.long()], start)
    elif op == "norm":
        flat = torch.empty(far * 2 + 4096, dtype=bf, device="cuda")
        x = torch.as_strided(flat, (2, 3, 256), (far * 2, 300, 1))
        x.copy_(randn(g, 2, 3, 256, dtype=bf))
        assert torch.equal(ssd.ssd_group_norm_fwd(x, 4), ssd.ssd_group_norm_fwd(x.contiguous(), 4))
    else:
        # codes of 2^32 + 2^16 bytes, all of one value but the last outputs'
        K = 1 << 17
        O = (1 << 33) // K + 8
        codes = torch.full((O, K // 2), 0x99, dtype=torch.uint8, device="cuda")
        scales = torch.ones(O, K // 128, dtype=bf, device="cuda")
        codes[-3:] = 0x77
        x = torch.zeros(20, K, dtype=bf, device="cuda")
        x[:, -128:] = 1.0
        for rows in (1, 20):
            y = ssd.ssd_w4_linear(x[:rows], codes, scales)
            assert (y[:, :-3] == 128.0).all() and (y[:, -3:] == -128.0).all()
        w = ssd.ssd_w4_dequantize(codes[-8:], scales[-8:])
        again, _ = ssd.ssd_w4_quantize(w.repeat(O // 8, 1)[:O], 128)
        assert (again[-3:] == 0x11).all() and (again[-8:-3] == 0xff).all()
