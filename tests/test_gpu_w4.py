"""4-bit weights: codes and scales against the rule in float64, bit for bit; the values they
stand for; products with every number of rows, group, type, odd output counts, strides."""

import pytest
import torch

from selective_state_space_amd import ssd
from _block import TYPES, U, assert_near, gen, randn, w4_ref, w4_values

pytestmark = pytest.mark.gpu


def packed(g, O, K, group):
    """Random codes (0 and 15 among them) and scales."""
    codes = torch.randint(0, 256, (O, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(O, K // group, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    return codes, scales


def whole(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(1).double() - 8.0


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("O,K,group", [(1, 64, 64), (3, 128, 64), (5, 128, 128), (33, 640, 128),
                                       (100, 2560, 64), (17, 5120, 128)])
def test_quantize(O, K, group, io):
    g = gen(O)
    w = randn(g, O, K, dtype=TYPES[io]) * torch.exp(randn(g, O, 1)).to(TYPES[io])
    codes, scales = ssd.ssd_w4_quantize(w, group)
    code, scale = w4_ref(w, group)
    assert codes.dtype == torch.uint8 and scales.dtype == torch.bfloat16
    assert torch.equal(scales.double(), scale)
    assert torch.equal(whole(codes), code.flatten(1))
    for t in TYPES.values():
        back = ssd.ssd_w4_dequantize(codes, scales, dtype=t)
        assert torch.equal(back, w4_values(codes, scales).to(t))


def test_quantize_borders():
    """Halves go to the even number, and the nearest floats on either side of a half to theirs;
    scales over the whole range."""
    ks = torch.arange(-6.5, 7.0, 1.0, device="cuda")
    rows = []
    for s in (1.0, 0.8125, 1.9921875, 2.0 ** -90, 3.0 * 2.0 ** 100):
        # 7 s is the largest of the group, so its scale is s
        for v in (ks * s, torch.nextafter(ks * s, ks * 0 + 1e38), torch.nextafter(ks * s, ks * 0 - 1e38)):
            row = torch.zeros(64, device="cuda")
            row[:14], row[63] = v, 7.0 * s
            rows.append(row)
    w = torch.stack(rows)
    codes, scales = ssd.ssd_w4_quantize(w, 64)
    code, scale = w4_ref(w, 64)
    assert torch.equal(scales.double(), scale) and torch.equal(whole(codes), code.flatten(1))


def test_quantize_edges():
    """Zeros, tiny groups, the largest float32, infinities and NaN."""
    w = torch.randn(6, 128, device="cuda")
    w[0] = 0.0
    w[1, :64] = 2.0 ** -101
    w[2, 5] = float("inf")
    w[3, 100] = float("nan")
    w[4] = torch.finfo(torch.float32).max
    w[5, ::2] = -torch.finfo(torch.float32).max
    codes, scales = ssd.ssd_w4_quantize(w, 64)
    back = ssd.ssd_w4_dequantize(codes, scales, dtype=torch.float32)
    assert not back[0].any() and not back[1, :64].any() and back[1, 64:].any()
    assert back[2, :64].isnan().all() and torch.isfinite(back[2, 64:]).all()
    assert back[3, 64:].isnan().all() and torch.isfinite(back[3, :64]).all()
    assert torch.isfinite(scales[4:].float()).all() and (whole(codes)[4] == 7).all()


def check(x, codes, scales, bias=None, **kw):
    y = ssd.ssd_w4_linear(x, codes, scales, bias, **kw)
    assert y.dtype == x.dtype
    w = w4_values(codes, scales)
    ref = (x.double().reshape(-1, w.shape[1])[:, None] * w).sum(-1)
    if bias is not None:
        ref = ref + bias.double()
    # float32 sums over K of terms that stand up to 24 / 4.6 times as high before 24 times the
    # sum of x is taken off (codes are read as 16 + code): 2^-24 5.2 sqrt(K), and the output's.
    # That is of what a sum of K such terms is on the average, the root of their squares' sum:
    # one output may come out smaller by chance while its terms' roundings do not.
    K = w.shape[1]
    size = float((x.double().reshape(-1, K).square() @ w.square().t()).sum()) ** 0.5
    off = float((y.reshape(-1, w.shape[0]).double() - ref).norm())
    bar = 2.0 ** -24 * 5.2 * K ** 0.5 * size
    if x.dtype == torch.bfloat16:
        bar += U[x.dtype] * float(ref.norm())
    print("  y off %.3g of %.3g" % (off, bar), flush=True)
    assert off <= bar
    return y


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("rows", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 48, 64, 65, 130])
def test_rows(rows, group, io):
    g = gen(rows)
    codes, scales = packed(g, 75, 640, group)
    check(randn(g, rows, 640, dtype=TYPES[io]), codes, scales, randn(g, 75))


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("O,K,group", [(1, 64, 64), (1, 128, 128), (15, 192, 64), (16, 384, 128),
                                       (17, 896, 128), (63, 1088, 64), (64, 2560, 64),
                                       (65, 5120, 128), (4098, 320, 64), (10576, 256, 128),
                                       (300, 8192, 128), (40, 16448, 64)])
def test_sizes(O, K, group, rows, io):
    g = gen(O + K)
    codes, scales = packed(g, O, K, group)
    check(randn(g, rows, K, dtype=TYPES[io]), codes, scales)


@pytest.mark.parametrize("io", TYPES)
def test_rows_agree(io):
    """A row's product does not depend on the rows beside it."""
    g = gen(3)
    codes, scales = packed(g, 100, 1280, 128)
    x = randn(g, 70, 1280, dtype=TYPES[io])
    y = ssd.ssd_w4_linear(x, codes, scales)
    for r in (0, 1, 15, 16, 64, 69):
        one = ssd.ssd_w4_linear(x[r], codes, scales)
        assert one.shape == (100,)
        assert_near(one, y[r].double(), 2 * U[torch.float32] * 5.2 * 1280 ** 0.5
                    + 2 * (io == "bf16") * U[torch.bfloat16], "row %d" % r)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strided(off, io):
    """Rows of a wider tensor, in place or (off 16 bytes) copied, and one row for all."""
    g = gen(6)
    codes, scales = packed(g, 50, 256, 64)
    wide = randn(g, 9, 256 + 32, dtype=TYPES[io])
    x = wide[:, off:off + 256]
    a = ssd.ssd_w4_linear(x, codes, scales)
    assert torch.equal(a, ssd.ssd_w4_linear(x.contiguous(), codes, scales))
    a = ssd.ssd_w4_linear(x[:1].expand(5, -1), codes, scales)
    assert torch.equal(a, a[:1].expand(5, -1))


@pytest.mark.parametrize("io", TYPES)
def test_columns_alone(io):
    """One input at a time gives the weights themselves, exactly: no code, place or scale can
    stand in for another."""
    g = gen(7)
    O, K, group = 37, 256, 64
    codes, scales = packed(g, O, K, group)
    x = torch.eye(K, device="cuda", dtype=TYPES[io])
    y = ssd.ssd_w4_linear(x, codes, scales)
    assert torch.equal(y.t(), w4_values(codes, scales).to(TYPES[io]))


def test_empty_and_reruns():
    g = gen(8)
    codes, scales = packed(g, 40, 128, 64)
    assert ssd.ssd_w4_linear(torch.zeros(0, 128, device="cuda"), codes, scales).shape == (0, 40)
    x = randn(g, 33, 128, dtype=torch.bfloat16)
    out = torch.empty(33, 40, dtype=torch.bfloat16, device="cuda")
    a = ssd.ssd_w4_linear(x, codes, scales, y=out)
    assert a is out and torch.equal(a, ssd.ssd_w4_linear(x, codes, scales))
