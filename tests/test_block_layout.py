"""The forms that the tests take for the sizes' are the library's own."""

import ctypes
import os

import pytest

from selective_state_space_amd import ssd

from block_forms import ATTN_BWD, ATTN_FWD

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH),
                                reason="libssd.so not built (python -m selective_state_space_amd.build)")


def layout(Bt, T, H, G, K, V, io):
    return ssd.linear_attn_layout(ssd.AttnDims(Bt, T, H, G, K, V, 0, 0, 0, 0, 0, 0, io, 1.0))


@pytest.mark.parametrize("io", [ssd.SSD_F32, ssd.SSD_BF16])
@pytest.mark.parametrize("sizes,cols,segments", ATTN_FWD)
def test_linear_attn_fwd(sizes, cols, segments, io):
    lay = layout(*sizes, io)
    assert (lay.fwd_cols, lay.fwd_segments) == (cols, segments[io])


@pytest.mark.parametrize("io", [ssd.SSD_F32, ssd.SSD_BF16])
@pytest.mark.parametrize("sizes,cols,segments,one", ATTN_BWD)
def test_linear_attn_bwd(sizes, cols, segments, one, io):
    Bt, T, H, G, K, V = sizes
    lay = layout(*sizes, io)
    assert (lay.bwd_cols, lay.bwd_segments) == (64 if io else cols, segments[io])
    if io == ssd.SSD_BF16:
        assert one == (3 * Bt * H * segments[io] * ((max(K, V) + 63) // 64) <= 256)


def test_every_form_is_among_them():
    pad = lambda d: 64 if d <= 64 else 128 if d <= 128 else 256
    fwd = {(pad(s[4]), c, n[1] > 1) for s, c, n in ATTN_FWD}
    assert fwd >= {(64, 64, False), (64, 128, False), (128, 64, False), (128, 128, False),
                   (256, 64, False), (64, 64, True), (128, 64, True), (256, 64, True)}
    bwd = {(pad(max(s[4:])), s[3] < s[2], c, n[1] > 1, one) for s, c, n, one in ATTN_BWD}
    assert bwd >= {(128, shared, c, False, False) for shared in (False, True) for c in (64, 128)}
