"""Which form of its kernel a call of the convolution or the selective scan takes: the query,
and that the sizes of the GPU tests reach every form."""

import ctypes
import os

import pytest

from selective_state_space_amd import ssd

import layer_forms as forms

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH),
                                reason="libssd.so not built (python -m selective_state_space_amd.build)")


def conv_layout(Bt, T, splits, W=4):
    return ssd.conv1d_layout(ssd.ConvDims(Bt, T, W, (ctypes.c_int64 * 3)(*splits), 0, 0,
                                          ssd.SSD_BF16, 1))


def scan_layout(Bt, T, Dm, N):
    return ssd.selective_scan_layout(ssd.ScanDims(Bt, T, Dm, N, ssd.SSD_BF16))


def test_sizes_of_the_gpu_tests_take_their_forms():
    for sizes, states, cut in forms.SCAN_FWD:
        v = scan_layout(*sizes)
        assert (v.fwd_states, v.fwd_segments > 1) == (states, cut), sizes
    for sizes, states, cut in forms.SCAN_BWD:
        v = scan_layout(*sizes)
        assert (v.bwd_states, v.bwd_segments > 1) == (states, cut), sizes
        assert sizes[1] > 2 * 16          # several tiles
    for (Bt, Dm, N), channels in forms.SCAN_STEP:
        assert scan_layout(Bt, 1, Dm, N).step_channels == channels, (Bt, Dm, N)
    for sizes, run in forms.CONV_FWD:
        assert conv_layout(*sizes).fwd_run == run, sizes
    for sizes, run in forms.CONV_BWD:
        assert conv_layout(*sizes).bwd_run == run, sizes
    for (Bt, splits), rows in forms.CONV_STEP:
        assert conv_layout(Bt, 1, splits).step_rows == rows, (Bt, splits)


def test_every_form_is_among_them():
    """Every (N, states, cut, width) that any size takes is in the list."""
    held = {"fwd": set(), "bwd": set()}
    for key, cases in (("fwd", forms.SCAN_FWD), ("bwd", forms.SCAN_BWD)):
        for (Bt, T, Dm, N), states, cut in cases:
            held[key].add((N, states, cut, Dm % 4 > 0))
    for N in (8, 16, 32, 64):
        for Bt in (1, 3, 16, 64, 200, 1500):
            for T in (1, 40, 130, 500, 4096):
                for Dm in (5, 64, 515, 2048, 5120):
                    v = scan_layout(Bt, T, Dm, N)
                    assert v.fwd_segments >= 1 and v.bwd_segments >= 1
                    odd = Dm % 4 > 0
                    assert (N, v.fwd_states, v.fwd_segments > 1, odd) in held["fwd"]
                    assert (N, v.bwd_states, v.bwd_segments > 1, odd) in held["bwd"]
    runs = [conv_layout(Bt, T, (C, 0, 0)) for Bt in (1, 16, 300) for T in (1, 300, 9000)
            for C in (3, 64, 5000)]
    assert {v.fwd_run for v in runs} <= {r for _, r in forms.CONV_FWD}
    assert {v.bwd_run for v in runs} <= {r for _, r in forms.CONV_BWD}
    assert {v.step_rows for v in runs} <= {r for _, r in forms.CONV_STEP}


def test_refusals():
    lib = ssd.load_library()
    detail = lambda: lib.ssd_last_error_detail().decode()
    conv = ssd.ConvDims(1, 1, 4, (ctypes.c_int64 * 3)(8, 0, 0), 0, 0, 0, 0)
    scan = ssd.ScanDims(1, 1, 8, 16, 0)
    cl, sl = ssd.ConvLayout(), ssd.ScanLayout()
    assert lib.ssd_conv1d_layout(ctypes.byref(conv), None) == -1 and "layout" in detail()
    assert lib.ssd_selective_scan_layout(ctypes.byref(scan), None) == -1 and "layout" in detail()
    assert lib.ssd_conv1d_layout(None, ctypes.byref(cl)) == -1 and "dims" in detail()
    assert lib.ssd_selective_scan_layout(None, ctypes.byref(sl)) == -1 and "dims" in detail()
    conv.width, scan.dstate = 9, 12
    with pytest.raises(ssd.SSDError, match="width"):
        ssd.conv1d_layout(conv)
    with pytest.raises(ssd.SSDError, match="dstate"):
        ssd.selective_scan_layout(scan)
    v = scan_layout(0, 5, 8, 16)
    assert v.fwd_segments == 1 and v.bwd_segments == 1
