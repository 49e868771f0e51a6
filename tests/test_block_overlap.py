"""Linear attention's states that would be written while others of them are still to be read are
refused on the host, before any HIP call."""

import ctypes
import os

import pytest

from selective_state_space_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH),
                                reason="libssd.so not built (python -m selective_state_space_amd.build)")

# Fake, aligned, never dereferenced: every call below fails validation.
P16 = 0x10000000
STATES = 2 * 4 * 64 * 32 * 4   # bytes


def dims(T=30):
    return ssd.AttnDims(2, T, 4, 2, 64, 32, 8000, 256, 8000, 128, 8000, 64, ssd.SSD_BF16, 0.125)


def fwd(d, init, fin):
    return ssd.load_library().ssd_linear_attn_fwd(P16, P16, P16, P16, init, None, P16, fin,
                                                  ctypes.byref(d), P16, 1 << 40, None)


def bwd(d, init, dfinal, dinit):
    return ssd.load_library().ssd_linear_attn_bwd(P16, P16, P16, P16, init, None, P16, dfinal, P16,
                                                  P16, P16, dinit, ctypes.byref(d), P16, 1 << 40,
                                                  None)


def refused(status, *words):
    detail = ssd.load_library().ssd_last_error_detail().decode()
    return status == -3 and all(w in detail for w in words + ("overlaps",))


@pytest.mark.parametrize("T", [0, 30])
@pytest.mark.parametrize("off", [0, 16, STATES - 16, 16 - STATES])
def test_dinit(off, T):
    assert refused(bwd(dims(T), None, P16, P16 + off), "dinit", "dfinal")
    assert refused(bwd(dims(T), P16, None, P16 + off), "dinit", "init_state")
    assert refused(bwd(dims(T), P16, P16 + 4 * STATES, P16 + off), "dinit", "init_state")


@pytest.mark.parametrize("off", [16, STATES - 16, 16 - STATES])
def test_final_state(off):
    assert refused(fwd(dims(), P16, P16 + off), "final_state", "init_state")


def test_states_apart_are_taken():
    """Side by side; with no sequences nothing is launched."""
    none = ssd.AttnDims(0, 30, 4, 2, 64, 32, 0, 0, 0, 0, 0, 0, ssd.SSD_BF16, 0.125)
    assert fwd(none, P16, P16) == 0 and fwd(none, P16, P16 + 16) == 0
    assert bwd(none, P16, P16, P16) == 0
