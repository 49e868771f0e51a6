"""A workspace passed to the binding is refused unless its memory is the GPU's and as long
as its element count says: the library sees an address and a size alone.

Without a GPU the calls are driven with host tensors: the device check of x and the
library call are replaced, and a call that gets as far as the library fails the test."""

import os

import pytest
import torch

from selective_state_space_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH),
                                reason="libssd.so not built (python -m selective_state_space_amd.build)")


def scan_args(device):
    z = lambda *s: torch.zeros(*s, device=device)
    return z(1, 200, 8), z(1, 200, 8), z(8, 16), z(1, 200, 16), z(1, 200, 16), z(8)


def calls(device):
    x, dt, A, B, C, D = scan_args(device)
    return {
        "conv_bwd": lambda ws: ssd.ssd_conv1d_bwd(x, torch.zeros(8, 4, device=device), x,
                                                  workspace=ws),
        "scan_fwd": lambda ws: ssd.ssd_selective_scan_fwd(x, dt, A, B, C, D, workspace=ws),
        "scan_bwd": lambda ws: ssd.ssd_selective_scan_bwd(x, dt, A, B, C, D, x, workspace=ws),
    }


LAYER = ["conv_bwd", "scan_fwd", "scan_bwd"]


def refused(call, device, elsewhere):
    n = 1 << 20
    with pytest.raises(ValueError, match="workspace is on"):
        call(torch.empty(n, dtype=torch.uint8, device=elsewhere))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(torch.empty(1, dtype=torch.uint8, device=device).expand(n))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(torch.empty(2 * n, dtype=torch.uint8, device=device)[::2])
    with pytest.raises(TypeError, match="workspace"):
        call(n)


@pytest.mark.parametrize("name", LAYER)
def test_refused_before_the_library_is_called(name, monkeypatch):
    reached = []
    monkeypatch.setattr(ssd, "_on_gpu", lambda t, name: t.device)
    monkeypatch.setattr(ssd, "_call", lambda fn, *a: reached.append(fn))
    call = calls("cpu")[name]
    refused(call, "cpu", "meta")
    assert not reached
    call(torch.empty(1 << 20, dtype=torch.uint8))
    assert len(reached) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("name", LAYER + ["chunked_fwd", "chunked_bwd"])
def test_refused_on_the_gpu(name):
    if name in LAYER:
        call = calls("cuda")[name]
    else:
        z = lambda *s: torch.zeros(*s, device="cuda")
        args = (z(1, 64, 2, 64), z(1, 64, 2), z(2), z(1, 64, 1, 64), z(1, 64, 1, 64), z(2), 64)
        if name == "chunked_fwd":
            call = lambda ws: ssd.ssd_chunked_fwd(*args, workspace=ws)
        else:
            call = lambda ws: ssd.ssd_chunked_bwd(*args, args[0], workspace=ws)
    refused(call, "cuda", "cpu")
