"""The C-ABI boundary of the operators around the scan, without a GPU: every
invalid call is refused on the host, with its status and the name of what is
wrong, before any HIP call."""

import ctypes
import os

import pytest
import torch

from selective_state_space_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH),
                                reason="libssd.so not built (python -m selective_state_space_amd.build)")

# Fake, aligned, never dereferenced: every call below fails validation first.
P16 = 0x1000
P_MIS = 0x1004
BIG = 1 << 40


def lib():
    return ssd.load_library()


def detail():
    return lib().ssd_last_error_detail().decode()


def parts(*p):
    return (ctypes.c_void_p * 3)(*p)


def conv_dims(Bt=2, T=30, W=4, ch=(64, 8, 8), sb=2400, stt=80, io=ssd.SSD_BF16, silu=1):
    return ssd.ConvDims(Bt, T, W, (ctypes.c_int64 * 3)(*ch), sb, stt, io, silu)


def conv_fwd(d, x=P16, weight=P16, bias=P16, init=P16, lens=P16, y=parts(P16, P16, P16),
             fin=P16):
    return lib().ssd_conv1d_fwd(x, weight, bias, init, lens, y, fin,
                                None if d is None else ctypes.byref(d), None)


def conv_step(d, state=P16, num=8, slots=P16, x=P16, weight=P16, bias=P16,
              y=parts(P16, P16, P16)):
    return lib().ssd_conv1d_step(state, num, slots, x, weight, bias, y,
                                 None if d is None else ctypes.byref(d), None)


def conv_bwd(d, x=P16, weight=P16, bias=P16, init=P16, dy=parts(P16, P16, P16), dfinal=P16,
             dx=P16, dweight=P16, dbias=P16, dinit=P16, ws=P16, wsb=BIG):
    return lib().ssd_conv1d_bwd(x, weight, bias, init, dy, dfinal, dx, dweight, dbias, dinit,
                                None if d is None else ctypes.byref(d), ws, wsb, None)


@pytest.mark.parametrize("call", [conv_fwd, conv_step, conv_bwd])
@pytest.mark.parametrize("kw,code,word", [
    (dict(Bt=-1), -2, "batch"), (dict(Bt=(1 << 30) + 1), -2, "batch"),
    (dict(W=1), -3, "width"), (dict(W=5), -3, "width"),
    (dict(ch=(0, 8, 8)), -2, "channels[0]"), (dict(ch=(8, -1, 8)), -2, "channels[1]"),
    (dict(ch=(8, 8, (1 << 24) + 1)), -2, "channels[2]"),
    (dict(sb=-1), -2, "stride"), (dict(stt=-1), -2, "stride"), (dict(io=2), -3, "io_dtype"),
    (dict(Bt=1 << 30, T=1 << 30, ch=(1 << 24, 0, 0)), -2, "too large"),
    (dict(Bt=1 << 24, T=1, ch=(1024, 0, 0)), -2, "too large"),
])
def test_conv_dims(call, kw, code, word):
    assert call(conv_dims(**kw)) == code
    assert word in detail()


def test_conv_seqlen():
    for call in (conv_fwd, conv_bwd):
        assert call(conv_dims(T=-1)) == -2 and "seqlen" in detail()
        assert call(None) == -1 and "dims" in detail()
    assert conv_step(None) == -1


@pytest.mark.parametrize("call,required,optional", [
    (conv_fwd, ["weight"], ["bias", "init", "lens", "fin"]),
    (conv_step, ["state", "weight"], ["bias", "slots"]),
    (conv_bwd, ["weight", "dx", "dweight", "ws"], ["bias", "init", "dfinal", "dbias", "dinit"]),
])
def test_conv_pointers(call, required, optional):
    for f in required:
        assert call(conv_dims(), **{f: None}) == -1, f
    for f in required + optional:
        assert call(conv_dims(), **{f: P_MIS}) == -4, f
    # x needs the alignment of its elements only
    assert call(conv_dims(), x=None) == -1 and "x" in detail()
    assert call(conv_dims(), x=0x1001) == -4 and "x" in detail()
    assert call(conv_dims(io=ssd.SSD_F32), x=0x1002) == -4
    outs = "dy" if call is conv_bwd else "y"
    assert call(conv_dims(), **{outs: parts(P16, None, P16)}) == -1 and "[1]" in detail()
    assert call(conv_dims(), **{outs: parts(P16, P16, P_MIS)}) == -4 and "[2]" in detail()
    assert call(conv_dims(), **{outs: None}) == -1


def test_conv_step_slots():
    assert conv_step(conv_dims(), num=1, slots=None) == -2 and "num_slots" in detail()
    assert conv_step(conv_dims(), num=-1) == -2


def test_conv_workspace():
    d = conv_dims()
    need = ssd.ssd_conv1d_bwd_workspace_size(d)
    assert need >= 5 * 80 * 4
    assert conv_bwd(d, wsb=need - 1) == -5 and str(need) in detail()
    assert ssd.ssd_conv1d_bwd_workspace_size(conv_dims(W=9)) == 0


def scan_dims(Bt=2, T=30, Dm=64, N=16, io=ssd.SSD_BF16):
    return ssd.ScanDims(Bt, T, Dm, N, io)


def opts(bias=P16, softplus=1, yio=0, z=P16):
    return ssd.LayerOpts(bias, softplus, yio, z)


def scan_fwd(d, x=P16, dt=P16, A=P16, B=P16, C=P16, D=P16, init=P16, lens=P16, y=P16, fin=P16,
             o=None, ws=P16, wsb=BIG):
    return lib().ssd_selective_scan_fwd(x, dt, A, B, C, D, init, lens, y, fin, o,
                                        None if d is None else ctypes.byref(d), ws, wsb, None)


def scan_step(d, state=P16, num=8, slots=P16, x=P16, dt=P16, A=P16, B=P16, C=P16, D=P16, y=P16,
              o=None):
    return lib().ssd_selective_scan_step(state, num, slots, x, dt, A, B, C, D, y, o,
                                         None if d is None else ctypes.byref(d), None)


def scan_bwd(d, x=P16, dt=P16, A=P16, B=P16, C=P16, D=P16, init=P16, dy=P16, dfinal=P16, dx=P16,
             ddt=P16, dA=P16, dB=P16, dC=P16, dD=P16, dbias=P16, dz=P16, dinit=P16, o=None,
             ws=P16, wsb=BIG):
    return lib().ssd_selective_scan_bwd(x, dt, A, B, C, D, init, dy, dfinal, dx, ddt, dA, dB, dC,
                                        dD, dbias, dz, dinit, o,
                                        None if d is None else ctypes.byref(d), ws, wsb, None)


@pytest.mark.parametrize("call", [scan_fwd, scan_step, scan_bwd])
@pytest.mark.parametrize("kw,code,word", [
    (dict(Bt=-1), -2, "batch"), (dict(Dm=0), -2, "dim"), (dict(Dm=(1 << 24) + 1), -2, "dim"),
    (dict(N=12), -3, "dstate"), (dict(N=128), -3, "dstate"), (dict(io=5), -3, "io_dtype"),
    (dict(Bt=1 << 28, Dm=1 << 20), -2, "too large"),
    (dict(Bt=1 << 24, Dm=64), -2, "too large"),
])
def test_scan_dims(call, kw, code, word):
    assert call(scan_dims(**kw)) == code
    assert word in detail()


def test_scan_too_many_sums():
    assert scan_bwd(scan_dims(Bt=1 << 10, T=1 << 20, N=64)) == -2 and "too large" in detail()


def test_scan_seqlen():
    for call in (scan_fwd, scan_bwd):
        assert call(scan_dims(T=-1)) == -2 and "seqlen" in detail()
    for call in (scan_fwd, scan_bwd, scan_step):
        assert call(None) == -1 and "dims" in detail()


@pytest.mark.parametrize("call,required,optional", [
    (scan_fwd, ["x", "dt", "A", "B", "C", "D", "y"], ["init", "lens", "fin", "ws"]),
    (scan_step, ["state", "x", "dt", "A", "B", "C", "D", "y"], ["slots"]),
    (scan_bwd, ["x", "dt", "A", "B", "C", "D", "dy", "dx", "ddt", "dA", "dB", "dC", "dD", "ws"],
     ["init", "dfinal", "dbias", "dinit"]),
])
def test_scan_pointers(call, required, optional):
    for f in required:
        assert call(scan_dims(), **{f: None}) == -1, f
    for f in required + optional:
        assert call(scan_dims(), **{f: P_MIS}) == -4, f
    for kw, code, word in [(dict(bias=P_MIS), -4, "dt_bias"), (dict(z=P_MIS), -4, "z"),
                           (dict(yio=2), -3, "y_io_dtype")]:
        assert call(scan_dims(), o=ctypes.byref(opts(**kw))) == code
        assert word in detail()
    if call is scan_bwd:   # a gate needs its gradient
        assert call(scan_dims(), o=ctypes.byref(opts()), dz=None) == -1 and "dz" in detail()


def test_scan_step_slots():
    assert scan_step(scan_dims(), num=1, slots=None) == -2 and "num_slots" in detail()


def test_scan_workspaces():
    few = scan_dims(Bt=1, T=4096, Dm=64)
    need = ssd.ssd_selective_scan_workspace_size(few)
    assert need > 0 and scan_fwd(few, wsb=need - 1) == -5 and str(need) in detail()
    assert scan_fwd(few, ws=None) == -1 and "workspace" in detail()
    assert ssd.ssd_selective_scan_workspace_size(scan_dims(Bt=64, T=4096, Dm=5120)) == 0
    assert ssd.ssd_selective_scan_workspace_size(scan_dims(N=5)) == 0
    need = ssd.ssd_selective_scan_bwd_workspace_size(few)
    assert need > 0 and scan_bwd(few, wsb=need - 1) == -5
    assert ssd.ssd_selective_scan_bwd_workspace_size(scan_dims(Bt=0)) == 0


def cache_write(state=P16, n=2, size=64, slots=P16, num=4, codes=P16, scales=P16, fmt=0):
    return lib().ssd_cache_write(state, n, size, slots, num, codes, scales, fmt, None)


def cache_read(state=P16, n=2, size=64, slots=P16, num=4, codes=P16, scales=P16, fmt=0):
    return lib().ssd_cache_read(codes, scales, n, size, slots, num, state, fmt, None)


@pytest.mark.parametrize("call", [cache_write, cache_read])
def test_cache(call):
    for kw, code, word in [(dict(n=-1), -2, "n ="), (dict(size=0), -2, "size"),
                           (dict(size=12), -2, "size"), (dict(fmt=2), -3, "format"),
                           (dict(num=-1), -2, "num_slots"),
                           (dict(slots=None, num=1), -2, "num_slots"),
                           (dict(n=1 << 30, size=1 << 20), -2, "too large"),
                           (dict(state=None), -1, "state"), (dict(codes=None), -1, "codes"),
                           (dict(scales=None), -1, "scales"), (dict(state=P_MIS), -4, "state"),
                           (dict(codes=P_MIS), -4, "codes"), (dict(scales=P_MIS), -4, "scales"),
                           (dict(slots=P_MIS), -4, "slots")]:
        assert call(**kw) == code, kw
        assert word in detail(), kw
    assert call(n=0, state=None, codes=None, scales=None, slots=None, num=0) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 2, 8)
    w = torch.zeros(8, 4)
    for f in (lambda: ssd.ssd_conv1d_fwd(x, w),
              lambda: ssd.ssd_conv1d_step(torch.zeros(1, 3, 8), x[:, 0], w),
              lambda: ssd.ssd_conv1d_bwd(x, w, x),
              lambda: ssd.ssd_selective_scan_fwd(x, x, w, w[None, :2], w[None, :2], w[:, 0]),
              lambda: ssd.ssd_cache_read(torch.zeros(1, 64, dtype=torch.int8),
                                         torch.zeros(1, 1))):
        with pytest.raises(ValueError):
            f()
