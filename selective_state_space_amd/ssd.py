"""Python binding of libssd.so (ctypes).

Argument marshalling only: shapes and dtypes are checked, tensors made
contiguous, output and workspace memory allocated with torch on the input's
device, and the C entry points of ``include/ssd.h`` called with raw device
pointers and torch's current stream.  Every step of the computation runs in
the HIP kernels of libssd.so; if the library is missing this module raises,
it never falls back to another implementation.

The functions carry the C names:

* :func:`ssd_chunked_fwd` -- chunked forward, with the layer options (dt bias,
  softplus, z gate, y in the io dtype) when given;
* :func:`ssd_chunked_fwd_noalloc` -- the same on the library's static
  workspace (no allocation in the library);
* :func:`ssd_chunk_cumsum`, :func:`ssd_chunk_state`, :func:`ssd_state_passing`,
  :func:`ssd_state_fwd`, :func:`ssd_chunk_scan` -- the stages one at a time,
  on a shared workspace;
* :func:`ssd_decode_step` -- one recurrent token, state updated in place;
* :func:`ssd_decode_multi` -- K tokens per sequence, with snapshots and
  draft-tree parents;
* :func:`ssd_decode_step_lp` -- the decode step on a 16-bit state;
* :func:`ssd_chunked_bwd` -- every gradient of the chunked forward;
* :func:`ssd_conv1d_fwd`, :func:`ssd_conv1d_step`, :func:`ssd_conv1d_bwd` -- the
  short causal convolution in front of the scan;
* :func:`ssd_selective_scan_fwd`, :func:`ssd_selective_scan_step`,
  :func:`ssd_selective_scan_bwd` -- the scan with a decay rate per channel and
  state;
* :func:`ssd_cache_write`, :func:`ssd_cache_read` -- recurrent states in a slot
  pool at 8 bits per element;
* :func:`ssd_chunked_fwd_workspace_size`, :func:`ssd_chunked_fwd_workspace_layout`,
  :func:`ssd_chunked_bwd_workspace_size`, :func:`fwd_path` and
  :func:`set_path_override` (which path the forward takes, and a switch for
  tests); :func:`conv1d_layout` and :func:`selective_scan_layout` (which forms of
  their kernels the convolution and the selective scan take).
"""

from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Tuple

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libssd.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "ssd.h")

SSD_F32, SSD_BF16 = 0, 1
STATUS = {0: "SSD_OK", -1: "SSD_ERR_NULL", -2: "SSD_ERR_SHAPE", -3: "SSD_ERR_UNSUPPORTED",
          -4: "SSD_ERR_ALIGN", -5: "SSD_ERR_WORKSPACE", -6: "SSD_ERR_HIP"}


class SSDError(RuntimeError):
    """A libssd.so entry point returned a non-zero ssd_status."""

    def __init__(self, fn: str, status: int, detail: str):
        super().__init__("%s -> %s (%d): %s" % (fn, STATUS.get(status, "?"), status, detail))
        self.status = status
        self.detail = detail


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32)]


class StateFormat(ctypes.Structure):
    """ssd_state_format."""
    _fields_ = [("dtype", ctypes.c_int32), ("philox_rounds", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("scale", ctypes.c_void_p)]


STATE_DTYPES = {"f32": (0, torch.float32), "f16": (1, torch.float16), "bf16": (2, torch.bfloat16),
                "int16": (3, torch.int16)}


class LayerOpts(ctypes.Structure):
    """ssd_layer_opts: dt_bias [H] f32 (or NULL), dt_softplus, y_io_dtype, z (or NULL)."""
    _fields_ = [("dt_bias", ctypes.c_void_p), ("dt_softplus", ctypes.c_int32),
                ("y_io_dtype", ctypes.c_int32), ("z", ctypes.c_void_p)]


class ConvDims(ctypes.Structure):
    """ssd_conv_dims."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("width", ctypes.c_int64),
                ("channels", ctypes.c_int64 * 3), ("x_batch_stride", ctypes.c_int64),
                ("x_token_stride", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("silu", ctypes.c_int32)]


class ScanDims(ctypes.Structure):
    """ssd_scan_dims."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("io_dtype", ctypes.c_int32)]


class ConvLayout(ctypes.Structure):
    """ssd_conv_layout."""
    _fields_ = [("fwd_run", ctypes.c_int32), ("bwd_run", ctypes.c_int32),
                ("step_rows", ctypes.c_int32)]


class ScanLayout(ctypes.Structure):
    """ssd_scan_layout."""
    _fields_ = [("fwd_states", ctypes.c_int32), ("bwd_states", ctypes.c_int32),
                ("step_channels", ctypes.c_int32), ("fwd_segments", ctypes.c_int64),
                ("bwd_segments", ctypes.c_int64)]


CACHE_BLOCK = 64   # SSD_CACHE_BLOCK
CACHE_FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}   # ssd_cache_format by the codes' dtype

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libssd.so (built in-tree by ``python -m selective_state_space_amd.build``)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libssd.so is not built (%s); run `python -m "
                           "selective_state_space_amd.build` -- there is no fallback" % path)
    lib = ctypes.CDLL(path)
    vp, i64, sz, dp = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER(Dims)
    cdp, sdp = ctypes.POINTER(ConvDims), ctypes.POINTER(ScanDims)
    lop = ctypes.POINTER(LayerOpts)
    st = ctypes.c_int
    sig = {
        "ssd_chunked_fwd": ([vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, dp, vp, sz, vp], st),
        "ssd_chunked_fwd_workspace_size": ([dp, i64], sz),
        "ssd_chunked_fwd_workspace_layout": ([dp, i64, ctypes.POINTER(ctypes.c_size_t)], st),
        "ssd_chunk_cumsum": ([vp, vp, i64, dp, vp, sz, vp], st),
        "ssd_chunk_state": ([vp, vp, i64, dp, vp, sz, vp], st),
        "ssd_state_passing": ([vp, vp, i64, dp, vp, sz, vp], st),
        "ssd_chunk_scan": ([vp, vp, vp, vp, vp, i64, dp, vp, sz, vp], st),
        "ssd_state_fwd": ([vp, vp, vp, vp, i64, dp, vp, sz, vp], st),
        "ssd_chunked_fwd_opts": ([vp, vp, vp, vp, vp, vp, i64, vp, vp, vp,
                                  ctypes.POINTER(LayerOpts), dp, vp, sz, vp], st),
        "ssd_decode_step_opts": ([vp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(LayerOpts), dp,
                                  vp], st),
        "ssd_chunked_fwd_path": ([dp, i64, ctypes.POINTER(ctypes.c_int)], st),
        "ssd_set_path_override": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int32], st),
        "ssd_chunked_fwd_noalloc": ([vp, vp, vp, vp, vp, vp, i64, vp, vp, vp,
                                     ctypes.POINTER(LayerOpts), dp, vp], st),
        "ssd_decode_step": ([vp, vp, vp, vp, vp, vp, vp, vp, dp, vp], st),
        "ssd_decode_multi": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_uint32,
                              ctypes.POINTER(LayerOpts), dp, vp], st),
        "ssd_chunked_bwd_workspace_size": ([dp, i64], sz),
        "ssd_chunked_bwd": ([vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                             vp, dp, vp, sz, vp], st),
        "ssd_decode_step_lp": ([vp, ctypes.POINTER(StateFormat), vp, vp, vp, vp, vp, vp, vp,
                                ctypes.POINTER(LayerOpts), dp, vp], st),
        "ssd_conv1d_fwd": ([vp, vp, vp, vp, vp, vp, vp, cdp, vp], st),
        "ssd_conv1d_step": ([vp, i64, vp, vp, vp, vp, vp, cdp, vp], st),
        "ssd_conv1d_bwd_workspace_size": ([cdp], sz),
        "ssd_conv1d_layout": ([cdp, ctypes.POINTER(ConvLayout)], st),
        "ssd_selective_scan_layout": ([sdp, ctypes.POINTER(ScanLayout)], st),
        "ssd_conv1d_bwd": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, cdp, vp, sz, vp], st),
        "ssd_selective_scan_workspace_size": ([sdp], sz),
        "ssd_selective_scan_fwd": ([vp] * 10 + [lop, sdp, vp, sz, vp], st),
        "ssd_selective_scan_step": ([vp, i64] + [vp] * 8 + [lop, sdp, vp], st),
        "ssd_selective_scan_bwd_workspace_size": ([sdp], sz),
        "ssd_selective_scan_bwd": ([vp] * 18 + [lop, sdp, vp, sz, vp], st),
        "ssd_cache_write": ([vp, i64, i64, vp, i64, vp, vp, ctypes.c_int32, vp], st),
        "ssd_cache_read": ([vp, vp, i64, i64, vp, i64, vp, ctypes.c_int32, vp], st),
        "ssd_status_string": ([st], ctypes.c_char_p),
        "ssd_last_error_detail": ([], ctypes.c_char_p),
        "ssd_version": ([], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    if path == LIB_PATH:
        _lib = lib
    return lib


def header_functions(path: str = HEADER):
    """Names of the functions ``include/ssd.h`` declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ssd_[a-z_0-9]+)\s*\(", text)))


def _check(fn: str, status: int):
    if status != 0:
        detail = load_library().ssd_last_error_detail().decode()
        raise SSDError(fn, status, detail)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _io_code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return SSD_F32
    if dtype == torch.bfloat16:
        return SSD_BF16
    raise TypeError("x, B, C must be float32 or bfloat16, got %s" % dtype)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t.contiguous()


def _need_out(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device) -> torch.Tensor:
    """An output the library writes into: a contiguous copy would lose the result."""
    if isinstance(t, torch.Tensor) and not t.is_contiguous():
        raise ValueError("%s must be contiguous (the library writes into it)" % name)
    return _need(t, name, dtype, shape, device)


def _own_workspace(t: torch.Tensor, device) -> torch.Tensor:
    """A workspace of the caller's.  The library checks its size and alignment but sees
    an address alone: that the memory is the GPU's, and as long as its element count
    says, is checked here."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if t.device != device:
        raise ValueError("workspace is on %s, expected %s" % (t.device, device))
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t


def fwd_dims(x: torch.Tensor, B: torch.Tensor) -> Dims:
    Bt, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return Dims(Bt, T, H, P, N, G, _io_code(x.dtype))


def ssd_chunked_fwd_workspace_size(dims: Dims, chunk_size: int) -> int:
    return int(load_library().ssd_chunked_fwd_workspace_size(ctypes.byref(dims), chunk_size))


def ssd_chunked_fwd_workspace_layout(dims: Dims, chunk_size: int) -> Tuple[int, int, int, int]:
    off = (ctypes.c_size_t * 4)()
    _check("ssd_chunked_fwd_workspace_layout",
           load_library().ssd_chunked_fwd_workspace_layout(ctypes.byref(dims), chunk_size, off))
    return tuple(int(v) for v in off)


class FwdArgs:
    """Checked, contiguous arguments of one chunked forward (shared by the stage calls)."""

    def __init__(self, x, dt, A, B, C, D, chunk_size, init_state=None, y=None,
                 final_state=None, want_final=True, workspace=None, dt_bias=None,
                 dt_softplus=False, z=None, y_io_dtype=False):
        if x.dim() != 4 or B.dim() != 4:
            raise ValueError("x must be [Bt,T,H,P] and B, C [Bt,T,G,N]")
        dev = x.device
        if dev.type != "cuda":
            raise ValueError("tensors must live on a GPU device, got %s" % dev)
        Bt, T, H, P = x.shape
        G, N = B.shape[2], B.shape[3]
        io = x.dtype
        self.x = x.contiguous()
        self.dt = _need(dt, "dt", torch.float32, (Bt, T, H), dev)
        self.A = _need(A, "A", torch.float32, (H,), dev)
        self.B = _need(B, "B", io, (Bt, T, G, N), dev)
        self.C = _need(C, "C", io, (Bt, T, G, N), dev)
        self.D = _need(D, "D", torch.float32, (H,), dev)
        self.init = None if init_state is None else _need(init_state, "init_state", torch.float32,
                                                         (Bt, H, P, N), dev)
        self.y_io_dtype = bool(y_io_dtype)
        ydt = io if self.y_io_dtype else torch.float32
        self.y = (torch.empty((Bt, T, H, P), dtype=ydt, device=dev) if y is None
                  else _need_out(y, "y", ydt, (Bt, T, H, P), dev))
        if final_state is not None:
            self.final = _need_out(final_state, "final_state", torch.float32, (Bt, H, P, N), dev)
        elif want_final:
            self.final = torch.empty((Bt, H, P, N), dtype=torch.float32, device=dev)
        else:
            self.final = None
        self.L = int(chunk_size)
        self.dt_bias = None if dt_bias is None else _need(dt_bias, "dt_bias", torch.float32,
                                                          (H,), dev)
        self.z = None if z is None else _need(z, "z", io, (Bt, T, H, P), dev)
        self.dt_softplus = bool(dt_softplus)
        self.dims = fwd_dims(self.x, self.B)
        need = ssd_chunked_fwd_workspace_size(self.dims, self.L)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        else:
            workspace = _own_workspace(workspace, dev)
        self.ws = workspace
        self.device = dev


def _layer_opts(dt_bias, dt_softplus, z, y_io_dtype=False):
    if dt_bias is None and not dt_softplus and z is None and not y_io_dtype:
        return None
    return LayerOpts(_ptr(dt_bias), int(bool(dt_softplus)), int(bool(y_io_dtype)), _ptr(z))


def ssd_chunked_fwd(x, dt=None, A=None, B=None, C=None, D=None, chunk_size=None,
                    init_state=None, y=None, final_state=None, want_final: bool = True,
                    workspace=None, dt_bias=None, dt_softplus: bool = False, z=None,
                    y_io_dtype: bool = False):
    """Chunked forward.  Returns (y, final_state or None).

    x [Bt,T,H,P] (float32 or bfloat16), dt [Bt,T,H] f32, A/D [H] f32,
    B/C [Bt,T,G,N] (x's dtype), init_state [Bt,H,P,N] f32 or None.  y is
    [Bt,T,H,P], float32 whatever the input dtype unless ``y_io_dtype``.  ``y``,
    ``final_state`` and ``workspace`` may be passed in to avoid allocation;
    ``final_state`` may be the same tensor as ``init_state``.  ``x`` may
    instead be a prepared FwdArgs (then the other arguments are ignored).
    ``dt_bias`` [H] f32, ``dt_softplus`` and the gate ``z`` (x's shape and
    dtype) are the optional layer interface (ssd_layer_opts); ``y_io_dtype``
    stores y in x's dtype instead of float32.
    """
    if isinstance(x, FwdArgs):
        a = x
    else:
        if any(v is None for v in (dt, A, B, C, D, chunk_size)):
            raise ValueError("ssd_chunked_fwd needs x, dt, A, B, C, D and chunk_size")
        a = FwdArgs(x, dt, A, B, C, D, chunk_size, init_state, y, final_state, want_final,
                    workspace, dt_bias, dt_softplus, z, y_io_dtype)
    lib = load_library()
    opts = _layer_opts(a.dt_bias, a.dt_softplus, a.z, a.y_io_dtype)
    if opts is None:
        st = lib.ssd_chunked_fwd(_ptr(a.x), _ptr(a.dt), _ptr(a.A), _ptr(a.B), _ptr(a.C),
                                 _ptr(a.D), a.L, _ptr(a.init), _ptr(a.y), _ptr(a.final),
                                 ctypes.byref(a.dims), _ptr(a.ws), a.ws.numel(),
                                 _stream(a.device))
        _check("ssd_chunked_fwd", st)
    else:
        st = lib.ssd_chunked_fwd_opts(_ptr(a.x), _ptr(a.dt), _ptr(a.A), _ptr(a.B), _ptr(a.C),
                                      _ptr(a.D), a.L, _ptr(a.init), _ptr(a.y), _ptr(a.final),
                                      ctypes.byref(opts), ctypes.byref(a.dims), _ptr(a.ws),
                                      a.ws.numel(), _stream(a.device))
        _check("ssd_chunked_fwd_opts", st)
    return a.y, a.final


NOALLOC_SCRATCH_BYTES = 64 << 20   # SSD_NOALLOC_SCRATCH_BYTES


def ssd_chunked_fwd_noalloc(x, dt, A, B, C, D, chunk_size, init_state=None, y=None,
                            final_state=None, want_final: bool = True, dt_bias=None,
                            dt_softplus: bool = False, z=None, y_io_dtype: bool = False):
    """ssd_chunked_fwd on the library's static scratch (no workspace is
    allocated or passed).  Returns (y, final_state or None).  Shapes whose
    workspace exceeds NOALLOC_SCRATCH_BYTES raise SSDError (SSD_ERR_WORKSPACE)."""
    a = FwdArgs(x, dt, A, B, C, D, chunk_size, init_state, y, final_state, want_final,
                torch.empty(0, dtype=torch.uint8, device=x.device), dt_bias, dt_softplus, z,
                y_io_dtype)
    opts = _layer_opts(a.dt_bias, a.dt_softplus, a.z, a.y_io_dtype)
    st = load_library().ssd_chunked_fwd_noalloc(
        _ptr(a.x), _ptr(a.dt), _ptr(a.A), _ptr(a.B), _ptr(a.C), _ptr(a.D), a.L, _ptr(a.init),
        _ptr(a.y), _ptr(a.final), None if opts is None else ctypes.byref(opts),
        ctypes.byref(a.dims), _stream(a.device))
    _check("ssd_chunked_fwd_noalloc", st)
    return a.y, a.final


def ssd_chunk_cumsum(a: FwdArgs):
    lib = load_library()
    _check("ssd_chunk_cumsum", lib.ssd_chunk_cumsum(_ptr(a.dt), _ptr(a.A), a.L,
                                                    ctypes.byref(a.dims), _ptr(a.ws),
                                                    a.ws.numel(), _stream(a.device)))


def ssd_chunk_state(a: FwdArgs):
    lib = load_library()
    _check("ssd_chunk_state", lib.ssd_chunk_state(_ptr(a.x), _ptr(a.B), a.L, ctypes.byref(a.dims),
                                                  _ptr(a.ws), a.ws.numel(), _stream(a.device)))


def ssd_state_passing(a: FwdArgs):
    lib = load_library()
    _check("ssd_state_passing", lib.ssd_state_passing(_ptr(a.init), _ptr(a.final), a.L,
                                                      ctypes.byref(a.dims), _ptr(a.ws),
                                                      a.ws.numel(), _stream(a.device)))


def ssd_state_fwd(a: FwdArgs):
    """chunk_state + state_passing in one pass (bf16): h_prev and final_state."""
    lib = load_library()
    _check("ssd_state_fwd", lib.ssd_state_fwd(_ptr(a.x), _ptr(a.B), _ptr(a.init), _ptr(a.final),
                                              a.L, ctypes.byref(a.dims), _ptr(a.ws),
                                              a.ws.numel(), _stream(a.device)))


PATH_FOUR_STAGE, PATH_STATE_FWD, PATH_FUSED = 0, 1, 2   # ssd_fwd_path


def fwd_path(dims: Dims, chunk_size: int) -> int:
    """The ssd_fwd_path ssd_chunked_fwd takes for this shape."""
    out = ctypes.c_int(-1)
    _check("ssd_chunked_fwd_path", load_library().ssd_chunked_fwd_path(
        ctypes.byref(dims), chunk_size, ctypes.byref(out)))
    return out.value


def set_path_override(fwd: int = -1, state_rows: int = 0, adj_rows: int = 0):
    """Test hook (ssd_set_path_override): force a forward path and row splits
    for later calls in this process; (-1, 0, 0) restores the default."""
    _check("ssd_set_path_override",
           load_library().ssd_set_path_override(int(fwd), int(state_rows), int(adj_rows)))


def ssd_chunk_scan(a: FwdArgs):
    """The chunk_scan stage (no layer options): writes y in float32."""
    if a.y.dtype != torch.float32:
        raise ValueError("the stage call ssd_chunk_scan writes y in float32; these arguments "
                         "hold a %s y (y_io_dtype): use ssd_chunked_fwd" % a.y.dtype)
    lib = load_library()
    _check("ssd_chunk_scan", lib.ssd_chunk_scan(_ptr(a.x), _ptr(a.B), _ptr(a.C), _ptr(a.D),
                                                _ptr(a.y), a.L, ctypes.byref(a.dims), _ptr(a.ws),
                                                a.ws.numel(), _stream(a.device)))


def workspace_views(a: FwdArgs):
    """Views of the intermediates a forward left in ``a.ws``: G, DT, S, h_prev."""
    Bt, T, H, P = a.x.shape
    N = a.B.shape[3]
    nc = -(-T // a.L)
    off = ssd_chunked_fwd_workspace_layout(a.dims, a.L)

    def view(o, n, dtype, shape):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return a.ws[o:o + nbytes].view(dtype).view(shape)

    units = Bt * H * nc
    return {
        "G": view(off[0], units * a.L, torch.float32, (Bt, H, nc, a.L)),
        "DT": view(off[1], units * a.L, torch.float32, (Bt, H, nc, a.L)),
        "S": view(off[2], units * P * N, torch.float32, (Bt, H, nc, P, N)),
        "h_prev": view(off[3], units * P * N, a.x.dtype, (Bt, H, nc, P, N)),
    }


def ssd_decode_step(state, x_t, dt_t, B_t, C_t, A, D, y_t=None, dt_bias=None,
                    dt_softplus: bool = False, z_t=None, y_io_dtype: bool = False):
    """One decode step; ``state`` [Bt,H,P,N] f32 is updated in place.  Returns y_t [Bt,H,P] f32.

    ``dt_bias`` [H], ``dt_softplus`` and the gate ``z_t`` [Bt,H,P] (x_t's dtype)
    are the optional layer interface (ssd_layer_opts); ``y_io_dtype`` stores
    y_t in x_t's dtype instead of float32.
    """
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device, got %s" % dev)
    if not state.is_contiguous() or state.dtype != torch.float32 or state.dim() != 4:
        raise ValueError("state must be a contiguous float32 [Bt,H,P,N] tensor (updated in place)")
    Bt, H, P, N = state.shape
    io = x_t.dtype
    G = B_t.shape[1]
    x_t = _need(x_t, "x_t", io, (Bt, H, P), dev)
    dt_t = _need(dt_t, "dt_t", torch.float32, (Bt, H), dev)
    B_t = _need(B_t, "B_t", io, (Bt, G, N), dev)
    C_t = _need(C_t, "C_t", io, (Bt, G, N), dev)
    A = _need(A, "A", torch.float32, (H,), dev)
    D = _need(D, "D", torch.float32, (H,), dev)
    ydt = io if y_io_dtype else torch.float32
    y_t = (torch.empty((Bt, H, P), dtype=ydt, device=dev) if y_t is None
           else _need_out(y_t, "y_t", ydt, (Bt, H, P), dev))
    dims = Dims(Bt, 1, H, P, N, G, _io_code(io))
    if dt_bias is not None:
        dt_bias = _need(dt_bias, "dt_bias", torch.float32, (H,), dev)
    if z_t is not None:
        z_t = _need(z_t, "z_t", io, (Bt, H, P), dev)
    lib = load_library()
    opts = _layer_opts(dt_bias, dt_softplus, z_t, y_io_dtype)
    if opts is None:
        _check("ssd_decode_step", lib.ssd_decode_step(_ptr(state), _ptr(x_t), _ptr(dt_t),
                                                      _ptr(B_t), _ptr(C_t), _ptr(A), _ptr(D),
                                                      _ptr(y_t), ctypes.byref(dims),
                                                      _stream(dev)))
    else:
        _check("ssd_decode_step_opts", lib.ssd_decode_step_opts(
            _ptr(state), _ptr(x_t), _ptr(dt_t), _ptr(B_t), _ptr(C_t), _ptr(A), _ptr(D),
            _ptr(y_t), ctypes.byref(opts), ctypes.byref(dims), _stream(dev)))
    return y_t


DECODE_NO_STATE_UPDATE = 1   # SSD_DECODE_NO_STATE_UPDATE


def ssd_decode_multi(state, x, dt, B, C, A, D, y=None, snapshots=None, parent=None,
                     update_state: bool = True, dt_bias=None, dt_softplus: bool = False, z=None,
                     y_io_dtype: bool = False):
    """K decode steps per sequence (speculative decoding); returns (y, snapshots).

    state [Bt,H,P,N] f32 (updated in place unless ``update_state`` is False),
    x [Bt,K,H,P], dt [Bt,K,H] f32, B/C [Bt,K,G,N] (x's dtype), A/D [H] f32.
    ``snapshots``: None (not written), True (allocated here) or a float32
    [Bt,K,H,P,N] tensor that receives the state after every step.  ``parent``
    [Bt,K] int32: step k restarts from the snapshot of step parent[b,k] when
    0 <= parent[b,k] < k (needs snapshots).  y [Bt,K,H,P] f32.
    """
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device, got %s" % dev)
    if not state.is_contiguous() or state.dtype != torch.float32 or state.dim() != 4:
        raise ValueError("state must be a contiguous float32 [Bt,H,P,N] tensor")
    Bt, H, P, N = state.shape
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [Bt,K,H,P] and B, C [Bt,K,G,N]")
    io = x.dtype
    K, G = x.shape[1], B.shape[2]
    x = _need(x, "x", io, (Bt, K, H, P), dev)
    dt = _need(dt, "dt", torch.float32, (Bt, K, H), dev)
    B = _need(B, "B", io, (Bt, K, G, N), dev)
    C = _need(C, "C", io, (Bt, K, G, N), dev)
    A = _need(A, "A", torch.float32, (H,), dev)
    D = _need(D, "D", torch.float32, (H,), dev)
    ydt = io if y_io_dtype else torch.float32
    y = (torch.empty((Bt, K, H, P), dtype=ydt, device=dev) if y is None
         else _need_out(y, "y", ydt, (Bt, K, H, P), dev))
    if snapshots is True:
        snapshots = torch.empty((Bt, K, H, P, N), dtype=torch.float32, device=dev)
    elif snapshots is not None:
        snapshots = _need_out(snapshots, "snapshots", torch.float32, (Bt, K, H, P, N), dev)
    if parent is not None:
        parent = _need(parent, "parent", torch.int32, (Bt, K), dev)
    if dt_bias is not None:
        dt_bias = _need(dt_bias, "dt_bias", torch.float32, (H,), dev)
    if z is not None:
        z = _need(z, "z", io, (Bt, K, H, P), dev)
    opts = _layer_opts(dt_bias, dt_softplus, z, y_io_dtype)
    dims = Dims(Bt, K, H, P, N, G, _io_code(io))
    flags = 0 if update_state else DECODE_NO_STATE_UPDATE
    _check("ssd_decode_multi", load_library().ssd_decode_multi(
        _ptr(state), _ptr(x), _ptr(dt), _ptr(B), _ptr(C), _ptr(A), _ptr(D), _ptr(y),
        _ptr(snapshots), _ptr(parent), flags, None if opts is None else ctypes.byref(opts),
        ctypes.byref(dims), _stream(dev)))
    return y, snapshots


def ssd_decode_step_lp(state, x_t, dt_t, B_t, C_t, A, D, fmt: str, scale=None,
                       philox_rounds: int = 0, seed: int = 0, y_t=None, dt_bias=None,
                       dt_softplus: bool = False, z_t=None, y_io_dtype: bool = False):
    """One decode step on a 16-bit state (``fmt`` "f16", "bf16" or "int16"; "f32"
    is the plain step), updated in place.  state [Bt,H,P,N] of fp16 / bf16 /
    int16; ``scale`` [Bt,H,P] f32 decode scales (int16 only, updated in place);
    ``philox_rounds`` > 0 (10 is standard) and ``seed`` select fp16
    stochastic rounding.  Returns y_t
    [Bt,H,P] f32."""
    if fmt not in STATE_DTYPES:
        raise ValueError("fmt must be one of %s" % sorted(STATE_DTYPES))
    code, sdt = STATE_DTYPES[fmt]
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU device, got %s" % dev)
    if not state.is_contiguous() or state.dtype != sdt or state.dim() != 4:
        raise ValueError("state must be a contiguous %s [Bt,H,P,N] tensor" % sdt)
    Bt, H, P, N = state.shape
    io = x_t.dtype
    G = B_t.shape[1]
    x_t = _need(x_t, "x_t", io, (Bt, H, P), dev)
    dt_t = _need(dt_t, "dt_t", torch.float32, (Bt, H), dev)
    B_t = _need(B_t, "B_t", io, (Bt, G, N), dev)
    C_t = _need(C_t, "C_t", io, (Bt, G, N), dev)
    A = _need(A, "A", torch.float32, (H,), dev)
    D = _need(D, "D", torch.float32, (H,), dev)
    ydt = io if y_io_dtype else torch.float32
    y_t = (torch.empty((Bt, H, P), dtype=ydt, device=dev) if y_t is None
           else _need_out(y_t, "y_t", ydt, (Bt, H, P), dev))
    if scale is not None:
        scale = _need_out(scale, "scale", torch.float32, (Bt, H, P), dev)
    if dt_bias is not None:
        dt_bias = _need(dt_bias, "dt_bias", torch.float32, (H,), dev)
    if z_t is not None:
        z_t = _need(z_t, "z_t", io, (Bt, H, P), dev)
    f = StateFormat(code, int(philox_rounds), int(seed) & 0xFFFFFFFFFFFFFFFF,
                    None if scale is None else scale.data_ptr())
    opts = _layer_opts(dt_bias, dt_softplus, z_t, y_io_dtype)
    dims = Dims(Bt, 1, H, P, N, G, _io_code(io))
    _check("ssd_decode_step_lp", load_library().ssd_decode_step_lp(
        _ptr(state), ctypes.byref(f), _ptr(x_t), _ptr(dt_t), _ptr(B_t), _ptr(C_t), _ptr(A),
        _ptr(D), _ptr(y_t), None if opts is None else ctypes.byref(opts), ctypes.byref(dims),
        _stream(dev)))
    return y_t


def ssd_chunked_bwd_workspace_size(dims: Dims, chunk_size: int) -> int:
    return int(load_library().ssd_chunked_bwd_workspace_size(ctypes.byref(dims), chunk_size))


def ssd_chunked_bwd(x, dt, A, B, C, D, chunk_size, dy, init_state=None, dfinal=None,
                    want_dinit: bool = True, workspace=None):
    """Backward of ssd_chunked_fwd (no layer options).  Returns a dict of float32
    gradients: dx [Bt,T,H,P], ddt [Bt,T,H], dA [H], dB and dC [Bt,T,G,N], dD [H],
    dinit [Bt,H,P,N] (None unless ``want_dinit``).  dy [Bt,T,H,P] f32; dfinal
    [Bt,H,P,N] f32 or None."""
    a = FwdArgs(x, dt, A, B, C, D, chunk_size, init_state, want_final=False,
                workspace=torch.empty(256, dtype=torch.uint8, device=x.device))
    Bt, T, H, P = a.x.shape
    G, N = a.B.shape[2], a.B.shape[3]
    dev = a.device
    dy = _need(dy, "dy", torch.float32, (Bt, T, H, P), dev)
    if dfinal is not None:
        dfinal = _need(dfinal, "dfinal", torch.float32, (Bt, H, P, N), dev)
    need = ssd_chunked_bwd_workspace_size(a.dims, a.L)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    else:
        workspace = _own_workspace(workspace, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dx=torch.empty((Bt, T, H, P), **f32), ddt=torch.empty((Bt, T, H), **f32),
               dA=torch.empty((H,), **f32), dB=torch.empty((Bt, T, G, N), **f32),
               dC=torch.empty((Bt, T, G, N), **f32), dD=torch.empty((H,), **f32),
               dinit=torch.empty((Bt, H, P, N), **f32) if want_dinit else None)
    _check("ssd_chunked_bwd", load_library().ssd_chunked_bwd(
        _ptr(a.x), _ptr(a.dt), _ptr(a.A), _ptr(a.B), _ptr(a.C), _ptr(a.D), a.L, _ptr(a.init),
        _ptr(dy), _ptr(dfinal), _ptr(out["dx"]), _ptr(out["ddt"]), _ptr(out["dA"]),
        _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["dD"]), _ptr(out["dinit"]),
        ctypes.byref(a.dims), _ptr(workspace), workspace.numel(), _stream(dev)))
    return out


# ---------------------------------------------------------------------------
# The operators around the scan.

def _on_gpu(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("tensors must live on a GPU device, got %s" % t.device)
    return t.device


def _current_stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# torch's raw handle of the current stream (what current_stream wraps, at a tenth of its
# cost per call) and its current device, where this torch has them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn: str, dev: torch.device, *args):
    """One library call on dev's current stream, with dev the current device."""
    f = getattr(load_library(), fn)
    stream = _current_stream(dev) if _raw_stream is None else _raw_stream(dev.index)
    if _raw_device() == dev.index:
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st != 0:
        _check(fn, st)


def _in(t, name, dtype, shape, device):
    """An input the library can read: contiguous, and a copy where a view starts off a
    16-byte boundary."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        t = _need(t, name, dtype, shape, device)
    return t.clone() if t.data_ptr() & 15 else t


def _opt(t, name, dtype, shape, device):
    return None if t is None else _in(t, name, dtype, shape, device)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_Ptr3 = ctypes.c_void_p * 3


def _parts3(ts):
    return _Ptr3(*[None if t is None or not t.numel() else t.data_ptr() for t in ts])


def _conv_args(x, weight, bias, splits, silu, tokens: int):
    """(dims, x, weight, bias, splits) of a convolution call; x [Bt, T, C] (tokens = 1)
    or [Bt, C] (tokens = 0) keeps its strides as long as its channels are consecutive."""
    dev = _on_gpu(x, "x")
    io = _io_code(x.dtype)
    if x.dim() != 2 + tokens:
        raise ValueError("x must be %s" % ("[Bt,T,C]" if tokens else "[Bt,C]"))
    C = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    weight = _in(weight, "weight", torch.float32, (C, weight.shape[1]), dev)
    bias = _opt(bias, "bias", torch.float32, (C,), dev)
    splits = (C,) if splits is None else tuple(int(c) for c in splits)
    if not 1 <= len(splits) <= 3 or sum(splits) != C or min(splits) < 0:
        raise ValueError("splits %s must be one to three channel counts that sum to %d"
                         % (splits, C))
    if C > 1 and x.stride(-1) != 1:
        x = x.contiguous()
    dims = ConvDims(x.shape[0], x.shape[1] if tokens else 1, weight.shape[1],
                    (ctypes.c_int64 * 3)(*(splits + (0, 0))[:3]), x.stride(0),
                    x.stride(1) if tokens else 0, io, 1 if silu else 0)
    return dims, x, weight, bias, splits, dev


# (torch.empty takes sizes one by one faster than as a tuple, 1.0 us against 1.4: of a short
# call's 14 us two thirds are the host's)
def _outs(y, name, dtype, shapes, dev):
    if y is None:
        return tuple([torch.empty(*s, dtype=dtype, device=dev) for s in shapes])
    if isinstance(y, torch.Tensor):
        y = (y,)
    if len(y) != len(shapes):
        raise ValueError("%s must hold %d tensors" % (name, len(shapes)))
    return tuple([_need_out(t, "%s[%d]" % (name, i), dtype, s, dev)
                  for i, (t, s) in enumerate(zip(y, shapes))])


def ssd_conv1d_fwd(x, weight, bias=None, silu: bool = True, splits=None, init_state=None,
                   final_state=None, want_final: bool = True, seq_lens=None, y=None):
    """Short causal convolution of a prompt.  Returns (tuple of outputs, final_state or None).

    x [Bt,T,C] (float32 or bfloat16; its channels consecutive, its rows at any
    stride: a slice of a projection is read in place), weight [C,W] f32 with W
    2, 3 or 4, bias [C] f32 or None.  ``splits``: one to three channel counts
    that sum to C, one dense output [Bt,T,splits[i]] each (None = one output).
    init_state [Bt,W-1,C] holds the inputs before the first token, oldest first
    (None = zeros); ``final_state`` may be the same tensor.  ``seq_lens`` [Bt]
    int32: outputs past a sequence's length are zero and its final state is
    that at its length.
    """
    dims, x, weight, bias, splits, dev = _conv_args(x, weight, bias, splits, silu, 1)
    Bt, T, C = x.shape
    W = weight.shape[1]
    init_state = _opt(init_state, "init_state", x.dtype, (Bt, W - 1, C), dev)
    seq_lens = _opt(seq_lens, "seq_lens", torch.int32, (Bt,), dev)
    if final_state is not None:
        final_state = _need_out(final_state, "final_state", x.dtype, (Bt, W - 1, C), dev)
    elif want_final:
        final_state = torch.empty(Bt, W - 1, C, dtype=x.dtype, device=dev)
    y = _outs(y, "y", x.dtype, [(Bt, T, c) for c in splits], dev)
    _call("ssd_conv1d_fwd", dev, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(init_state),
          _addr(seq_lens), _parts3(y + (None,) * (3 - len(y))), _addr(final_state),
          ctypes.byref(dims))
    return y, final_state


def ssd_conv1d_step(conv_state, x_t, weight, bias=None, silu: bool = True, splits=None,
                    slots=None, y_t=None):
    """One token of the convolution per sequence; returns the tuple of outputs [Bt,splits[i]].

    conv_state [num_slots,W-1,C] (x_t's dtype, updated in place) and slots [Bt]
    int32 (None = sequence b has state b): a slot outside the pool marks a
    padded row (output zero, no state touched); a slot may be named once.
    x_t [Bt,C] may be a slice of wider rows.
    """
    dims, x_t, weight, bias, splits, dev = _conv_args(x_t, weight, bias, splits, silu, 0)
    Bt, C = x_t.shape
    if conv_state.dim() != 3:
        raise ValueError("conv_state must be [num_slots,W-1,C]")
    conv_state = _need_out(conv_state, "conv_state", x_t.dtype,
                           (conv_state.shape[0], weight.shape[1] - 1, C), dev)
    slots = _opt(slots, "slots", torch.int32, (Bt,), dev)
    y_t = _outs(y_t, "y_t", x_t.dtype, [(Bt, c) for c in splits], dev)
    _call("ssd_conv1d_step", dev, conv_state.data_ptr(), conv_state.shape[0], _addr(slots),
          x_t.data_ptr(), weight.data_ptr(), _addr(bias), _parts3(y_t + (None,) * (3 - len(y_t))),
          ctypes.byref(dims))
    return y_t


def ssd_conv1d_bwd_workspace_size(dims: ConvDims) -> int:
    return int(load_library().ssd_conv1d_bwd_workspace_size(ctypes.byref(dims)))


def conv1d_layout(dims: ConvDims) -> ConvLayout:
    """How convolution calls of these dims are laid over the chip (ssd_conv1d_layout)."""
    out = ConvLayout()
    _check("ssd_conv1d_layout",
           load_library().ssd_conv1d_layout(ctypes.byref(dims), ctypes.byref(out)))
    return out


def ssd_conv1d_bwd(x, weight, dy, bias=None, silu: bool = True, init_state=None, dfinal=None,
                   want_dinit: bool = True, workspace=None):
    """Gradients of ssd_conv1d_fwd (without seq_lens), float32: a dict of dx [Bt,T,C],
    dweight [C,W], dbias [C] (None without bias) and dinit [Bt,W-1,C] (None unless
    ``want_dinit``).  dy: one tensor or a tuple of one to three, [Bt,T,splits[i]] f32;
    dfinal [Bt,W-1,C] f32 or None."""
    dy = (dy,) if isinstance(dy, torch.Tensor) else tuple(dy)
    dims, x, weight, bias, splits, dev = _conv_args(x, weight, bias, [d.shape[-1] for d in dy],
                                                    silu, 1)
    Bt, T, C = x.shape
    W = weight.shape[1]
    dy = tuple([_in(d, "dy[%d]" % i, torch.float32, (Bt, T, c), dev)
                for i, (d, c) in enumerate(zip(dy, splits))])
    init_state = _opt(init_state, "init_state", x.dtype, (Bt, W - 1, C), dev)
    dfinal = _opt(dfinal, "dfinal", torch.float32, (Bt, W - 1, C), dev)
    if workspace is None:
        workspace = torch.empty(max(ssd_conv1d_bwd_workspace_size(dims), 16), dtype=torch.uint8,
                                device=dev)
    else:
        workspace = _own_workspace(workspace, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dx=torch.empty(Bt, T, C, **f32), dweight=torch.empty(C, W, **f32),
               dbias=None if bias is None else torch.empty(C, **f32),
               dinit=torch.empty(Bt, W - 1, C, **f32) if want_dinit else None)
    _call("ssd_conv1d_bwd", dev, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(init_state),
          _parts3(dy + (None,) * (3 - len(dy))), _addr(dfinal), out["dx"].data_ptr(),
          out["dweight"].data_ptr(), _addr(out["dbias"]), _addr(out["dinit"]), ctypes.byref(dims),
          _addr(workspace), workspace.numel() * workspace.element_size())
    return out


def _scan_layer(x, dt_bias, dt_softplus, z, zname, y_io_dtype, Dm, dev):
    """(options or None, tensors to keep) of a selective-scan call."""
    dt_bias = _opt(dt_bias, "dt_bias", torch.float32, (Dm,), dev)
    z = _opt(z, zname, x.dtype, tuple(x.shape), dev)
    if dt_bias is None and z is None and not dt_softplus and not y_io_dtype:
        return None, None, None
    return (LayerOpts(_addr(dt_bias), 1 if dt_softplus else 0, 1 if y_io_dtype else 0, _addr(z)),
            dt_bias, z)


def _scan_tokens(x, dt, A, B, C, D, names):
    dev = _on_gpu(x, names[0])
    lead, Dm = tuple(x.shape[:-1]), x.shape[-1]
    if A.dim() != 2:
        raise ValueError("A must be [Dm,N]")
    N = A.shape[1]
    return (dev, _in(x, names[0], x.dtype, lead + (Dm,), dev),
            _in(dt, names[1], x.dtype, lead + (Dm,), dev),
            _in(A, "A", torch.float32, (Dm, N), dev),
            _in(B, names[2], x.dtype, lead + (N,), dev),
            _in(C, names[3], x.dtype, lead + (N,), dev),
            _in(D, "D", torch.float32, (Dm,), dev))


def ssd_selective_scan_workspace_size(dims: ScanDims) -> int:
    return int(load_library().ssd_selective_scan_workspace_size(ctypes.byref(dims)))


def ssd_selective_scan_fwd(x, dt, A, B, C, D, init_state=None, y=None, final_state=None,
                           want_final: bool = True, seq_lens=None, dt_bias=None,
                           dt_softplus: bool = False, z=None, y_io_dtype: bool = False,
                           workspace=None):
    """Selective scan of a prompt.  Returns (y, final_state or None).

    x, dt [Bt,T,Dm] (float32 or bfloat16), A [Dm,N] f32 with N 8, 16, 32 or 64,
    B, C [Bt,T,N] (x's dtype), D [Dm] f32, init_state [Bt,Dm,N] f32 or None;
    ``final_state`` may be the same tensor.  y is [Bt,T,Dm] float32, x's dtype
    with ``y_io_dtype``.  ``dt_bias`` [Dm] f32, ``dt_softplus`` and the gate
    ``z`` (x's shape and dtype) are the layer options.  ``seq_lens`` [Bt]
    int32: y past a sequence's length is zero and its final state is that at
    its length.
    """
    if x.dim() != 3:
        raise ValueError("x must be [Bt,T,Dm]")
    dev, x, dt, A, B, C, D = _scan_tokens(x, dt, A, B, C, D, ("x", "dt", "B", "C"))
    Bt, T, Dm = x.shape
    N = A.shape[1]
    dims = ScanDims(Bt, T, Dm, N, _io_code(x.dtype))
    opts, dt_bias, z = _scan_layer(x, dt_bias, dt_softplus, z, "z", y_io_dtype, Dm, dev)
    init_state = _opt(init_state, "init_state", torch.float32, (Bt, Dm, N), dev)
    seq_lens = _opt(seq_lens, "seq_lens", torch.int32, (Bt,), dev)
    ydt = x.dtype if y_io_dtype else torch.float32
    y = (torch.empty(Bt, T, Dm, dtype=ydt, device=dev) if y is None
         else _need_out(y, "y", ydt, (Bt, T, Dm), dev))
    if final_state is not None:
        final_state = _need_out(final_state, "final_state", torch.float32, (Bt, Dm, N), dev)
    elif want_final:
        final_state = torch.empty(Bt, Dm, N, dtype=torch.float32, device=dev)
    if workspace is None:
        need = ssd_selective_scan_workspace_size(dims)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        workspace = _own_workspace(workspace, dev)
    _call("ssd_selective_scan_fwd", dev, x.data_ptr(), dt.data_ptr(), A.data_ptr(),
          B.data_ptr(), C.data_ptr(), D.data_ptr(), _addr(init_state), _addr(seq_lens),
          y.data_ptr(), _addr(final_state),
          None if opts is None else ctypes.byref(opts), ctypes.byref(dims), _addr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size())
    return y, final_state


def ssd_selective_scan_step(state, x_t, dt_t, A, B_t, C_t, D, slots=None, y_t=None, dt_bias=None,
                            dt_softplus: bool = False, z_t=None, y_io_dtype: bool = False):
    """One token of the selective scan per sequence; returns y_t [Bt,Dm].

    state [num_slots,Dm,N] f32 is updated in place; slots [Bt] int32 (None =
    sequence b has state b): a slot outside the pool marks a padded row (y
    zero, no state touched); a slot may be named once.  x_t, dt_t [Bt,Dm],
    B_t, C_t [Bt,N]; the other arguments as for ssd_selective_scan_fwd.
    """
    if x_t.dim() != 2:
        raise ValueError("x_t must be [Bt,Dm]")
    dev, x_t, dt_t, A, B_t, C_t, D = _scan_tokens(x_t, dt_t, A, B_t, C_t, D,
                                                  ("x_t", "dt_t", "B_t", "C_t"))
    Bt, Dm = x_t.shape
    N = A.shape[1]
    if state.dim() != 3:
        raise ValueError("state must be [num_slots,Dm,N]")
    state = _need_out(state, "state", torch.float32, (state.shape[0], Dm, N), dev)
    slots = _opt(slots, "slots", torch.int32, (Bt,), dev)
    opts, dt_bias, z_t = _scan_layer(x_t, dt_bias, dt_softplus, z_t, "z_t", y_io_dtype, Dm, dev)
    ydt = x_t.dtype if y_io_dtype else torch.float32
    y_t = (torch.empty(Bt, Dm, dtype=ydt, device=dev) if y_t is None
           else _need_out(y_t, "y_t", ydt, (Bt, Dm), dev))
    dims = ScanDims(Bt, 1, Dm, N, _io_code(x_t.dtype))
    _call("ssd_selective_scan_step", dev, state.data_ptr(), state.shape[0], _addr(slots),
          x_t.data_ptr(), dt_t.data_ptr(), A.data_ptr(), B_t.data_ptr(), C_t.data_ptr(),
          D.data_ptr(), y_t.data_ptr(),
          None if opts is None else ctypes.byref(opts), ctypes.byref(dims))
    return y_t


def ssd_selective_scan_bwd_workspace_size(dims: ScanDims) -> int:
    return int(load_library().ssd_selective_scan_bwd_workspace_size(ctypes.byref(dims)))


def selective_scan_layout(dims: ScanDims) -> ScanLayout:
    """How selective-scan calls of these dims are laid over the chip
    (ssd_selective_scan_layout)."""
    out = ScanLayout()
    _check("ssd_selective_scan_layout",
           load_library().ssd_selective_scan_layout(ctypes.byref(dims), ctypes.byref(out)))
    return out


def ssd_selective_scan_bwd(x, dt, A, B, C, D, dy, init_state=None, dfinal=None, dt_bias=None,
                           dt_softplus: bool = False, z=None, want_dinit: bool = True,
                           workspace=None):
    """Gradients of ssd_selective_scan_fwd (without seq_lens), float32: a dict of dx, ddt
    [Bt,T,Dm], dA [Dm,N], dB, dC [Bt,T,N], dD [Dm], ddt_bias [Dm] (None without dt_bias),
    dz [Bt,T,Dm] (None without z) and dinit [Bt,Dm,N] (None unless ``want_dinit``).
    dy [Bt,T,Dm] f32; dfinal [Bt,Dm,N] f32 or None."""
    if x.dim() != 3:
        raise ValueError("x must be [Bt,T,Dm]")
    dev, x, dt, A, B, C, D = _scan_tokens(x, dt, A, B, C, D, ("x", "dt", "B", "C"))
    Bt, T, Dm = x.shape
    N = A.shape[1]
    dims = ScanDims(Bt, T, Dm, N, _io_code(x.dtype))
    opts, dt_bias, z = _scan_layer(x, dt_bias, dt_softplus, z, "z", False, Dm, dev)
    dy = _in(dy, "dy", torch.float32, (Bt, T, Dm), dev)
    init_state = _opt(init_state, "init_state", torch.float32, (Bt, Dm, N), dev)
    dfinal = _opt(dfinal, "dfinal", torch.float32, (Bt, Dm, N), dev)
    if workspace is None:
        workspace = torch.empty(max(ssd_selective_scan_bwd_workspace_size(dims), 16),
                                dtype=torch.uint8, device=dev)
    else:
        workspace = _own_workspace(workspace, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dx=torch.empty(Bt, T, Dm, **f32), ddt=torch.empty(Bt, T, Dm, **f32),
               dA=torch.empty(Dm, N, **f32), dB=torch.empty(Bt, T, N, **f32),
               dC=torch.empty(Bt, T, N, **f32), dD=torch.empty(Dm, **f32),
               ddt_bias=None if dt_bias is None else torch.empty(Dm, **f32),
               dz=None if z is None else torch.empty(Bt, T, Dm, **f32),
               dinit=torch.empty(Bt, Dm, N, **f32) if want_dinit else None)
    _call("ssd_selective_scan_bwd", dev, x.data_ptr(), dt.data_ptr(), A.data_ptr(),
          B.data_ptr(), C.data_ptr(), D.data_ptr(), _addr(init_state), dy.data_ptr(),
          _addr(dfinal), out["dx"].data_ptr(),
          out["ddt"].data_ptr(), out["dA"].data_ptr(), out["dB"].data_ptr(), out["dC"].data_ptr(),
          out["dD"].data_ptr(), _addr(out["ddt_bias"]), _addr(out["dz"]), _addr(out["dinit"]),
          None if opts is None else ctypes.byref(opts), ctypes.byref(dims), _addr(workspace),
          workspace.numel() * workspace.element_size())
    return out


def _cache_pool(codes, scales):
    dev = _on_gpu(codes, "codes")
    if codes.dtype not in CACHE_FORMATS:
        raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % codes.dtype)
    if codes.dim() != 2:
        raise ValueError("codes must be [num_slots,size]")
    nblk = -(-codes.shape[1] // CACHE_BLOCK)
    codes = _need_out(codes, "codes", codes.dtype, tuple(codes.shape), dev)
    scales = _need_out(scales, "scales", torch.float32, (codes.shape[0], nblk), dev)
    return codes, scales, dev


def ssd_cache_write(state, codes, scales, slots=None):
    """Stores states at 8 bits: state [n,...] f32 (size = elements of one state, a multiple
    of 8) into the rows ``slots`` [n] int32 of codes [num_slots,size] (int8 or
    float8_e4m3fn) and scales [num_slots,ceil(size/64)] f32, in place.  A slot outside the
    pool skips that state; a slot may be named once."""
    codes, scales, dev = _cache_pool(codes, scales)
    n, size = state.shape[0], codes.shape[1]
    state = _in(state, "state", torch.float32, tuple(state.shape), dev)
    if state.numel() != n * size:
        raise ValueError("a state holds %d elements, the pool's rows %d"
                         % (state.numel() // max(n, 1), size))
    slots = _opt(slots, "slots", torch.int32, (n,), dev)
    _call("ssd_cache_write", dev, state.data_ptr(), n, size, _addr(slots), codes.shape[0],
          codes.data_ptr(), scales.data_ptr(), CACHE_FORMATS[codes.dtype])


def ssd_cache_read(codes, scales, slots=None, shape=None, state=None):
    """Reads states back: returns state [n, *shape] f32 (shape None = [n,size]) from the rows
    ``slots`` [n] int32 of the pool (None = every row).  A slot may be named several times;
    one outside the pool reads as zeros."""
    codes, scales, dev = _cache_pool(codes, scales)
    size = codes.shape[1]
    n = codes.shape[0] if slots is None else slots.shape[0]
    slots = _opt(slots, "slots", torch.int32, (n,), dev)
    full = (n, size) if shape is None else (n,) + tuple(shape)
    state = (torch.empty(*full, dtype=torch.float32, device=dev) if state is None
             else _need_out(state, "state", torch.float32, full, dev))
    if state.numel() != n * size:
        raise ValueError("a state of shape %s does not hold the pool's %d elements"
                         % (full[1:], size))
    _call("ssd_cache_read", dev, codes.data_ptr(), scales.data_ptr(), n, size, _addr(slots),
          codes.shape[0], state.data_ptr(), CACHE_FORMATS[codes.dtype])
    return state
