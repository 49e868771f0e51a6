"""The C-ABI boundary of linear attention, the group norm and 4-bit projections,
without a GPU: every invalid call is refused on the host, with its status and the
name of what is wrong, before any HIP call."""

import ctypes
import os

import pytest
import torch

from selective_state_space_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH),
                                reason="libssd.so not built (python -m selective_state_space_amd.build)")

# Fake, aligned, never dereferenced: every call below fails validation first.
P16 = 0x1000
P_MIS = 0x1008
BIG = 1 << 40


def lib():
    return ssd.load_library()


def detail():
    return lib().ssd_last_error_detail().decode()


def ref(d):
    return None if d is None else ctypes.byref(d)


def attn_dims(Bt=2, T=30, H=4, G=2, K=64, V=32, qb=8000, qt=256, kb=8000, kt=128, vb=8000, vt=64,
              io=ssd.SSD_BF16, scale=0.125):
    return ssd.AttnDims(Bt, T, H, G, K, V, qb, qt, kb, kt, vb, vt, io, scale)


def attn_fwd(d, q=P16, k=P16, v=P16, decay=P16, init=P16, lens=P16, y=P16, fin=P16, ws=P16,
             wsb=BIG):
    return lib().ssd_linear_attn_fwd(q, k, v, decay, init, lens, y, fin, ref(d), ws, wsb, None)


def attn_step(d, state=P16, num=8, slots=P16, q=P16, k=P16, v=P16, decay=P16, y=P16):
    return lib().ssd_linear_attn_step(state, num, slots, q, k, v, decay, y, ref(d), None)


def attn_bwd(d, q=P16, k=P16, v=P16, decay=P16, init=P16, lens=P16, dy=P16, dfinal=P16, dq=P16,
             dk=P16, dv=P16, dinit=P16, ws=P16, wsb=BIG):
    return lib().ssd_linear_attn_bwd(q, k, v, decay, init, lens, dy, dfinal, dq, dk, dv, dinit,
                                     ref(d), ws, wsb, None)


@pytest.mark.parametrize("call", [attn_fwd, attn_step, attn_bwd])
@pytest.mark.parametrize("kw,code,word", [
    (dict(Bt=-1), -2, "batch"), (dict(Bt=(1 << 30) + 1), -2, "batch"),
    (dict(H=0), -2, "nheads"), (dict(H=65537, G=1), -2, "nheads"), (dict(G=0), -2, "ngroups"),
    (dict(G=3), -2, "ngroups"), (dict(G=8), -2, "ngroups"),
    (dict(K=0), -3, "dim_k"), (dict(K=12), -3, "dim_k"), (dict(K=264), -3, "dim_k"),
    (dict(V=4), -3, "dim_v"), (dict(V=-8), -3, "dim_v"), (dict(V=512), -3, "dim_v"),
    (dict(io=2), -3, "io_dtype"), (dict(scale=float("nan")), -2, "scale"),
    (dict(scale=float("inf")), -2, "scale"),
    (dict(qb=-8), -2, "q_batch_stride"), (dict(kb=(1 << 40) + 8), -2, "k_batch_stride"),
    (dict(vb=4), -4, "v_batch_stride"), (dict(qb=2, io=ssd.SSD_F32), -4, "q_batch_stride"),
    (dict(Bt=1 << 24), -2, "too large"),
])
def test_attn_dims(call, kw, code, word):
    assert call(attn_dims(**kw)) == code
    assert word in detail()


def test_attn_sequence():
    for call in (attn_fwd, attn_bwd):
        assert call(attn_dims(T=-1)) == -2 and "seqlen" in detail()
        assert call(attn_dims(qt=4)) == -4 and "q_token_stride" in detail()
        assert call(attn_dims(kt=-8)) == -2 and "k_token_stride" in detail()
        assert call(attn_dims(vt=12)) == -4 and "v_token_stride" in detail()
        assert call(attn_dims(Bt=1 << 12, T=1 << 30, G=4)) == -2 and "too large" in detail()
    for call in (attn_fwd, attn_bwd, attn_step):
        assert call(None) == -1 and "dims" in detail()


@pytest.mark.parametrize("call,required,optional", [
    (attn_fwd, ["q", "k", "v", "decay", "y"], ["init", "lens", "fin", "ws"]),
    (attn_step, ["state", "q", "k", "v", "decay", "y"], ["slots"]),
    (attn_bwd, ["q", "k", "v", "decay", "dy", "dq", "dk", "dv"],
     ["init", "lens", "dfinal", "dinit", "ws"]),
])
def test_attn_pointers(call, required, optional):
    for f in required:
        assert call(attn_dims(), **{f: None}) == -1, f
    for f in required + optional:
        assert call(attn_dims(), **{f: P_MIS}) == -4, f


def test_attn_slots():
    assert attn_step(attn_dims(), num=1, slots=None) == -2 and "num_slots" in detail()
    assert attn_step(attn_dims(), num=-1) == -2 and "num_slots" in detail()


def test_attn_workspaces():
    few = attn_dims(Bt=1, T=8192, H=2, G=2)
    for call, size in ((attn_fwd, ssd.ssd_linear_attn_workspace_size),
                       (attn_bwd, ssd.ssd_linear_attn_bwd_workspace_size)):
        need = size(few)
        assert need > 0 and call(few, wsb=need - 1) == -5 and str(need) in detail()
        assert call(few, ws=None) == -1 and "workspace" in detail()
        assert size(attn_dims(K=5)) == 0
        assert size(attn_dims(Bt=64, H=64, G=64, T=4096)) == 0    # the chip is full without cuts
    # the gradients of shared heads are held apart until they are summed
    many = attn_dims(Bt=64, H=64, G=32, T=100)
    assert ssd.ssd_linear_attn_bwd_workspace_size(many) == 64 * 64 * 100 * (64 + 32) * 4


def test_attn_layout():
    for kw in (dict(), dict(Bt=1, T=65536, H=1, G=1), dict(Bt=64, T=4096, H=64),
               dict(T=0), dict(Bt=0)):
        lay = ssd.linear_attn_layout(attn_dims(**kw))
        assert lay.fwd_cols in (64, 128) and lay.bwd_cols in (64, 128)
        assert lay.fwd_segments >= 1 and lay.bwd_segments >= 1
    assert ssd.linear_attn_layout(attn_dims(Bt=1, T=65536, H=1, G=1)).fwd_segments > 8
    assert lib().ssd_linear_attn_layout(ref(attn_dims()), None) == -1


def norm_dims(Bt=2, T=30, C=96, groups=3, xb=3000, xt=100, zb=3000, zt=100, io=ssd.SSD_BF16,
              form=2, rms=0, eps=1e-5):
    return ssd.NormDims(Bt, T, C, groups, xb, xt, zb, zt, io, form, rms, eps)


def norm_fwd(d, x=P16, z=P16, weight=P16, bias=P16, lens=P16, y=P16):
    return lib().ssd_group_norm_fwd(x, z, weight, bias, lens, y, ref(d), None)


def norm_bwd(d, x=P16, z=P16, weight=P16, bias=P16, lens=P16, dy=P16, dx=P16, dz=P16,
             dweight=P16, dbias=P16, ws=P16, wsb=BIG):
    return lib().ssd_group_norm_bwd(x, z, weight, bias, lens, dy, dx, dz, dweight, dbias, ref(d),
                                    ws, wsb, None)


@pytest.mark.parametrize("call", [norm_fwd, norm_bwd])
@pytest.mark.parametrize("kw,code,word", [
    (dict(Bt=-1), -2, "batch"), (dict(T=-1), -2, "seqlen"), (dict(C=0), -2, "channels"),
    (dict(C=(1 << 24) + 1, groups=1), -2, "channels"), (dict(groups=0), -2, "groups"),
    (dict(groups=5), -2, "groups"), (dict(groups=97), -2, "groups"),
    (dict(C=16385, groups=1), -3, "16384"), (dict(io=3), -3, "io_dtype"),
    (dict(form=4), -3, "form"), (dict(form=-1), -3, "form"), (dict(eps=0.0), -2, "eps"),
    (dict(eps=-1.0), -2, "eps"), (dict(eps=float("nan")), -2, "eps"),
    (dict(eps=float("inf")), -2, "eps"), (dict(xb=-1), -2, "x_batch_stride"),
    (dict(zt=(1 << 40) + 1), -2, "z_token_stride"), (dict(form=1), -3, "no gate"),
    (dict(Bt=1 << 20, T=1 << 10), -2, "too large"),
])
def test_norm_dims(call, kw, code, word):
    assert call(norm_dims(**kw)) == code
    assert word in detail()


@pytest.mark.parametrize("call,required,optional", [
    (norm_fwd, ["y"], ["weight", "bias", "lens"]),
    (norm_bwd, ["dy", "dx", "dz", "ws"], ["weight", "bias", "lens", "dweight", "dbias"]),
])
def test_norm_pointers(call, required, optional):
    assert call(None) == -1 and "dims" in detail()
    for f in required:
        assert call(norm_dims(), **{f: None}) == -1, f
    for f in required + optional:
        assert call(norm_dims(), **{f: P_MIS}) == -4, f
    # x and z need the alignment of their elements only
    for f in ("x", "z"):
        assert call(norm_dims(), **{f: None}) == -1 and f in detail()
        assert call(norm_dims(), **{f: 0x1001}) == -4 and f in detail()
        assert call(norm_dims(io=ssd.SSD_F32), **{f: 0x1002}) == -4


def test_norm_workspace():
    d = norm_dims()
    need = ssd.ssd_group_norm_bwd_workspace_size(d)
    assert need >= 96 * 4 and norm_bwd(d, wsb=need - 1) == -5 and str(need) in detail()
    assert ssd.ssd_group_norm_bwd_workspace_size(norm_dims(groups=5)) == 0
    assert ssd.ssd_group_norm_bwd_workspace_size(norm_dims(T=0)) == 0
    assert norm_fwd(norm_dims(T=0), x=None, z=None, y=None) == 0
    assert norm_bwd(norm_dims(Bt=0), x=None, z=None, dy=None, dx=None, dz=None, dweight=None,
                    dbias=None, ws=None, wsb=0) == 0


def w4_dims(rows=3, K=256, O=10, group=64, xs=256, io=ssd.SSD_BF16):
    return ssd.W4Dims(rows, K, O, group, xs, io)


def w4_linear(d, x=P16, codes=P16, scales=P16, bias=P16, y=P16):
    return lib().ssd_w4_linear(x, codes, scales, bias, y, ref(d), None)


def w4_quantize(d, weight=P16, codes=P16, scales=P16):
    return lib().ssd_w4_quantize(weight, codes, scales, ref(d), None)


def w4_dequantize(d, weight=P16, codes=P16, scales=P16):
    return lib().ssd_w4_dequantize(codes, scales, weight, ref(d), None)


@pytest.mark.parametrize("call", [w4_linear, w4_quantize, w4_dequantize])
@pytest.mark.parametrize("kw,code,word", [
    (dict(group=32), -3, "group"), (dict(group=0), -3, "group"), (dict(K=0), -2, "inputs"),
    (dict(K=96), -2, "inputs"), (dict(K=192, group=128), -2, "inputs"),
    (dict(K=(1 << 24) + 64), -2, "inputs"), (dict(O=0), -2, "outputs"),
    (dict(O=(1 << 24) + 1), -2, "outputs"), (dict(io=7), -3, "io_dtype"),
    (dict(K=1 << 24, O=1 << 24), -2, "too large"),
])
def test_w4_dims(call, kw, code, word):
    assert call(w4_dims(**kw)) == code
    assert word in detail()


@pytest.mark.parametrize("call,required", [(w4_linear, ["x", "codes", "scales", "y"]),
                                           (w4_quantize, ["weight", "codes", "scales"]),
                                           (w4_dequantize, ["weight", "codes", "scales"])])
def test_w4_pointers(call, required):
    assert call(None) == -1 and "dims" in detail()
    for f in required:
        assert call(w4_dims(), **{f: None}) == -1, f
        assert call(w4_dims(), **{f: P_MIS}) == -4, f
    if call is w4_linear:
        assert call(w4_dims(), bias=P_MIS) == -4
        assert call(w4_dims(rows=-1)) == -2 and "rows" in detail()
        assert call(w4_dims(xs=-8)) == -2 and "x_row_stride" in detail()
        assert call(w4_dims(xs=260)) == -4 and "x_row_stride" in detail()
        assert call(w4_dims(rows=0), x=None, y=None) == 0


# ---------------------------------------------------------------------------
# the binding, with the library call replaced

@pytest.fixture
def on_host(monkeypatch):
    calls = []
    monkeypatch.setattr(ssd, "_on_gpu", lambda t, name: t.device)
    monkeypatch.setattr(ssd, "_call", lambda fn, dev, *a: calls.append((fn, a)))
    return calls


def test_binding_refuses_host_tensors():
    q, x = torch.zeros(1, 2, 3, 8), torch.zeros(1, 2, 64)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.bfloat16)
    for f in (lambda: ssd.ssd_linear_attn_fwd(q, q, q, q[0, 0, :, 0]),
              lambda: ssd.ssd_linear_attn_bwd(q, q, q, q[0, 0, :, 0], q),
              lambda: ssd.ssd_linear_attn_step(q, q[0], q[0], q[0], q[0, 0, :, 0]),
              lambda: ssd.ssd_group_norm_fwd(x, 2), lambda: ssd.ssd_group_norm_bwd(x, 2, x),
              lambda: ssd.ssd_w4_quantize(x[0], 64),
              lambda: ssd.ssd_w4_dequantize(codes, scales),
              lambda: ssd.ssd_w4_linear(x[0], codes, scales)):
        with pytest.raises(ValueError, match="GPU"):
            f()


def test_binding_refuses_shapes(on_host):
    z = torch.zeros
    q, k, v, r = z(1, 2, 4, 8), z(1, 2, 2, 8), z(1, 2, 2, 16), z(4)
    bad = [
        lambda: ssd.ssd_linear_attn_fwd(q[0], k[0], v[0], r),
        lambda: ssd.ssd_linear_attn_fwd(q, k[0], v, r),
        lambda: ssd.ssd_linear_attn_fwd(q, k[..., :4], v, r),
        lambda: ssd.ssd_linear_attn_fwd(q, k, v[:, :1], r),
        lambda: ssd.ssd_linear_attn_fwd(q, k[:, :, :1], v, r),
        lambda: ssd.ssd_linear_attn_fwd(q, k, v, r[:2]),
        lambda: ssd.ssd_linear_attn_fwd(q, k, v, r, init_state=z(1, 4, 16, 8)),
        lambda: ssd.ssd_linear_attn_fwd(q, k, v, r, seq_lens=z(2, dtype=torch.int32)),
        lambda: ssd.ssd_linear_attn_fwd(q, k, v, r, y=z(1, 2, 16, 4).transpose(2, 3)),
        lambda: ssd.ssd_linear_attn_bwd(q, k, v, r, q),
        lambda: ssd.ssd_linear_attn_step(z(3, 4, 16, 8), q[:, 0], k[:, 0], v[:, 0], r),
        lambda: ssd.ssd_linear_attn_step(z(4, 8, 16), q[:, 0], k[:, 0], v[:, 0], r),
        lambda: ssd.ssd_group_norm_fwd(z(6), 2),
        lambda: ssd.ssd_group_norm_fwd(z(1, 2, 6), 2, z=z(1, 2, 5), form="gate"),
        lambda: ssd.ssd_group_norm_fwd(z(1, 2, 6), 2, weight=z(5)),
        lambda: ssd.ssd_group_norm_fwd(z(1, 2, 6), 2, form="relu"),
        lambda: ssd.ssd_group_norm_bwd(z(1, 2, 6), 2, z(1, 2, 5)),
        lambda: ssd.ssd_w4_quantize(z(4, 96), 64), lambda: ssd.ssd_w4_quantize(z(128), 64),
        lambda: ssd.ssd_w4_linear(z(2, 64), z(4, 64, dtype=torch.uint8),
                                  z(4, 1, dtype=torch.bfloat16)),
        lambda: ssd.ssd_w4_linear(z(2, 128), z(4, 64, dtype=torch.uint8),
                                  z(3, 1, dtype=torch.bfloat16)),
        lambda: ssd.ssd_w4_linear(z(2, 128), z(4, 64, dtype=torch.uint8),
                                  z(4, 0, dtype=torch.bfloat16)),
        lambda: ssd.ssd_w4_linear(z(2, 2, 128), z(4, 64, dtype=torch.uint8),
                                  z(4, 1, dtype=torch.bfloat16)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was taken" % i)
    half = torch.float16
    for f in (lambda: ssd.ssd_linear_attn_fwd(q.to(half), k.to(half), v.to(half), r),
              lambda: ssd.ssd_linear_attn_fwd(q, k.bfloat16(), v, r),
              lambda: ssd.ssd_linear_attn_fwd(q, k, v, r.double()),
              lambda: ssd.ssd_group_norm_fwd(z(1, 2, 6, dtype=half), 2),
              lambda: ssd.ssd_w4_linear(z(2, 128), z(4, 64, dtype=torch.int8),
                                        z(4, 1, dtype=torch.bfloat16)),
              lambda: ssd.ssd_w4_linear(z(2, 128), z(4, 64, dtype=torch.uint8), z(4, 1)),
              lambda: ssd.ssd_linear_attn_fwd(q, None, v, r)):
        with pytest.raises(TypeError):
            f()
    assert not on_host


def test_binding_reads_slices_in_place(on_host):
    """Rows of a projection are passed by their strides; what does not start on 16 bytes, or
    has other strides, as a dense copy."""
    proj = torch.zeros(2, 5, 4 * 8 + 2 * 8 + 2 * 16, dtype=torch.bfloat16)
    q, k, v = proj.split((32, 16, 32), 2)
    q, k, v = q.unflatten(2, (4, 8)), k.unflatten(2, (2, 8)), v.unflatten(2, (2, 16))
    ssd.ssd_linear_attn_fwd(q, k, v, torch.zeros(4))
    fn, a = on_host[-1]
    assert fn == "ssd_linear_attn_fwd"
    assert a[0] == q.data_ptr() and a[1] == k.data_ptr() and a[2] == v.data_ptr()
    d = a[8]._obj
    assert (d.q_batch_stride, d.q_token_stride, d.v_token_stride) == (400, 80, 80)
    ssd.ssd_linear_attn_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, torch.zeros(4))
    d = on_host[-1][1][8]._obj
    assert (d.q_batch_stride, d.q_token_stride) == (160, 32)
    x = torch.zeros(2, 5, 70)[:, :, 3:67]
    ssd.ssd_group_norm_fwd(x, 4)
    a = on_host[-1][1]
    assert a[0] == x.data_ptr() and a[6]._obj.x_token_stride == 70
