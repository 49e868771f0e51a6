"""Workspaces and strides of linear attention, the group norm and 4-bit projections at the
binding and the C ABI, without a GPU: the library call is replaced, or refuses."""

import ctypes
import os

import pytest
import torch

from selective_state_space_amd import ssd

from test_block_abi import attn_dims, attn_fwd, detail, norm_dims, norm_fwd, w4_dims, w4_linear

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH),
                                reason="libssd.so not built (python -m selective_state_space_amd.build)")


@pytest.fixture
def on_host(monkeypatch):
    calls = []
    monkeypatch.setattr(ssd, "_on_gpu", lambda t, name: t.device)
    monkeypatch.setattr(ssd, "_call", lambda fn, dev, *a: calls.append((fn, a)))
    return calls


def calls(device):
    z = lambda *s: torch.zeros(*s, device=device)
    q, k, v, r, x = z(1, 1024, 2, 8), z(1, 1024, 1, 8), z(1, 1024, 1, 8), z(2), z(1, 4, 8)
    return {
        "attn_fwd": lambda ws: ssd.ssd_linear_attn_fwd(q, k, v, r, workspace=ws),
        "attn_bwd": lambda ws: ssd.ssd_linear_attn_bwd(q, k, v, r, q, workspace=ws),
        "norm_bwd": lambda ws: ssd.ssd_group_norm_bwd(x, 2, x, z(8), workspace=ws),
    }


NAMES = ["attn_fwd", "attn_bwd", "norm_bwd"]


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


@pytest.mark.parametrize("name", NAMES)
def test_workspace_refused_before_the_library_is_called(name, on_host):
    call = calls("cpu")[name]
    refused(call, "cpu", "meta")
    assert not on_host
    call(torch.empty(1 << 20, dtype=torch.uint8))
    assert len(on_host) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_workspace_refused_on_the_gpu(name):
    call = calls("cuda")[name]
    refused(call, "cuda", "cpu")
    with pytest.raises(ssd.SSDError, match="workspace"):
        call(torch.empty(16, dtype=torch.uint8, device="cuda"))
    call(None)
    call(torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


def test_token_strides_past_the_limit():
    """Rows of one access lie at most 2^24 elements apart; the library refuses more, and the
    binding passes a dense copy."""
    top = 1 << 24
    for name in ("qt", "kt", "vt"):
        assert attn_fwd(attn_dims(**{name: top + 8}), ws=None) == -2
        assert name[0] + "_token_stride" in detail()
    assert w4_linear(w4_dims(xs=top + 8)) == -2 and "x_row_stride" in detail()


def test_binding_refuses_what_is_no_tensor(on_host):
    q, r = torch.zeros(1, 2, 1, 8), torch.zeros(1)
    for f in (lambda: ssd.ssd_linear_attn_fwd(q, None, q, r),
              lambda: ssd.ssd_linear_attn_bwd(q, q, [1.0], r, q),
              lambda: ssd.ssd_group_norm_fwd(q[0], 1, z=3.0, form="gate"),
              lambda: ssd.ssd_linear_attn_fwd(q, q, q, 0.5)):
        with pytest.raises((TypeError, ValueError)):
            f()
    for f in (lambda: ssd.ssd_linear_attn_step(None, q[0], q[0], q[0], r),
              lambda: ssd.ssd_linear_attn_step(torch.zeros(1, 1, 8, 8), q, q, q, r),
              lambda: ssd.ssd_linear_attn_fwd(q[0], q[0], q[0], r),
              lambda: ssd.ssd_linear_attn_fwd(q[None], q[None], q[None], r)):
        with pytest.raises(ValueError):
            f()
    assert not on_host


def test_binding_refuses_a_first_argument_that_is_no_tensor():
    q, r = torch.zeros(1, 2, 1, 8), torch.zeros(1)
    for f in (lambda: ssd.ssd_linear_attn_fwd(None, q, q, r),
              lambda: ssd.ssd_linear_attn_bwd([1.0], q, q, r, q),
              lambda: ssd.ssd_group_norm_fwd(None, 1), lambda: ssd.ssd_w4_quantize(1.0, 64),
              lambda: ssd.ssd_w4_linear(None, q, q)):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            f()


def test_binding_copies_rows_that_lie_far_apart(on_host):
    far = torch.empty(1).expand(1)     # (a shape alone: nothing of it is read)
    far = torch.as_strided(torch.empty((1 << 24) + 8 + 16, dtype=torch.bfloat16), (1, 2, 1, 16),
                           (0, (1 << 24) + 8, 16, 1))
    near = torch.zeros(1, 2, 1, 16, dtype=torch.bfloat16)
    ssd.ssd_linear_attn_fwd(far, near, near, torch.zeros(1))
    a = on_host[-1][1]
    assert a[0] != far.data_ptr() and a[8]._obj.q_token_stride == 16
    # between sequences any distance is read in place
    ssd.ssd_linear_attn_step(torch.zeros(2, 1, 16, 16), far[0], near[0], near[0], torch.zeros(1))
    a = on_host[-1][1]
    assert a[3] == far.data_ptr() and a[8]._obj.q_batch_stride == (1 << 24) + 8
    x = torch.as_strided(torch.empty((1 << 24) + 8 + 64), (2, 64), ((1 << 24) + 8, 1))
    ssd.ssd_w4_linear(x, torch.zeros(4, 32, dtype=torch.uint8),
                      torch.zeros(4, 1, dtype=torch.bfloat16))
    a = on_host[-1][1]
    assert a[0] != x.data_ptr() and a[5]._obj.x_row_stride == 64


def test_sizes_that_one_launch_holds():
    """Large calls that the grids hold are taken, those that they do not are refused, before
    anything is launched (a NULL tensor is found after the sizes)."""
    none = dict(q=None)
    for kw, code in ((dict(Bt=8192, H=32, G=32, T=4096), -1), (dict(Bt=1 << 21, H=8, G=8), -2),
                     (dict(Bt=1 << 15, T=1 << 20), -1), (dict(Bt=1 << 15, T=1 << 25), -2)):
        assert attn_fwd(attn_dims(**kw), **none) == code, (kw, detail())
    for kw, code in ((dict(Bt=8, T=65536, C=5120, groups=40), -1),
                     (dict(Bt=8, T=1 << 20, C=2048, groups=1), -1),
                     (dict(Bt=1 << 20, T=1 << 20), -2), (dict(Bt=1 << 15, T=1 << 15), -2)):
        assert norm_fwd(norm_dims(**kw), x=None, z=None) == code, (kw, detail())
    for kw, code in ((dict(rows=65535 * 16), -1), (dict(rows=65535 * 16 + 1), -2)):
        assert w4_linear(w4_dims(**kw), x=None) == code, (kw, detail())


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 2, 5, 20, 40])
def test_a_row_that_is_not_finite_is_alone(rows):
    """An infinity or a NaN in a row of x leaves the other rows' products as they are."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    codes, scales = ssd.ssd_w4_quantize(torch.randn(100, 256, generator=g, device="cuda"), 64)
    for io in (torch.float32, torch.bfloat16):
        x = torch.randn(rows, 256, generator=g, device="cuda").to(io)
        want = ssd.ssd_w4_linear(x, codes, scales)
        for bad in (float("inf"), float("nan")):
            y = x.clone()
            y[rows // 2, 70] = bad
            got = ssd.ssd_w4_linear(y, codes, scales)
            keep = [r for r in range(rows) if r != rows // 2]
            assert torch.equal(got[keep], want[keep])
            code = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, 70]
            assert not torch.isfinite(got[rows // 2][code != 8]).any()
