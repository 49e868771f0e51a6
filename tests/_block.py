"""Plain float64 forms of linear attention, the group norm and 4-bit weights, and
the tolerances that the GPU tests hold the library to."""

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def rel(got, ref):
    """2-norm of the difference over the reference's; infinite where one is not finite."""
    if not ref.numel():
        return 0.0
    got, ref = got.double(), ref.double()
    if not bool(torch.isfinite(got).all()):
        return math.inf
    n = float(ref.norm())
    d = float((got - ref).norm())
    return d / n if n else (math.inf if d else 0.0)


def assert_near(got, ref, bar, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    r = rel(got, ref)
    print("  %-12s rel %.3g of %.3g" % (what, r, bar), flush=True)
    assert r <= bar, "%s: %.3g off, %.3g allowed" % (what, r, bar)


# ---------------------------------------------------------------------------
# linear attention, token by token

def attn_bar(io, terms):
    """Relative 2-norm of the error: `terms` roundings of independent signs, each half a
    step at most, in float32; for bf16 outputs three of half a bf16 step that reach 0.58 of it
    on the average of a step's range (the pairs' weights, the state as an operand, the
    output), 0.58 sqrt(3) = 1."""
    f = 2.0 ** -24 * math.sqrt(terms)
    return f if io == torch.float32 else U[io] + f


def heads(t, H):
    return t.double().repeat_interleave(H // t.shape[-2], -2)


def attn_ref(q, k, v, log_decay, scale, init=None, lens=None, dy=None, dfinal=None):
    """(y, final), or the dict of gradients where dy is given."""
    Bt, T, H, K = q.shape
    G, V = v.shape[-2:]
    a = torch.exp(log_decay.double())[:, None, None]
    q, k, v = heads(q, H), heads(k, H), heads(v, H)
    zero = q.new_zeros(Bt, H, K, V)
    s = zero if init is None else init.double()
    n = torch.full((Bt,), T, device=q.device) if lens is None else lens.long().clamp(0, T)
    live = (torch.arange(T, device=q.device)[None] < n[:, None])[:, :, None, None]   # [Bt,T,1,1]
    y, dq = q.new_zeros(Bt, T, H, V), torch.zeros_like(q)
    for t in range(T):
        new = a * s + k[:, t, :, :, None] * v[:, t, :, None]
        on = live[:, t, :, :, None]
        s = torch.where(on, new, s)
        if dy is None:
            y[:, t] = torch.where(live[:, t], scale * (q[:, t, :, :, None] * new).sum(2), 0.0)
        else:
            dq[:, t] = torch.where(live[:, t], scale * (new * dy[:, t, :, None].double()).sum(3),
                                   0.0)
    if dy is None:
        return y, s
    d = zero if dfinal is None else dfinal.double()
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in reversed(range(T)):
        full = d + scale * q[:, t, :, :, None] * dy[:, t, :, None].double()
        dk[:, t] = torch.where(live[:, t], (full * v[:, t, :, None]).sum(3), 0.0)
        dv[:, t] = torch.where(live[:, t], (full * k[:, t, :, :, None]).sum(2), 0.0)
        d = torch.where(live[:, t, :, :, None], a * full, d)
    share = lambda t: t.unflatten(2, (G, H // G)).sum(3)
    return dict(dq=dq, dk=share(dk), dv=share(dv), dinit=d)


def attn_inputs(seed, Bt, T, H, G, K, V, io, init=False, lens=None, grads=False):
    g = gen(seed)
    c = dict(q=randn(g, Bt, T, H, K, dtype=io), k=randn(g, Bt, T, G, K, dtype=io),
             v=randn(g, Bt, T, G, V, dtype=io))
    h = torch.arange(H, device="cuda", dtype=torch.float32)
    c["log_decay"] = -torch.exp2(-1.0 - 7.0 * h / max(H, 1))
    kw = dict(scale=K ** -0.5)
    if init:
        kw["init_state"] = randn(g, Bt, H, K, V)
    if lens is not None:
        kw["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if grads:
        c["dy"] = randn(g, Bt, T, H, V, dtype=io)
        if init:
            kw["dfinal"] = randn(g, Bt, H, K, V)
    return c, kw


# ---------------------------------------------------------------------------
# group norm

def norm_ref(x, groups, weight=None, bias=None, z=None, form="plain", rms=False, eps=1e-5,
             lens=None, dy=None):
    """y, or the dict of gradients where dy is given (float64 autograd)."""
    leaf = {n: t.double().detach().requires_grad_(True)
            for n, t in (("x", x), ("z", z), ("weight", weight), ("bias", bias)) if t is not None}
    u = leaf["x"]
    if form == "gated_input":
        u = u * torch.nn.functional.silu(leaf["z"])
    u = u.unflatten(-1, (groups, -1))
    c = u if rms else u - u.mean(-1, keepdim=True)
    n = (c / torch.sqrt(c.square().mean(-1, keepdim=True) + eps)).flatten(-2)
    if weight is not None:
        n = n * leaf["weight"]
    if bias is not None:
        n = n + leaf["bias"]
    y = n
    if form == "silu":
        y = torch.nn.functional.silu(n)
    elif form == "gate":
        y = n * torch.nn.functional.silu(leaf["z"])
    if lens is not None:
        keep = torch.arange(x.shape[1], device=x.device)[None] < lens[:, None]
        y = torch.where(keep[..., None], y, torch.zeros_like(y))
    if dy is None:
        return y.detach()
    grads = torch.autograd.grad(y, list(leaf.values()), dy.double())
    return {"d" + n: t for n, t in zip(leaf, grads)}


# ---------------------------------------------------------------------------
# 4-bit weights

def w4_ref(weight, group):
    """(whole numbers, scales in float64) of weights, ties to even."""
    w = weight.double().unflatten(1, (-1, group))
    most = w.abs().amax(-1)
    scale = (most.float() / 7.0).to(torch.bfloat16).double()
    scale = torch.where(most >= 2.0 ** -100, scale, torch.zeros_like(scale))
    by = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = torch.where((scale > 0)[..., None], (w / by[..., None]).round(), torch.zeros_like(w))
    return code, scale


def w4_values(codes, scales):
    """The weights that codes and scales stand for, in float64."""
    v = torch.stack([codes & 15, codes >> 4], -1).flatten(1).double() - 8.0
    return (v.unflatten(1, (scales.shape[1], -1)) * scales.double()[..., None]).flatten(1)
