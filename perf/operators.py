"""Cases, plain forms and exact values of the operators around the layer scan:
the short causal convolution, the per-channel selective scan, and the 8-bit
cache of recurrent states.

``own`` is False: ``run`` computes the operators from their formulas with
elementary torch operations.  ``own`` is True: ``run`` calls the package.

Formulas (b batch row, t token, c channel, n state element):

* convolution: pre = bias_c + sum_k w[c, k] x[t - (W-1) + k, c], tokens before
  the first from init_state (or 0); y = pre * sigmoid(pre) with SiLU.
* selective scan: d = softplus(dt + bias_c); a = exp(d A[c, n]);
  h = a h + d x B[n]; y = (sum_n h C[n] + D_c x) * z * sigmoid(z).
* cache: per block of 64 consecutive state elements, scale = max|v| / q and
  code = round(v q / max|v|), q = 127 (int8) or 448 (fp8 e4m3).
"""

import math

import torch

own = False

BLOCK = 64          # state elements that share one scale
QMAX = {"int8": 127.0, "fp8": 448.0}
CODE_DTYPE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
TINY = 2.0 ** -100  # blocks below this magnitude are stored as zeros

IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def _named(name, **values):
    return values if name is None else dict(name=name, **values)


def _conv(name, op, Bt, T, ch, width, io, silu=True, bias=True, init=True, lens=False):
    return _named(name, op=op, Bt=Bt, T=T, c0=ch[0], c1=ch[1], c2=ch[2], width=width, io=io,
                  silu=silu, bias=bias, init=init, lens=lens)


def _scan(name, op, Bt, T, dim, N, io, gate=True, init=True, lens=False):
    return _named(name, op=op, Bt=Bt, T=T, dim=dim, N=N, io=io, gate=gate, init=init, lens=lens)


def _cache(name, op, n, pool, size, fmt):
    return _named(name, op=op, n=n, pool=pool, size=size, fmt=fmt)


def listed():
    return [
        # prompts through the 2.7B-shaped layer's convolution: x, B and C are one slice of
        # the input projection's rows and come out as three dense tensors
        _conv("conv_prompt", "conv_fwd", 8, 4096, (5120, 128, 128), 4, "bf16", init=False),
        # right-padded prompts of odd lengths that continue a cached prefix, float32, odd widths
        _conv("conv_ragged", "conv_fwd", 3, 509, (515, 64, 64), 3, "f32", lens=True),
        # gradients of the 370M-shaped layer's convolution, from the scan's float32 gradients
        _conv("conv_train", "conv_bwd", 4, 2048, (2048, 128, 128), 4, "bf16"),
        # one decoded token for 256 sequences of the 128-head layer, states in a slot pool
        _conv("conv_step", "conv_step", 256, 1, (8192, 1024, 1024), 4, "bf16"),
        # gated per-channel scan of long prompts, 5120 channels
        _scan("scan_prompt", "scan_fwd", 8, 4096, 5120, 16, "bf16", init=False),
        # one long sequence: few rows, so the work has to be split over time
        _scan("scan_long", "scan_fwd", 1, 65536, 2048, 16, "bf16"),
        # a short chat turn on top of a cached state, float32, odd sizes, padded
        _scan("scan_turn", "scan_fwd", 2, 37, 515, 16, "f32", lens=True),
        # training step of a 2048-channel layer
        _scan("scan_train", "scan_bwd", 4, 2048, 2048, 16, "bf16"),
        # gradients at an odd length and width, wider state, no gate, float32
        _scan("scan_train_odd", "scan_bwd", 2, 333, 777, 32, "f32", gate=False),
        # one decoded token for 256 sequences
        _scan("scan_step", "scan_step", 256, 1, 5120, 16, "bf16"),
        # 64 sequences of an 80-head layer swapped out to the 8-bit pool and back
        _cache("cache_swap", "cache_write", 64, 96, 80 * 64 * 128, "int8"),
        # a few cached prefixes read by many new sequences of a 32-head layer
        _cache("cache_prefix", "cache_read", 48, 16, 32 * 64 * 128, "fp8"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step",
                     "cache_write", "cache_read"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("conv"):
        bc = rng.choice([64, 128, 256, 1024])
        c0 = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            c0 = max(64, c0 // 64 * 64)
        Bt = _log_int(rng, 1, 16) if op != "conv_step" else _log_int(rng, 1, 512)
        total = c0 + 2 * bc
        cap = 160_000_000 if op == "conv_fwd" else 40_000_000
        T = 1 if op == "conv_step" else min(_log_int(rng, 1, 16384), max(1, cap // (Bt * total)))
        return _conv(None, op, Bt, T, (c0, bc, bc), rng.choice([2, 3, 4, 4]), io,
                     silu=rng.random() < 0.8, bias=rng.random() < 0.8, init=rng.random() < 0.5,
                     lens=op == "conv_fwd" and rng.random() < 0.4)
    if op.startswith("scan"):
        N = rng.choice([8, 16, 16, 32, 64])
        dim = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            dim = max(64, dim // 64 * 64)
        Bt = _log_int(rng, 1, 16) if op != "scan_step" else _log_int(rng, 1, 512)
        cap, most = {"scan_fwd": (1_500_000_000, 65536), "scan_bwd": (260_000_000, 8192),
                     "scan_step": (1, 1)}[op]
        T = min(_log_int(rng, 1, most), max(1, cap // (Bt * dim * N)))
        if op == "scan_step":
            Bt = min(Bt, max(1, 40_000_000 // (dim * N)))
        return _scan(None, op, Bt, T, dim, N, io, gate=rng.random() < 0.7,
                     init=rng.random() < 0.5,
                     lens=op == "scan_fwd" and rng.random() < 0.4)
    size = 8 * _log_int(rng, 64, 131072)
    n = max(1, min(_log_int(rng, 1, 128), 40_000_000 // size))
    pool = n + rng.randint(0, 32) if op == "cache_write" else max(1, n // rng.randint(1, 4))
    return _cache(None, op, n, pool, size, rng.choice(["int8", "fp8"]))


# ---------------------------------------------------------------------------
# inputs

def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _lengths(g, case):
    """Lengths of right-padded prompts: any from 0 to T, one of them whole."""
    if not case["lens"]:
        return None
    lens = torch.randint(0, case["T"] + 1, (case["Bt"],), generator=g, device="cuda",
                         dtype=torch.int32)
    lens[0] = case["T"]
    return lens


def _slots(g, n, pool):
    return torch.randperm(pool, generator=g, device="cuda")[:n].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op.startswith("conv"):
        io = IO[case["io"]]
        Bt, T, W = case["Bt"], case["T"], case["width"]
        ch = (case["c0"], case["c1"], case["c2"])
        total = sum(ch)
        # the input projection's rows hold [z | x B C | dt]; the convolution reads the middle
        row = 2 * case["c0"] + case["c1"] + case["c2"] + 80
        proj = _randn(g, Bt, T, row, dtype=io)
        x = proj[:, :, case["c0"]:case["c0"] + total]
        st["splits"] = ch
        st["weight"] = _randn(g, total, W, scale=W ** -0.5)
        st["bias"] = _randn(g, total, scale=0.1) if case["bias"] else None
        if op == "conv_step":
            pool = Bt + 16
            st["x"] = x[:, 0]
            st["state"] = _randn(g, pool, W - 1, total, dtype=io)
            st["slots"] = _slots(g, Bt, pool)
            return st
        st["x"] = x
        st["init"] = _randn(g, Bt, W - 1, total, dtype=io) if case["init"] else None
        if op == "conv_fwd":
            st["lens"] = _lengths(g, case)
        else:
            st["dy"] = tuple(_randn(g, Bt, T, c) for c in ch)
            st["dfinal"] = _randn(g, Bt, W - 1, total) if case["init"] else None
        return st
    if op.startswith("scan"):
        io = IO[case["io"]]
        Bt, T, Dm, N = case["Bt"], case["T"], case["dim"], case["N"]
        n = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
        st["A"] = -n * torch.exp(_randn(g, Dm, N, scale=0.2))
        st["D"] = _randn(g, Dm)
        dt0 = torch.exp(torch.rand(Dm, generator=g, device="cuda") * math.log(100.0)) * 1e-3
        st["dt_bias"] = torch.log(torch.expm1(dt0))
        if op == "scan_step":
            pool = Bt + 16
            st["x"] = _randn(g, Bt, Dm, dtype=io)
            st["dt"] = _randn(g, Bt, Dm, dtype=io)
            st["B"] = _randn(g, Bt, N, scale=N ** -0.5, dtype=io)
            st["C"] = _randn(g, Bt, N, scale=N ** -0.5, dtype=io)
            st["z"] = _randn(g, Bt, Dm, dtype=io) if case["gate"] else None
            st["state"] = _randn(g, pool, Dm, N, scale=0.5)
            st["slots"] = _slots(g, Bt, pool)
            return st
        st["x"] = _randn(g, Bt, T, Dm, dtype=io)
        st["dt"] = _randn(g, Bt, T, Dm, dtype=io)
        st["B"] = _randn(g, Bt, T, N, scale=N ** -0.5, dtype=io)
        st["C"] = _randn(g, Bt, T, N, scale=N ** -0.5, dtype=io)
        st["z"] = _randn(g, Bt, T, Dm, dtype=io) if case["gate"] else None
        st["init"] = _randn(g, Bt, Dm, N, scale=0.1) if case["init"] else None
        if op == "scan_fwd":
            st["lens"] = _lengths(g, case)
        else:
            st["dy"] = _randn(g, Bt, T, Dm)
            st["dfinal"] = _randn(g, Bt, Dm, N) if case["init"] else None
        return st
    nblk = -(-case["size"] // BLOCK)
    if op == "cache_write":
        st["codes"] = torch.zeros(case["pool"], case["size"], device="cuda",
                                  dtype=torch.int8).view(CODE_DTYPE[case["fmt"]])
        st["scales"] = torch.zeros(case["pool"], nblk, device="cuda")
        st["slots"] = _slots(g, case["n"], case["pool"])
        # states differ in size by channel
        state = _randn(g, case["n"], case["size"])
        state *= torch.exp(_randn(g, nblk)).repeat_interleave(BLOCK)[:case["size"]]
        st["state"] = state
    else:
        state = _randn(g, case["pool"], case["size"])
        st["codes"], st["scales"] = _quantise(state, case["fmt"])
        st["slots"] = torch.randint(0, case["pool"], (case["n"],), generator=g, device="cuda",
                                    dtype=torch.int32)
        if case["n"] >= 4:  # a sequence without a cached prefix starts from zeros
            st["slots"][0] = -1
    return st


# ---------------------------------------------------------------------------
# plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _token_mask(lens, T, t0=0, t1=None):
    t = torch.arange(t0, T if t1 is None else t1, device="cuda")
    return (t[None, :] < lens[:, None]).float()[:, :, None]


def _conv_fwd(st):
    case, x = st["case"], st["x"]
    Bt, T, total = x.shape
    W = case["width"]
    head = torch.zeros(Bt, W - 1, total, device="cuda") if st["init"] is None else st["init"].float()
    xp = torch.cat([head, x.float()], 1)
    pre = xp[:, 0:T] * st["weight"][:, 0]
    for k in range(1, W):
        pre += xp[:, k:k + T] * st["weight"][:, k]
    if st["bias"] is not None:
        pre += st["bias"]
    y = pre * _sigmoid(pre) if case["silu"] else pre
    if st["lens"] is None:
        final = xp[:, T:]
    else:
        y = y * _token_mask(st["lens"], T)
        rows = st["lens"].long()[:, None] + torch.arange(W - 1, device="cuda")
        final = torch.gather(xp, 1, rows[:, :, None].expand(-1, -1, total))
    parts = y.split(st["splits"], dim=2)
    return [p.to(x.dtype).contiguous() for p in parts] + [final.to(x.dtype).contiguous()]


def _conv_step(st):
    case, x = st["case"], st["x"]
    W = case["width"]
    slots = st["slots"].long()
    win = torch.cat([st["state"][slots], x[:, None]], 1)          # [Bt, W, total]
    pre = (win.float() * st["weight"].t()).sum(1)
    if st["bias"] is not None:
        pre += st["bias"]
    y = pre * _sigmoid(pre) if case["silu"] else pre
    st["state"][slots] = win[:, 1:]
    return [p.to(x.dtype).contiguous() for p in y.split(st["splits"], dim=1)] + [st["state"]]


def _conv_bwd(st):
    case, x = st["case"], st["x"]
    Bt, T, total = x.shape
    W = case["width"]
    head = torch.zeros(Bt, W - 1, total, device="cuda") if st["init"] is None else st["init"].float()
    xp = torch.cat([head, x.float()], 1)
    dpre = torch.cat(st["dy"], 2)
    if case["silu"]:
        pre = xp[:, 0:T] * st["weight"][:, 0]
        for k in range(1, W):
            pre += xp[:, k:k + T] * st["weight"][:, k]
        if st["bias"] is not None:
            pre += st["bias"]
        s = _sigmoid(pre)
        dpre = dpre * (s * (1.0 + pre * (1.0 - s)))
    dxp = torch.zeros_like(xp)
    if st["dfinal"] is not None:
        dxp[:, T:] += st["dfinal"]
    dw = torch.empty(total, W, device="cuda")
    for k in range(W):
        dxp[:, k:k + T] += dpre * st["weight"][:, k]
        dw[:, k] = (dpre * xp[:, k:k + T]).sum((0, 1), dtype=torch.float64).float()
    out = dict(dx=dxp[:, W - 1:].contiguous(), dweight=dw)
    if st["bias"] is not None:
        out["dbias"] = dpre.sum((0, 1), dtype=torch.float64).float()
    if st["init"] is not None:
        out["dinit"] = dxp[:, :W - 1].contiguous()
    return out


def _prefix(a, b, h0):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h0, by doubling."""
    b = b.clone()
    b[:, 0] += a[:, 0] * h0
    s, L = 1, a.shape[1]
    while s < L:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        if 2 * s < L:
            a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _scan_chunk(st, t0, t1):
    """d, d x and a of tokens t0..t1 (a padded token: d = 0)."""
    d = _softplus(st["dt"][:, t0:t1].float() + st["dt_bias"])
    if st.get("lens") is not None:
        d = d * _token_mask(st["lens"], None, t0, t1)
    a = torch.exp(d[..., None] * st["A"])
    return d, a


def _chunk_len(case):
    return max(8, min(128, 2 ** 26 // (case["Bt"] * case["dim"] * case["N"])))


def _scan_init(st):
    case = st["case"]
    if st["init"] is not None:
        return st["init"]
    return torch.zeros(case["Bt"], case["dim"], case["N"], device="cuda")


def _scan_fwd(st):
    case, io = st["case"], st["x"].dtype
    T, L = case["T"], _chunk_len(case)
    h = _scan_init(st)
    ys = []
    for t0 in range(0, T, L):
        t1 = min(T, t0 + L)
        x = st["x"][:, t0:t1].float()
        d, a = _scan_chunk(st, t0, t1)
        hs = _prefix(a, (d * x)[..., None] * st["B"][:, t0:t1, None, :].float(), h)
        y = (hs * st["C"][:, t0:t1, None, :].float()).sum(-1) + st["D"] * x
        if st["z"] is not None:
            z = st["z"][:, t0:t1].float()
            y = y * (z * _sigmoid(z))
        if st["lens"] is not None:
            y = y * _token_mask(st["lens"], None, t0, t1)
        ys.append(y.to(io))
        h = hs[:, -1]
    return [torch.cat(ys, 1), h.contiguous()]


def _scan_bwd(st):
    case = st["case"]
    Bt, T, Dm, N = case["Bt"], case["T"], case["dim"], case["N"]
    L = _chunk_len(case)
    h = _scan_init(st)
    starts = []
    for t0 in range(0, T, L):
        t1 = min(T, t0 + L)
        starts.append(h)
        d, a = _scan_chunk(st, t0, t1)
        u = d * st["x"][:, t0:t1].float()
        h = _prefix(a, u[..., None] * st["B"][:, t0:t1, None, :].float(), h)[:, -1]
    dx = torch.empty(Bt, T, Dm, device="cuda")
    ddt = torch.empty_like(dx)
    dz = torch.empty_like(dx) if st["z"] is not None else None
    dB = torch.empty(Bt, T, N, device="cuda")
    dC = torch.empty_like(dB)
    dA = torch.zeros(Dm, N, device="cuda", dtype=torch.float64)
    dD = torch.zeros(Dm, device="cuda", dtype=torch.float64)
    carry = st["dfinal"] if st["dfinal"] is not None else torch.zeros(Bt, Dm, N, device="cuda")
    for t0 in reversed(range(0, T, L)):
        t1 = min(T, t0 + L)
        h0 = starts.pop()
        x = st["x"][:, t0:t1].float()
        Bv = st["B"][:, t0:t1, None, :].float()
        Cv = st["C"][:, t0:t1, None, :].float()
        d, a = _scan_chunk(st, t0, t1)
        hs = _prefix(a, (d * x)[..., None] * Bv, h0)
        hp = torch.cat([h0[:, None], hs[:, :-1]], 1)
        dy = st["dy"][:, t0:t1]
        if dz is not None:
            z = st["z"][:, t0:t1].float()
            s = _sigmoid(z)
            y = (hs * Cv).sum(-1) + st["D"] * x
            dz[:, t0:t1] = dy * y * (s * (1.0 + z * (1.0 - s)))
            dy = dy * (z * s)
        # g_t = dy_t C_t + a_{t+1} g_{t+1}
        coef = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
        gr = _prefix(coef, (dy[..., None] * Cv).flip(1), carry).flip(1)
        ga = gr * a
        carry = ga[:, 0]
        gah = ga * hp
        gb = (gr * Bv).sum(-1)
        dx[:, t0:t1] = d * gb + st["D"] * dy
        dd = x * gb + (gah * st["A"]).sum(-1)
        raw = st["dt"][:, t0:t1].float() + st["dt_bias"]
        ddt[:, t0:t1] = torch.where(raw > 20.0, dd, dd * _sigmoid(raw))
        dB[:, t0:t1] = (gr * (d * x)[..., None]).sum(2)
        dC[:, t0:t1] = (hs * dy[..., None]).sum(2)
        dA += (gah * d[..., None]).sum((0, 1), dtype=torch.float64)
        dD += (dy * x).sum((0, 1), dtype=torch.float64)
    out = dict(dx=dx, ddt=ddt, dA=dA.float(), dB=dB, dC=dC, dD=dD.float(),
               ddt_bias=ddt.sum((0, 1), dtype=torch.float64).float())
    if dz is not None:
        out["dz"] = dz
    if st["init"] is not None:
        out["dinit"] = carry.contiguous()
    return out


def _scan_step(st):
    slots = st["slots"].long()
    x = st["x"].float()
    d = _softplus(st["dt"].float() + st["dt_bias"])
    h = torch.exp(d[..., None] * st["A"]) * st["state"][slots]
    h += (d * x)[..., None] * st["B"].float()[:, None, :]
    y = (h * st["C"].float()[:, None, :]).sum(-1) + st["D"] * x
    if st["z"] is not None:
        z = st["z"].float()
        y = y * (z * _sigmoid(z))
    st["state"][slots] = h
    return [y.to(st["x"].dtype), st["state"]]


def _quantise(state, fmt):
    """Codes and scales; the quotients in 64 bits, so that a value next to the border
    between two codes goes to the nearer one."""
    n, size = state.shape
    nblk = -(-size // BLOCK)
    v = torch.zeros(n, nblk * BLOCK, device="cuda")
    v[:, :size] = state
    v = v.view(n, nblk, BLOCK)
    amax = v.abs().amax(-1)
    keep = amax >= TINY
    scale = torch.where(keep, amax / QMAX[fmt], torch.zeros_like(amax))
    q = v.double() * QMAX[fmt] / torch.where(keep, amax, torch.ones_like(amax)).double()[..., None]
    q = torch.where(keep[..., None], q, torch.zeros_like(q))
    if fmt == "int8":
        q = q.round()
    else:   # e4m3 keeps 4 significant bits, and steps of 2^-9 below 2^-6
        shift = 4 - torch.frexp(q)[1].clamp(min=-5)
        q = torch.ldexp(torch.ldexp(q, shift).round(), -shift)
    codes = q.float().to(CODE_DTYPE[fmt]).view(n, -1).view(torch.int8)[:, :size].contiguous()
    return codes.view(CODE_DTYPE[fmt]), scale


def _read(st):
    case = st["case"]
    keep = (st["slots"] >= 0)[:, None, None]
    slots = st["slots"].long().clamp(min=0)
    nblk = st["scales"].shape[1]
    v = torch.zeros(case["n"], nblk * BLOCK, device="cuda")
    v[:, :case["size"]] = st["codes"].view(torch.int8)[slots].view(CODE_DTYPE[case["fmt"]]).float()
    v = v.view(case["n"], nblk, BLOCK) * st["scales"][slots][..., None]
    v = torch.where(keep, v, torch.zeros_like(v))
    return v.view(case["n"], -1)[:, :case["size"]].contiguous()


def _cache_write(st):
    codes, scale = _quantise(st["state"], st["case"]["fmt"])
    slots = st["slots"].long()
    st["codes"].view(torch.int8)[slots] = codes.view(torch.int8)
    st["scales"][slots] = scale
    return [_read(st), st["scales"]]


# ---------------------------------------------------------------------------
# one pass

def run(st):
    op = st["case"]["op"]
    if not own:
        return {"conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd, "conv_step": _conv_step,
                "scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd, "scan_step": _scan_step,
                "cache_write": _cache_write, "cache_read": lambda s: [_read(s)]}[op](st)
    from selective_state_space_amd import ssd
    case = st["case"]
    if op == "conv_fwd":
        ys, final = ssd.ssd_conv1d_fwd(st["x"], st["weight"], st["bias"], silu=case["silu"],
                                       splits=st["splits"], init_state=st["init"],
                                       seq_lens=st["lens"])
        return list(ys) + [final]
    if op == "conv_step":
        ys = ssd.ssd_conv1d_step(st["state"], st["x"], st["weight"], st["bias"],
                                 silu=case["silu"], splits=st["splits"], slots=st["slots"])
        return list(ys) + [st["state"]]
    if op == "conv_bwd":
        out = ssd.ssd_conv1d_bwd(st["x"], st["weight"], st["dy"], st["bias"], silu=case["silu"],
                                 init_state=st["init"], dfinal=st["dfinal"],
                                 want_dinit=st["init"] is not None)
        return {k: v for k, v in out.items() if v is not None}
    if op == "scan_fwd":
        y, final = ssd.ssd_selective_scan_fwd(
            st["x"], st["dt"], st["A"], st["B"], st["C"], st["D"], init_state=st["init"],
            seq_lens=st["lens"], dt_bias=st["dt_bias"], dt_softplus=True, z=st["z"],
            y_io_dtype=True)
        return [y, final]
    if op == "scan_bwd":
        out = ssd.ssd_selective_scan_bwd(
            st["x"], st["dt"], st["A"], st["B"], st["C"], st["D"], st["dy"],
            init_state=st["init"], dfinal=st["dfinal"], dt_bias=st["dt_bias"], dt_softplus=True,
            z=st["z"], want_dinit=st["init"] is not None)
        return {k: v for k, v in out.items() if v is not None}
    if op == "scan_step":
        y = ssd.ssd_selective_scan_step(
            st["state"], st["x"], st["dt"], st["A"], st["B"], st["C"], st["D"],
            slots=st["slots"], dt_bias=st["dt_bias"], dt_softplus=True, z_t=st["z"],
            y_io_dtype=True)
        return [y, st["state"]]
    if op == "cache_write":
        ssd.ssd_cache_write(st["state"], st["codes"], st["scales"], st["slots"])
        return [ssd.ssd_cache_read(st["codes"], st["scales"], st["slots"]), st["scales"]]
    return [ssd.ssd_cache_read(st["codes"], st["scales"], st["slots"])]


# ---------------------------------------------------------------------------
# the work of one pass

def work(case):
    op = case["op"]
    if op.startswith("conv"):
        e = IO[case["io"]].itemsize
        total = case["c0"] + case["c1"] + case["c2"]
        W, Bt, T = case["width"], case["Bt"], case["T"]
        tok, state = Bt * T * total, Bt * (W - 1) * total
        if op == "conv_fwd":
            return {"bytes": 2 * tok * e + 2 * state * e + total * (W + 1) * 4,
                    "flops": tok * (2 * W + 5)}
        if op == "conv_step":
            return {"bytes": 2 * tok * e + 2 * state * e + total * (W + 1) * 4,
                    "flops": tok * (2 * W + 5)}
        return {"bytes": tok * (e + 8) + state * (e + 8) + 2 * total * (W + 1) * 4,
                "flops": tok * (6 * W + 12)}
    if op.startswith("scan"):
        e = IO[case["io"]].itemsize
        Bt, T, Dm, N = case["Bt"], case["T"], case["dim"], case["N"]
        tok, bc, state = Bt * T * Dm, Bt * T * N, Bt * Dm * N
        gate = 1 if case["gate"] else 0
        if op == "scan_bwd":
            return {"bytes": tok * (2 * e + 4 + 8 + gate * (e + 4)) + 2 * bc * (e + 4)
                    + 4 * state * 4 + 2 * Dm * N * 4 + 4 * Dm * 4,
                    "flops": tok * (N * 20 + 20)}
        return {"bytes": tok * e * (3 + gate) + 2 * bc * e + 2 * state * 4 + Dm * N * 4 + 2 * Dm * 4,
                "flops": tok * (N * 7 + 12)}
    n, size = case["n"], case["size"]
    nblk = -(-size // BLOCK)
    held = size + nblk * 4
    if op == "cache_write":     # quantised once, read back once
        return {"bytes": n * (size * 8 + 2 * held), "flops": n * size * 4}
    return {"bytes": n * size * 4 + min(n, case["pool"]) * held, "flops": n * size}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits

def _sig64(v):
    return torch.sigmoid(v.double())


def _conv_exact(st):
    case, op = st["case"], st["case"]["op"]
    W, w = case["width"], st["weight"].double()
    bias = 0.0 if st["bias"] is None else st["bias"].double()
    if op == "conv_step":
        slots = st["slots"].long()
        state = st["state"].double()
        seq = torch.cat([state[slots], st["x"].double()[:, None]], 1)
        state[slots] = seq[:, 1:]
    else:
        x = st["x"].double()
        head = x.new_zeros(x.shape[0], W - 1, x.shape[2]) if st["init"] is None else st["init"].double()
        seq = torch.cat([head, x], 1)
    pre = (seq.unfold(1, W, 1) * w).sum(-1) + bias
    s = torch.sigmoid(pre)
    if op == "conv_step":
        y = (pre * s if case["silu"] else pre)[:, 0]
        return [p.contiguous() for p in y.split(st["splits"], dim=1)] + [state]
    if op == "conv_fwd":
        y = pre * s if case["silu"] else pre
        T = case["T"]
        lens = [T] * case["Bt"] if st["lens"] is None else st["lens"].tolist()
        final = torch.stack([seq[b, n:n + W - 1] for b, n in enumerate(lens)])
        for b, n in enumerate(lens):
            y[b, n:] = 0.0
        return [p.contiguous() for p in y.split(st["splits"], dim=2)] + [final]
    dpre = torch.cat([d.double() for d in st["dy"]], 2)
    if case["silu"]:
        dpre = dpre * (s + pre * s * (1.0 - s))
    # every x[t] enters the windows of tokens t .. t + W - 1, at taps W - 1 .. 0
    padded = torch.nn.functional.pad(dpre, (0, 0, W - 1, W - 1))
    dseq = (padded.unfold(1, W, 1) * w.flip(1)).sum(-1)
    if st["dfinal"] is not None:
        dseq[:, case["T"]:] += st["dfinal"].double()
    out = dict(dx=dseq[:, W - 1:].contiguous(),
               dweight=(dpre[..., None] * seq.unfold(1, W, 1)).sum((0, 1)))
    if st["bias"] is not None:
        out["dbias"] = dpre.sum((0, 1))
    if st["init"] is not None:
        out["dinit"] = dseq[:, :W - 1].contiguous()
    return out


def _softplus64(v):
    return torch.where(v > 20.0, v, torch.nn.functional.softplus(v.double()))


def _scan_exact(st):
    case, op = st["case"], st["case"]["op"]
    A, D = st["A"].double(), st["D"].double()
    raw = st["dt"].double() + st["dt_bias"].double()
    d = _softplus64(raw)
    x, B, C = st["x"].double(), st["B"].double(), st["C"].double()
    if op == "scan_step":
        slots = st["slots"].long()
        state = st["state"].double()
        h = torch.exp(d[..., None] * A) * state[slots] + (d * x)[..., None] * B[:, None]
        y = (h * C[:, None]).sum(-1) + D * x
        if st["z"] is not None:
            y = y * torch.nn.functional.silu(st["z"].double())
        state[slots] = h
        return [y, state]
    Bt, T, Dm, N = case["Bt"], case["T"], case["dim"], case["N"]
    h = x.new_zeros(Bt, Dm, N) if st["init"] is None else st["init"].double()
    if op == "scan_fwd":
        y = torch.empty_like(x)
        live = None if st["lens"] is None else [
            (st["lens"] > t)[:, None, None] for t in range(T)]
        for t in range(T):
            nh = torch.exp(d[:, t, :, None] * A) * h
            nh.addcmul_((d[:, t] * x[:, t])[..., None], B[:, t, None])
            h = nh if live is None else torch.where(live[t], nh, h)
            torch.sum(h * C[:, t, None], -1, out=y[:, t])
        y += D * x
        if st["z"] is not None:
            y *= torch.nn.functional.silu(st["z"].double())
        if st["lens"] is not None:
            for b, n in enumerate(st["lens"].tolist()):
                y[b, n:] = 0.0
        return [y, h]
    hist = x.new_empty(T + 1, Bt, Dm, N)
    hist[0] = h
    for t in range(T):
        torch.mul(torch.exp(d[:, t, :, None] * A), hist[t], out=hist[t + 1])
        hist[t + 1].addcmul_((d[:, t] * x[:, t])[..., None], B[:, t, None])
    dy = st["dy"].double()
    out = {}
    if st["z"] is not None:
        z = st["z"].double()
        s = _sig64(z)
        y = torch.stack([(hist[t + 1] * C[:, t, None]).sum(-1) for t in range(T)], 1) + D * x
        out["dz"] = dy * y * (s + z * s * (1.0 - s))
        dy = dy * z * s
    dx, dd = torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.empty_like(B), torch.empty_like(C)
    dA = torch.zeros_like(A)
    g = x.new_zeros(Bt, Dm, N) if st["dfinal"] is None else st["dfinal"].double()
    for t in reversed(range(T)):
        g = g + dy[:, t, :, None] * C[:, t, None]
        dC[:, t] = (dy[:, t, :, None] * hist[t + 1]).sum(1)
        dB[:, t] = ((d[:, t] * x[:, t])[..., None] * g).sum(1)
        gB = (g * B[:, t, None]).sum(-1)
        g = g * torch.exp(d[:, t, :, None] * A)
        gh = g * hist[t]
        dx[:, t] = d[:, t] * gB + D * dy[:, t]
        dd[:, t] = x[:, t] * gB + (gh * A).sum(-1)
        dA += (gh * d[:, t, :, None]).sum(0)
    ddt = torch.where(raw > 20.0, dd, dd * _sig64(raw))
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum((0, 1)),
               ddt_bias=ddt.sum((0, 1)))
    if st["init"] is not None:
        out["dinit"] = g
    return out


def _cache_exact(st):
    """The values that come back, from each block's largest magnitude."""
    case = st["case"]
    if case["op"] == "cache_read":
        out = torch.zeros(case["n"], case["size"], device="cuda", dtype=torch.float64)
        values = st["codes"].to(torch.float32).double()
        scale = st["scales"].double().repeat_interleave(BLOCK, 1)[:, :case["size"]]
        for i, s in enumerate(st["slots"].tolist()):
            if s >= 0:
                out[i] = values[s] * scale[s]
        return [out]
    n, size, q = case["n"], case["size"], QMAX[case["fmt"]]
    scales = st["scales"].double()
    back = torch.empty(n, size, device="cuda", dtype=torch.float64)
    for i, s in enumerate(st["slots"].tolist()):
        row = st["state"][i].double()
        blocks = torch.nn.functional.pad(row, (0, -size % BLOCK)).view(-1, BLOCK)
        scale = blocks.abs().max(1).values / q
        units = blocks / scale[:, None]
        if case["fmt"] == "int8":
            units = units.round()
        else:   # e4m3: 3 mantissa bits from exponent -6 up, steps of 2^-9 below
            e = torch.floor(torch.log2(units.abs().clamp(min=2.0 ** -6)))
            step = torch.exp2(e - 3)
            units = (units / step).round() * step
        back[i] = (units * scale[:, None]).view(-1)[:size]
        scales[s] = scale
    return [back, scales]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("conv"):
        return _conv_exact(st)
    if case["op"].startswith("scan"):
        return _scan_exact(st)
    return _cache_exact(st)
