"""Cases, plain forms and exact values of a layer's further operators: linear attention
with a decay for each head, the group norm behind a mixer with its gate, and projections
with 4-bit weights.

``own`` is False: ``run`` computes the operators from their formulas with elementary torch
operations.  ``own`` is True: ``run`` calls the package.

Formulas (b batch row, t token, h head, g = h / (H / G) its key and value head):

* linear attention: S_t = exp(r_h) S_{t-1} + k_t (outer) v_t;  y_t = scale q_t S_t, with the
  state S [K, V] and r the heads' log decays.  A sequence ends at its length: what lies
  behind it is not read, gives y = 0 and leaves the state.
* group norm: u = x, or x silu(z); n = (u - mean) / sqrt(var + eps) w + b over each token's
  groups of consecutive channels (rms: u / sqrt(mean u^2 + eps) w + b); y = n, silu(n) or
  n silu(z).
* 4-bit weights: per output and group of consecutive inputs, scale = max|w| / 7 rounded to
  bfloat16 and code = round(w / scale) + 8, two codes to a byte (the even input in the low
  half); the weight is (code - 8) scale, and a projection y = x w^T + bias.
"""

import math

import torch

own = False

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 128          # tokens that the plain form takes at a time
TINY = 2.0 ** -100   # groups of weights below this magnitude are stored as zeros
EPS = 1e-5


def _named(name, **values):
    return values if name is None else dict(name=name, **values)


def _attn(name, op, Bt, T, H, G, K, V, io, init=True, lens=False):
    return _named(name, op=op, Bt=Bt, T=T, H=H, G=G, K=K, V=V, io=io, init=init, lens=lens)


def _norm(name, op, Bt, T, C, groups, io, form, rms, affine=True, lens=False):
    return _named(name, op=op, Bt=Bt, T=T, C=C, groups=groups, io=io, form=form, rms=rms,
                  affine=affine, lens=lens)


def _w4(name, op, rows, inputs, outputs, group, io, bias=False):
    return _named(name, op=op, rows=rows, inputs=inputs, outputs=outputs, group=group, io=io,
                  bias=bias)


def listed():
    return [
        # prompts through a 5120-channel layer: 40 heads of 128
        _attn("attn_prompt", "attn_fwd", 8, 4096, 40, 40, 128, 128, "bf16", init=False),
        # one long document on top of a cached state: few rows, so time has to be split
        _attn("attn_long", "attn_fwd", 1, 65536, 16, 16, 128, 128, "bf16"),
        # a short chat turn, float32, odd sizes, padded, keys and values shared by heads
        _attn("attn_turn", "attn_fwd", 2, 37, 6, 2, 80, 48, "f32", lens=True),
        # training step of a 2048-channel layer
        _attn("attn_train", "attn_bwd", 4, 2048, 16, 16, 128, 128, "bf16", init=False),
        # gradients at an odd length and of shared keys and values, float32, from a state
        _attn("attn_train_odd", "attn_bwd", 2, 333, 6, 3, 64, 96, "f32", lens=True),
        # one decoded token for 256 sequences of a 32-head layer, states in a slot pool
        _attn("attn_step", "attn_step", 256, 1, 32, 8, 128, 128, "bf16"),
        # each head of a prompt's 5120 channels normalised and gated
        _norm("norm_prompt", "norm_fwd", 8, 4096, 5120, 40, "bf16", "gate", False),
        # training step of a 2048-channel layer, the gate in front of an rms norm
        _norm("norm_train", "norm_bwd", 4, 2048, 2048, 1, "bf16", "gated_input", True),
        # one decoded token for 5 sequences, float32, an odd width
        _norm("norm_token", "norm_fwd", 5, 1, 2100, 4, "f32", "silu", False),
        # one decoded token through a 2560-channel layer's input projection
        _w4("w4_token", "w4_linear", 1, 2560, 10576, 64, "bf16"),
        # 48 decoded tokens through an output projection
        _w4("w4_batch", "w4_linear", 48, 5120, 2560, 128, "bf16", bias=True),
        # a projection's weights brought to 4 bits when a model is loaded, and read back
        _w4("w4_load", "w4_pack", 0, 2560, 10576, 64, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step", "norm_fwd",
                     "norm_bwd", "w4_linear", "w4_linear", "w4_pack"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("attn"):
        K, V = (rng.choice([64, 128, 128, 256, 8 * rng.randint(2, 32)]) for _ in range(2))
        if rng.random() < 0.6:
            V = K
        G = _log_int(rng, 1, 40)
        H = G * rng.choice([1, 1, 1, 2, 4])
        step = op == "attn_step"
        Bt = _log_int(rng, 1, 16) if not step else _log_int(rng, 1, 512)
        if step:
            Bt, T = min(Bt, max(1, 130_000_000 // (H * K * V))), 1
        else:
            cap, most = ((20_000_000_000, 65536) if op == "attn_fwd" else (2_000_000_000, 8192))
            T = min(_log_int(rng, 1, most), max(1, cap // (Bt * H * K * V)),
                    max(1, cap // 64 // (Bt * H * (K + V))))
        return _attn(None, op, Bt, T, H, G, K, V, io, init=rng.random() < 0.5,
                     lens=not step and rng.random() < 0.4)
    if op.startswith("norm"):
        groups = rng.choice([1, 1, 2, 8, _log_int(rng, 1, 64)])
        size = _log_int(rng, 16, 8192)
        if rng.random() < 0.6:
            size = max(16, size // 16 * 16)
        size = min(size, 8192 // groups if groups < 512 else 16)
        C = groups * size
        cap = 160_000_000 if op == "norm_fwd" else 16_000_000
        Bt = _log_int(rng, 1, 16)
        T = min(_log_int(rng, 1, 8192), max(1, cap // (Bt * C)))
        form = rng.choice(["plain", "silu", "gate", "gated_input"])
        return _norm(None, op, Bt, T, C, groups, io, form, rng.random() < 0.5,
                     affine=rng.random() < 0.8, lens=rng.random() < 0.3)
    group = rng.choice([64, 128])
    inputs = group * _log_int(rng, 1, 8192 // group)
    outputs = min(_log_int(rng, 16, 32768), 54_000_000 // inputs)
    if op == "w4_pack":
        return _w4(None, op, 0, inputs, min(outputs, 27_000_000 // inputs), group, io)
    return _w4(None, op, rng.choice([1, 1, 2, 4, 8, 16, rng.randint(1, 64)]), inputs, outputs,
               group, io, bias=rng.random() < 0.5)


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


def _attn_inputs(g, case):
    io, op = IO[case["io"]], case["op"]
    Bt, T, H, G, K, V = (case[n] for n in ("Bt", "T", "H", "G", "K", "V"))
    st = dict(case=case, scale=K ** -0.5)
    # slopes from strong to weak over the heads
    h = torch.arange(1, H + 1, device="cuda", dtype=torch.float32)
    st["log_decay"] = -torch.exp2(-8.0 * h / H)
    # q, k and v are slices of one projection's rows
    proj = _randn(g, Bt, T, H * K + G * K + G * V, dtype=io)
    q, k, v = proj.split((H * K, G * K, G * V), dim=2)
    st["q"], st["k"], st["v"] = q.unflatten(2, (H, K)), k.unflatten(2, (G, K)), v.unflatten(2, (G, V))
    if op == "attn_step":
        for n in ("q", "k", "v"):
            st[n] = st[n][:, 0]
        pool = Bt + 16
        st["state"] = _randn(g, pool, H, K, V)
        st["slots"] = torch.randperm(pool, generator=g, device="cuda")[:Bt].to(torch.int32)
        return st
    st["init"] = _randn(g, Bt, H, K, V) if case["init"] else None
    st["lens"] = _lengths(g, case)
    if op == "attn_bwd":
        st["dy"] = _randn(g, Bt, T, H, V, dtype=io)
        st["dfinal"] = _randn(g, Bt, H, K, V, scale=0.1) if case["init"] else None
    return st


def _norm_inputs(g, case):
    io = IO[case["io"]]
    Bt, T, C = case["Bt"], case["T"], case["C"]
    st = dict(case=case)
    st["x"] = _randn(g, Bt, T, C).add_(0.3).mul_(torch.exp(_randn(g, C, scale=0.3))).to(io)
    # the gate is a slice of the input projection's rows
    st["z"] = None
    if case["form"].startswith("gate"):
        st["z"] = _randn(g, Bt, T, C + 80, dtype=io)[:, :, 80:]
    st["weight"] = 1.0 + _randn(g, C, scale=0.1) if case["affine"] else None
    st["bias"] = _randn(g, C, scale=0.1) if case["affine"] and not case["rms"] else None
    st["lens"] = _lengths(g, case)
    if case["op"] == "norm_bwd":
        st["dy"] = _randn(g, Bt, T, C, dtype=io)
    return st


def _w4_inputs(g, case):
    io = IO[case["io"]]
    K, O = case["inputs"], case["outputs"]
    weight = _randn(g, O, K, scale=K ** -0.5)
    st = dict(case=case)
    if case["op"] == "w4_pack":
        st["weight"] = weight.to(io)
        return st
    st["codes"], st["scales"] = _pack(weight, case["group"])
    st["bias"] = _randn(g, O) if case["bias"] else None
    st["x"] = _randn(g, case["rows"], K, dtype=io)
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["op"].split("_")[0]
    return {"attn": _attn_inputs, "norm": _norm_inputs, "w4": _w4_inputs}[kind](g, case)


# ---------------------------------------------------------------------------
# plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _live(lens, T):
    """1 for tokens before their sequence's length, 0 behind it: [Bt, T]."""
    t = torch.arange(T, device=lens.device)
    return (t[None] < lens[:, None]).float()


def _heads(t, H):
    """[Bt, T, G, d] to float32 [Bt, H, T, d], each shared head repeated."""
    return t.float().repeat_interleave(H // t.shape[2], 2).transpose(1, 2).contiguous()


def _powers(log_decay, n):
    """exp(n log_decay) per head, the exponents in 64 bits: [H, *n.shape]."""
    r = log_decay.double().view(-1, *[1] * n.dim())
    return torch.exp(r * n.double()).float()


def _recur(q, k, v, log_decay):
    """sum over j <= i of exp(r (i - j)) (q_i . k_j) v_j, by chunks: the pairs within a
    chunk, and the states between chunks."""
    Bt, H, T, K = q.shape
    L = min(CHUNK, T)
    nc = -(-T // L)
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, nc * L - T)).view(Bt, H, nc, L, -1)
               for t in (q, k, v))
    n = torch.arange(L, device=q.device)
    gap = n[:, None] - n[None]
    pair = _powers(log_decay, gap.clamp(min=0)) * (gap >= 0)
    out = (q @ k.transpose(-1, -2).contiguous() * pair[:, None]) @ v
    ends = (k * _powers(log_decay, L - 1 - n)[:, None, :, None]).transpose(-1, -2).contiguous() @ v
    c = torch.arange(nc, device=q.device)
    gap = c[:, None] - 1 - c[None]
    carry = _powers(log_decay, L * gap.clamp(min=0)) * (gap >= 0)
    states = (carry @ ends.view(Bt, H, nc, -1)).view_as(ends)
    out += (q * _powers(log_decay, n + 1)[:, None, :, None]) @ states
    return out.view(Bt, H, nc * L, -1)[:, :, :T]


def _from_start(lens, T, Bt, device):
    """Tokens from the start up to and with each one, [T]; tokens behind each one up to its
    sequence's end, [Bt, T]; lengths, [Bt]."""
    t = torch.arange(T, device=device)
    n = torch.full((Bt,), T, device=device) if lens is None else lens.long()
    return t + 1, (n[:, None] - 1 - t).clamp(min=0), n


def _masked(t, lens):
    return t if lens is None else t * _live(lens, t.shape[2])[:, None, :, None]


def _out(t, io):
    return t.transpose(1, 2).to(io).contiguous()


def _attn_fwd(st):
    r, lens, io, H = st["log_decay"], st["lens"], st["q"].dtype, st["case"]["H"]
    q, k, v = _heads(st["q"], H), _masked(_heads(st["k"], H), lens), _heads(st["v"], H)
    Bt, _, T, _ = q.shape
    y = _recur(q, k, v, r)
    ahead, behind, n = _from_start(lens, T, Bt, q.device)
    weight = _powers(r, behind).transpose(0, 1)[..., None]
    final = (k * weight).transpose(-1, -2).contiguous() @ v
    if st["init"] is not None:
        y += (q * _powers(r, ahead)[:, :, None]) @ st["init"]
        final += _powers(r, n).t()[:, :, None, None] * st["init"]
    return [_out(_masked(y * st["scale"], lens), io), final]


def _shared(t, G, io):
    """Gradients of shared heads: the sum over the heads that share one."""
    Bt, H, T, d = t.shape
    return _out(t.view(Bt, G, H // G, T, d).sum(2), io)


def _attn_bwd(st):
    r, lens, io, scale = st["log_decay"], st["lens"], st["q"].dtype, st["scale"]
    H, G = st["case"]["H"], st["case"]["G"]
    q, k, v, dy = (_masked(_heads(st[n], H), lens) for n in ("q", "k", "v", "dy"))
    Bt, _, T, _ = q.shape
    dq = _recur(dy, v, k, r) * scale
    dk = _recur(v.flip(2), dy.flip(2), q.flip(2), r).flip(2) * scale
    dv = _recur(k.flip(2), q.flip(2), dy.flip(2), r).flip(2) * scale
    ahead, behind, n = _from_start(lens, T, Bt, q.device)
    first = _powers(r, ahead)[:, :, None]
    out = {}
    if st["init"] is not None:
        dq += (dy * first * scale) @ st["init"].transpose(-1, -2).contiguous()
        last = _powers(r, behind).transpose(0, 1)[..., None]
        dk += (v * last) @ st["dfinal"].transpose(-1, -2).contiguous()
        dv += (k * last) @ st["dfinal"]
        out["dinit"] = ((q * first * scale).transpose(-1, -2).contiguous() @ dy
                        + _powers(r, n).t()[:, :, None, None] * st["dfinal"])
    out.update(dq=_out(_masked(dq, lens), io), dk=_shared(_masked(dk, lens), G, io),
               dv=_shared(_masked(dv, lens), G, io))
    return out


def _attn_step(st):
    H, slots = st["case"]["H"], st["slots"].long()
    q, k, v = (t.float().repeat_interleave(H // t.shape[1], 1) for t in (st["q"], st["k"], st["v"]))
    s = torch.exp(st["log_decay"])[:, None, None] * st["state"][slots]
    s += k[..., None] * v[:, :, None]
    st["state"][slots] = s
    return [((q * st["scale"])[..., None] * s).sum(2).to(st["q"].dtype), st["state"]]


def _grouped(t, groups):
    return t.unflatten(2, (groups, -1))


def _normal(u, groups, rms):
    """(the normalised u, 1 / its deviation), over each token's groups."""
    u = _grouped(u, groups)
    if not rms:
        u = u - u.mean(-1, keepdim=True)
    inv = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    return u * inv, inv


def _affine(st, n):
    if st["weight"] is not None:
        n = n * st["weight"]
    return n if st["bias"] is None else n + st["bias"]


def _norm_fwd(st):
    case, x = st["case"], st["x"].float()
    form = case["form"]
    z = None if st["z"] is None else st["z"].float()
    u = x * z * _sigmoid(z) if form == "gated_input" else x
    n = _affine(st, _normal(u, case["groups"], case["rms"])[0].flatten(2))
    y = n * _sigmoid(n) if form == "silu" else n * (z * _sigmoid(z)) if form == "gate" else n
    if st["lens"] is not None:
        y = y * _live(st["lens"], case["T"])[..., None]
    return [y.to(st["x"].dtype)]


def _norm_bwd(st):
    case, x, io = st["case"], st["x"].float(), st["x"].dtype
    form, groups = case["form"], case["groups"]
    dn = st["dy"].float()
    if st["lens"] is not None:
        dn = dn * _live(st["lens"], case["T"])[..., None]
    out, u = {}, x
    if st["z"] is not None:
        z = st["z"].float()
        s = _sigmoid(z)
        gate, slope = z * s, s * (1.0 + z * (1.0 - s))
        u = x * gate if form == "gated_input" else x
    normal, inv = _normal(u, groups, case["rms"])
    flat = normal.flatten(2)
    if form != "gated_input":
        n = _affine(st, flat)
        if form == "silu":
            s = _sigmoid(n)
            dn = dn * (s * (1.0 + n * (1.0 - s)))
        elif form == "gate":
            out["dz"] = (dn * n * slope).to(io)
            dn = dn * gate
    if st["weight"] is not None:
        out["dweight"] = (dn * flat).sum((0, 1), dtype=torch.float64).float()
        if st["bias"] is not None:
            out["dbias"] = dn.sum((0, 1), dtype=torch.float64).float()
        dn = dn * st["weight"]
    d = _grouped(dn, groups)
    along = normal * (d * normal).mean(-1, keepdim=True)
    if not case["rms"]:
        d = d - d.mean(-1, keepdim=True)
    du = ((d - along) * inv).flatten(2)
    if form == "gated_input":
        out["dz"] = (du * x * slope).to(io)
        du = du * gate
    out["dx"] = du.to(io)
    return out


def _pack(weight, group):
    """Codes and scales; the quotients in 64 bits, so that a weight next to the border between
    two codes goes to the nearer one."""
    O, K = weight.shape
    w = weight.float().view(O, K // group, group)
    most = w.abs().amax(-1)
    keep = most >= TINY
    scales = torch.where(keep, most / 7.0, torch.zeros_like(most)).to(torch.bfloat16)
    by = torch.where(keep, scales.double(), torch.ones_like(most, dtype=torch.float64))
    code = (w.double() / by[..., None]).round()
    code = torch.where(keep[..., None], code, torch.zeros_like(code))
    code = (code + 8.0).to(torch.uint8).view(O, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scales


def _unpack(codes, scales):
    """The weights in float32."""
    O, half = codes.shape
    w = torch.stack([codes & 15, codes >> 4], -1).float() - 8.0
    return (w.view(O, scales.shape[1], -1) * scales.float()[..., None]).view(O, 2 * half)


def _w4_linear(st):
    w = _unpack(st["codes"], st["scales"])
    y = st["x"].float() @ w.t().contiguous()
    if st["bias"] is not None:
        y = y + st["bias"]
    return [y.to(st["x"].dtype)]


def _w4_pack(st):
    codes, scales = _pack(st["weight"], st["case"]["group"])
    return [_unpack(codes, scales).to(st["weight"].dtype), scales]


# ---------------------------------------------------------------------------
# one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"attn_fwd": _attn_fwd, "attn_bwd": _attn_bwd, "attn_step": _attn_step,
                "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "w4_linear": _w4_linear,
                "w4_pack": _w4_pack}[op](st)
    from selective_state_space_amd import ssd
    if op == "attn_fwd":
        y, final = ssd.ssd_linear_attn_fwd(st["q"], st["k"], st["v"], st["log_decay"],
                                           scale=st["scale"], init_state=st["init"],
                                           seq_lens=st["lens"])
        return [y, final]
    if op == "attn_bwd":
        out = ssd.ssd_linear_attn_bwd(st["q"], st["k"], st["v"], st["log_decay"], st["dy"],
                                      scale=st["scale"], init_state=st["init"],
                                      dfinal=st["dfinal"], seq_lens=st["lens"],
                                      want_dinit=st["init"] is not None)
        return {n: t for n, t in out.items() if t is not None}
    if op == "attn_step":
        y = ssd.ssd_linear_attn_step(st["state"], st["q"], st["k"], st["v"], st["log_decay"],
                                     scale=st["scale"], slots=st["slots"])
        return [y, st["state"]]
    if op == "norm_fwd":
        return [ssd.ssd_group_norm_fwd(st["x"], case["groups"], st["weight"], st["bias"],
                                       z=st["z"], form=case["form"], rms=case["rms"], eps=EPS,
                                       seq_lens=st["lens"])]
    if op == "norm_bwd":
        out = ssd.ssd_group_norm_bwd(st["x"], case["groups"], st["dy"], st["weight"], st["bias"],
                                     z=st["z"], form=case["form"], rms=case["rms"], eps=EPS,
                                     seq_lens=st["lens"])
        return {n: t for n, t in out.items() if t is not None}
    if op == "w4_linear":
        return [ssd.ssd_w4_linear(st["x"], st["codes"], st["scales"], st["bias"])]
    codes, scales = ssd.ssd_w4_quantize(st["weight"], case["group"])
    return [ssd.ssd_w4_dequantize(codes, scales, dtype=st["weight"].dtype), scales]


# ---------------------------------------------------------------------------
# the work of one pass

def work(case):
    op, e = case["op"], IO[case["io"]].itemsize
    if op.startswith("attn"):
        Bt, T, H, G, K, V = (case[n] for n in ("Bt", "T", "H", "G", "K", "V"))
        tok, state = Bt * T, Bt * H * K * V * 4
        qkv, y = tok * (H * K + G * (K + V)) * e, tok * H * V * e
        if op == "attn_step":
            return {"bytes": qkv + y + 2 * state, "flops": tok * H * K * V * 5}
        pairs = (min(T, 64) + 1) * (K + V)
        if op == "attn_fwd":
            return {"bytes": qkv + y + state * (1 + bool(case["init"])),
                    "flops": tok * H * (4 * K * V + pairs)}
        return {"bytes": 2 * qkv + y + state * 3 * bool(case["init"]),
                "flops": tok * H * (10 * K * V + 2.5 * pairs)}
    if op.startswith("norm"):
        n = case["Bt"] * case["T"] * case["C"]
        gate = case["form"].startswith("gate")
        if op == "norm_fwd":
            return {"bytes": n * e * (2 + gate) + 8 * case["C"], "flops": n * 12}
        return {"bytes": n * e * (3 + 2 * gate) + 16 * case["C"], "flops": n * 30}
    K, O, R = case["inputs"], case["outputs"], case["rows"]
    held = O * K / 2 + O * (K // case["group"]) * 2
    if op == "w4_linear":
        return {"bytes": held + R * (K + O) * e + 4 * O * case["bias"], "flops": 2 * R * K * O}
    return {"bytes": 2 * (O * K * e + held), "flops": 6 * O * K}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits

def _attn_exact(st):
    """Token by token."""
    case, op, scale = st["case"], st["case"]["op"], st["scale"]
    H, K, V, Bt, T = (case[n] for n in ("H", "K", "V", "Bt", "T"))
    a = torch.exp(st["log_decay"].double())[:, None, None]

    def each(t):
        return torch.repeat_interleave(t.double(), H // t.shape[-2], -2)

    q, k, v = each(st["q"]), each(st["k"]), each(st["v"])
    if op == "attn_step":
        state, slots = st["state"].double(), st["slots"].long()
        new = a * state[slots] + torch.einsum("bhk,bhv->bhkv", k, v)
        state[slots] = new
        return [torch.einsum("bhk,bhkv->bhv", q, new) * scale, state]
    zero = q.new_zeros(Bt, H, K, V)
    s = zero if st["init"] is None else st["init"].double()
    lens = st["lens"]
    live = None if lens is None else [(lens > t).view(-1, 1, 1, 1) for t in range(T)]
    dy = st["dy"].double() if op == "attn_bwd" else None
    y, dq = q.new_zeros(Bt, T, H, V), torch.zeros_like(q)
    for t in range(T):
        new = a * s + k[:, t, :, :, None] * v[:, t, :, None]
        if dy is None:
            out, at = (q[:, t, :, :, None] * new).sum(2), y
        else:
            out, at = (new * dy[:, t, :, None]).sum(3), dq
        if live is None:
            s = new
        else:
            s = torch.where(live[t], new, s)
            out = out * live[t][..., 0]
        at[:, t] = out * scale
    if dy is None:
        return [y, s]
    d = zero if st["dfinal"] is None else st["dfinal"].double()
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in reversed(range(T)):
        full = d + scale * q[:, t, :, :, None] * dy[:, t, :, None]
        gk, gv = (full * v[:, t, :, None]).sum(3), (full * k[:, t, :, :, None]).sum(2)
        if live is None:
            d = a * full
        else:
            d = torch.where(live[t], a * full, d)
            gk, gv = gk * live[t][..., 0], gv * live[t][..., 0]
        dk[:, t], dv[:, t] = gk, gv
    G = case["G"]
    out = dict(dq=dq, dk=dk.unflatten(2, (G, H // G)).sum(3),
               dv=dv.unflatten(2, (G, H // G)).sum(3))
    if st["init"] is not None:
        out["dinit"] = d
    return out


def _norm_exact(st):
    case = st["case"]
    form, rms = case["form"], case["rms"]
    leaf = {n: st[n].double().requires_grad_(True) for n in ("x", "z", "weight", "bias")
            if st[n] is not None}
    u = leaf["x"]
    if form == "gated_input":
        u = u * torch.nn.functional.silu(leaf["z"])
    u = u.unflatten(2, (case["groups"], -1))
    var = u.square().mean(-1, keepdim=True) if rms else u.var(-1, unbiased=False, keepdim=True)
    n = ((u if rms else u - u.mean(-1, keepdim=True)) / (var + EPS).sqrt()).flatten(2)
    if "weight" in leaf:
        n = n * leaf["weight"]
    if "bias" in leaf:
        n = n + leaf["bias"]
    y = {"silu": lambda: torch.nn.functional.silu(n), "plain": lambda: n, "gated_input": lambda: n,
         "gate": lambda: n * torch.nn.functional.silu(leaf["z"])}[form]()
    if st["lens"] is not None:
        keep = torch.arange(case["T"], device="cuda")[None] < st["lens"][:, None]
        y = torch.where(keep[..., None], y, torch.zeros_like(y))
    if case["op"] == "norm_fwd":
        return [y.detach()]
    grads = torch.autograd.grad(y, list(leaf.values()), st["dy"].double())
    return {"d" + n: t for n, t in zip(leaf, grads)}


def _w4_exact(st):
    case = st["case"]
    if case["op"] == "w4_linear":
        low, high = st["codes"].to(torch.int64) % 16, st["codes"].to(torch.int64) // 16
        w = torch.empty(case["outputs"], case["inputs"], device="cuda", dtype=torch.float64)
        w[:, 0::2], w[:, 1::2] = low - 8, high - 8
        w *= st["scales"].double().repeat_interleave(case["group"], 1)
        y = torch.matmul(st["x"].double(), w.t())
        return [y if st["bias"] is None else y + st["bias"].double()]
    w = st["weight"].double().unflatten(1, (-1, case["group"]))
    most = w.abs().amax(-1)
    # bfloat16 keeps 8 significant bits
    e = torch.floor(torch.log2(most / 7.0)) - 7.0
    scale = torch.round(most / 7.0 / torch.exp2(e)) * torch.exp2(e)
    return [(torch.round(w / scale[..., None]) * scale[..., None]).flatten(1), scale]


def exact(case, seed):
    st = prepare(case, seed)
    with torch.enable_grad():
        if case["op"].startswith("norm"):
            return _norm_exact(st)
    return _attn_exact(st) if case["op"].startswith("attn") else _w4_exact(st)
