"""The operators around the scan run together, as a layer uses them: a prompt
through the convolution and a scan, its state into the 8-bit cache and back,
decoded tokens on top, and the gradients of convolution and scan chained.
float32 io; outputs to the framework's float32 bar, max|gpu - ref| <= 1e-4
max|ref|, against float64 on the CPU."""

import pytest
import torch

import oracle
from selective_state_space_amd import inputs as gen
from selective_state_space_amd import ssd

from _gpu import assert_close, host, log

pytestmark = pytest.mark.gpu


def conv64(x, w, b, state):
    """(silu(conv), new state) in float64; x [Bt,T,C], state [Bt,W-1,C]."""
    W, T = w.shape[1], x.shape[1]
    xp = torch.cat([state.double(), x.double()], 1)
    pre = b.double() + sum(xp[:, k:k + T] * w[:, k].double() for k in range(W))
    return pre * torch.sigmoid(pre), xp[:, T:]


def scan64(x, dt, A, B, C, D, dt_bias, z, h):
    x, dt, A, B, C, D, z, h = (t.double() for t in (x, dt, A, B, C, D, z, h))
    d = torch.nn.functional.softplus(dt + dt_bias.double())
    ys = []
    for t in range(x.shape[1]):
        h = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * x[:, t])[..., None] * B[:, t, None]
        ys.append((h * C[:, t, None]).sum(-1) + D * x[:, t])
    y = torch.stack(ys, 1)
    return y * z * torch.sigmoid(z), h


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_prefix_cache_then_padded_prompt_then_tokens(fmt):
    """Per-channel layer: two cached prefixes continue as four right-padded prompts (one of
    them new), then three decoded tokens each, with a padded row in the decode batch."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)
    Dm, N, W, T, K = 96, 16, 4, 21, 3
    w, b, D = r(Dm, W) * 0.5, r(Dm) * 0.1, r(Dm)
    A = -torch.arange(1, N + 1).float() * torch.exp(0.2 * r(Dm, N))
    dt_bias = torch.full((Dm,), -4.0)
    c = lambda t: t.cuda()
    kw = dict(dt_bias=c(dt_bias), dt_softplus=True)
    # the prefixes, each once
    px, pdt, pB, pC, pz = r(2, 40, Dm), r(2, 40, Dm), r(2, 40, N), r(2, 40, N), r(2, 40, Dm)
    (xc,), conv_state = ssd.ssd_conv1d_fwd(c(px), c(w), c(b))
    _, state = ssd.ssd_selective_scan_fwd(xc, c(pdt), c(A), c(pB), c(pC), c(D), z=c(pz), **kw)
    codes = torch.zeros(6, Dm * N, dtype=torch.int8).view(fmt).cuda()
    scales = torch.zeros(6, Dm * N // 64).cuda()
    at = torch.tensor([4, 1], dtype=torch.int32).cuda()
    ssd.ssd_cache_write(state, codes, scales, at)
    # four prompts: prefix 1, prefix 0, prefix 1 again, a new sequence
    use = [1, 0, 1, None]
    slots = torch.tensor([1, 4, 1, -1], dtype=torch.int32).cuda()
    pool = ssd.ssd_cache_read(codes, scales, slots, shape=(Dm, N))
    conv = torch.zeros(4, W - 1, Dm, device="cuda")
    for i, u in enumerate(use):
        if u is not None:
            conv[i] = conv_state[u]
    # (an 8-bit code is off by at most half a step: 1/254 of its block's largest, or 2^-4)
    worst = (pool[0] - state[1]).abs().max() / state[1].abs().max()
    assert float(worst) <= (0.5 / 127 if fmt == torch.int8 else 2.0 ** -4)
    lens = [21, 5, 0, 17]
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    x, dt, B, C, z = r(4, T + K, Dm), r(4, T + K, Dm), r(4, T + K, N), r(4, T + K, N), r(4, T + K, Dm)
    h64, s64 = host_t(pool), host_t(conv)
    ref = []
    for i, n in enumerate(lens):       # tokens 0..n-1 of the prompt, then T..T+K-1
        keep = list(range(n)) + list(range(T, T + K))
        cut = lambda t: t[i:i + 1, keep]
        xc64, _ = conv64(cut(x), w, b, s64[i:i + 1])
        ref.append(scan64(xc64, cut(dt), A, cut(B), cut(C), D, dt_bias, cut(z), h64[i:i + 1]))
    p = lambda t: c(t)[:, :T].contiguous()
    (xc,), _ = ssd.ssd_conv1d_fwd(p(x), c(w), c(b), init_state=conv, final_state=conv, seq_lens=ln)
    y, _ = ssd.ssd_selective_scan_fwd(xc, p(dt), c(A), p(B), p(C), c(D), init_state=pool,
                                      final_state=pool, seq_lens=ln, z=p(z), **kw)
    for i, n in enumerate(lens):
        if n:
            assert_close(host(y[i, :n]), ref[i][0][0, :n].numpy(), gen.F32, "prompt %d" % i)
        assert not y[i, n:].any()
    # decode: a batch of five rows, the third padded
    rows = [2, 0, None, 3, 1]
    sl = torch.tensor([-1 if q is None else q for q in rows], dtype=torch.int32).cuda()
    idx = torch.tensor([0 if q is None else q for q in rows])
    for k in range(K):
        t = lambda a: c(a)[:, T + k][idx.cuda()]
        (xt,) = ssd.ssd_conv1d_step(conv, t(x), c(w), c(b), slots=sl)
        yt = ssd.ssd_selective_scan_step(pool, xt, t(dt), c(A), t(B), t(C), c(D), slots=sl,
                                         z_t=t(z), **kw)
        for j, q in enumerate(rows):
            if q is None:
                assert not yt[j].any() and not xt[j].any()
            else:
                assert_close(host(yt[j]), ref[q][0][0, lens[q] + k].numpy(), gen.F32,
                             "token %d of %d" % (k, q))
    for i in range(4):
        assert_close(host(pool[i]), ref[i][1][0].numpy(), gen.F32, "state %d" % i)


def host_t(t):
    return t.detach().cpu().double()


def test_convolution_into_the_ssd_scan_and_decode():
    """The convolution's three outputs are x, B and C of the chunked scan; the prompt's last
    tokens once more as decode steps from the prompt's prefix."""
    Bt, T, H, P, N, G, K = 2, 150, 4, 64, 64, 1, 5
    C3 = (H * P, G * N, G * N)
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)
    proj = r(Bt, T, 2 * H * P + 2 * G * N + H)     # rows [z | x B C | dt]
    w, b = r(sum(C3), 4) * 0.5, r(sum(C3)) * 0.1
    A, D = -torch.exp(r(H)), r(H)
    dt = torch.exp(r(Bt, T, H) * 0.5 - 3)
    dev = proj.cuda()
    xbc = dev[..., H * P:H * P + sum(C3)]
    (x, B, C), conv = ssd.ssd_conv1d_fwd(xbc, w.cuda(), b.cuda(), splits=C3)
    y, fin = ssd.ssd_chunked_fwd(x.view(Bt, T, H, P), dt.cuda(), A.cuda(), B.view(Bt, T, G, N),
                                 C.view(Bt, T, G, N), D.cuda(), 64)
    c64, _ = conv64(xbc.cpu(), w, b, torch.zeros(Bt, 3, sum(C3)))
    x64, B64, C64 = (t.numpy() for t in c64.split(C3, 2))
    yr, fr, _ = oracle.token_fwd(x64.reshape(Bt, T, H, P), dt.numpy(), A.numpy(),
                                 B64.reshape(Bt, T, G, N), C64.reshape(Bt, T, G, N), D.numpy())
    yr = yr.reshape(Bt, H, T, P).transpose(0, 2, 1, 3)
    assert_close(host(y), yr, gen.F32, "y")
    assert_close(host(fin), fr.reshape(fin.shape), gen.F32, "state")
    # prefix, then tokens
    n = T - K
    (x, B, C), conv = ssd.ssd_conv1d_fwd(xbc[:, :n], w.cuda(), b.cuda(), splits=C3)
    _, st = ssd.ssd_chunked_fwd(x.view(Bt, n, H, P), dt[:, :n].cuda(), A.cuda(),
                                B.view(Bt, n, G, N), C.view(Bt, n, G, N), D.cuda(), 64)
    for t in range(n, T):
        x, B, C = ssd.ssd_conv1d_step(conv, xbc[:, t], w.cuda(), b.cuda(), splits=C3)
        yt = ssd.ssd_decode_step(st, x.view(Bt, H, P), dt[:, t].cuda(), B.view(Bt, G, N),
                                 C.view(Bt, G, N), A.cuda(), D.cuda())
        assert_close(host(yt), yr[:, t], gen.F32, "token %d" % t)
    assert_close(host(st), fr.reshape(fin.shape), gen.F32, "state after the tokens")


@pytest.mark.parametrize("kind", ["ssd", "selective"])
def test_chained_gradients(kind):
    """d(loss) of convolution and scan together, against autograd in float64."""
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g)
    if kind == "ssd":
        Bt, T, H, P, N = 1, 70, 2, 64, 64
        C3 = (H * P, N, N)
    else:
        Bt, T, Dm, N = 2, 45, 40, 16
        C3 = (Dm,)
    Ct = sum(C3)
    xin, w, b = r(Bt, T, Ct), r(Ct, 4) * 0.5, r(Ct) * 0.1
    dy = r(Bt, T, C3[0])
    leaf = [t.double().requires_grad_() for t in (xin, w, b)]
    pre = torch.nn.functional.pad(leaf[0], (0, 0, 3, 0)).unfold(1, 4, 1)
    pre = (pre * leaf[1]).sum(-1) + leaf[2]
    act = pre * torch.sigmoid(pre)
    ys, _ = ssd.ssd_conv1d_fwd(xin.cuda(), w.cuda(), b.cuda(), splits=C3)
    if kind == "ssd":
        A, D, dt = -torch.exp(r(H)), r(H), torch.exp(r(Bt, T, H) * 0.5 - 3)
        x, B, C = act.split(C3, 2)
        h = torch.zeros(Bt, H, P, N, dtype=torch.float64)
        out = []
        for t in range(T):
            d = dt[:, t].double()
            xt = x[:, t].reshape(Bt, H, P)
            h = (torch.exp(d * A.double())[..., None, None] * h
                 + (d[..., None] * xt)[..., None] * B[:, t, None, None])
            out.append(((h * C[:, t, None, None]).sum(-1) + D.double()[:, None] * xt).reshape(Bt, -1))
        x, B, C = ys
        gr = ssd.ssd_chunked_bwd(x.view(Bt, T, H, P), dt.cuda(), A.cuda(), B.view(Bt, T, 1, N),
                                 C.view(Bt, T, 1, N), D.cuda(), 64, dy.cuda().view(Bt, T, H, P))
        dconv = (gr["dx"].view(Bt, T, -1), gr["dB"].view(Bt, T, N), gr["dC"].view(Bt, T, N))
    else:
        A = -torch.arange(1, N + 1).float() * torch.exp(0.2 * r(Dm, N))
        D, dt, B, C, z = r(Dm), r(Bt, T, Dm), r(Bt, T, N), r(Bt, T, N), r(Bt, T, Dm)
        bias = torch.full((Dm,), -3.0)
        h = torch.zeros(Bt, Dm, N, dtype=torch.float64)
        d = torch.nn.functional.softplus(dt.double() + bias.double())
        out = []
        for t in range(T):
            h = (torch.exp(d[:, t, :, None] * A.double()) * h
                 + (d[:, t] * act[:, t])[..., None] * B[:, t, None].double())
            y = (h * C[:, t, None].double()).sum(-1) + D.double() * act[:, t]
            out.append(y * torch.nn.functional.silu(z[:, t].double()))
        gr = ssd.ssd_selective_scan_bwd(ys[0], dt.cuda(), A.cuda(), B.cuda(), C.cuda(), D.cuda(),
                                        dy.cuda(), dt_bias=bias.cuda(), dt_softplus=True, z=z.cuda())
        dconv = (gr["dx"],)
    (torch.stack(out, 1) * dy.double()).sum().backward()
    got = ssd.ssd_conv1d_bwd(xin.cuda(), w.cuda(), dconv, b.cuda())
    log("chained gradients", kind)
    for k, t in zip(("dx", "dweight", "dbias"), leaf):
        assert_close(host(got[k]), t.grad.numpy(), gen.F32, k)


def test_calls_at_once_on_two_streams():
    """Calls in flight on two streams, each with workspaces of its own, equal the same calls
    one after another."""
    torch.manual_seed(21)
    bf = torch.bfloat16
    sets = []
    for T in (2049, 1111):
        x, z = (torch.randn(1, T, 96, device="cuda").to(bf) for _ in range(2))
        B, C = (torch.randn(1, T, 16, device="cuda").to(bf) for _ in range(2))
        sets.append(dict(x=x, dt=(torch.randn(1, T, 96, device="cuda") - 3).to(bf),
                         A=-torch.rand(96, 16, device="cuda"), B=B, C=C,
                         D=torch.randn(96, device="cuda"), z=z, dt_softplus=True))
    w = torch.randn(96, 4, device="cuda")
    dy = [torch.randn(1, m["x"].shape[1], 96, device="cuda") for m in sets]

    def calls(m, g):
        (u,), _ = ssd.ssd_conv1d_fwd(m["x"], w)
        n = dict(m, x=u)
        y, fin = ssd.ssd_selective_scan_fwd(**n)
        out = ssd.ssd_selective_scan_bwd(dy=g, **n)
        return [u, y, fin] + [out[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz")]

    want = [calls(m, g) for m, g in zip(sets, dy)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(calls(sets[i], dy[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i]))
