"""Linear attention, the group norm and 4-bit projections run together, as a layer uses them,
with the convolution and the 8-bit cache beside them: prompts, decoded tokens, gradients,
captured graphs, calls at once.  float32 outputs to the framework's float32 bar, max|gpu - ref|
<= 1e-4 max|ref|, against float64."""

import pytest
import torch

from selective_state_space_amd import inputs as gen
from selective_state_space_amd import ssd

from _block import attn_ref, norm_ref, w4_values
from _gpu import assert_close, host, log

pytestmark = pytest.mark.gpu

H, G, K, V, C = 4, 2, 32, 48, 256      # C: the model's channels
SPLIT = (H * K, G * K, G * V, H * V)    # q, k, v, z of the first projection's outputs


def layer(seed):
    """Weights of a layer: 4-bit projections in and out, decays, the norm's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return dict(win=ssd.ssd_w4_quantize(r(sum(SPLIT), C) * C ** -0.5, 64), bin=r(sum(SPLIT)) * 0.1,
                wout=ssd.ssd_w4_quantize(r(C, H * V) * (H * V) ** -0.5, 64),
                decay=-torch.exp2(-1.0 - 5.0 * torch.arange(H, device="cuda").float() / H),
                weight=1 + 0.1 * r(H * V), bias=0.1 * r(H * V)), r


def tensors(p, lead):
    q, k, v, z = p.split(SPLIT, -1)
    return (q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V)), z)


def prompt(m, x, lens=None, state=None):
    """(y, state) of x [Bt,T,C]; q, k, v and the gate z are slices of one projection."""
    Bt, T = x.shape[:2]
    p = ssd.ssd_w4_linear(x.reshape(Bt * T, C), *m["win"], m["bin"]).view(Bt, T, -1)
    q, k, v, z = tensors(p, (Bt, T))
    y, state = ssd.ssd_linear_attn_fwd(q, k, v, m["decay"], init_state=state, seq_lens=lens)
    y = ssd.ssd_group_norm_fwd(y.view(Bt, T, H * V), H, m["weight"], m["bias"], z=z, form="gate",
                               seq_lens=lens)
    return ssd.ssd_w4_linear(y.view(Bt * T, H * V), *m["wout"]).view(Bt, T, C), state


def token(m, x, state, slots):
    q, k, v, z = tensors(ssd.ssd_w4_linear(x, *m["win"], m["bin"]), x.shape[:1])
    y = ssd.ssd_linear_attn_step(state, q, k, v, m["decay"], slots=slots)
    y = ssd.ssd_group_norm_fwd(y.view(-1, H * V), H, m["weight"], m["bias"], z=z, form="gate")
    return ssd.ssd_w4_linear(y, *m["wout"])


def layer64(m, x, state):
    """One sequence [T,C] in float64."""
    p = x.double() @ w4_values(*m["win"]).t() + m["bin"].double()
    q, k, v, z = (t[None] for t in tensors(p, x.shape[:1]))
    y, state = attn_ref(q, k, v, m["decay"], K ** -0.5, state[None])
    y = norm_ref(y.flatten(2), H, m["weight"], m["bias"], z, "gate")
    return y[0] @ w4_values(*m["wout"]).t(), state[0]


@pytest.mark.parametrize("fmt", [None, torch.int8, torch.float8_e4m3fn])
def test_prompts_then_tokens(fmt):
    """Four right-padded prompts, their states (through the 8-bit cache where one is named) into
    a pool, and five decoded tokens each with a padded row in the batch."""
    m, r = layer(3)
    lens, T, n = [70, 33, 1, 64], 70, 5
    x, more = r(4, T, C), r(n, 4, C)
    y, state = prompt(m, x, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    pool = r(7, H, K, V)
    keep = pool.clone()
    slots = torch.tensor([5, 0, -1, 6, 2], dtype=torch.int32, device="cuda")   # row 2 is padding
    rows, at = [0, 1, 3, 4], [5, 0, 6, 2]
    if fmt is None:
        pool[at] = state
    else:
        codes = torch.zeros(9, H * K * V, dtype=torch.int8, device="cuda").view(fmt)
        scales = torch.zeros(9, H * K * V // 64, device="cuda")
        saved = torch.tensor([8, 1, 4, 3], dtype=torch.int32, device="cuda")
        ssd.ssd_cache_write(state, codes, scales, saved)
        pool[at] = ssd.ssd_cache_read(codes, scales, saved, shape=(H, K, V))
    from64 = pool[at].double()
    xs = torch.zeros(n, 5, C, device="cuda")
    xs[:, rows] = more
    out = torch.stack([token(m, xs[i], pool, slots) for i in range(n)])
    log("layer", fmt)
    for b, ln in enumerate(lens):
        want, s = layer64(m, x[b, :ln], torch.zeros(H, K, V, device="cuda"))
        assert_close(host(y[b, :ln]), want.cpu().numpy(), gen.F32, "prompt %d" % b)
        assert not y[b, ln:].any()
        if fmt is None:
            assert_close(host(state[b]), s.cpu().numpy(), gen.F32, "state %d" % b)
        want, s = layer64(m, more[:, b], from64[b])
        assert_close(host(out[:, rows[b]]), want.cpu().numpy(), gen.F32, "tokens %d" % b)
        assert_close(host(pool[at[b]]), s.cpu().numpy(), gen.F32, "pool %d" % b)
    for s in (1, 3, 4):
        assert torch.equal(pool[s], keep[s])


def test_prompt_in_parts():
    """A prompt, the same in two parts with the state between, and its last tokens one by one."""
    m, r = layer(4)
    x = r(2, 90, C)
    whole, end = prompt(m, x)
    first, state = prompt(m, x[:, :41].contiguous())
    second, state = prompt(m, x[:, 41:85].contiguous(), state=state)
    out = [token(m, x[:, t].contiguous(), state, None)[:, None] for t in range(85, 90)]
    log("parts")
    assert_close(host(torch.cat([first, second] + out, 1)), host(whole), gen.F32, "y")
    assert_close(host(state), host(end), gen.F32, "state")


@pytest.mark.parametrize("form", ["gate", "gated_input"])
def test_chained_gradients(form):
    """Gradients through convolution, linear attention (padded, shared heads) and the group
    norm, against float64 autograd."""
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)
    Bt, T = 2, 75
    lens = torch.tensor([75, 40], dtype=torch.int32)
    cs = SPLIT[:3]
    xin, w, b = r(Bt, T, sum(cs)), r(sum(cs), 4) * 0.5, r(sum(cs)) * 0.1
    z, nw, nb, dy = r(Bt, T, H * V), 1 + 0.1 * r(H * V), 0.1 * r(H * V), r(Bt, T, H * V)
    decay = -torch.exp2(-1.0 - 5.0 * torch.arange(H).float() / H)
    kw = dict(z=z.cuda(), form=form, seq_lens=lens.cuda())
    (q, k, v), _ = ssd.ssd_conv1d_fwd(xin.cuda(), w.cuda(), b.cuda(), splits=cs,
                                      seq_lens=lens.cuda())
    q, k, v = (t.view(Bt, T, n, d) for t, n, d in ((q, H, K), (k, G, K), (v, G, V)))
    y, _ = ssd.ssd_linear_attn_fwd(q, k, v, decay.cuda(), seq_lens=lens.cuda())
    y = y.view(Bt, T, H * V)
    gn = ssd.ssd_group_norm_bwd(y, H, dy.cuda(), nw.cuda(), nb.cuda(), **kw)
    ga = ssd.ssd_linear_attn_bwd(q, k, v, decay.cuda(), gn["dx"].view(Bt, T, H, V),
                                 seq_lens=lens.cuda())
    # (zero behind the lengths, so that the convolution's gradients need none)
    gc = ssd.ssd_conv1d_bwd(xin.cuda(), w.cuda(),
                            tuple(ga[n].flatten(2) for n in ("dq", "dk", "dv")), b.cuda())
    # float64, token by token
    leaf = [t.double().requires_grad_() for t in (xin, w, b, z, nw, nb)]
    pre = torch.nn.functional.pad(leaf[0], (0, 0, 3, 0)).unfold(1, 4, 1)
    pre = (pre * leaf[1]).sum(-1) + leaf[2]
    q, k, v = (pre * torch.sigmoid(pre)).split(cs, 2)
    q = q.unflatten(2, (H, K))
    k, v = (t.unflatten(2, (G, -1)).repeat_interleave(H // G, 2) for t in (k, v))
    s = torch.zeros(Bt, H, K, V, dtype=torch.float64)
    a, ys = torch.exp(decay.double())[:, None, None], []
    for t in range(T):
        s = a * s + k[:, t, :, :, None] * v[:, t, :, None]
        ys.append(K ** -0.5 * (q[:, t, :, :, None] * s).sum(2).flatten(1))
    u = torch.stack(ys, 1)
    gate = torch.nn.functional.silu(leaf[3])
    if form == "gated_input":
        u = u * gate
    u = u.unflatten(2, (H, V))
    c = u - u.mean(-1, keepdim=True)
    n = (c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5)).flatten(2) * leaf[4] + leaf[5]
    out = n * gate if form == "gate" else n
    live = (torch.arange(T)[None] < lens[:, None])[..., None]
    (torch.where(live, out, 0.0) * dy.double()).sum().backward()
    log("chained gradients", form)
    for got, t, name in ((gc["dx"], leaf[0], "dx"), (gc["dweight"], leaf[1], "conv weight"),
                         (gc["dbias"], leaf[2], "conv bias"), (gn["dz"], leaf[3], "dz"),
                         (gn["dweight"], leaf[4], "norm weight"), (gn["dbias"], leaf[5], "norm bias")):
        assert_close(host(got), t.grad.numpy(), gen.F32, name)


def work(seed, T):
    """Every operator's calls on inputs of their own, as (inputs to refresh, the calls)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bf = torch.bfloat16
    r = lambda *s, dtype=bf: torch.randn(*s, generator=g, device="cuda").to(dtype)
    q, k, v, dy = r(1, T, 4, 64), r(1, T, 2, 64), r(1, T, 2, 96), r(1, T, 4, 96)
    decay = torch.tensor([-0.5, -0.1, -0.01, -0.001], device="cuda")
    x, z, nw, nb = r(1, T, 384), r(1, T, 384), r(384, dtype=torch.float32), r(384, dtype=torch.float32)
    w, rows = r(300, 256), r(20, 256)
    pool = torch.zeros(3, 4, 64, 96, device="cuda")

    def calls(pool):
        y, fin = ssd.ssd_linear_attn_fwd(q, k, v, decay)
        ga = ssd.ssd_linear_attn_bwd(q, k, v, decay, dy)
        t = ssd.ssd_linear_attn_step(pool, q[0, :3], k[0, :3], v[0, :3], decay)
        n = ssd.ssd_group_norm_fwd(x, 4, nw, nb, z=z, form="gate")
        gn = ssd.ssd_group_norm_bwd(x, 4, n, nw, nb, z=z, form="gated_input")
        codes, scales = ssd.ssd_w4_quantize(w, 64)
        return [y, fin, t, n, codes, scales, ssd.ssd_w4_linear(rows, codes, scales),
                ssd.ssd_w4_linear(rows[0], codes, scales), ssd.ssd_w4_dequantize(codes, scales)
                ] + [ga[n] for n in ("dq", "dk", "dv", "dinit")] + [
                    gn[n] for n in ("dx", "dz", "dweight", "dbias")]
    return [q, k, v, dy, x, z, w, rows], pool, calls


def test_graph_replays_follow_the_inputs():
    """All calls (the attention cut over time) in one graph: every replay equals the eager calls
    on that replay's inputs, with eager work between."""
    inputs, pool, calls = work(7, 1111)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(pool)
    for _ in range(4):
        for t in inputs:
            t.copy_(torch.randn(t.shape, device="cuda"))
        eager_pool = pool.clone()
        want = [t.clone() for t in calls(eager_pool)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), i
        assert torch.equal(pool, eager_pool)


def test_two_graphs_and_eager_calls_at_once():
    """Two captured graphs, each with the workspaces of its own capture, replayed on two streams
    with eager calls on a third."""
    sets = [work(11 + i, T) for i, T in enumerate((1111, 2049, 777))]
    want = [calls(pool.clone()) for _, pool, calls in sets]
    torch.cuda.synchronize()
    graphs, outs, pools = [], [], []
    for _, pool, calls in sets[:2]:
        pools.append(pool.clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(calls(pools[-1]))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for p in pools:
            p.zero_()
        eager = sets[2][1].clone()
        torch.cuda.synchronize()
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            third = sets[2][2](eager)
        torch.cuda.synchronize()
        for got, ref in zip(outs + [third], want):
            for i, (a, b) in enumerate(zip(got, ref)):
                assert torch.equal(a, b), i


def test_calls_at_once_on_two_streams():
    sets = [work(21 + i, T) for i, T in enumerate((2049, 1111))]
    want = [calls(pool.clone()) for _, pool, calls in sets]
    pools = [[pool.clone() for _ in range(4)] for _, pool, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for n in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(sets[i][2](pools[i][n]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i]))


def test_a_long_cut_sequence_with_far_tokens():
    """Token offsets past 2^32 elements within one sequence, cut over time."""
    T, d, far = 1100, 64, 1 << 22
    flat = torch.empty((T - 1) * far + 3 * d, dtype=torch.bfloat16, device="cuda")
    q, k, v = (torch.as_strided(flat, (1, T, 1, d), (0, far, d, 1), i * d) for i in range(3))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dense = [torch.randn(1, T, 1, d, generator=g, device="cuda").bfloat16() for _ in range(3)]
    for t, s in zip((q, k, v), dense):
        t.copy_(s)
    r = torch.tensor([-0.01], device="cuda")
    dy = torch.randn(1, T, 1, d, generator=g, device="cuda").bfloat16()
    for a, b in zip(ssd.ssd_linear_attn_fwd(q, k, v, r), ssd.ssd_linear_attn_fwd(*dense, r)):
        assert torch.equal(a, b)
    got, want = (ssd.ssd_linear_attn_bwd(*t, r, dy) for t in ((q, k, v), dense))
    assert all(torch.equal(got[n], want[n]) for n in got)
