"""Long memories: a state that lives through tens of thousands of tokens at a slow decay
weighs what the float64 formula says, in a prompt that is not cut over time, in the gradients, in
one that is cut, and over single tokens."""

import pytest
import torch

from selective_state_space_amd import ssd
from _block import TYPES, attn_bar, gen, randn

pytestmark = pytest.mark.gpu

RATES = [0.0, -1e-6, -3e-6, -1.7e-5, -3e-5, -2.3e-4, -3e-4, -4.7e-3]
K = V = 8


def over_tokens(a, b, w):
    """sum over t of w[h, t] a_t (outer) b_t: a, b [Bt,T,H,d], w [H,T] float64."""
    a = (a.double() * w.t()[None, :, :, None]).permute(0, 2, 3, 1).contiguous()
    return torch.matmul(a, b.double().transpose(1, 2).contiguous())


def weights(T):
    """e^{r n} for n tokens [H,T+1]; the rates as the float32 that the library reads."""
    r = torch.tensor(RATES, device="cuda")
    n = torch.arange(T + 1, device="cuda", dtype=torch.float64)
    return r, torch.exp(r.double()[:, None] * n)


def near_each(got, ref, bar, what):
    """Each head on its own, relative 2-norms.  What has decayed below float32's normal numbers
    (at -4.7e-3 e^-154 is left after 32768 tokens) is held to steps of 2^-149: each factor
    f = e^{32 r} rounds by half of one, which comes to 2^-150 / (1 - f) at most, 3.6 steps for
    f = 0.86; 2^-126 an element covers it."""
    assert torch.isfinite(got).all()
    for h, r in enumerate(RATES):
        a, b = got[:, h].double(), ref[:, h]
        off, size = float((a - b).norm()), float(b.norm())
        print("  %-8s %-8g off %.3g of %.3g, %.3g allowed" % (what, r, off, size, bar * size),
              flush=True)
        assert off <= bar * size + 2.0 ** -126 * b.numel() ** 0.5, (what, r)


def roundings(n):
    return attn_bar(torch.float32, n)   # n roundings of independent signs


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("Bt,T", [(17, 32768), (17, 65536 + 7), (1, 300000)])
def test_states_after_many_tokens(Bt, T, io):
    """17 x 8 sequences and heads walk their whole length, 1 x 8 are cut."""
    H = len(RATES)
    dims = ssd.AttnDims(Bt, T, H, H, K, V, 0, 0, 0, 0, 0, 0, 1 if io == "bf16" else 0, 1.0)
    lay = ssd.linear_attn_layout(dims)
    assert (lay.fwd_segments == 1) == (lay.bwd_segments == 1) == (Bt > 1)
    g = gen(T)
    r, w = weights(T)
    q, k, v, dy = (randn(g, Bt, T, H, d, dtype=TYPES[io]) for d in (K, K, V, V))
    init, dfinal = randn(g, Bt, H, K, V), randn(g, Bt, H, K, V)
    # what is left of the start alone: a rounding for each 32 tokens' factor (cut: fewer)
    _, fin = ssd.ssd_linear_attn_fwd(q, k, torch.zeros_like(v), r, init_state=init)
    near_each(fin, w[:, T][None, :, None, None] * init.double(), roundings(T // 32 + 64), "start")
    got = ssd.ssd_linear_attn_bwd(q, k, v, r, torch.zeros_like(dy), dfinal=dfinal)
    near_each(got["dinit"], w[:, T][None, :, None, None] * dfinal.double(), roundings(T // 32 + 64),
              "end")
    # and what all tokens add: a rounding for each
    _, fin = ssd.ssd_linear_attn_fwd(q, k, v, r, scale=0.5)
    near_each(fin, over_tokens(k, v, w[:, :T].flip(1)), roundings(T + 64), "final")
    got = ssd.ssd_linear_attn_bwd(q, k, v, r, dy, scale=0.5)
    near_each(got["dinit"], 0.5 * over_tokens(q, dy, w[:, 1:]), roundings(T + 64), "dinit")


def test_state_after_many_steps():
    """Three roundings a token: of k v, of what the factor lacks, of the state.  Where nothing
    is added the state's are not of independent signs: at -1e-6 a token takes 8 to 17 steps off
    a number, the same count and the same fraction of a step for thousands of tokens, so each
    may leave half a step, 2^-24 of the number, to the same side."""
    H, T = len(RATES), 4000
    g = gen(5)
    r, w = weights(T)
    q, k, v = (randn(g, T, 1, H, d) for d in (K, K, V))
    start = randn(g, 1, H, K, V)
    state, kept = start.clone(), start.clone()
    none = torch.zeros_like(v[0])
    for t in range(T):
        ssd.ssd_linear_attn_step(state, q[t], k[t], v[t], r)
        ssd.ssd_linear_attn_step(kept, q[t], k[t], none, r)
    left = w[:, T][None, :, None, None] * start.double()
    near_each(kept, left, T * 2.0 ** -24, "start")
    added = over_tokens(k.transpose(0, 1), v.transpose(0, 1), w[:, :T].flip(1))
    near_each(state, left + added, roundings(3 * T), "state")


@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_infinite_states_stay_infinite(bad):
    """A state that is infinite decays to itself, at any rate."""
    H = len(RATES)
    state = torch.full((1, H, K, V), bad, device="cuda")
    q = torch.ones(1, H, K, device="cuda")
    y = ssd.ssd_linear_attn_step(state, q, q, q, torch.tensor(RATES, device="cuda"))
    assert (state == bad).all() and (y == bad).all()
