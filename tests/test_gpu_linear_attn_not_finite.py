"""An infinity or a NaN in q, k, v or dy of a gradient call reaches what its formula says and
nothing else:

    dq_t = scale sum over s <= t of e^{r(t-s)} (dy_t . v_s) k_s, and the start state's
    dk_s = scale sum over t >= s of e^{r(t-s)} (dy_t . v_s) q_t, and the end's adjoint
    dv_s = scale sum over t >= s of e^{r(t-s)} (q_t . k_s) dy_t, likewise
"""

import pytest
import torch

from selective_state_space_amd import ssd
from _block import TYPES, assert_near, attn_bar, attn_inputs

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), -float("inf")]
T, H = 70, 4


def same_but(got, want, heads, tokens, columns, bar, what):
    """Sequence 0, other heads, and sequence 1's tokens and columns that a mask leaves out."""
    assert torch.equal(got[0], want[0]), what
    rest = [h for h in range(got.shape[2]) if h not in heads]
    assert torch.equal(got[1][:, rest], want[1][:, rest]), what
    reached = torch.zeros(got.shape[1], got.shape[3], dtype=torch.bool, device="cuda")
    reached[tokens, columns] = True
    for h in heads:
        a, b = got[1, :, h], want[1, :, h]
        if not reached.all():
            assert_near(a[~reached], b[~reached], bar, what)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("K,V", [(64, 64), (128, 72), (64, 136)])
@pytest.mark.parametrize("G", [2, 4])
@pytest.mark.parametrize("at", [0, 1, 16, 31, 32, 50, 69])
def test_gradients(at, G, K, V, io):
    c, kw = attn_inputs(9, 2, T, H, G, K, V, TYPES[io], init=True, grads=True)
    want = ssd.ssd_linear_attn_bwd(**c, **kw)
    bar = 2 * attn_bar(TYPES[io], T + 2 * max(K, V) + 64)
    own, upto, after, every, col = slice(at, at + 1), slice(0, at + 1), slice(at, T), slice(None), 3
    rep = H // G
    head, group = 1, 1             # of q and dy; of k and v
    readers = list(range(group * rep, group * rep + rep))
    shared = [head // rep]
    for i, name in enumerate(("q", "k", "v", "dy")):
        d = {n: t.clone() for n, t in c.items()}
        d[name][1, at, head if name in ("q", "dy") else group, col] = BAD[(i + at) % 3]
        got = ssd.ssd_linear_attn_bwd(**d, **kw)
        what = lambda n: "%s of %s" % (n, name)
        if name == "q":
            assert torch.equal(got["dq"], want["dq"])
            same_but(got["dk"], want["dk"], shared, upto, col, bar, what("dk"))
            same_but(got["dv"], want["dv"], shared, upto, every, bar, what("dv"))
            hit = [got["dk"][1, at, shared, col], got["dv"][1, at, shared]]
        elif name == "k":
            assert torch.equal(got["dk"], want["dk"])
            same_but(got["dq"], want["dq"], readers, after, col, bar, what("dq"))
            same_but(got["dv"], want["dv"], [group], own, every, bar, what("dv"))
            hit = [got["dq"][1, at, readers, col], got["dv"][1, at, group]]
        elif name == "v":
            assert torch.equal(got["dv"], want["dv"])
            same_but(got["dq"], want["dq"], readers, after, every, bar, what("dq"))
            same_but(got["dk"], want["dk"], [group], own, every, bar, what("dk"))
            hit = [got["dq"][1, at, readers], got["dk"][1, at, group]]
        else:
            same_but(got["dq"], want["dq"], [head], own, every, bar, what("dq"))
            same_but(got["dk"], want["dk"], shared, upto, every, bar, what("dk"))
            same_but(got["dv"], want["dv"], shared, upto, col, bar, what("dv"))
            hit = [got["dq"][1, at, head], got["dk"][1, at, shared], got["dv"][1, at, shared, col]]
        assert not any(bool(torch.isfinite(t).any()) for t in hit), name
        other = [h for h in range(H) if h != head]
        if name in ("k", "v"):
            assert torch.equal(got["dinit"], want["dinit"])
        else:
            assert torch.equal(got["dinit"][0], want["dinit"][0])
            assert torch.equal(got["dinit"][1, other], want["dinit"][1, other])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("name", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("bad", BAD)
def test_cut_over_time(name, bad, io):
    """The same between the parts of a sequence that is cut."""
    n, at, K = 1100, 500, 64
    c, kw = attn_inputs(3, 1, n, 2, 1, K, K, TYPES[io], init=True, grads=True)
    want = ssd.ssd_linear_attn_bwd(**c, **kw)
    dims = ssd.AttnDims(1, n, 2, 1, K, K, 0, 0, 0, 0, 0, 0, 1 if io == "bf16" else 0, 1.0)
    assert ssd.linear_attn_layout(dims).bwd_segments > 2
    d = {m: t.clone() for m, t in c.items()}
    d[name][0, at, 0, 5] = bad
    got = ssd.ssd_linear_attn_bwd(**d, **kw)
    bar = 2 * attn_bar(TYPES[io], n + 2 * K + 64)
    forward = {"k": slice(0, at), "v": slice(0, at)}.get(name)
    if forward:
        assert_near(got["dq"][:, forward], want["dq"][:, forward], bar, "dq")
        for m in ("dk", "dv"):
            keep = [t for t in range(n) if t != at]
            assert_near(got[m][:, keep], want[m][:, keep], bar, m)
        assert torch.equal(got["dinit"], want["dinit"])
    else:
        for m in ("dk", "dv"):
            assert_near(got[m][:, at + 1:], want[m][:, at + 1:], bar, m)
        keep = [t for t in range(n) if t != at]
        assert_near(got["dq"][:, keep], want["dq"][:, keep], bar, "dq")


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("Bt,K", [(40, 64), (40, 128), (65, 128)])
@pytest.mark.parametrize("at", [0, 17, 40, 44])
def test_prompts_of_many_sequences(at, Bt, K, io):
    """Workgroups of 128 columns (65 sequences: in bf16 alone): a bad k, v or q leaves the tokens
    before it, other heads, other sequences and, in v, other columns."""
    V, n = 128, 45
    lay = ssd.linear_attn_layout(ssd.AttnDims(Bt, n, H, H, K, V, 0, 0, 0, 0, 0, 0,
                                              1 if io == "bf16" else 0, 1.0))
    assert lay.fwd_cols == (128 if Bt == 40 or io == "bf16" else 64)
    c, kw = attn_inputs(4, Bt, n, H, H, K, V, TYPES[io], init=True)
    y, _ = ssd.ssd_linear_attn_fwd(**c, **kw)
    bar = 2 * attn_bar(TYPES[io], n + 2 * max(K, V) + 64)
    for i, name in enumerate("kvq"):
        d = {m: t.clone() for m, t in c.items()}
        d[name][1, at, 2, 3] = BAD[(i + at) % 3]
        got, _ = ssd.ssd_linear_attn_fwd(**d, **kw)
        tokens, columns = slice(at, at + 1 if name == "q" else n), 3 if name == "v" else slice(None)
        same_but(got[:2], y[:2], [2], tokens, columns, bar, name)
        assert torch.equal(got[2:], y[2:])
        assert not torch.isfinite(got[1, tokens, 2, columns]).any()
