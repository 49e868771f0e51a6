"""How many bits bf16 linear attention keeps: its outputs and gradients are the float64
values rounded to bf16 once, but for those next to a border between two bf16 numbers."""

import pytest
import torch

from selective_state_space_amd import ssd
from _block import assert_near, attn_inputs, attn_ref

pytestmark = pytest.mark.gpu


def bar(T, K, V):
    """Relative 2-norm of (rounded output - rounded float64 value).

    Before it is rounded an output is off by d: two operands held in two bf16 terms (hi cut,
    which leaves anything below 2^-7 of an element, 0.58 of that root mean square; of it the
    rounding of lo 2^-8 at the worst, 0.58 of that root mean square: 0.33 2^-15, below 2^-16)
    and float32 roundings of T + 2 max(K, V) + 64 terms, of independent signs:
    d <= sqrt(2) 2^-16 + 2^-24 sqrt(terms) of the norm.  The rounded numbers then differ by a
    step, at most 2^-7 of the value, with probability d / step: the square of the difference
    is on average step d, of the norms' squares 2^-7 d."""
    d = 2.0 ** 0.5 * 2.0 ** -16 + 2.0 ** -24 * (T + 2 * max(K, V) + 64) ** 0.5
    return (2.0 ** -7 * d) ** 0.5


# (Bt, T, H, G, K, V): 64 and 128 columns of a state of 64, 128 and 256 rows, cut over time,
# shared heads, a launch for all gradients and one for each row count
SIZES = [(2, 70, 3, 3, 64, 64), (2, 150, 3, 1, 128, 128), (40, 45, 5, 5, 64, 128),
         (50, 45, 4, 2, 128, 72), (2, 100, 2, 2, 256, 200), (1, 1100, 4, 2, 128, 128),
         (24, 40, 4, 1, 128, 128)]


@pytest.mark.parametrize("sizes", SIZES)
def test_outputs_are_rounded_once(sizes):
    Bt, T, H, G, K, V = sizes
    c, kw = attn_inputs(T + K, Bt, T, H, G, K, V, torch.bfloat16, init=True, grads=True)
    dy, df = c.pop("dy"), kw.pop("dfinal")
    args = (c["q"], c["k"], c["v"], c["log_decay"], kw["scale"], kw["init_state"])
    y, _ = ssd.ssd_linear_attn_fwd(**c, **kw)
    yr, _ = attn_ref(*args)
    assert_near(y, yr.bfloat16(), bar(T, K, V), "y")
    got = ssd.ssd_linear_attn_bwd(**c, dy=dy, dfinal=df, **kw)
    ref = attn_ref(*args, dy=dy, dfinal=df)
    for n in ("dq", "dk", "dv"):
        assert_near(got[n], ref[n].bfloat16(), bar(T, K, V), n)
