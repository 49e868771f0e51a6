"""bf16 prompts of many sequences and heads: 128 columns of the state a workgroup, by the
library's own answer, and what they give against float64."""

import pytest
import torch

from selective_state_space_amd import ssd
from _block import assert_near, attn_bar, attn_inputs, attn_ref

pytestmark = pytest.mark.gpu

# (Bt, T, H, G, K, V), columns in float32, in bf16
SIZES = [((65, 40, 4, 4, 128, 128), (64, 128)), ((65, 70, 4, 2, 72, 96), (64, 128)),
         ((97, 33, 4, 1, 64, 128), (64, 128)), ((96, 33, 4, 4, 64, 128), (64, 64)),
         ((65, 35, 4, 4, 128, 200), (64, 128)), ((65, 35, 4, 4, 136, 128), (64, 64)),
         ((65, 40, 4, 4, 128, 64), (64, 64))]


@pytest.mark.parametrize("io", [ssd.SSD_F32, ssd.SSD_BF16])
@pytest.mark.parametrize("sizes,columns", SIZES)
def test_many_rows(sizes, columns, io):
    Bt, T, H, G, K, V = sizes
    lay = ssd.linear_attn_layout(ssd.AttnDims(Bt, T, H, G, K, V, 0, 0, 0, 0, 0, 0, io, 1.0))
    assert (lay.fwd_cols, lay.fwd_segments) == (columns[io], 1)
    dtype = torch.bfloat16 if io else torch.float32
    lens = [T, 0, 1, T - 1, T // 2] * (Bt // 5) + [T] * (Bt % 5)
    c, kw = attn_inputs(K + V, Bt, T, H, G, K, V, dtype, init=True, lens=lens)
    y, fin = ssd.ssd_linear_attn_fwd(**c, **kw)
    yr, fr = attn_ref(c["q"], c["k"], c["v"], c["log_decay"], kw["scale"], kw["init_state"],
                      kw["seq_lens"])
    terms = T + 2 * max(K, V) + 64
    assert_near(y, yr, attn_bar(dtype, terms), "y")
    assert_near(fin, fr, attn_bar(torch.float32, terms), "final")
