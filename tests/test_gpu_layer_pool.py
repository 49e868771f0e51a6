"""The SSD scan's states through the 8-bit pool: prompts leave their states in slots, later
prompts and decoded tokens continue from what reads back.  float32 io; outputs to the
framework's float32 bar against the float64 oracle started from the values read back, and
those within half a code's step of the states written."""

import pytest
import torch

import oracle
from selective_state_space_amd import inputs as gen
from selective_state_space_amd import ssd

from _gpu import assert_close, host, log

pytestmark = pytest.mark.gpu


def token_fwd(m, t0, t1, rows, init):
    """(y [rows,T,H,P], final [rows,H,P,N]) of tokens t0..t1 in float64."""
    cut = lambda k: m[k][rows, t0:t1].numpy()
    H, P = m["x"].shape[2:]
    y, fin, _ = oracle.token_fwd(cut("x"), cut("dt"), m["A"].numpy(), cut("B"), cut("C"),
                                 m["D"].numpy(), None if init is None else init.numpy())
    n = len(rows)
    return y.reshape(n, H, t1 - t0, P).transpose(0, 2, 1, 3), fin.reshape(n, H, P, -1)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("H,P,N,G", [(4, 64, 64, 1), (2, 64, 128, 2)])
def test_prompts_and_tokens_on_pooled_states(fmt, H, P, N, G):
    log("ssd states through the pool", fmt, H, P, N, G)
    g = torch.Generator().manual_seed(H * N)
    r = lambda *s: torch.randn(*s, generator=g)
    Bt, T0, T1, K, L = 3, 130, 70, 3, 64
    T = T0 + T1 + K
    m = dict(x=r(Bt, T, H, P), dt=torch.exp(r(Bt, T, H) * 0.5 - 3), A=-torch.exp(r(H)),
             B=r(Bt, T, G, N), C=r(Bt, T, G, N), D=r(H))
    c = lambda k, t0, t1, rows: m[k][rows, t0:t1].contiguous().cuda()
    A, D = m["A"].cuda(), m["D"].cuda()

    def prompt(t0, t1, rows, init):
        return ssd.ssd_chunked_fwd(c("x", t0, t1, rows), c("dt", t0, t1, rows), A,
                                   c("B", t0, t1, rows), c("C", t0, t1, rows), D, L,
                                   init_state=init)

    every = [0, 1, 2]
    _, state = prompt(0, T0, every, None)
    size = H * P * N
    codes = torch.full((6, size), 3, dtype=torch.int8).view(fmt).cuda()
    scales = torch.full((6, size // 64), 0.5).cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    ssd.ssd_cache_write(state, codes, scales, slots)
    # the pool serves two of them and a new sequence
    rows = [2, 0, 1]
    at = torch.tensor([2, 4, -1], dtype=torch.int32).cuda()
    back = ssd.ssd_cache_read(codes, scales, at, shape=(H, P, N))
    assert not back[2].any()
    for i, b in ((0, 2), (1, 0)):
        block = state[b].view(-1, 64)
        scale = block.abs().amax(1, keepdim=True) / (127.0 if fmt == torch.int8 else 448.0)
        step = 0.5 * scale if fmt == torch.int8 else torch.maximum(2.0 ** -4 * block.abs(),
                                                                   2.0 ** -10 * scale)
        # (and the roundings of the scale and of the product)
        assert ((back[i].view(-1, 64) - block).abs() <= step + 2.0 ** -22 * block.abs()).all()
    start = back.cpu().double()
    y, fin = prompt(T0, T0 + T1, rows, back)
    yr, fr = token_fwd(m, T0, T, rows, start)
    assert_close(host(y), yr[:, :T1], gen.F32, "y on pooled states")
    for k in range(K):
        t = T0 + T1 + k
        one = lambda key: c(key, t, t + 1, rows)[:, 0].contiguous()
        yt = ssd.ssd_decode_step(fin, one("x"), one("dt"), one("B"), one("C"), A, D)
        assert_close(host(yt), yr[:, T1 + k], gen.F32, "token %d" % k)
    assert_close(host(fin), fr, gen.F32, "state")
    # a state written back into its slot leaves the others as they were
    before = codes.view(torch.int8).clone(), scales.clone()
    ssd.ssd_cache_write(fin[:1], codes, scales, at[:1])
    others = [0, 1, 3, 4, 5]
    assert torch.equal(codes.view(torch.int8)[others], before[0][others])
    assert torch.equal(scales[others], before[1][others])
    assert not torch.equal(codes.view(torch.int8)[2], before[0][2])
