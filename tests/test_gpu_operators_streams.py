"""Calls at once on two streams of the block norm and the rotary positions, each its own workspace: the bits of calls by
themselves."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def normal(*shape, to=torch.float32):
    return torch.randn(*shape, device="cuda").to(to)


def at_once(a, b):
    """a and b by themselves, then ten times on a stream each, given as the current one and as an argument."""
    wa, wb = a(None), b(None)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s):
            ga = a(None)
        got.append((ga, b(t)))
    torch.cuda.synchronize()
    for ga, gb in got:
        assert all(torch.equal(p, q) for p, q in zip(wa, ga))
        assert all(torch.equal(p, q) for p, q in zip(wb, gb))


# widths: several rows a workgroup, a row each, rows that the registers do not hold
@pytest.mark.parametrize("n,C,other", [(20000, 64, 2048), (3000, 4096, 100), (400, 20000, 9000)])
def test_block_norm(n, C, other):
    from state_space_sequence_amd import m3
    torch.manual_seed(1)

    def call(n, C, io, res):
        x, z, r, dy, dR = normal(n, C, to=io), normal(n, C, to=io), normal(n, C, to=res), normal(n, C, to=io), normal(n, C, to=res)
        w, wp, sc = normal(C), normal(C), normal(C)
        kw = dict(z=z, scale=sc, post_norm=True, post_weight=w, pre_weight=wp, residual_scale=0.5)

        def f(stream):
            y, R = m3.block_norm_fwd(x, r, stream=stream, **kw)
            g = m3.block_norm_bwd(x, R, dy, dR, stream=stream, **kw)
            return [y, R] + [g[k] for k in sorted(g)]
        return f

    at_once(call(n, C, BF, BF), call(n // 2, other, BF, torch.float32))


def test_rotary():
    from state_space_sequence_amd import m3
    torch.manual_seed(2)

    def call(b, L, H, G, D, io, layout):
        q, k = normal(b, L, H, D, to=io), normal(b, L, G, D, to=io)
        freqs = m3.rotary_frequencies(D, device="cuda")
        return lambda stream: list(m3.rotary(q, k, freqs, layout=layout, stream=stream))

    at_once(call(2, 3000, 16, 4, 128, BF, "half"), call(3, 2000, 8, 1, 80, torch.float32, "interleaved"))
