"""bf16 linear attention keeps all 24 bits of what it computes in between: a state and a
score that enter the next product lose nothing that fp32 holds.

Each case is a sum of two terms near 1 whose difference is 2^-17: a bit that a state or a
score needs more than 16 bits for, and that the bf16 output holds exactly. Every product
and sum of these inputs is exact in fp32 (the terms have 18 bits at most), the decay is 1 and the scale is
1, so the output has to be 2^-17 itself, whatever the order of the sums."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BIT = 2.0 ** -17


def tensors(L, N, P):
    z = lambda *s: torch.zeros(1, L, 1, *s, dtype=torch.bfloat16, device="cuda")
    return z(N), z(N), z(P), torch.zeros(1, device="cuda")


@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 1, 63, 64, 100])
def test_states(N, at):
    """A carried state of 1 + 2^-9 + 2^-17 and -(1 + 2^-9) against a query of ones."""
    from state_space_sequence_amd import m3
    L, P = 101, 64
    q, k, v, ld = tensors(L, N, P)
    h0 = torch.zeros(1, 1, P, N, device="cuda")
    h0[0, 0, :, 3], h0[0, 0, :, N - 1] = 1 + 2.0 ** -9 + BIT, -(1 + 2.0 ** -9)
    q[0, at] = 1
    y, h = m3.linattn_fwd(q, k, v, ld, scale=1.0, h0=h0)
    torch.cuda.synchronize()
    assert torch.equal(h, h0)
    assert bool((y[0, at] == BIT).all()) and not y[0, :at].any() and not y[0, at + 1:].any()


# (earlier token, later token) of one chunk of 64
PAIRS = [(0, 1), (2, 63), (15, 16), (64, 100)]


def pair(N, i, j):
    """Scores of token j with itself and with i: 1 + 2^-9 and 1 + 2^-9 + 2^-17."""
    a, b = torch.zeros(101, N), torch.zeros(101, N)
    a[j, [0, 7, N - 1]] = 1.0
    b[i, 0], b[i, 7], b[i, N - 1] = 1.0, 2.0 ** -9, BIT
    b[j, 0], b[j, 7] = 1.0, 2.0 ** -9
    to = lambda t: t.to(torch.bfloat16).cuda()[None, :, None].contiguous()
    return to(a), to(b)


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("i,j", PAIRS)
def test_scores(N, i, j):
    from state_space_sequence_amd import m3
    _, _, v, ld = tensors(101, N, 64)
    q, k = pair(N, i, j)
    v[0, i], v[0, j] = 1, -1
    y, _ = m3.linattn_fwd(q, k, v, ld, scale=1.0)
    torch.cuda.synchronize()
    assert bool((y[0, j] == BIT).all()), y[0, j]


@pytest.mark.parametrize("i,j", PAIRS)
def test_gradients(i, j):
    """dq of (dy, v, k) forwards, dk of (v, dy, q) and dv of (k, q, dy) backwards in time."""
    from state_space_sequence_amd import m3
    D = 64
    one = torch.zeros(1, 101, 1, D, dtype=torch.bfloat16, device="cuda")
    one[0, i], one[0, j] = 1, -1
    ld = torch.zeros(1, device="cuda")
    late, early = pair(D, i, j)  # forwards: token j meets i and itself
    g = m3.linattn_bwd(late, one, early, ld, late, scale=1.0)
    torch.cuda.synchronize()
    assert bool((g["q"][0, j] == BIT).all()), g["q"][0, j]
    # backwards token i meets j and itself
    flip = lambda t: torch.stack([t[0, j], t[0, i]]).clone()
    a, b = late.clone(), early.clone()
    a[0, [i, j]], b[0, [i, j]] = flip(late), flip(early)
    back = one.clone()
    back[0, i], back[0, j] = -1, 1
    g = m3.linattn_bwd(back, a, a, ld, b, scale=1.0)
    torch.cuda.synchronize()
    assert bool((g["k"][0, i] == BIT).all()), g["k"][0, i]
    g = m3.linattn_bwd(b, a, a, ld, back, scale=1.0)
    torch.cuda.synchronize()
    assert bool((g["v"][0, i] == BIT).all()), g["v"][0, i]
