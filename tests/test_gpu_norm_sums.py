"""The group norm's weight gradients over many rows, and its sums over long sequences.

Equal terms are the worst case of a sum: every addition of a binade is off the same way. A thread adds
at most 256 rows or positions in fp32, n / 2 2^-24 of the sum for equal terms = 128 2^-24; the joining of
a workgroup's threads (8 additions at most), the terms themselves (xh and du: a dozen roundings) and the
result's rounding leave it below 160 2^-24. What lies beyond is summed in 64 bits."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

F = 160 * 2.0 ** -24
EPS = 1e-5


def near(name, got, want):
    off = float(((got.double() - want) / want).abs().max())
    print("  %s: %.1f * 2^-24" % (name, off * 2 ** 24), flush=True)
    assert off <= F, (name, off)


def test_tokens_of_many_rows():
    """2^21 rows of 129 groups of two channels: 1 and -1, dy 0.1."""
    from state_space_sequence_amd import m3
    rows, G = 1 << 21, 129
    x = torch.tensor([1.0, -1.0], device="cuda").repeat(G).expand(rows, 2 * G).contiguous()
    dy = torch.full_like(x, 0.1)
    w = torch.ones(2 * G, device="cuda")
    g = m3.group_norm_bwd(x, G, dy, w, w, activation="none", eps=EPS)
    torch.cuda.synchronize()
    d = float(torch.tensor(0.1))
    near("bias", g["bias"], torch.full((2 * G,), rows * d, dtype=torch.float64, device="cuda"))
    near("weight", g["weight"], rows * d / (1 + EPS) ** 0.5 * x[0].double())


@pytest.mark.parametrize("ragged", [False, True])
def test_many_long_sequences(ragged):
    """512 rows of 4096 positions of 43 groups of three channels: 1, -1 and 0, dy 0.1."""
    from state_space_sequence_amd import m3
    rows, S, G = 512, 4096, 43
    x = torch.tensor([1.0, -1.0, 0.0], device="cuda").repeat(G).expand(rows, S, 3 * G).contiguous()
    dy = torch.full_like(x, 0.1)
    w = torch.ones(3 * G, device="cuda")
    lengths = torch.arange(S, S - rows, -1, dtype=torch.int32, device="cuda") if ragged else None
    g = m3.group_norm_bwd(x, G, dy, w, w, activation="none", eps=EPS, over="sequence", lengths=lengths)
    torch.cuda.synchronize()
    n = int(lengths.sum()) if ragged else rows * S
    d = float(torch.tensor(0.1))
    near("bias", g["bias"], torch.full((3 * G,), n * d, dtype=torch.float64, device="cuda"))
    live = x[0, 0] != 0
    near("weight", g["weight"][live], (n * d / (2.0 / 3 + EPS) ** 0.5 * x[0, 0].double())[live])
