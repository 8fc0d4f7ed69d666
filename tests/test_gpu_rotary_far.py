"""Rotary positions far out and frequencies above 1: cosine and sine against angles reduced in whole numbers of 400 bits.

Bound: 2^-22 for each. The fraction of a turn reaches the fp32 functions whole (its rounding, at most 2^-26 of a turn, goes
in by the sums of angles); cosine and sine are off by at most two steps of 2^-24, that sum by 2^-48, and its rounding is
half a step: 2^-23 + 2^-25 in all. A head of (1, 0) pairs returns them as they are."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BITS = 400


def arctan_of_one_over(n):
    """arctan(1 / n) 2^BITS, by its series."""
    x = s = (1 << BITS) // n
    k = 1
    while x:
        x = -x // (n * n)
        k += 2
        s += x // k
    return s


TURN = 8 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239))  # 2 pi 2^BITS, by Machin's formula


def angle(pos, freq):
    """pos * freq less whole turns, in 64 bits, between -pi and pi."""
    n, d = float(freq).as_integer_ratio()  # (d is a power of 2)
    a = ((pos * n << BITS) // d) % TURN
    return (a - TURN if 2 * a > TURN else a) / (1 << BITS)


def check(oq, pos, freqs, layout, back):
    """oq [tokens, 1, 2 n] from pairs (1, 0)."""
    n = len(freqs)
    t = torch.tensor([[angle(p, f) for f in freqs] for p in pos], dtype=torch.float64)
    got = oq.double().cpu()[:, 0]
    c, s = (got[:, :n], got[:, n:]) if layout == "half" else (got[:, 0::2], got[:, 1::2])
    worst = max(float((c - t.cos()).abs().max()), float((s - (-t.sin() if back else t.sin())).abs().max()))
    print("  off by %.3f of 2^-22" % (worst * 2 ** 22), flush=True)
    assert worst <= 2.0 ** -22, (layout, worst)


def unit(tokens, n, layout):
    q = torch.zeros(tokens, 1, 2 * n)
    q[..., slice(0, n) if layout == "half" else slice(0, None, 2)] = 1
    return q.cuda()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
# frequencies: those of a model, of a long context's, between 0 and 1, above 1, far above
@pytest.mark.parametrize("which", ["base", "scaled", "below", "above", "far"])
def test_far_positions(which, layout):
    from state_space_sequence_amd import m3
    print("rotary far", which, layout, flush=True)
    gen = torch.Generator().manual_seed(5)
    n, tokens = 64, 48
    u = torch.rand(n, generator=gen)
    freqs = {"base": m3.rotary_frequencies(2 * n), "scaled": m3.rotary_frequencies(2 * n, 5e5, scaling="base", factor=8.0),
             "below": u, "above": 1 + 99 * u, "far": 2.0 ** (33 * u)}[which]
    freqs[0] = {"below": 0.8435195, "above": 100.0, "far": 2.0 ** 33}.get(which, freqs[0])
    pos = torch.randint(1 << 30, (1 << 31) - 1, (tokens,), generator=gen, dtype=torch.int64)
    pos[::5] = torch.randint(-(1 << 31), -(1 << 30), pos[::5].shape, generator=gen)
    pos[:4] = torch.tensor([(1 << 31) - 1, -(1 << 31), 2145487393, 1000000007])
    for back in (False, True):
        oq, _ = m3.rotary(unit(tokens, n, layout), None, freqs.cuda(), positions=pos.int().cuda(), layout=layout, backward=back)
        check(oq, pos.tolist(), freqs.tolist(), layout, back)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_offsets_that_pass_31_bits(layout):
    """Tokens behind an offset of the largest int32, and behind the smallest."""
    from state_space_sequence_amd import m3
    n, L = 32, 20
    freqs = m3.rotary_frequencies(2 * n)
    off = torch.tensor([(1 << 31) - 1, -(1 << 31)])
    q = unit(2 * L, n, layout).view(2, L, 1, 2 * n)
    oq, _ = m3.rotary(q, None, freqs.cuda(), offsets=off.int().cuda(), layout=layout)
    for row in range(2):
        check(oq[row], [int(off[row]) + t for t in range(L)], freqs.tolist(), layout, False)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_every_part_of_a_turn(layout):
    """Positions of one turn and around: fractions near 0, the eighths and the halves."""
    from state_space_sequence_amd import m3
    n, tokens = 4, 4096
    freqs = [2 * math.pi / 4096, 1.0, 2.0 ** -12, math.pi / 4]
    freqs = torch.tensor(freqs, dtype=torch.float32)
    pos = torch.arange(tokens)
    oq, _ = m3.rotary(unit(tokens, n, layout), None, freqs.cuda(), positions=pos.int().cuda(), layout=layout)
    check(oq, pos.tolist(), freqs.tolist(), layout, False)
