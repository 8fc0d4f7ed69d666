"""Edges of the linear attention calls on the host (no GPU needed): what a step does not use, and
tensors without keys."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "state_space_sequence_amd", "libm3.so")


@pytest.fixture(scope="module")
def m3():
    if not os.path.exists(LIB):
        from state_space_sequence_amd import build
        build.build()
    from state_space_sequence_amd import m3 as mod
    return mod


@pytest.mark.parametrize("seqlen,nsegments", [(-1, 0), (1, -1), (1 << 40, 7), (1 << 32, 0)])
def test_a_step_does_not_use_the_length(m3, seqlen, nsegments):
    """An empty batch is accepted whatever the two hold, and what is wrong otherwise is still refused."""
    s = m3.make_shape(0, seqlen, 4, 2, 64, 128, 1, 1, m3.M3_BF16, 0.0, 0, nsegments)
    io = m3.LinattnStepIO()
    io.scale = 0.5
    step = lambda: m3.lib.m3_linattn_step(ctypes.byref(s), ctypes.byref(io), None)
    assert step() == 0
    s.batch = 2
    assert step() == -1  # no tensors
    s.dstate = 257
    assert step() == -2


def test_no_keys(m3):
    """Tensors without a key dimension are refused like other sizes, not by the default scale's division."""
    b, L, H, G, P = 2, 10, 4, 2, 16
    q, k, v = torch.zeros(b, L, H, 0), torch.zeros(b, L, G, 0), torch.zeros(b, L, G, P)
    ld, dy = torch.zeros(H), torch.zeros(b, L, H, P)
    with pytest.raises(ValueError, match="q"):
        m3.linattn_fwd(q, k, v, ld)
    with pytest.raises(ValueError, match="q"):
        m3.linattn_bwd(q, k, v, ld, dy)
    with pytest.raises(ValueError, match="q"):
        m3.linattn_step(q[:, 0], k[:, 0], v[:, 0], ld, torch.zeros(b, H, P, 0))
