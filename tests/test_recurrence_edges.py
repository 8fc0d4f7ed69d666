"""Edges of the gated linear recurrence on the host (no GPU needed): what a step does not use."""
from __future__ import annotations

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "state_space_sequence_amd", "libm3.so")


@pytest.fixture(scope="module")
def m3():
    if not os.path.exists(LIB):
        from state_space_sequence_amd import build
        build.build()
    from state_space_sequence_amd import m3 as mod
    return mod


@pytest.mark.parametrize("seqlen", [-1, 0, (1 << 40) + 1, (1 << 63) - 1, -(1 << 63)])
def test_a_step_does_not_use_the_length(m3, seqlen):
    """An empty batch is accepted whatever it holds, and what is wrong otherwise is still refused."""
    s = m3.RecShape(0, seqlen, 24, m3.M3_BF16, 0)
    io = m3.RecStepIO()
    step = lambda: m3.lib.m3_recurrence_step(ctypes.byref(s), ctypes.byref(io), None)
    assert step() == 0
    s.batch = 2
    assert step() == -1  # no tensors
    s.batch = (1 << 31) + 1
    assert step() == -2
    s.batch, s.flags = 2, 2
    assert step() == -1
    assert m3.lib.m3_recurrence_step(None, ctypes.byref(io), None) == -1
