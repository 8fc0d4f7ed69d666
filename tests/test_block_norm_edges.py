"""Edges of the block norm's sizes on the host (no GPU needed): every size that its header promises is accepted."""
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


@pytest.mark.parametrize("io,res", [(0, 0), (1, 0), (1, 1)])
@pytest.mark.parametrize("channels", [1, 2, 63, 64, 65, 129, 257, 513, 1025, 1281, 1537, 2049, 4097, 8192, 8193, 1 << 20])
def test_the_most_rows(m3, channels, io, res):
    """Without tensors the call is refused for them, not for its size."""
    most = (1 << 41) // max(channels, 64)
    if channels > 8192:
        most = min(most, 1 << 23)
    for rows in (most, most - 1, most // 2 + 1):
        s = m3.BlockNormShape(rows, channels, io, res, 1, 1e-5, 1.0, 3)
        io_, g = m3.BlockNormIO(), m3.BlockNormGrads()
        assert m3.lib.m3_block_norm_fwd(ctypes.byref(s), ctypes.byref(io_), None) == -1
        assert m3.lib.m3_block_norm_bwd(ctypes.byref(s), ctypes.byref(io_), ctypes.byref(g), None, 0, None) == -1
        assert m3.lib.m3_block_norm_bwd_workspace_bytes(ctypes.byref(s)) >= 12 * channels
