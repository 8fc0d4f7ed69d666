"""Workspace of the group norm's gradients (no GPU needed): it is bounded by the card and the tensors, not by the
number of rows or of positions that a workgroup takes at a time."""
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


@pytest.mark.parametrize("lengths", [0, 1])
@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("rows,positions,channels,groups", [
    (100000, 2, 8, 1), (100000, 4, 64, 1), (32768, 1, 4096, 1), (262144, 1, 4096, 1), (4096, 16, 64, 4), (8, 4096, 4096, 64),
    (2, 4000, 2048, 16), (512, 4096, 129, 43), (64, 16384, 8192, 64), (1, 1 << 24, 8, 1), (1 << 21, 1, 64, 1), (1, 1, 1, 1),
    (1 << 22, 3, 12, 4), (3, 1001, 1280, 32), (1, 100, 1 << 20, 1)])
def test_gradients(m3, rows, positions, channels, groups, io, lengths):
    s = m3.NormShape(rows, positions, channels, groups, io, 1, 1e-5, 0)
    need = int(m3.lib.m3_group_norm_bwd_workspace_bytes(ctypes.byref(s), lengths))
    x = rows * positions * channels * (2 if io else 4)
    # partial sums: 8 bytes a channel and workgroup, of at most 2048 channels and 2048 workgroups, or of 64 positions and
    # more each; 16 bytes a group and slice; the statistics of a row and group
    bound = (48 << 20) + x // 8 + 64 * rows * groups + 4096
    assert 0 < need <= bound, (need, bound, x)
