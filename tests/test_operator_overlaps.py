"""A pointer given twice to the linear attention and group norm calls, where one of the two
is written, is refused on the host before any HIP call (no GPU needed), but for the pairs
that the headers allow."""
from __future__ import annotations

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "state_space_sequence_amd", "libm3.so")
WS = 0x40000000


@pytest.fixture(scope="module")
def m3():
    if not os.path.exists(LIB):
        from state_space_sequence_amd import build
        build.build()
    from state_space_sequence_amd import m3 as mod
    return mod


def filled(*structs):
    """Every pointer of the structs its own."""
    at = 0x100000
    for s in structs:
        for name, kind in s._fields_:
            if kind is ctypes.c_void_p:
                setattr(s, name, at)
                at += 0x1000
        if hasattr(s, "scale"):
            s.scale = 0.5
    return structs


def shared(structs, names):
    for s in structs:
        for name, kind in s._fields_:
            if name in names and kind is ctypes.c_void_p:
                setattr(s, name, 0x900000)


def linattn(m3, nsegments):
    return m3.make_shape(2, 4096, 4, 2, 64, 128, 1, 1, m3.M3_BF16, 0.0, 0, nsegments)


FWD_OUT, FWD_IN = ("y", "h_final"), ("q", "k", "v", "log_decay", "h0", "lengths")
BWD_OUT = ("dq", "dk", "dv", "dlog_decay", "dh0")
BWD_IN = ("q", "k", "v", "log_decay", "h0", "lengths", "dy", "dh_final")


@pytest.mark.parametrize("nsegments", [1, 4])
def test_linattn_fwd(m3, nsegments):
    s = linattn(m3, nsegments)
    n = m3.linattn_workspace_bytes(s)
    call = lambda io, ws=WS: m3.lib.m3_linattn_fwd(ctypes.byref(s), ctypes.byref(io), ws, n, None)
    for out in FWD_OUT:
        for other in FWD_IN + FWD_OUT:
            if other == out or (out, other) == ("h_final", "h0"):
                continue
            io, = filled(m3.LinattnIO())
            shared([io], (out, other))
            assert call(io) == -1, (out, other)
    if n:  # the workspace is written too
        for other in FWD_IN + FWD_OUT:
            io, = filled(m3.LinattnIO())
            assert call(io, getattr(io, other)) == -1, other


@pytest.mark.parametrize("nsegments", [1, 4])
def test_linattn_bwd(m3, nsegments):
    s = linattn(m3, nsegments)
    n = m3.linattn_bwd_workspace_bytes(s)
    call = lambda io, g, ws=WS: m3.lib.m3_linattn_bwd(ctypes.byref(s), ctypes.byref(io), ctypes.byref(g), ws, n, None)
    for out in BWD_OUT:
        for other in BWD_IN + BWD_OUT:
            if other != out:
                io, g = both = filled(m3.LinattnIO(), m3.LinattnGrads())
                shared(both, (out, other))
                assert call(io, g) == -1, (out, other)
    for other in BWD_IN + BWD_OUT:
        io, g = filled(m3.LinattnIO(), m3.LinattnGrads())
        assert call(io, g, getattr(g if hasattr(g, other) else io, other)) == -1, other


def test_linattn_step(m3):
    s = m3.make_shape(2, 1, 4, 2, 64, 128, 1, 1, m3.M3_BF16, 0.0)
    for out in ("h", "y"):
        for other in ("q", "k", "v", "log_decay", "h", "y"):
            if other != out:
                io, = filled(m3.LinattnStepIO())
                shared([io], (out, other))
                assert m3.lib.m3_linattn_step(ctypes.byref(s), ctypes.byref(io), None) == -1, (out, other)


def norm(m3, positions):
    return m3.NormShape(4, positions, 64, 4, m3.M3_BF16, 1, 1e-5, 0)


NORM_IN = ("x", "z", "weight", "bias", "lengths")
NORM_OUT = ("dx", "dz", "dweight", "dbias")


@pytest.mark.parametrize("positions", [1, 100])
def test_group_norm_fwd(m3, positions):
    s = norm(m3, positions)
    n = int(m3.lib.m3_group_norm_workspace_bytes(ctypes.byref(s), 1))
    call = lambda io, ws=WS: m3.lib.m3_group_norm_fwd(ctypes.byref(s), ctypes.byref(io), ws, n, None)
    for other in ("weight", "bias", "lengths"):
        io, = filled(m3.NormIO())
        shared([io], ("y", other))
        assert call(io) == -1, other
    for other in NORM_IN + ("y",):
        io, = filled(m3.NormIO())
        assert call(io, getattr(io, other)) == -1, other


@pytest.mark.parametrize("positions", [1, 100])
def test_group_norm_bwd(m3, positions):
    s = norm(m3, positions)
    n = int(m3.lib.m3_group_norm_bwd_workspace_bytes(ctypes.byref(s), 1))
    call = lambda io, g, ws=WS: m3.lib.m3_group_norm_bwd(ctypes.byref(s), ctypes.byref(io), ctypes.byref(g), ws, n, None)
    allowed = {("dx", "x"), ("dx", "dy"), ("dz", "z")}
    for out in NORM_OUT:
        for other in NORM_IN + ("dy",) + NORM_OUT:
            if other != out and (out, other) not in allowed:
                io, g = both = filled(m3.NormIO(), m3.NormGrads())
                shared(both, (out, other))
                assert call(io, g) == -1, (out, other)
    for other in NORM_IN + ("dy",) + NORM_OUT:
        io, g = filled(m3.NormIO(), m3.NormGrads())
        assert call(io, g, getattr(g if hasattr(g, other) else io, other)) == -1, other
