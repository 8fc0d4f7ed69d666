"""Host-side checks of the norms around a block (no GPU needed): what the C ABI refuses
before any HIP call, and what the binding refuses before the library."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

from tests.test_operator_overlaps import shared

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "state_space_sequence_amd", "libm3.so")
BIG = (0x40000000, 1 << 40)


def filled(*structs):
    """Every pointer of the structs its own."""
    at = 0x100000
    for s in structs:
        for name, _ in s._fields_:
            setattr(s, name, at)
            at += 0x1000
    return structs


@pytest.fixture(scope="module")
def m3():
    if not os.path.exists(LIB):
        from state_space_sequence_amd import build
        build.build()
    from state_space_sequence_amd import m3 as mod
    return mod


def shape(m3, **kw):
    d = dict(rows=40, channels=64, io_dtype=m3.M3_BF16, residual_dtype=m3.M3_F32, activation=1, eps=1e-5, residual_scale=1.0,
             flags=3)
    d.update(kw)
    return m3.BlockNormShape(*(d[n] for n, _ in m3.BlockNormShape._fields_))


def fwd(m3, s, io):
    return m3.lib.m3_block_norm_fwd(ctypes.byref(s), io and ctypes.byref(io), None)


def bwd(m3, s, io, g, ws=BIG):
    return m3.lib.m3_block_norm_bwd(ctypes.byref(s), io and ctypes.byref(io), g and ctypes.byref(g), *ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(channels=0), -1), (dict(io_dtype=2), -1), (dict(residual_dtype=2), -1),
    (dict(io_dtype=0, residual_dtype=1), -1), (dict(activation=3), -1), (dict(activation=-1), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(residual_scale=float("inf")), -1), (dict(residual_scale=float("nan")), -1),
    (dict(flags=4), -1), (dict(rows=(1 << 40) + 1), -2), (dict(channels=(1 << 20) + 1), -2),
    (dict(rows=1 << 39), -2), (dict(rows=1 << 30, channels=1 << 15), -2), (dict(rows=1 << 25, channels=8193), -2)])
def test_refused_shapes(m3, kw, code):
    s = shape(m3, **kw)
    assert fwd(m3, s, *filled(m3.BlockNormIO())) == code
    assert bwd(m3, s, *filled(m3.BlockNormIO(), m3.BlockNormGrads())) == code
    assert m3.lib.m3_block_norm_bwd_workspace_bytes(ctypes.byref(s)) == 0


def test_required_aligned_and_workspace(m3):
    s = shape(m3)
    for name, _ in m3.BlockNormIO._fields_:
        io, = filled(m3.BlockNormIO())
        setattr(io, name, None)
        if name in ("x", "y"):
            assert fwd(m3, s, io) == -1, name
        setattr(io, name, 0x900004)
        assert fwd(m3, s, io) == -3, name
    for name, _ in m3.BlockNormGrads._fields_:
        io, g = filled(m3.BlockNormIO(), m3.BlockNormGrads())
        setattr(g, name, None)
        if name in ("dy", "dx", "dz"):
            assert bwd(m3, s, io, g) == -1, name
        setattr(g, name, 0x900004)
        assert bwd(m3, s, io, g) == -3, name
    io, = filled(m3.BlockNormIO())
    io.y = io.pre_weight = io.residual_out = None  # nothing to write
    assert fwd(m3, shape(m3, flags=1), io) == -1
    io, g = filled(m3.BlockNormIO(), m3.BlockNormGrads())
    io.z = None  # a gate and its gradient go together
    assert bwd(m3, s, io, g) == -1
    # what belongs to a norm that the call does not have
    for flags, names in ((1, ("pre_weight", "y")), (2, ("post_weight",))):
        for name in names:
            io, = filled(m3.BlockNormIO())
            for other in ("pre_weight", "post_weight", "y"):
                if other != name and not (other == "y" and flags == 2):
                    setattr(io, other, None)
            assert fwd(m3, shape(m3, flags=flags), io) == -1, (flags, name)
    for flags, names in ((1, ("dpre_weight", "dy")), (2, ("dpost_weight",))):
        for name in names:
            io, g = filled(m3.BlockNormIO(), m3.BlockNormGrads())
            io.pre_weight = io.post_weight = None
            for other in ("dpre_weight", "dpost_weight", "dy"):
                if other != name and not (other == "dy" and flags == 2):
                    setattr(g, other, None)
            assert bwd(m3, shape(m3, flags=flags), io, g) == -1, (flags, name)
    io, g = filled(m3.BlockNormIO(), m3.BlockNormGrads())
    io.pre_weight = g.dpre_weight = g.dy = g.dresidual_out = None
    assert bwd(m3, shape(m3, flags=1), io, g) == -1  # no gradient comes in
    need = int(m3.lib.m3_block_norm_bwd_workspace_bytes(ctypes.byref(s)))
    io, g = filled(m3.BlockNormIO(), m3.BlockNormGrads())
    assert need > 0 and bwd(m3, s, io, g, (BIG[0], need - 1)) == -4 and bwd(m3, s, io, g, (None, need)) == -4
    assert bwd(m3, s, io, g, (BIG[0] + 4, need)) == -3
    assert fwd(m3, s, None) == -1 and bwd(m3, s, None, g) == -1 and bwd(m3, s, io, None) == -1
    assert m3.lib.m3_block_norm_fwd(None, ctypes.byref(io), None) == -1
    assert fwd(m3, shape(m3, rows=0), m3.BlockNormIO()) == 0


def test_workspace_is_bounded(m3):
    for rows, C in ((1, 1), (100, 4096), (32768, 2048), (10_000_000, 64), (1 << 20, 16384), (100, 1 << 20)):
        for res in (0, 1):
            s = shape(m3, rows=rows, channels=C, residual_dtype=res)
            assert int(m3.lib.m3_block_norm_bwd_workspace_bytes(ctypes.byref(s))) <= 12 * C * (768 + rows // 256 + 1) + 16 * rows + 256


IN = ("x", "z", "residual", "post_weight", "pre_weight", "scale")


def test_a_pointer_given_twice(m3):
    s = shape(m3)
    allowed = {("residual_out", "residual"), ("y", "x"), ("y", "z")}
    for out in ("residual_out", "y"):
        for other in IN + ("residual_out", "y"):
            if other != out and (out, other) not in allowed:
                io, = filled(m3.BlockNormIO())
                shared([io], (out, other))
                assert fwd(m3, s, io) == -1, (out, other)
    outs = ("dx", "dz", "dresidual", "dpost_weight", "dpre_weight", "dscale")
    ins = ("x", "z", "post_weight", "pre_weight", "scale", "residual_out", "dy", "dresidual_out")
    allowed = {("dx", "x"), ("dx", "dy"), ("dz", "z"), ("dresidual", "dresidual_out")}
    for out in outs:
        for other in ins + outs:
            if other != out and (out, other) not in allowed:
                both = filled(m3.BlockNormIO(), m3.BlockNormGrads())
                shared(both, (out, other))
                assert bwd(m3, s, *both) == -1, (out, other)
    for other in ins + outs:
        io, g = filled(m3.BlockNormIO(), m3.BlockNormGrads())
        assert bwd(m3, s, io, g, (getattr(g if hasattr(g, other) else io, other), 1 << 40)) == -1, other


@pytest.fixture
def quiet(m3, monkeypatch):
    def boom(*a, **k):
        raise AssertionError("the library was called")
    for name in ("m3_block_norm_fwd", "m3_block_norm_bwd"):
        monkeypatch.setattr(m3.lib, name, boom)
    return m3


X, W = torch.zeros(2, 5, 24), torch.zeros(24)


@pytest.mark.parametrize("kw,match", [
    (dict(x=None), "x"), (dict(x=X.half()), "io tensors"), (dict(x=torch.zeros(2, 0)), "channels"),
    (dict(x=X.bfloat16()[..., ::2]), "contiguous|residual"), (dict(residual=X.half()), "residual"), (dict(residual=X.bfloat16()), "residual"),
    (dict(residual=X[:1]), "residual"), (dict(z=X.bfloat16()), "z"), (dict(z=X[0]), "z"), (dict(activation="gelu"), "activation"),
    (dict(scale=torch.zeros(23)), "scale"), (dict(scale=W.bfloat16()), "scale"), (dict(post_weight=W), "post_weight"),
    (dict(pre_norm=False, pre_weight=W), "pre_weight"), (dict(post_norm=True, post_weight=W.double()), "post_weight"),
    (dict(pre_weight=torch.zeros(24, 1)), "pre_weight"), (dict(), "GPU")])
def test_binding_refuses(quiet, kw, match):
    kw = dict(kw)
    x, r = kw.pop("x", X), kw.pop("residual", X)
    with pytest.raises((TypeError, ValueError), match=match):
        quiet.block_norm_fwd(x, r, **kw)
    with pytest.raises((TypeError, ValueError), match=match):
        quiet.block_norm_bwd(x, r, X if kw.get("pre_norm", True) else None, X, **kw)


def test_binding_refuses_outputs_and_gradients(quiet):
    m3 = quiet
    with pytest.raises(ValueError, match="y"):
        m3.block_norm_fwd(X, X, pre_norm=False, y=X)
    with pytest.raises(TypeError, match="y"):
        m3.block_norm_fwd(X, X, y=X.bfloat16())
    with pytest.raises(TypeError, match="residual_out"):
        m3.block_norm_fwd(X, X, residual_out=X.bfloat16())
    with pytest.raises(TypeError, match="residual"):
        m3.block_norm_fwd(X, None, residual_dtype=torch.bfloat16)
    b = lambda *a, **k: m3.block_norm_bwd(X, X, *a, **k)
    for a, kw, match in (((None,), {}, "dy"), ((X.bfloat16(),), {}, "dy"), ((X, X.bfloat16()), {}, "dresidual_out"),
                         ((X, X), dict(pre_norm=False), "dy"), ((None, None), dict(pre_norm=False), "dresidual_out"),
                         ((X,), dict(grads={"x": X, "z": X}), "unknown"), ((X,), dict(grads={"x": X, "scale": W}), "unknown"),
                         ((X,), dict(grads={}), "required"), ((X,), dict(z=X, grads={"x": X}), "required"),
                         ((X,), dict(grads={"x": X, "residual": X.bfloat16()}), "grads"),
                         ((X,), dict(workspace=torch.zeros(8)), "workspace")):
        with pytest.raises((TypeError, ValueError), match=match):
            b(*a, **kw)
