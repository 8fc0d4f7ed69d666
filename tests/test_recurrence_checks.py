"""Host-side checks of the gated linear recurrence (no GPU needed): what the C ABI refuses
before any HIP call, and what the binding refuses before the library."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

from tests.test_operator_overlaps import filled, shared

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "state_space_sequence_amd", "libm3.so")
BIG = (0x40000000, 1 << 40)


@pytest.fixture(scope="module")
def m3():
    if not os.path.exists(LIB):
        from state_space_sequence_amd import build
        build.build()
    from state_space_sequence_amd import m3 as mod
    return mod


def shape(m3, **kw):
    d = dict(batch=2, seqlen=1000, channels=64, io_dtype=m3.M3_BF16, flags=0)
    d.update(kw)
    return m3.RecShape(*(d[n] for n, _ in m3.RecShape._fields_))


def fwd(m3, s, io, ws=BIG):
    return m3.lib.m3_recurrence_fwd(ctypes.byref(s), io and ctypes.byref(io), *ws, None)


def bwd(m3, s, io, g, ws=BIG):
    return m3.lib.m3_recurrence_bwd(ctypes.byref(s), io and ctypes.byref(io), g and ctypes.byref(g), *ws, None)


def step(m3, s, io):
    return m3.lib.m3_recurrence_step(ctypes.byref(s), io and ctypes.byref(io), None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(seqlen=-1), -1), (dict(channels=0), -1), (dict(io_dtype=2), -1), (dict(flags=2), -1),
    (dict(channels=(1 << 20) + 1), -2), (dict(batch=1 << 32), -2),
    (dict(seqlen=1 << 41), -2), (dict(batch=1 << 20, seqlen=1 << 21), -2), (dict(batch=1 << 24), -2),
    (dict(batch=1 << 13, channels=1 << 17, seqlen=1 << 10), -2), (dict(seqlen=1 << 30, batch=1), -2)])
def test_refused_shapes(m3, kw, code):
    s = shape(m3, **kw)
    assert fwd(m3, s, *filled(m3.RecIO())) == code
    assert bwd(m3, s, *filled(m3.RecIO(), m3.RecGrads())) == code
    assert m3.recurrence_workspace_bytes(s) == 0
    assert m3.recurrence_bwd_workspace_bytes(s) == 0 and m3.recurrence_bwd_workspace_bytes(s, True) == 0


def test_required_aligned_and_workspace(m3):
    s = shape(m3)
    for name in ("x", "decay_gate", "log_decay", "y", "input_gate", "h0", "lengths", "h_final", "states"):
        io, = filled(m3.RecIO())
        setattr(io, name, None)
        if name in ("x", "decay_gate", "log_decay", "y"):
            assert fwd(m3, s, io) == -1, name
        setattr(io, name, 0x900004)
        assert fwd(m3, s, io) == -3, name
    for name in ("dy", "dx", "ddecay_gate", "dinput_gate"):
        io, g = filled(m3.RecIO(), m3.RecGrads())
        setattr(g, name, None)
        assert bwd(m3, s, io, g) == -1, name
    for name, _ in m3.RecGrads._fields_:
        io, g = filled(m3.RecIO(), m3.RecGrads())
        setattr(g, name, 0x900004)
        assert bwd(m3, s, io, g) == -3, name
    io, g = filled(m3.RecIO(), m3.RecGrads())
    io.input_gate = None  # a gate and its gradient go together
    assert bwd(m3, s, io, g) == -1
    for name in ("x", "decay_gate", "log_decay", "h", "y"):
        io, = filled(m3.RecStepIO())
        setattr(io, name, None)
        assert step(m3, s, io) == -1, name
        setattr(io, name, 0x900004)
        assert step(m3, s, io) == -3, name
    # workspace: too little, misaligned, missing
    need = m3.recurrence_workspace_bytes(s)
    io, g = filled(m3.RecIO(), m3.RecGrads())
    assert need > 0 and fwd(m3, s, io, (BIG[0], need - 1)) == -4 and fwd(m3, s, io, (None, need)) == -4
    assert fwd(m3, s, io, (BIG[0] + 8, need)) == -3
    with_states, without = m3.recurrence_bwd_workspace_bytes(s, True), m3.recurrence_bwd_workspace_bytes(s)
    assert 0 < with_states < without
    assert bwd(m3, s, io, g, (BIG[0], with_states - 1)) == -4
    io.states = None
    assert bwd(m3, s, io, g, (BIG[0], without - 1)) == -4
    assert m3.recurrence_workspace_bytes(shape(m3, seqlen=128)) == 0
    for f, a in ((fwd, (None,)), (bwd, (None, g)), (bwd, (io, None)), (step, (None,))):
        assert f(m3, s, *a) == -1
    assert m3.lib.m3_recurrence_fwd(None, ctypes.byref(io), *BIG, None) == -1
    assert fwd(m3, shape(m3, batch=0), m3.RecIO()) == 0 and step(m3, shape(m3, batch=0), m3.RecStepIO()) == 0


def test_workspace_is_bounded(m3):
    """The kept states, the segments' maps and the sums: a small part of the tensors."""
    for b, L, C in ((1, 1 << 20, 64), (8, 4096, 4096), (1, 1, 1 << 20), (64, 100, 1000), (1, 65536, 8)):
        s = shape(m3, batch=b, seqlen=L, channels=C)
        # maps and states of tiles of 128 tokens (64 with gradients), and what the chain starts from
        fwd = 12 * b * C * (L // 128 + 1) + 8 * b * C + 1024
        assert m3.recurrence_workspace_bytes(s) <= fwd
        # and kept states and sums of 64 tokens
        assert m3.recurrence_bwd_workspace_bytes(s) <= fwd + (4 + 12 + 4) * b * C * (L // 64 + 1) + 8 * b * C + 2048


IN = ("x", "decay_gate", "input_gate", "log_decay", "h0", "lengths")


@pytest.mark.parametrize("seqlen", [60, 1000])
def test_a_pointer_given_twice(m3, seqlen):
    s = shape(m3, seqlen=seqlen)
    for out in ("y", "h_final", "states"):
        for other in IN + ("y", "h_final", "states"):
            if other == out or (out, other) == ("h_final", "h0"):
                continue
            io, = filled(m3.RecIO())
            shared([io], (out, other))
            assert fwd(m3, s, io) == -1, (out, other)
    outs, ins = ("dx", "ddecay_gate", "dinput_gate", "dlog_decay", "dh0"), IN + ("states", "dy", "dh_final")
    for out in outs:
        for other in ins + outs:
            if other == out or (out, other) == ("dh0", "dh_final"):
                continue
            both = filled(m3.RecIO(), m3.RecGrads())
            shared(both, (out, other))
            assert bwd(m3, s, *both) == -1, (out, other)
    for other in IN + ("y", "h_final", "states"):
        io, = filled(m3.RecIO())
        if m3.recurrence_workspace_bytes(s):
            assert fwd(m3, s, io, (getattr(io, other), 1 << 40)) == -1, other
    for other in ins + outs:
        io, g = filled(m3.RecIO(), m3.RecGrads())
        assert bwd(m3, s, io, g, (getattr(g if hasattr(g, other) else io, other), 1 << 40)) == -1, other
    for out in ("h", "y"):
        for other in ("x", "decay_gate", "input_gate", "log_decay", "h", "y"):
            if other != out:
                io, = filled(m3.RecStepIO())
                shared([io], (out, other))
                assert step(m3, s, io) == -1, (out, other)


@pytest.fixture
def quiet(m3, monkeypatch):
    def boom(*a, **k):
        raise AssertionError("the library was called")
    for name in ("m3_recurrence_fwd", "m3_recurrence_bwd", "m3_recurrence_step"):
        monkeypatch.setattr(m3.lib, name, boom)
    return m3


X, LD = torch.zeros(2, 70, 24), torch.zeros(24)


@pytest.mark.parametrize("kw,match", [
    (dict(x=None), "x"), (dict(x=X[0]), "x"), (dict(x=X.half()), "io tensors"), (dict(x=torch.zeros(2, 3, 0)), "channels"),
    (dict(decay_gate=None), "decay_gate"), (dict(decay_gate=X.bfloat16()), "decay_gate"), (dict(decay_gate=X[:, :5]), "decay_gate"),
    (dict(decay_gate=torch.zeros(2, 24, 70).transpose(1, 2)), "contiguous"), (dict(log_decay=None), "log_decay"),
    (dict(log_decay=LD.double()), "log_decay"), (dict(log_decay=torch.zeros(23)), "log_decay"),
    (dict(input_gate=X[:1]), "input_gate"), (dict(h0=torch.zeros(2, 23)), "h0"), (dict(h0=torch.zeros(2, 24).bfloat16()), "h0"),
    (dict(lengths=torch.zeros(2)), "lengths"), (dict(lengths=torch.zeros(3, dtype=torch.int32)), "lengths"),
    (dict(states=torch.zeros(2, 1, 24)), "states"), (dict(workspace=torch.zeros(8)), "workspace"), (dict(), "GPU")])
def test_binding_refuses(quiet, kw, match):
    kw = dict(kw)
    a = [kw.pop(n, d) for n, d in (("x", X), ("decay_gate", X), ("log_decay", LD))]
    with pytest.raises((TypeError, ValueError), match=match):
        quiet.recurrence_fwd(*a, **kw)
    with pytest.raises((TypeError, ValueError), match=match):
        quiet.recurrence_bwd(*a, X, **kw)


def test_binding_refuses_outputs_and_gradients(quiet):
    f, b = (lambda **k: quiet.recurrence_fwd(X, X, LD, **k)), (lambda **k: quiet.recurrence_bwd(X, X, LD, X, **k))
    for kw in (dict(y=X.bfloat16()), dict(y=X[:, :3]), dict(h_final=torch.zeros(24))):
        with pytest.raises((TypeError, ValueError), match="y|h_final"):
            f(**kw)
    with pytest.raises(ValueError, match="dy"):
        quiet.recurrence_bwd(X, X, LD, None)
    with pytest.raises(ValueError, match="unknown"):
        b(grads={"x": X, "decay_gate": X, "input_gate": X})
    with pytest.raises(ValueError, match="required"):
        b(grads={"x": X})
    with pytest.raises(ValueError, match="required"):
        b(input_gate=X, grads={"x": X, "decay_gate": X})
    with pytest.raises(ValueError, match="grads"):
        b(grads={"x": X, "decay_gate": X, "h0": X})
    T, h = torch.zeros(2, 24), torch.zeros(2, 24)
    for a, kw, match in (((X, X, LD, h), {}, "x"), ((T, None, LD, h), {}, "decay_gate"), ((T, T, None, h), {}, "log_decay"),
                         ((T, T, LD, None), {}, "h"), ((T, T, LD, h.bfloat16()), {}, "h"), ((T, T, LD, h), dict(y=h[:1]), "y"),
                         ((T, T, LD, h), dict(input_gate=X), "input_gate"), ((T, T, LD, h), {}, "GPU")):
        with pytest.raises((TypeError, ValueError), match=match):
            quiet.recurrence_step(*a, **kw)
