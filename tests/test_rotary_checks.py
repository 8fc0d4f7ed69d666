"""Host-side checks of rotary positions (no GPU needed): what the C ABI refuses
before any HIP call, and what the binding refuses before the library."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

from tests.test_operator_overlaps import filled, shared

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "state_space_sequence_amd", "libm3.so")


@pytest.fixture(scope="module")
def m3():
    if not os.path.exists(LIB):
        from state_space_sequence_amd import build
        build.build()
    from state_space_sequence_amd import m3 as mod
    return mod


def shape(m3, **kw):
    d = dict(batch=2, seqlen=10, nheads=4, ngroups=2, headdim=64, rotary=32, io_dtype=m3.M3_BF16, flags=0, scale=1.0, reserved=0)
    d.update(kw)
    return m3.RotaryShape(*(d[n] for n, _ in m3.RotaryShape._fields_))


def full(m3, **kw):
    io, = filled(m3.RotaryIO())
    io.offsets = None
    for n, v in kw.items():
        setattr(io, n, v)
    return io


def call(m3, s, io):
    return m3.lib.m3_rotary(ctypes.byref(s), io and ctypes.byref(io), None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(seqlen=-1), -1), (dict(nheads=0), -1), (dict(ngroups=0), -1), (dict(headdim=0), -1),
    (dict(rotary=-2), -1), (dict(rotary=3), -1), (dict(rotary=66), -1), (dict(io_dtype=2), -1), (dict(flags=4), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(reserved=1), -1), (dict(headdim=1025), -2),
    (dict(nheads=4097), -2), (dict(ngroups=4097), -2), (dict(batch=1 << 40), -2), (dict(seqlen=1 << 40), -2),
    (dict(batch=1 << 20, seqlen=1 << 20), -2), (dict(batch=1 << 62, seqlen=1 << 62), -2)])
def test_refused_shapes(m3, kw, code):
    assert call(m3, shape(m3, **kw), full(m3)) == code


def test_required_and_aligned(m3):
    s = shape(m3)
    for name in ("q", "freqs", "q_out", "k", "k_out"):
        assert call(m3, s, full(m3, **{name: None})) == -1, name
    for name, _ in m3.RotaryIO._fields_:
        assert call(m3, s, full(m3, **({"positions": None} if name == "offsets" else {}), **{name: 0x900004})) == -3, name
    assert call(m3, s, full(m3, offsets=0x800000)) == -1  # positions and offsets
    assert call(m3, s, None) == -1 and m3.lib.m3_rotary(None, ctypes.byref(full(m3)), None) == -1
    assert call(m3, shape(m3, batch=0), m3.RotaryIO()) == 0
    # without keys their number of heads is not looked at
    assert call(m3, shape(m3, batch=0, ngroups=0), m3.RotaryIO()) == 0


def test_a_pointer_given_twice(m3):
    s = shape(m3)
    for out in ("q_out", "k_out"):
        for other, _ in m3.RotaryIO._fields_:
            if other == out or (out[0] == other[0] and other in "qk"):
                continue
            io = full(m3, **({"positions": None, "offsets": 0x700000} if other == "offsets" else {}))
            shared([io], (out, other))
            assert call(m3, s, io) == -1, (out, other)


@pytest.fixture
def quiet(m3, monkeypatch):
    def boom(*a, **k):
        raise AssertionError("the library was called")
    monkeypatch.setattr(m3.lib, "m3_rotary", boom)
    return m3


Q, K, F = torch.zeros(2, 5, 4, 16), torch.zeros(2, 5, 2, 16), torch.zeros(8)
I32 = torch.int32


@pytest.mark.parametrize("kw,match", [
    (dict(q=None), "q"), (dict(q=Q[0, 0]), "q"), (dict(q=Q.half()), "io tensors"), (dict(q=torch.zeros(2, 5, 0, 16)), "q"),
    (dict(q=Q.transpose(1, 2)), "q|k"), (dict(k=K.bfloat16()), "k"), (dict(k=K[:, 0]), "k"), (dict(k=K[..., :8]), "k"),
    (dict(k=K[:, :, :0]), "k"), (dict(freqs=None), "freqs"), (dict(freqs=torch.zeros(9)), "freqs"), (dict(freqs=F.double()), "freqs"),
    (dict(freqs=torch.zeros(2, 4)), "freqs"), (dict(layout="pairs"), "layout"), (dict(positions=torch.zeros(2, 5)), "positions"),
    (dict(positions=torch.zeros(2, dtype=I32)), "positions"), (dict(offsets=torch.zeros(5, dtype=I32)), "offsets"),
    (dict(offsets=torch.zeros(2, dtype=torch.int64)), "offsets"),
    (dict(offsets=torch.zeros(2, dtype=I32), positions=torch.zeros(2, 5, dtype=I32)), "both"), (dict(q_out=Q.bfloat16()), "q_out"),
    (dict(k_out=Q), "k_out"), (dict(k=None, k_out=K), "k_out"), (dict(), "GPU")])
def test_binding_refuses(quiet, kw, match):
    kw = dict(kw)
    a = [kw.pop(n, d) for n, d in (("q", Q), ("k", K), ("freqs", F))]
    with pytest.raises((TypeError, ValueError), match=match):
        quiet.rotary(*a, **kw)


@pytest.mark.parametrize("a,kw", [((3,), {}), ((-2,), {}), ((2.0,), {}), ((True,), {}), ((8,), dict(scaling="more")), ((8,), dict(base=0.0)),
                                  ((8,), dict(factor=0.0)), ((2,), dict(scaling="base")), ((8,), dict(scaling="parts")),
                                  ((8,), dict(scaling="parts", trained_length=64, fast=1.0, slow=1.0))])
def test_frequencies_refuse(m3, a, kw):
    with pytest.raises(ValueError):
        m3.rotary_frequencies(*a, **kw)
