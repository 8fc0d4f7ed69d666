"""Host-side checks of the group norm calls (no GPU needed): what the C ABI refuses
before any HIP call, and what the binding refuses before the library."""
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


def shape(m3, **kw):
    d = dict(rows=4, positions=1, channels=64, groups=4, io_dtype=m3.M3_BF16, activation=1, eps=1e-5, flags=0)
    d.update(kw)
    return m3.NormShape(*(d[n] for n, _ in m3.NormShape._fields_))


def fill(io, skip=("z", "weight", "bias", "lengths", "dz", "dweight", "dbias"), drop=None, misalign=None):
    for i, (name, _) in enumerate(io._fields_):
        if name not in skip and name != drop:
            setattr(io, name, 0x100000 + 0x1000 * i)
    if misalign:
        setattr(io, misalign, 0x900004)
    return io


def fwd(m3, s, io, ws=None, n=0):
    return m3.lib.m3_group_norm_fwd(ctypes.byref(s), ctypes.byref(io), ws, n, None)


def bwd(m3, s, io, g, ws=None, n=0):
    return m3.lib.m3_group_norm_bwd(ctypes.byref(s), ctypes.byref(io), ctypes.byref(g), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(positions=-1), -1), (dict(channels=0), -1), (dict(groups=0), -1), (dict(groups=5), -1),
    (dict(io_dtype=2), -1), (dict(activation=2), -1), (dict(activation=-1), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(flags=1), -1),
    (dict(channels=1 << 21, groups=1), -2), (dict(rows=1 << 32), -2), (dict(rows=1 << 20, positions=1 << 21), -2),
    (dict(rows=1 << 24, positions=2, groups=64), -2)])
def test_refused_shapes(m3, kw, code):
    s = shape(m3, **kw)
    assert fwd(m3, s, fill(m3.NormIO())) == code
    assert bwd(m3, s, fill(m3.NormIO()), fill(m3.NormGrads())) == code
    assert m3.lib.m3_group_norm_workspace_bytes(ctypes.byref(s), 0) == 0
    assert m3.lib.m3_group_norm_bwd_workspace_bytes(ctypes.byref(s), 0) == 0


def test_required_aligned_and_workspace(m3):
    s = shape(m3)
    big = (0x40000000, 1 << 30)
    for name in ("x", "y"):
        assert fwd(m3, s, fill(m3.NormIO(), drop=name)) == -1, name
    for name in ("x", "z", "weight", "bias", "lengths", "y"):
        assert fwd(m3, s, fill(m3.NormIO(), misalign=name)) == -3, name
    for name in ("dy", "dx"):
        assert bwd(m3, s, fill(m3.NormIO()), fill(m3.NormGrads(), drop=name), *big) == -1, name
    for name in ("dy", "dx", "dweight", "dbias"):
        assert bwd(m3, s, fill(m3.NormIO()), fill(m3.NormGrads(), misalign=name), *big) == -3, name
    # a gate and its gradient go together
    gate = fill(m3.NormIO(), skip=("weight", "bias", "lengths"))
    assert bwd(m3, s, gate, fill(m3.NormGrads()), *big) == -1
    assert bwd(m3, s, fill(m3.NormIO()), fill(m3.NormGrads(), skip=("dweight", "dbias")), *big) == -1
    # a token's norm needs no workspace forwards; its gradients and a sequence's norm do
    size = lambda f, sh, n: int(getattr(m3.lib, f)(ctypes.byref(sh), n))
    assert size("m3_group_norm_workspace_bytes", s, 0) == 0
    assert size("m3_group_norm_workspace_bytes", s, 1) > 0
    need = size("m3_group_norm_bwd_workspace_bytes", s, 0)
    assert need > 0 and bwd(m3, s, fill(m3.NormIO()), fill(m3.NormGrads()), 0x40000000, need - 1) == -4
    seq = shape(m3, positions=100)
    need = size("m3_group_norm_workspace_bytes", seq, 0)
    assert need > 0 and fwd(m3, seq, fill(m3.NormIO())) == -4 and fwd(m3, seq, fill(m3.NormIO()), 0x40000008, need) == -3
    assert fwd(m3, seq, fill(m3.NormIO()), 0x40000000, need - 1) == -4
    assert m3.lib.m3_group_norm_fwd(None, ctypes.byref(fill(m3.NormIO())), None, 0, None) == -1
    assert m3.lib.m3_group_norm_fwd(ctypes.byref(s), None, None, 0, None) == -1
    assert m3.lib.m3_group_norm_bwd(ctypes.byref(s), ctypes.byref(fill(m3.NormIO())), None, None, 0, None) == -1
    assert fwd(m3, shape(m3, rows=0), m3.NormIO()) == 0


@pytest.fixture
def quiet(m3, monkeypatch):
    def boom(*a, **k):
        raise AssertionError("the library was called")
    for name in ("m3_group_norm_fwd", "m3_group_norm_bwd"):
        monkeypatch.setattr(m3.lib, name, boom)
    return m3


X = torch.zeros(2, 5, 24)


@pytest.mark.parametrize("kw,match", [
    (dict(groups=5), "groups"), (dict(groups=0), "groups"), (dict(groups=True), "groups"), (dict(groups=2.0), "groups"),
    (dict(x=torch.zeros(24)), "x"), (dict(x=X.half()), "io tensors"), (dict(x=None), "x"), (dict(activation="gelu"), "activation"),
    (dict(over="batch"), "over"), (dict(x=torch.zeros(5, 24), over="sequence"), "x"),
    (dict(lengths=torch.zeros(2, dtype=torch.int32)), "lengths"),
    (dict(over="sequence", lengths=torch.zeros(2, dtype=torch.int64)), "lengths"),
    (dict(over="sequence", lengths=torch.zeros(5, dtype=torch.int32)), "lengths"),
    (dict(z=X.bfloat16()), "z"), (dict(z=X[:1]), "z"), (dict(weight=torch.zeros(5)), "weight"),
    (dict(bias=torch.zeros(24, dtype=torch.bfloat16)), "bias"), (dict(y=X.bfloat16()), "y"),
    (dict(workspace=torch.zeros(8)), "workspace"), (dict(), "GPU")])
def test_binding_refuses(quiet, kw, match):
    kw = dict(kw)
    x, groups = kw.pop("x", X), kw.pop("groups", 4)
    with pytest.raises((TypeError, ValueError), match=match):
        quiet.group_norm_fwd(x, groups, **kw)


def test_binding_refuses_wrong_gradients(quiet):
    with pytest.raises(ValueError, match="dy"):
        quiet.group_norm_bwd(X, 4, None)
    with pytest.raises(TypeError, match="dy"):
        quiet.group_norm_bwd(X, 4, X.bfloat16())
    with pytest.raises(ValueError, match="unknown"):
        quiet.group_norm_bwd(X, 4, X, grads={"x": X, "z": X})
    with pytest.raises(ValueError, match="required"):
        quiet.group_norm_bwd(X, 4, X, z=X, grads={"x": X})
    with pytest.raises(ValueError, match="grads"):
        quiet.group_norm_bwd(X, 4, X, grads={"x": X, "weight": torch.zeros(5)})
