"""Host-side checks of the linear attention calls (no GPU needed): what the C ABI
refuses before any HIP call, and what the binding refuses before the library."""
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
    d = dict(batch=2, seqlen=100, nheads=4, ngroups=2, headdim=64, dstate=128, rank=1, chunk=1, io_dtype=m3.M3_BF16,
             eps=0.0, flags=0, nsegments=0)
    d.update(kw)
    return m3.make_shape(d["batch"], d["seqlen"], d["nheads"], d["ngroups"], d["headdim"], d["dstate"], d["rank"],
                         d["chunk"], d["io_dtype"], d["eps"], d["flags"], d["nsegments"])


OPTIONAL = ("h0", "lengths", "h_final", "dh_final", "dlog_decay", "dh0")


def fill(io, drop=None, misalign=None):
    for i, (name, kind) in enumerate(io._fields_):
        if kind is ctypes.c_void_p and name not in OPTIONAL and name != drop:
            setattr(io, name, 0x100000 + 0x1000 * i)
    if hasattr(io, "scale"):
        io.scale = 0.5
    if misalign:
        setattr(io, misalign, 0x900004)
    return io


def fwd(m3, s, io, ws=None, n=0):
    return m3.lib.m3_linattn_fwd(ctypes.byref(s), ctypes.byref(io), ws, n, None)


def bwd(m3, s, io, g, ws=None, n=0):
    return m3.lib.m3_linattn_bwd(ctypes.byref(s), ctypes.byref(io), ctypes.byref(g), ws, n, None)


def step(m3, s, io):
    return m3.lib.m3_linattn_step(ctypes.byref(s), ctypes.byref(io), None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(seqlen=-1), -1), (dict(nheads=0), -1), (dict(ngroups=3), -1), (dict(dstate=0), -1),
    (dict(headdim=0), -1), (dict(rank=0), -1), (dict(io_dtype=2), -1), (dict(nsegments=-1), -1), (dict(flags=1), -1),
    (dict(flags=2), -1), (dict(rank=2), -2), (dict(dstate=257), -2), (dict(headdim=257), -2),
    (dict(nheads=65538), -2), (dict(batch=1 << 31, nheads=4), -2), (dict(batch=1 << 20, seqlen=1 << 21), -2),
    (dict(seqlen=1 << 32), -2)])
def test_refused_shapes(m3, kw, code):
    s = shape(m3, **kw)
    io = fill(m3.LinattnIO())
    assert fwd(m3, s, io) == code
    assert bwd(m3, s, io, fill(m3.LinattnGrads())) == code
    assert m3.linattn_workspace_bytes(s) == 0 and m3.linattn_bwd_workspace_bytes(s) == 0
    if kw.get("flags") != 2 and "seqlen" not in kw and "nsegments" not in kw:
        assert step(m3, s, fill(m3.LinattnStepIO())) == code


def test_required_aligned_and_finite(m3):
    s = shape(m3)
    for name in ("q", "k", "v", "log_decay", "y"):
        assert fwd(m3, s, fill(m3.LinattnIO(), drop=name)) == -1, name
    for name in ("q", "k", "v", "log_decay", "h0", "lengths", "y", "h_final"):
        assert fwd(m3, s, fill(m3.LinattnIO(), misalign=name)) == -3, name
    for name in ("dy", "dq", "dk", "dv"):
        assert bwd(m3, s, fill(m3.LinattnIO()), fill(m3.LinattnGrads(), drop=name)) == -1, name
    for name in ("dy", "dh_final", "dq", "dk", "dv", "dlog_decay", "dh0"):
        assert bwd(m3, s, fill(m3.LinattnIO()), fill(m3.LinattnGrads(), misalign=name)) == -3, name
    for name in ("q", "k", "v", "log_decay", "h", "y"):
        assert step(m3, s, fill(m3.LinattnStepIO(), drop=name)) == -1, name
        assert step(m3, s, fill(m3.LinattnStepIO(), misalign=name)) == -3, name
    for bad in (float("nan"), float("inf")):
        io, st = fill(m3.LinattnIO()), fill(m3.LinattnStepIO())
        io.scale = st.scale = bad
        assert fwd(m3, s, io) == -1 and step(m3, s, st) == -1 and bwd(m3, s, io, fill(m3.LinattnGrads())) == -1
    assert m3.lib.m3_linattn_fwd(None, ctypes.byref(fill(m3.LinattnIO())), None, 0, None) == -1
    assert m3.lib.m3_linattn_fwd(ctypes.byref(s), None, None, 0, None) == -1
    assert m3.lib.m3_linattn_bwd(ctypes.byref(s), ctypes.byref(fill(m3.LinattnIO())), None, None, 0, None) == -1
    assert m3.lib.m3_linattn_step(ctypes.byref(s), None, None) == -1
    assert fwd(m3, shape(m3, batch=0), m3.LinattnIO()) == 0
    assert step(m3, shape(m3, batch=0), m3.LinattnStepIO()) == 0


def test_workspace(m3):
    one = shape(m3, nsegments=1)
    assert m3.linattn_workspace_bytes(one) == 0
    split = shape(m3, seqlen=4096, nsegments=4)
    need = m3.linattn_workspace_bytes(split)
    assert need == 2 * 4 * 4 * 64 * 128 * 4
    io = fill(m3.LinattnIO())
    assert fwd(m3, split, io) == -4 and fwd(m3, split, io, 0x200000, need - 1) == -4
    assert fwd(m3, split, io, 0x200008, need) == -3
    need = m3.linattn_bwd_workspace_bytes(split)
    assert bwd(m3, split, io, fill(m3.LinattnGrads()), 0x200000, need - 1) == -4
    # no more segments than chunks, and a long sequence on few chains is split by itself
    assert m3.linattn_workspace_bytes(shape(m3, seqlen=130, nsegments=1000)) == 2 * 4 * 3 * 64 * 128 * 4
    assert m3.linattn_workspace_bytes(shape(m3, seqlen=32768)) > 0


def test_outputs_that_are_inputs(m3):
    """A pointer given as an output and an input, or as two outputs, is refused (h_final may be h0)."""
    s = shape(m3, nsegments=1)
    for out, other in (("y", "q"), ("y", "v"), ("y", "h0"), ("h_final", "k"), ("y", "h_final")):
        io = fill(m3.LinattnIO())
        io.h0, io.h_final = 0x700000, 0x800000
        setattr(io, out, getattr(io, other))
        assert fwd(m3, s, io) == -1, (out, other)
    need = m3.linattn_bwd_workspace_bytes(s)
    for out, other in (("dq", "q"), ("dv", "v"), ("dq", "dy"), ("dk", "dv"), ("dh0", "dh_final"), ("dh0", "h0")):
        io, g = fill(m3.LinattnIO()), m3.LinattnGrads()
        io.h0 = 0x700000
        for i, name in enumerate(("dy", "dh_final", "dq", "dk", "dv", "dlog_decay", "dh0")):
            setattr(g, name, 0xa00000 + 0x1000 * i)
        setattr(g, out, getattr(g if hasattr(g, other) else io, other))
        assert bwd(m3, s, io, g, 0x200000, need) == -1, (out, other)
    for out, other in (("y", "q"), ("y", "v"), ("h", "k"), ("y", "h")):
        io = fill(m3.LinattnStepIO())
        setattr(io, out, getattr(io, other))
        assert step(m3, s, io) == -1, (out, other)


def test_sizes_whose_tensors_no_memory_holds(m3):
    s = shape(m3, batch=2, nheads=4096, ngroups=1, seqlen=1 << 31)
    assert fwd(m3, s, fill(m3.LinattnIO())) == -2
    assert m3.linattn_bwd_workspace_bytes(s) == 0


b, L, H, G, N, P = 2, 10, 4, 2, 32, 16


def tensors(io=torch.bfloat16):
    return dict(q=torch.zeros(b, L, H, N, dtype=io), k=torch.zeros(b, L, G, N, dtype=io),
                v=torch.zeros(b, L, G, P, dtype=io), log_decay=torch.zeros(H))


@pytest.fixture
def quiet(m3, monkeypatch):
    def boom(*a, **k):
        raise AssertionError("the library was called")
    for name in ("m3_linattn_fwd", "m3_linattn_bwd", "m3_linattn_step"):
        monkeypatch.setattr(m3.lib, name, boom)
    return m3


@pytest.mark.parametrize("key,bad", [
    ("q", lambda d: d["q"].half()), ("q", lambda d: d["q"][0]), ("k", lambda d: d["k"].float()),
    ("k", lambda d: d["k"][:, :, :1].contiguous()), ("v", lambda d: d["v"][:, 1:].contiguous()),
    ("log_decay", lambda d: d["log_decay"].double()), ("log_decay", lambda d: torch.zeros(H + 1)),
    ("log_decay", lambda d: None), ("h0", lambda d: torch.zeros(b, H, N, P)),
    ("lengths", lambda d: torch.zeros(b, dtype=torch.int64)), ("lengths", lambda d: torch.zeros(b + 1, dtype=torch.int32)),
    ("y", lambda d: torch.zeros(b, L, H, P)), ("h_final", lambda d: torch.zeros(b, H, P, N, dtype=torch.bfloat16)),
    ("workspace", lambda d: torch.zeros(4))])
def test_binding_refuses_a_mismatch(quiet, key, bad):
    d = tensors()
    value = bad(d)
    kw = {}
    if key in d:
        d[key] = value
    else:
        kw[key] = value
    with pytest.raises((TypeError, ValueError), match="io tensors" if key == "q" and value.dim() == 4 else key):
        quiet.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], **kw)


def test_binding_refuses_wrong_gradients_and_states(quiet):
    d = tensors()
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    dy = torch.zeros(b, L, H, P, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dy"):
        quiet.linattn_bwd(*args, None)
    with pytest.raises(TypeError, match="dy"):
        quiet.linattn_bwd(*args, dy.float())
    with pytest.raises(ValueError, match="unknown"):
        quiet.linattn_bwd(*args, dy, grads={"x": dy})
    with pytest.raises(ValueError, match="grads"):
        quiet.linattn_bwd(*args, dy, grads={"q": d["q"], "k": d["k"]})
    with pytest.raises(TypeError, match="grads"):
        quiet.linattn_bwd(*args, dy, grads={"q": d["q"].float(), "k": d["k"], "v": d["v"]})
    one = [t[:, 0].contiguous() for t in args[:3]]
    with pytest.raises(ValueError, match="h is required"):
        quiet.linattn_step(*one, d["log_decay"], None)
    with pytest.raises(TypeError, match="h"):
        quiet.linattn_step(*one, d["log_decay"], torch.zeros(b, H, P, N, dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        quiet.linattn_fwd(*args)
    with pytest.raises(ValueError, match="GPU"):
        quiet.linattn_step(*one, d["log_decay"], torch.zeros(b, H, P, N))
