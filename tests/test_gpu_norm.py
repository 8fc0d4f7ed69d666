"""GPU parity of the group norm with an activation (m3_group_norm_fwd, _bwd) with its
definition in 64 bits on the CPU.

Bounds, elementwise. fp32 arithmetic: the mean and the variance are sums of n terms whose
roundings are at most log2-many on any path plus the 32 values that one lane adds in a row, so a normalised value is
off by at most 64 * 2^-24 of (|x - mean| + max|x|) / std; F below is that with the activation's
exponential (|u| 2^-24 relative, |u| <= 32 here) and a dozen roundings more. Outputs
stored in bf16 are rounded by at most 2^-8 of themselves; the fast exponential of bf16
calls adds the same |u| 2^-24. Sums over rows are held in fp32 within a thread (at most 4096 rows) and in
64 bits beyond, of terms that are off as above."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F = 160 * 2.0 ** -24


def reference(x, G, w, b, z, act, over, lengths, eps, dy=None):
    """Outputs and, for each, the size that the fp32 bound is relative to."""
    x, w, b, z, dy = (None if t is None else t.double().cpu() for t in (x, w, b, z, dy))
    C = x.shape[-1]
    if over == "token":
        xs = x.reshape(-1, 1, C)
    else:
        xs = x.reshape(x.shape[0], -1, C)
    like = lambda t: None if t is None else t.reshape(xs.shape)
    z, dy = like(z), like(dy)
    w = torch.ones(C).double() if w is None else w
    b = torch.zeros(C).double() if b is None else b
    y, dx, dz = torch.zeros_like(xs), torch.zeros_like(xs), torch.zeros_like(xs)
    sy, sx, sz = torch.zeros_like(xs), torch.zeros_like(xs), torch.zeros_like(xs)
    dw, db, sw, sb = (torch.zeros(C).double() for _ in range(4))
    for i in range(xs.shape[0]):
        n = xs.shape[1] if lengths is None else max(0, min(xs.shape[1], int(lengths[i])))
        if n == 0:
            continue
        v = xs[i, :n].reshape(n, G, C // G)
        mu = v.mean((0, 2), keepdim=True)
        r = 1 / torch.sqrt(((v - mu) ** 2).mean((0, 2), keepdim=True) + eps)
        xh = ((v - mu) * r).reshape(n, C)
        # what xh's error is relative to: a difference of values up to max|x|, over std
        sh = (((v - mu).abs() + v.abs().amax((0, 2), keepdim=True)) * r).reshape(n, C)
        u, su = xh * w + b, sh * w.abs() + b.abs()
        t = u if z is None else z[i, :n]
        s = torch.sigmoid(t) if act == "silu" else torch.ones_like(t)
        slope = s * (1 + t * (1 - s)) if act == "silu" else s
        y[i, :n] = t * s if z is None else u * t * s
        # |silu'| <= 1.1, |silu''| <= 0.5
        sy[i, :n] = 1.1 * su + t.abs() * s if z is None else (su + u.abs()) * (t * s).abs()
        if dy is None:
            continue
        d = dy[i, :n]
        if z is None:
            du, sdu = d * slope, d.abs() * (1.1 + 0.5 * su)
        else:
            du, sdu = d * t * s, d.abs() * (t * s).abs() + 0 * su
            dz[i, :n] = d * u * slope
            sz[i, :n] = d.abs() * ((su + u.abs()) * 1.1)
        g = lambda q: q.reshape(n, G, C // G)
        dxh, sdxh = g(du * w), g(sdu * w.abs())
        m = lambda q: q.mean((0, 2), keepdim=True)
        dx[i, :n] = (r * (dxh - m(dxh) - g(xh) * m(dxh * g(xh)))).reshape(n, C)
        sx[i, :n] = (r * (sdxh + m(sdxh) + (g(sh) + 1) * m(sdxh * (g(sh) + 1)))).reshape(n, C)
        dw += (du * xh).sum(0)
        db += du.sum(0)
        sw += (sdu * (sh + 1)).sum(0)
        sb += sdu.sum(0)
    out = {"y": (y, sy)}
    if dy is not None:
        out.update(x=(dx, sx), z=(dz, sz), weight=(dw, sw), bias=(db, sb))
    return {k: (a.reshape(x.shape) if a.dim() == 3 else a, c.reshape(x.shape) if c.dim() == 3 else c)
            for k, (a, c) in out.items()}


def check(name, got, ref, f=F):
    want, size = ref
    e = (got.double().cpu() - want).abs()
    bound = HALF[got.dtype] * want.abs() + f * size + 1e-300
    worst = float((e / bound).max()) if e.numel() else 0.0
    print("  %s: %.3f of the bound" % (name, worst), flush=True)
    assert torch.isfinite(got).all() and worst <= 1, (name, worst)


def draw(seed, shape, io, gate, affine, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (2 * r(*shape) + offset).to(io).cuda()
    z = (3 * r(*shape)).to(io).cuda() if gate else None
    dy = r(*shape).to(io).cuda()
    w, b = ((1 + 0.3 * r(shape[-1])).cuda(), (0.3 * r(shape[-1])).cuda()) if affine else (None, None)
    return x, z, dy, w, b


# (shape, groups): widths of a group from 1 to more than a workgroup holds, odd ones among them
TOKEN = [((1, 8), 1), ((3, 5, 64), 8), ((7, 24), 8), ((2, 9, 4096), 64), ((5, 300), 4), ((129, 40), 40), ((33, 51), 3),
         ((4, 1000), 2), ((2, 2048), 1), ((3, 4104), 1), ((70, 16), 2), ((2, 3, 6000), 3), ((1025, 128), 1)]
SEQ = [((1, 1, 8), 1), ((3, 37, 64), 8), ((2, 5, 7, 24), 3), ((2, 300, 51), 3), ((1, 1000, 256), 32), ((2, 65, 2056), 1),
       ((3, 19, 1024), 4), ((2, 4000, 16), 1)]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate,act,affine", [(False, "silu", True), (True, "silu", True), (False, "none", False),
                                             (True, "none", True)])
@pytest.mark.parametrize("over,shape,groups", [("token",) + c for c in TOKEN] + [("sequence",) + c for c in SEQ])
def test_forward_and_backward(over, shape, groups, gate, act, affine, io):
    from state_space_sequence_amd import m3
    print("norm", over, shape, groups, gate, act, affine, io, flush=True)
    x, z, dy, w, b = draw(len(shape) + shape[-1], shape, io, gate, affine)
    kw = dict(z=z, activation=act, over=over)
    y = m3.group_norm_fwd(x, groups, w, b, **kw)
    g = m3.group_norm_bwd(x, groups, dy, w, b, **kw)
    torch.cuda.synchronize()
    ref = reference(x, groups, w, b, z, act, over, None, 1e-5, dy)
    check("y", y, ref["y"])
    assert set(g) == {"x"} | ({"z"} if gate else set()) | ({"weight", "bias"} if affine else set())
    for name in g:
        check(name, g[name], ref[name])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [False, True])
def test_lengths(gate, io):
    from state_space_sequence_amd import m3
    x, z, dy, w, b = draw(4, (4, 90, 48), io, gate, True)
    lengths = torch.tensor([90, 0, 1, 37], dtype=torch.int32).cuda()
    kw = dict(z=z, over="sequence", lengths=lengths)
    y, g = m3.group_norm_fwd(x, 6, w, b, **kw), m3.group_norm_bwd(x, 6, dy, w, b, **kw)
    ref = reference(x, 6, w, b, z, "silu", "sequence", lengths, 1e-5, dy)
    check("y", y, ref["y"])
    for name in g:
        check(name, g[name], ref[name])
    # what lies behind the lengths reaches nothing; lengths are clamped
    for t in [x, dy] + ([z] if gate else []):
        t[1], t[2, 1:], t[3, 37:] = float("nan"), float("inf"), float("nan")
    kw["lengths"] = torch.tensor([1 << 30, -3, 1, 37], dtype=torch.int32).cuda()
    y2, g2 = m3.group_norm_fwd(x, 6, w, b, **kw), m3.group_norm_bwd(x, 6, dy, w, b, **kw)
    assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)
    assert not y[1].any() and not y[3, 37:].any() and not g["x"][2, 1:].any()


@pytest.mark.parametrize("over,shape", [("token", (6, 256)), ("sequence", (2, 200, 32))])
def test_values_far_from_zero(over, shape):
    """The variance survives a mean of a thousand deviations (the bound grows with max|x| / std alone)."""
    from state_space_sequence_amd import m3
    x, _, dy, w, b = draw(5, shape, torch.float32, False, True, offset=2000.0)
    y, g = m3.group_norm_fwd(x, 2, w, b, over=over), m3.group_norm_bwd(x, 2, dy, w, b, over=over)
    ref = reference(x, 2, w, b, None, "silu", over, None, 1e-5, dy)
    check("y", y, ref["y"])
    for name in g:
        check(name, g[name], ref[name])


def test_constant_groups_and_empty_calls():
    from state_space_sequence_amd import m3
    for over in ("token", "sequence"):
        x = torch.full((3, 4, 32), 7.0, device="cuda")
        assert not m3.group_norm_fwd(x, 4, activation="none", over=over).any()
        e = torch.zeros(3, 0, 32, device="cuda")
        w = torch.ones(32, device="cuda")
        assert m3.group_norm_fwd(e, 4, w, w, over=over).shape == (3, 0, 32)
        g = m3.group_norm_bwd(e, 4, e, w, w, over=over)
        assert g["x"].shape == (3, 0, 32) and not g["weight"].any() and not g["bias"].any()


def test_gradients_against_differences():
    from state_space_sequence_amd import m3
    gen = torch.Generator().manual_seed(3)
    for over, shape in (("token", (9, 32)), ("sequence", (2, 7, 32))):
        for gate in (False, True):
            x, z, dy, w, b = draw(6, shape, torch.float32, gate, True)
            g = m3.group_norm_bwd(x, 4, dy, w, b, z=z, over=over)
            base = {"x": x, "weight": w, "bias": b, **({"z": z} if gate else {})}
            base = {k: t.double().cpu() for k, t in base.items()}

            def loss(t):
                y = reference(t["x"], 4, t["weight"], t["bias"], t.get("z"), "silu", over, None, 1e-5)["y"][0]
                return float((y * dy.double().cpu()).sum())

            for name in base:
                way = torch.randn(base[name].shape, generator=gen, dtype=torch.float64)
                h = 1e-5
                num = (loss({**base, name: base[name] + h * way}) - loss({**base, name: base[name] - h * way})) / (2 * h)
                terms = g[name].double().cpu() * way
                # differences in 64 bits: h^2 of third derivatives and 1e-16 / h of the loss; fp32 gradients
                assert abs(float(terms.sum()) - num) <= 1e-5 * float(terms.abs().sum()), (over, gate, name)


def test_in_place_captured_and_on_another_stream():
    from state_space_sequence_amd import m3
    for over in ("token", "sequence"):
        x, z, dy, w, b = draw(7, (2, 50, 64), torch.bfloat16, True, True)
        kw = dict(z=z, over=over)
        call = lambda: [m3.group_norm_fwd(x, 8, w, b, **kw)] + [t for _, t in sorted(m3.group_norm_bwd(x, 8, dy, w, b, **kw).items())]
        want = call()
        a, d, e = x.clone(), dy.clone(), z.clone()
        assert torch.equal(m3.group_norm_fwd(a, 8, w, b, y=a, **kw), want[0])
        g = m3.group_norm_bwd(x, 8, d, w, b, z=e, over=over, grads={"x": d, "z": e})
        assert torch.equal(g["x"], want[3]) and torch.equal(g["z"], want[4])
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        other = [m3.group_norm_fwd(x, 8, w, b, stream=s, **kw) for _ in range(3)]
        s.synchronize()
        assert all(torch.equal(o, want[0]) for o in other)
        with torch.cuda.stream(s):
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for k in range(3):
            x.copy_(torch.randn_like(x))
            eager = [t.clone() for t in call()]
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(eager, out)), (over, k)


def test_mixer_layer_of_linear_attention_and_norm():
    """The operators as a layer uses them: linear attention, the gated norm of its heads, and back."""
    from state_space_sequence_amd import m3
    from tests.linattn_reference import reference as attention
    gen = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()
    b, L, H, G, N, P = 2, 70, 4, 2, 32, 16
    q, k, v, z, dy = r(b, L, H, N), r(b, L, G, N), r(b, L, G, P), r(b, L, H * P), r(b, L, H * P)
    w, bias, ld = 1 + 0.1 * r(H * P), 0.1 * r(H * P), torch.tensor([-0.5, -0.1, -0.02, 0.0]).cuda()
    y, _ = m3.linattn_fwd(q, k, v, ld)
    o = m3.group_norm_fwd(y.view(b, L, H * P), H, w, bias, z=z)
    gn = m3.group_norm_bwd(y.view(b, L, H * P), H, dy, w, bias, z=z)
    ga = m3.linattn_bwd(q, k, v, ld, gn["x"].view(b, L, H, P))
    torch.cuda.synchronize()
    fwd = attention(q, k, v, ld, N ** -0.5)["y"].reshape(b, L, H * P)
    ref = reference(fwd, H, w, bias, z, "silu", "token", None, 1e-5, dy)
    back = attention(q, k, v, ld, N ** -0.5, dy=ref["x"][0].reshape(b, L, H, P))
    # two fp32 calls in a row: the norm passes its input's error (2e-5 of its size) on, divided by the deviation
    near = lambda got, want: float((got.double().cpu() - want).norm() / want.norm()) < 1e-4
    assert near(o, ref["y"][0]) and near(gn["z"], ref["z"][0]) and near(gn["weight"], ref["weight"][0])
    assert all(near(ga[n], back[n]) for n in ("q", "k", "v", "log_decay"))


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_tensors_larger_than_the_caches(io):
    """Rows of a call whose tensors fit no cache are those of a small call, bit by bit."""
    from state_space_sequence_amd import m3
    torch.manual_seed(4)
    C, G, n = 1024, 8, 50000
    x, z, dy = (torch.randn(n, C, device="cuda").to(io) for _ in range(3))
    w, b = torch.randn(C, device="cuda"), torch.randn(C, device="cuda")
    y = m3.group_norm_fwd(x, G, w, b, z=z)
    g = m3.group_norm_bwd(x, G, dy, w, b, z=z)
    for s in (slice(0, 100), slice(31000, 31077), slice(n - 50, n)):
        assert torch.equal(y[s], m3.group_norm_fwd(x[s], G, w, b, z=z[s]))
        small = m3.group_norm_bwd(x[s], G, dy[s], w, b, z=z[s])
        assert torch.equal(g["x"][s], small["x"]) and torch.equal(g["z"][s], small["z"])
