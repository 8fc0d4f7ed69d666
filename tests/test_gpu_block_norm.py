"""GPU parity of the norms around a block (m3_block_norm_fwd, _bwd) with their definition in 64 bits on the CPU.

Bounds, elementwise. A row's sums are sums of up to 32768 fp32 terms: 32 roundings in a lane's own, 6 in a wave's and 16 in a
row's, so a norm's factor is off by at most (54 / 2 + 8) 2^-24 relative, and a product of a dozen factors by F = 96 * 2^-24
of its absolute value; where a mean over the row is taken off, of the sum of both absolute values, the mean's
taken over absolute terms. Sums over rows are of fp32 terms, at most 256 roundings of 2^-24, those of halves of them on average, of
the sum of absolute terms: G = (96 + 256) * 2^-24. Outputs in bf16 are rounded by at most 2^-8 of themselves."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F, G = 96 * 2.0 ** -24, 352 * 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def act_of(z, act):
    if z is None:
        return 1.0, 0.0
    if act == "none":
        return z, torch.ones_like(z)
    s, s1 = torch.sigmoid(z), torch.sigmoid(-z)
    return (z * s, s * (1 + z * s1)) if act == "silu" else (s, s * s1)


def reference(x, r, z=None, act="silu", scale=None, post=False, w=None, pre=True, wp=None, alpha=1.0, eps=1e-5, dy=None,
              dR=None, R=None):
    """{name: (value, bound of the fp32 error)}; with R the gradients, from it."""
    d = lambda t: None if t is None else t.detach().double().cpu()
    x, r, z, scale, w, wp, dy, dR, R = map(d, (x, r, z, scale, w, wp, dy, dR, R))
    one = torch.ones(x.shape[-1]).double()
    scale, w, wp = (one if t is None else t for t in (scale, w, wp))
    mean = lambda t: t.mean(-1, keepdim=True)
    act, slope = act_of(z, act)
    rx = (mean(x * x) + eps) ** -0.5 if post else torch.ones_like(x[..., :1])
    n = x * rx
    v = n * w
    if R is None:
        e = scale * act * v
        R = e if r is None else alpha * r + e
        size = e.abs() if r is None else (alpha * r).abs() + e.abs()
        out = {"residual": (R, F * size)}
        if pre:
            rR = (mean(R * R) + eps) ** -0.5
            # the factor's error: that of the mean of R^2, half of it
            rel = mean(R.abs() * F * size) * rR * rR
            out["y"] = (R * rR * wp, (F * size * rR + R.abs() * rR * (rel + F)) * wp.abs())
        return out
    D = torch.zeros_like(x) if dR is None else dR
    sD = D.abs()
    out = {}
    if pre:
        rR = (mean(R * R) + eps) ** -0.5
        N, q = R * rR, dy * wp
        D = D + rR * (q - N * mean(q * N))
        sD = sD + rR * (q.abs() + N.abs() * mean((q * N).abs()))
        out["pre_weight"] = ((dy * N).flatten(0, -2).sum(0), G * (dy * N).abs().flatten(0, -2).sum(0))
    out["residual"] = (alpha * D, F * (alpha * sD).abs())
    t = lambda q: q.flatten(0, -2).sum(0)
    sact = act.abs() if z is not None else 1.0
    out["scale"] = (t(D * act * v), G * t(sD * sact * v.abs()))
    if z is not None:
        # a slope s (1 + z (1 - s)) is off by what its terms are
        sslope = slope.abs() + 1.0
        out["z"] = (D * scale * v * slope, F * sD * (scale * v).abs() * sslope)
    p, sp = D * scale * act, sD * scale.abs() * sact
    out["post_weight"] = (t(p * n), G * t(sp * n.abs()))
    g, sg = p * w, sp * w.abs()
    if post:
        out["x"] = (rx * (g - n * mean(g * n)), F * rx * (sg + n.abs() * mean(sg * n.abs())))
    else:
        out["x"] = (g, F * sg)
    return out


def check(name, got, ref):
    want, err = ref
    assert got.shape == want.shape, name
    e = (got.double().cpu() - want).abs()
    bound = HALF[got.dtype] * (want.abs() + err) + err + 1e-300
    worst = float((e / bound).max()) if e.numel() else 0.0
    print("  %s: %.3f of the bound" % (name, worst), flush=True)
    assert torch.isfinite(got).all() and worst <= 1, (name, worst)


def draw(seed, shape, io, res, gate=True, weights=True, scale=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    C = shape[-1]
    vec = lambda on, m: (m + 0.3 * r(C)).cuda() if on else None
    return dict(x=(2 * r(*shape)).to(io).cuda(), r=(3 * r(*shape)).to(res).cuda(), z=(2 * r(*shape)).to(io).cuda() if gate else None,
                w=vec(weights, 1.0), wp=vec(weights, 1.0), scale=vec(scale, 0.5), dy=r(*shape).to(io).cuda(),
                dR=r(*shape).to(res).cuda())


def run(d, act="silu", post=True, pre=True, alpha=0.75, residual=True, dR=True, **more):
    from state_space_sequence_amd import m3
    kw = dict(z=d["z"], activation=act, scale=d["scale"], post_norm=post, post_weight=d["w"] if post else None, pre_norm=pre,
              pre_weight=d["wp"] if pre else None, residual_scale=alpha)
    kw.update(more)
    y, R = m3.block_norm_fwd(d["x"], d["r"] if residual else None, residual_dtype=None if residual else d["r"].dtype, **kw)
    g = m3.block_norm_bwd(d["x"], R, d["dy"] if pre else None, d["dR"] if dR else None, **kw)
    torch.cuda.synchronize()
    ref = reference(d["x"], d["r"] if residual else None, d["z"], act, d["scale"], post, kw["post_weight"], pre, kw["pre_weight"],
                    alpha)
    back = reference(d["x"], None, d["z"], act, d["scale"], post, kw["post_weight"], pre, kw["pre_weight"], alpha,
                     dy=d["dy"] if pre else None, dR=d["dR"] if dR else None, R=R)
    check("R", R, ref["residual"])
    if pre:
        check("y", y, ref["y"])
    else:
        assert y is None
    want = {"x", "residual"} | ({"z"} if d["z"] is not None else set()) | ({"scale"} if d["scale"] is not None else set())
    want |= ({"post_weight"} if kw["post_weight"] is not None else set()) | ({"pre_weight"} if kw["pre_weight"] is not None else set())
    assert set(g) == want
    for name in g:
        check(name, g[name], back[name])
    return y, R, g


IO = [(BF, BF), (BF, FP), (FP, FP)]


@pytest.mark.parametrize("io,res", IO)
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 5, 16), (33, 128), (7, 130), (5, 512), (257, 264), (3, 1000), (4, 1001), (3, 2048),
                                   (2, 1280), (2, 1500), (2, 2560), (3, 2600), (2, 4096), (2, 4100), (3, 5000), (2, 8192), (1, 8191), (1, 9001),
                                   (2, 16384)])
def test_widths(shape, io, res):
    print("block norm", shape, io, res, flush=True)
    run(draw(sum(shape), shape, io, res))


@pytest.mark.parametrize("io,res", IO)
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_rows_that_the_registers_do_not_hold(post, pre, io, res):
    print("block norm wide", post, pre, io, res, flush=True)
    for shape in ((2, 32768), (300, 8193), (3, 20001)):
        run(draw(shape[1], shape, io, res, scale=pre), post=post, pre=pre)


def test_a_norm_alone():
    """Without the stream behind: the same y."""
    from state_space_sequence_amd import m3
    for shape in ((50, 264), (3, 20001)):
        d = draw(2, shape, BF, BF)
        kw = dict(z=d["z"], post_norm=True, pre_weight=d["wp"])
        y, R = m3.block_norm_fwd(d["x"], d["r"], **kw)
        y2, none = m3.block_norm_fwd(d["x"], d["r"], want_residual=False, **kw)
        assert none is None and torch.equal(y, y2)
        y, _ = m3.block_norm_fwd(d["x"], pre_weight=d["wp"], want_residual=False)
        check("y", y, reference(d["x"], None, wp=d["wp"])["y"])


def test_wide_rows_in_place():
    from state_space_sequence_amd import m3
    d = draw(8, (5, 17000), BF, BF)
    kw = dict(scale=d["scale"], post_norm=True, post_weight=d["w"], pre_weight=d["wp"], residual_scale=0.5)
    y, R = m3.block_norm_fwd(d["x"], d["r"], z=d["z"], **kw)
    ref = m3.block_norm_bwd(d["x"], R, d["dy"], d["dR"], z=d["z"], **kw)
    plain = m3.block_norm_bwd(d["x"], R, d["dy"], d["dR"], z=d["z"], grads={n: torch.empty_like(ref[n]) for n in ("x", "z")}, **kw)
    assert all(torch.equal(plain[n], ref[n]) for n in plain)
    e = {n: t.clone() for n, t in d.items()}
    m3.block_norm_fwd(e["x"], e["r"], z=e["z"], y=e["x"], residual_out=e["r"], **kw)
    assert torch.equal(e["x"], y) and torch.equal(e["r"], R)
    e = {n: t.clone() for n, t in d.items()}
    g = {n: torch.empty_like(t) for n, t in ref.items()}
    g.update(x=e["dy"], z=e["z"], residual=e["dR"])
    m3.block_norm_bwd(e["x"], R, e["dy"], e["dR"], z=e["z"], grads=g, **kw)
    assert all(torch.equal(g[n], ref[n]) for n in ref)


@pytest.mark.parametrize("io,res", IO)
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("act", ["silu", "sigmoid", "none", None])
def test_parts(act, post, pre, io, res):
    print("block norm parts", act, post, pre, io, res, flush=True)
    d = draw(5, (9, 96), io, res, gate=act is not None, scale=post)
    run(d, act or "silu", post, pre)
    run(d, act or "silu", post, pre, residual=False, dR=not pre)
    d["w"] = d["wp"] = None
    run(d, act or "silu", post, pre, alpha=1.0)


@pytest.mark.parametrize("io,res", IO)
@pytest.mark.parametrize("shape", [(3000, 24), (20011, 64), (5000, 300), (1300, 2048)])
def test_many_rows(shape, io, res):
    print("block norm rows", shape, io, res, flush=True)
    run(draw(shape[0], shape, io, res))


def test_more_rows_than_one_thread_sums():
    """Over 256 rows a thread the weights' gradients are summed by more workgroups."""
    torch.manual_seed(2)
    from state_space_sequence_amd import m3
    n, C = 9_000_000, 16
    x = torch.randn(n, C, device="cuda")
    dy, w = torch.ones_like(x), torch.ones(C, device="cuda")
    g = m3.block_norm_bwd(x, x.abs(), dy, pre_weight=w)
    N = x.abs().double()
    want = (N * (N.square().mean(-1, keepdim=True) + 1e-5).rsqrt()).sum(0)
    # (all terms positive: 256 roundings of a thread's sum, a few of each term)
    assert ((g["pre_weight"] - want).abs() <= G * want).all()


def test_extreme_values():
    from state_space_sequence_amd import m3
    x = torch.zeros(4, 64, device="cuda")
    y, R = m3.block_norm_fwd(x, x, post_norm=True, z=torch.full_like(x, -200.0), activation="silu")
    assert not y.any() and not R.any()
    g = m3.block_norm_bwd(x, R, x, x, post_norm=True, z=torch.full_like(x, 300.0), activation="sigmoid")
    assert all(torch.isfinite(t).all() for t in g.values())
    # a NaN or an infinity stays in its row
    d = draw(3, (70, 96), FP, FP)
    kw = dict(z=d["z"], post_norm=True, post_weight=d["w"], pre_weight=d["wp"])
    y, R = m3.block_norm_fwd(d["x"], d["r"], **kw)
    for name in ("x", "r", "z"):
        e = {k: t.clone() for k, t in d.items()}
        e[name][33, 5] = float("nan")
        kw["z"] = e["z"]
        y2, R2 = m3.block_norm_fwd(e["x"], e["r"], **kw)
        assert y2[33].isnan().all()
        keep = torch.arange(70) != 33
        assert torch.equal(y2[keep], y[keep]) and torch.equal(R2[keep], R[keep])
    # large values whose squares still fit
    big = draw(4, (3, 40), FP, FP)
    big["x"], big["r"] = big["x"] * 1e15, big["r"] * 1e15
    run(big)


def test_gradients_against_differences():
    for act, post, pre in (("silu", True, True), ("sigmoid", True, False), ("none", False, True)):
        from state_space_sequence_amd import m3
        d = draw(6, (5, 24), FP, FP)
        kw = dict(z=d["z"], activation=act, scale=d["scale"], post_norm=post, post_weight=d["w"] if post else None, pre_norm=pre,
                  pre_weight=d["wp"] if pre else None, residual_scale=0.6)
        y, R = m3.block_norm_fwd(d["x"], d["r"], **kw)
        g = m3.block_norm_bwd(d["x"], R, d["dy"] if pre else None, d["dR"], **kw)
        base = {"x": d["x"], "residual": d["r"], "z": d["z"], "scale": d["scale"]}
        if post:
            base["post_weight"] = d["w"]
        if pre:
            base["pre_weight"] = d["wp"]
        base = {k: t.double().cpu() for k, t in base.items()}
        gen = torch.Generator().manual_seed(1)

        def loss(t):
            o = reference(t["x"], t["residual"], t["z"], act, t["scale"], post, t.get("post_weight"), pre, t.get("pre_weight"), 0.6)
            s = (o["residual"][0] * d["dR"].double().cpu()).sum()
            return float(s + (o["y"][0] * d["dy"].double().cpu()).sum()) if pre else float(s)

        for name in base:
            way, h = torch.randn(base[name].shape, generator=gen, dtype=torch.float64), 1e-6
            num = (loss({**base, name: base[name] + h * way}) - loss({**base, name: base[name] - h * way})) / (2 * h)
            terms = g[name].double().cpu() * way
            # differences in 64 bits: h^2 of third derivatives, 1e-14 / h of the loss; fp32 gradients of a stored fp32 stream
            assert abs(float(terms.sum()) - num) <= 1e-5 * float(terms.abs().sum()) + 1e-6, (act, post, pre, name)


def test_empty_calls():
    from state_space_sequence_amd import m3
    e, w = torch.zeros(3, 0, 32, device="cuda"), torch.ones(32, device="cuda")
    y, R = m3.block_norm_fwd(e, e, post_norm=True, post_weight=w, pre_weight=w, scale=w)
    assert y.shape == R.shape == (3, 0, 32)
    g = m3.block_norm_bwd(e, e, e, e, post_norm=True, post_weight=w, pre_weight=w, scale=w)
    assert g["x"].shape == (3, 0, 32) and not any(g[n].any() for n in ("post_weight", "pre_weight", "scale"))


@pytest.mark.parametrize("io,res", IO)
def test_in_place_captured_and_on_another_stream(io, res):
    from state_space_sequence_amd import m3
    d = draw(7, (1200, 264), io, res)
    kw = dict(z=d["z"], scale=d["scale"], post_norm=True, post_weight=d["w"], pre_weight=d["wp"], residual_scale=0.5)

    def call(stream=None):
        y, R = m3.block_norm_fwd(d["x"], d["r"], stream=stream, **kw)
        g = m3.block_norm_bwd(d["x"], R, d["dy"], d["dR"], stream=stream, **kw)
        return [y, R] + [g[n] for n in sorted(g)]

    want = call()
    # y over x or z, the stream over itself; dx over x or dy, dz over z, dresidual over dresidual_out
    for over in ("x", "z"):
        e = {n: None if t is None else t.clone() for n, t in d.items()}
        m3.block_norm_fwd(e["x"], e["r"], y=e[over], residual_out=e["r"], **dict(kw, z=e["z"]))
        assert torch.equal(e[over], want[0]) and torch.equal(e["r"], want[1])
    ref = m3.block_norm_bwd(d["x"], want[1], d["dy"], d["dR"], **kw)
    for over in ("x", "dy"):
        e = {n: None if t is None else t.clone() for n, t in d.items()}
        g = {n: torch.empty_like(t) for n, t in ref.items()}
        g.update(x=e[over], z=e["z"], residual=e["dR"])
        m3.block_norm_bwd(e["x"], want[1], e["dy"], e["dR"], grads=g, **dict(kw, z=e["z"]))
        assert all(torch.equal(g[n], ref[n]) for n in ref)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = [call(s) for _ in range(2)]
    s.synchronize()
    assert all(torch.equal(a, b) for o in other for a, b in zip(want, o))
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        for n in ("x", "r", "z", "dy", "dR"):
            d[n].copy_(torch.randn_like(d[n]))
        eager = [t.clone() for t in call()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))
