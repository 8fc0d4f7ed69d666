"""GPU parity of the gated linear recurrence (m3_recurrence_fwd, _bwd, _step) with its definition
in 64 bits on the CPU, token by token.

Bounds, elementwise. A token's a, m and gates are off by at most E = 16 * 2^-24 relative (a rounded product, an
exponential, a reciprocal, a square root, each of at most 2 steps; ld s enters a with |ld s| <= 8 times that, so a with
at most 12 * 16 * 2^-24 of itself where it decays by much, and with the rounding 2^-24 where it does not). A
state is a sum of terms; its error is at most that of every term plus a rounding (2^-24 of the state) a
token, all carried on by the decays: the same recurrence, run on the absolute values with F = 256 * 2^-24 of every term as
its input, bounds it, and so do its adjoints for the gradients. Outputs in bf16 are rounded by at most 2^-8 of themselves."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F = 256 * 2.0 ** -24


def reference(x, r, ld, i=None, h0=None, lengths=None, scaled=True, dy=None, dh=None):
    """{name: (value, bound of the fp32 error)}: y, h, states, and with dy the gradients."""
    x, r, ld, i, h0, dy, dh = (None if t is None else t.detach().double().cpu() for t in (x, r, ld, i, h0, dy, dh))
    b, L, C = x.shape
    s, g = torch.sigmoid(r), torch.ones_like(x) if i is None else torch.sigmoid(i)
    s1, g1 = torch.sigmoid(-r), torch.zeros_like(x) if i is None else torch.sigmoid(-i)
    la = ld * s
    a = torch.exp(la)
    q = -torch.expm1(2 * la)
    m = q.sqrt() if scaled else torch.ones_like(q)
    inv = torch.where(q > 0, 1 / q.sqrt(), torch.zeros_like(q)) if scaled else torch.zeros_like(q)
    n = torch.full((b,), L) if lengths is None else lengths.cpu().long().clamp(0, L)
    live = (torch.arange(L)[None] < n[:, None])[..., None]
    zero = torch.zeros((), dtype=torch.float64)
    x = torch.where(live, x, zero)
    u = m * g * x
    h = torch.zeros(b, C).double() if h0 is None else h0
    e = h.abs() * 0
    before, eb = torch.zeros_like(x), torch.zeros_like(x)
    y, ey = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(L):
        on = live[:, t]
        before[:, t], eb[:, t] = h, e
        new = a[:, t] * h + u[:, t]
        e = torch.where(on, a[:, t] * e + F * (a[:, t] * h.abs() * (1 + la[:, t].abs()) + u[:, t].abs()), e)
        h = torch.where(on, new, h)
        y[:, t], ey[:, t] = h * on, e * on
    keep = lambda t: t[:, ::64]  # noqa: E731
    out = {"y": (y, ey), "h": (h, e), "states": (keep(before), keep(eb))}
    if dy is None:
        return out
    dy = torch.where(live, dy, zero)
    G = torch.zeros(b, C).double() if dh is None else dh
    eg = G.abs() * 0
    dx, dr, di, dl = (torch.zeros_like(x) for _ in range(4))
    ex, er, ei, el = (torch.zeros_like(x) for _ in range(4))
    for t in reversed(range(L)):
        on = live[:, t]
        E = dy[:, t] + G
        ee = eg + F * (dy[:, t].abs() + G.abs())
        c = a[:, t] * before[:, t] - g[:, t] * x[:, t] * a[:, t] ** 2 * inv[:, t]
        ec = a[:, t] * eb[:, t] + F * (a[:, t] * before[:, t].abs() * (1 + la[:, t].abs())
                                       + (g[:, t] * x[:, t] * a[:, t] ** 2 * inv[:, t]).abs() * (1 + la[:, t].abs()))
        def put(o, eo, f, ef):
            o[:, t] = torch.where(on, E * f, zero)
            eo[:, t] = torch.where(on, ee * f.abs() + E.abs() * ef + F * (E * f).abs(), zero)
        f = m[:, t] * g[:, t]
        put(dx, ex, f, F * f)
        f = u[:, t] * g1[:, t]
        put(di, ei, f, F * f.abs())
        put(dr, er, c * ld * s[:, t] * s1[:, t], ec * (ld * s[:, t] * s1[:, t]).abs())
        put(dl, el, c * s[:, t], ec * s[:, t])
        eg = torch.where(on, a[:, t] * ee + F * a[:, t] * E.abs() * (1 + la[:, t].abs()), eg)
        G = torch.where(on, a[:, t] * E, G)
    out.update(x=(dx, ex), decay_gate=(dr, er), log_decay=(dl.sum((0, 1)), el.sum((0, 1))), dh0=(G, eg))
    if i is not None:
        out["input_gate"] = (di, ei)
    return out


def check(name, got, ref):
    want, err = ref
    assert got.shape == want.shape, name
    e = (got.double().cpu() - want).abs()
    bound = HALF[got.dtype] * (want.abs() + err) + err + 1e-30
    worst = float((e / bound).max()) if e.numel() else 0.0
    print("  %s: %.3f of the bound" % (name, worst), flush=True)
    assert torch.isfinite(got).all() and worst <= 1, (name, worst)


def draw(seed, b, L, C, io, gate=True, h0=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    ld = (8 * torch.log(0.9 + 0.0995 * torch.rand(C, generator=g))).cuda()
    return dict(x=r(b, L, C).to(io).cuda(), r=(2 * r(b, L, C)).to(io).cuda(), ld=ld,
                i=(2 * r(b, L, C)).to(io).cuda() if gate else None, h0=r(b, C).cuda() if h0 else None,
                dy=r(b, L, C).to(io).cuda(), dh=r(b, C).cuda())


def run(d, lengths=None, scaled=True, kept=False):
    from state_space_sequence_amd import m3
    kw = dict(input_gate=d["i"], h0=d["h0"], lengths=lengths, scaled=scaled)
    y, h, states = m3.recurrence_fwd(d["x"], d["r"], d["ld"], want_states=True, **kw)
    if kept:
        kw["states"] = states
    g = m3.recurrence_bwd(d["x"], d["r"], d["ld"], d["dy"], dh_final=d["dh"], **kw)
    torch.cuda.synchronize()
    g["dh0"] = g.pop("h0")
    return dict(y=y, h=h, states=states, **g)


def compare(d, got, lengths=None, scaled=True):
    ref = reference(d["x"], d["r"], d["ld"], d["i"], d["h0"], lengths, scaled, d["dy"], d["dh"])
    assert set(got) == set(ref)
    for name in ref:
        check(name, got[name], ref[name])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate,scaled,h0", [(True, True, True), (False, True, False), (True, False, False), (False, False, True)])
@pytest.mark.parametrize("b,L,C", [(1, 1, 1), (2, 3, 7), (1, 64, 128), (2, 65, 130), (3, 200, 129), (1, 127, 64), (2, 256, 258)])
def test_forward_and_backward(b, L, C, gate, scaled, h0, io):
    print("recurrence", b, L, C, gate, scaled, h0, io, flush=True)
    d = draw(L + C, b, L, C, io, gate, h0)
    got = run(d, scaled=scaled)
    compare(d, got, scaled=scaled)
    kept = run(d, scaled=scaled, kept=True)
    assert all(torch.equal(got[n], kept[n]) for n in got)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [640, 700, 1024, 1025, 1100, 2177, 3300])
def test_long_chains(L, io):
    """Many tiles: within a group, at a group's end, over several groups."""
    print("recurrence long", L, io, flush=True)
    d = draw(L, 2, L, 66, io)
    lengths = torch.tensor([L, L // 3], dtype=torch.int32).cuda()
    compare(d, run(d, lengths), lengths)


@pytest.mark.parametrize("io,b,L,C", [(torch.bfloat16, 2, 130, 16384), (torch.float32, 3, 70, 8000), (torch.bfloat16, 1, 9000, 34),
                                      (torch.float32, 1, 5000, 65), (torch.bfloat16, 5, 300, 7682)])
def test_columns_from_one_to_more_than_the_card_holds(io, b, L, C):
    """Many columns, a workgroup each or a few; one or two columns, whose tiles are all taken at once."""
    print("recurrence columns", io, b, L, C, flush=True)
    d = draw(L, b, L, C, io)
    got = run(d)
    compare(d, got)
    for _ in range(5):  # whoever is first, the same bits
        again = run(d)
        assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_lengths(io):
    """Rows of no, one and all tokens; what lies behind the lengths reaches nothing; lengths are clamped."""
    d = draw(4, 5, 150, 40, io)
    lengths = torch.tensor([150, 0, 1, 64, 97], dtype=torch.int32).cuda()
    got = run(d, lengths)
    compare(d, got, lengths)
    for n in ("x", "r", "i", "dy"):
        d[n][1], d[n][2, 1:], d[n][3, 64:], d[n][4, 97:] = float("nan"), float("inf"), float("nan"), float("-inf")
    again = run(d, torch.tensor([1 << 30, -5, 1, 64, 97], dtype=torch.int32).cuda())
    assert all(torch.equal(got[n], again[n]) for n in got)
    assert torch.equal(got["h"][1], d["h0"][1]) and torch.equal(got["dh0"][1], d["dh"][1])
    assert not got["y"][2, 1:].any() and not got["decay_gate"][4, 97:].any()


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_extreme_gates_and_decays(io):
    """Gates far from 0 (infinite ones too), decays of nothing and of nearly everything."""
    d = draw(9, 2, 80, 64, io)
    d["ld"][:8] = torch.tensor([0.0, -1e-30, -1e-12, -1e-6, -60.0, -200.0, -1e4, -8.0])
    for n, k in (("r", 0), ("i", 1)):
        d[n][:, k::9] = 12.0
        d[n][:, k + 2::9] = -12.0
        d[n][:, k + 4::9] = float("inf")
        d[n][:, k + 6::9] = float("-inf")
        d[n][:, k + 7::9] = -80.0
    got = run(d)
    assert all(torch.isfinite(t).all() for t in got.values())
    ref = reference(d["x"], d["r"].clamp(-1e4, 1e4), d["ld"], d["i"].clamp(-1e4, 1e4), d["h0"], None, True, d["dy"], d["dh"])
    for name in ("y", "h", "states", "x", "input_gate", "dh0"):
        check(name, got[name], ref[name])
    # (below the smallest normal number, 1 - a^2 and its slope count as 0: the two gradients of the decay where it is above)
    for name in ("decay_gate", "log_decay"):
        check(name, got[name][..., 2:], tuple(t[..., 2:] for t in ref[name]))
    # a decay of 0 keeps the state
    assert torch.equal(got["h"][:, 0], d["h0"][:, 0]) and not got["x"][..., 0].any()


def test_a_nan_stays_in_its_row_and_channel():
    d = draw(5, 2, 130, 6, torch.float32)
    for n in ("x", "r", "i"):
        e = {k: None if t is None else t.clone() for k, t in d.items()}
        e[n][1, 70, 3] = float("nan")
        got = run(e)
        assert got["y"][1, 70:, 3].isnan().all() and got["y"][1, :70, 3].isfinite().all()
        assert got["y"][0].isfinite().all() and got["y"][1, :, :3].isfinite().all()
        assert got["h"][1, 3].isnan() and got["decay_gate"][0].isfinite().all()


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("L", [100, 1500])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_state_has_no_part_behind_the_lengths(bad, L, kept, io):
    """An empty row whose start state is not finite (the place of no sequence in a batch) adds nothing to d log_decay, and
    gradients behind a length are 0 also where the last token's state is not finite."""
    from state_space_sequence_amd import m3

    d = draw(12, 3, L, 70, io)
    lengths = torch.tensor([0, L // 2 + 3, L], dtype=torch.int32, device="cuda")
    names = ["x", "decay_gate", "input_gate"]

    def grads(h0, x):
        a = dict(input_gate=d["i"], h0=h0, lengths=lengths)
        st = m3.recurrence_fwd(x, d["r"], d["ld"], want_states=True, **a)[2] if kept else None
        return m3.recurrence_bwd(x, d["r"], d["ld"], d["dy"], dh_final=d["dh"], states=st, **a)

    h0 = d["h0"].clone()
    h0[0] = bad
    want, got = grads(d["h0"], d["x"]), grads(h0, d["x"])
    for k in want:
        assert torch.equal(got[k], want[k]) and got[k].isfinite().all(), k
    assert all((got[k][0] == 0).all() for k in names)
    x = d["x"].clone()
    x[1, L // 2 + 2] = bad
    got = grads(d["h0"], x)
    assert all((got[k][1, L // 2 + 3:] == 0).all() for k in names)
    assert all(torch.equal(got[k][2], want[k][2]) for k in names)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate,scaled", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("b,C", [(1, 1), (3, 7), (5, 256), (129, 130)])
def test_step(b, C, gate, scaled, io):
    from state_space_sequence_amd import m3
    d = draw(b + C, b, 1, C, io, gate)
    h = d["h0"].clone()
    t = lambda n: None if d[n] is None else d[n][:, 0].contiguous()
    y = m3.recurrence_step(t("x"), t("r"), d["ld"], h, input_gate=t("i"), scaled=scaled)
    ref = reference(d["x"], d["r"], d["ld"], d["i"], d["h0"], None, scaled)
    check("y", y, tuple(v[:, 0] for v in ref["y"]))
    check("h", h, ref["h"])


def test_prompt_continued_by_steps_is_the_prompt():
    from state_space_sequence_amd import m3
    d = draw(8, 2, 90, 34, torch.float32)
    y, h = m3.recurrence_fwd(d["x"], d["r"], d["ld"], input_gate=d["i"], h0=d["h0"])
    cut = lambda t, a, b: t[:, a:b].contiguous()
    state = d["h0"].clone()
    m3.recurrence_fwd(*(cut(d[n], 0, 70) for n in "xr"), d["ld"], input_gate=cut(d["i"], 0, 70), h0=state, h_final=state)
    outs = [m3.recurrence_step(d["x"][:, t].contiguous(), d["r"][:, t].contiguous(), d["ld"], state,
                               input_gate=d["i"][:, t].contiguous()) for t in range(70, 90)]
    ref = reference(d["x"], d["r"], d["ld"], d["i"], d["h0"])
    check("y", torch.stack(outs, 1), tuple(t[:, 70:] for t in ref["y"]))
    check("h", state, ref["h"])


@pytest.mark.parametrize("L", [60, 1600])
def test_state_in_place(L):
    """h_final may be h0 itself, dh0 dh_final: tiles that start later still see the first."""
    from state_space_sequence_amd import m3
    d = draw(3, 4, L, 700, torch.bfloat16)
    kw = dict(input_gate=d["i"])
    y, h = m3.recurrence_fwd(d["x"], d["r"], d["ld"], h0=d["h0"], **kw)
    g = m3.recurrence_bwd(d["x"], d["r"], d["ld"], d["dy"], h0=d["h0"], dh_final=d["dh"], **kw)
    for _ in range(3):
        s, e = d["h0"].clone(), d["dh"].clone()
        y2, _ = m3.recurrence_fwd(d["x"], d["r"], d["ld"], h0=s, h_final=s, **kw)
        g2 = {n: torch.empty_like(t) for n, t in g.items() if n != "h0"}
        m3.recurrence_bwd(d["x"], d["r"], d["ld"], d["dy"], h0=d["h0"], dh_final=e, grads=dict(g2, h0=e), **kw)
        assert torch.equal(y, y2) and torch.equal(h, s) and torch.equal(e, g["h0"])
        assert all(torch.equal(g[n], g2[n]) for n in g2)


def test_gradients_against_differences():
    for scaled, gate in ((True, True), (False, True), (True, False)):
        d = draw(6, 2, 20, 5, torch.float32, gate)
        got = run(d, scaled=scaled)
        base = {n: None if t is None else t.double().cpu() for n, t in d.items()}
        gen = torch.Generator().manual_seed(1)

        def loss(t):
            o = reference(t["x"], t["r"], t["ld"], t["i"], t["h0"], None, scaled)
            return float((o["y"][0] * base["dy"]).sum() + (o["h"][0] * base["dh"]).sum())

        for name, key in (("x", "x"), ("r", "decay_gate"), ("i", "input_gate"), ("ld", "log_decay"), ("h0", "dh0")):
            if base[name] is None:
                continue
            way, eps = torch.randn(base[name].shape, generator=gen, dtype=torch.float64), 1e-6
            num = (loss({**base, name: base[name] + eps * way}) - loss({**base, name: base[name] - eps * way})) / (2 * eps)
            terms = got[key].double().cpu() * way
            # differences in 64 bits: eps^2 of third derivatives, 1e-15 / eps of the loss; fp32 gradients
            assert abs(float(terms.sum()) - num) <= 1e-5 * float(terms.abs().sum()) + 1e-6, (scaled, gate, name)


def test_empty_calls():
    from state_space_sequence_amd import m3
    ld = -torch.ones(6, device="cuda")
    e, h0 = torch.zeros(2, 0, 6, device="cuda"), torch.randn(2, 6, device="cuda")
    y, h, states = m3.recurrence_fwd(e, e, ld, input_gate=e, h0=h0, want_states=True)
    assert y.shape == (2, 0, 6) and states.shape == (2, 0, 6) and torch.equal(h, h0)
    g = m3.recurrence_bwd(e, e, ld, e, input_gate=e, h0=h0, dh_final=h0)
    assert torch.equal(g["h0"], h0) and not g["log_decay"].any()
    n = torch.zeros(0, 5, 6, device="cuda")
    y, h = m3.recurrence_fwd(n, n, ld)
    assert y.shape == (0, 5, 6) and h.shape == (0, 6)
    assert not m3.recurrence_bwd(n, n, ld, n)["log_decay"].any()
    assert m3.recurrence_step(n[:, 0], n[:, 0], ld, n[:, 0]).shape == (0, 6)


@pytest.mark.parametrize("L", [50, 300])
def test_captured_and_on_another_stream(L):
    from state_space_sequence_amd import m3
    d = draw(7, 2, L, 64, torch.bfloat16)
    kw = dict(input_gate=d["i"], h0=d["h0"])
    state = torch.zeros(2, 64, device="cuda")

    def call(stream=None):
        y, h, s = m3.recurrence_fwd(d["x"], d["r"], d["ld"], want_states=True, stream=stream, **kw)
        g = m3.recurrence_bwd(d["x"], d["r"], d["ld"], d["dy"], states=s, dh_final=h, stream=stream, **kw)
        f = m3.recurrence_bwd(d["x"], d["r"], d["ld"], d["dy"], dh_final=h, stream=stream, **kw)
        o = m3.recurrence_step(d["x"][:, 0].contiguous(), d["r"][:, 0].contiguous(), d["ld"], h, stream=stream)
        return [y, h, s, o] + [g[n] for n in sorted(g)] + [f[n] for n in sorted(f)]

    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        other = call()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        for n in ("x", "r", "i", "dy"):
            d[n].copy_(torch.randn_like(d[n]))
        eager = [t.clone() for t in call()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))
