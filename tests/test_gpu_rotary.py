"""GPU parity of rotary positions (m3_rotary) with their definition in 64 bits on the CPU.

Bound, elementwise: the angle in turns is a product in fp64, of which the fraction is rounded to fp32: at most 2^-26 of a
turn, 2 pi 2^-26 < 2^-23 rad; cosine and sine of it, two steps at most: E = 2^-22 for each. Scale, two products and a sum
add 3 roundings: an output is off by at most scale (|u| + |w|) (2^-22 + 3 * 2^-24) and its own rounding, 2^-8 of
itself in bf16. Copied channels are equal."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 2.0 ** -22 + 3 * 2.0 ** -24


def reference(x, freqs, pos, layout, scale=1.0, back=False):
    """(value, bound of the fp32 error) of x [..., heads, D] at pos [...]."""
    x, f, n = x.detach().double().cpu(), freqs.double().cpu(), freqs.shape[0]
    t = pos.double().cpu()[..., None, None] * f * (-1 if back else 1)
    c, s = scale * torch.cos(t), scale * torch.sin(t)
    i = torch.arange(n)
    a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    u, w = x[..., a], x[..., b]
    out, err = x.clone(), torch.zeros_like(x)
    out[..., a], out[..., b] = u * c - w * s, u * s + w * c
    err[..., a] = err[..., b] = abs(scale) * (u.abs() + w.abs()) * E
    return out, err


def check(name, got, ref):
    want, err = ref
    assert got.shape == want.shape, name
    e = (got.double().cpu() - want).abs()
    bound = torch.where(err > 0, HALF[got.dtype] * (want.abs() + err) + err, torch.zeros_like(err))
    assert (e <= bound).all(), (name, float((e - bound).max()))
    assert torch.isfinite(got).all()


def draw(seed, b, L, H, G, D, io):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(io).cuda()
    return r(b, L, H, D), r(b, L, G, D)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("H,G,D,n", [(1, 1, 2, 2), (3, 1, 7, 4), (8, 2, 64, 64), (64, 8, 128, 128), (5, 5, 80, 40), (4, 2, 96, 32), (2, 1, 256, 256),
                                     (3, 2, 24, 6), (7, 1, 100, 100), (2, 2, 1024, 1024), (1, 1, 1000, 400), (4, 4, 16, 0), (1, 1, 1, 0), (2, 3, 96, 50),
                                     (3, 1, 72, 24), (2, 2, 100, 92), (5, 1, 36, 20)])
@pytest.mark.parametrize("where", ["none", "each", "offsets"])
def test_layouts_and_positions(where, H, G, D, n, layout, io):
    from state_space_sequence_amd import m3
    print("rotary", where, H, G, D, n, layout, io, flush=True)
    b, L = 3, 13
    q, k = draw(H + D, b, L, H, G, D, io)
    freqs = m3.rotary_frequencies(n, device="cuda")
    gen = torch.Generator().manual_seed(1)
    pos, kw = torch.arange(L).expand(b, L), {}
    if where == "each":
        pos = torch.randint(-1000, 1 << 27, (b, L), generator=gen, dtype=torch.int32)
        kw["positions"] = pos.cuda()
    elif where == "offsets":
        off = torch.tensor([0, 70000, (1 << 27) - 50], dtype=torch.int32)
        pos, kw["offsets"] = pos + off[:, None], off.cuda()
    for back, scale in ((False, 1.0), (True, 1.25)):
        oq, ok = m3.rotary(q, k, freqs, layout=layout, scale=scale, backward=back, **kw)
        torch.cuda.synchronize()
        check("q", oq, reference(q, freqs, pos, layout, scale, back))
        check("k", ok, reference(k, freqs, pos, layout, scale, back))
    # in place, q alone, and k in place beside q elsewhere: the same bits
    iq, ik = q.clone(), k.clone()
    m3.rotary(iq, ik, freqs, layout=layout, scale=scale, backward=True, q_out=iq, k_out=ik, **kw)
    assert torch.equal(iq, oq) and torch.equal(ik, ok)
    assert torch.equal(m3.rotary(q, None, freqs, layout=layout, scale=scale, backward=True, **kw)[0], oq)
    ik = k.clone()
    assert torch.equal(m3.rotary(q, ik, freqs, layout=layout, scale=scale, backward=True, k_out=ik, **kw)[0], oq)
    assert torch.equal(ik, ok)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,L,H,G,D,n", [(128, 1, 32, 4, 128, 128), (1, 1, 1, 1, 64, 32), (1, 5000, 3, 1, 64, 64), (2, 3000, 16, 4, 72, 48),
                                         (1, 2500, 40, 40, 32, 32)])
def test_many_and_few_tokens(b, L, H, G, D, n, io):
    from state_space_sequence_amd import m3
    q, k = draw(7, b, L, H, G, D, io)
    freqs = m3.rotary_frequencies(n, device="cuda")
    for layout in ("half", "interleaved"):
        oq, ok = m3.rotary(q, k, freqs, layout=layout)
        pos = torch.arange(L).expand(b, L)
        check("q", oq, reference(q, freqs, pos, layout))
        check("k", ok, reference(k, freqs, pos, layout))


def test_tokens_of_a_serving_batch():
    from state_space_sequence_amd import m3
    q, k = draw(3, 9, 1, 6, 2, 64, torch.bfloat16)
    freqs = m3.rotary_frequencies(64, device="cuda")
    pos = torch.arange(9, dtype=torch.int32).cuda() * 100003
    q3, k3 = q[:, 0].contiguous(), k[:, 0].contiguous()
    want = m3.rotary(q, k, freqs, positions=pos[:, None].contiguous())
    for kw in (dict(positions=pos), dict(offsets=pos)):
        got = m3.rotary(q3, k3, freqs, **kw)
        assert torch.equal(got[0], want[0][:, 0]) and torch.equal(got[1], want[1][:, 0])
    check("q", got[0], reference(q3, freqs, pos.cpu(), "half"))


def test_other_channels_pass_as_they_are():
    """NaN and infinity in channels that are not turned stay there, whatever shares their access."""
    from state_space_sequence_amd import m3
    for io in (torch.bfloat16, torch.float32):
        for n in (4, 6, 16):
            q, _ = draw(5, 2, 5, 3, 1, 32, io)
            q[..., n:] = float("nan")
            q[..., n + 1::3] = float("inf")
            freqs = m3.rotary_frequencies(n, device="cuda")
            for layout in ("half", "interleaved"):
                out, _ = m3.rotary(q, None, freqs, layout=layout)
                assert torch.isfinite(out[..., :n]).all()
                assert torch.equal(out[..., n:].isnan(), q[..., n:].isnan()) and torch.equal(out[..., n:].isinf(), q[..., n:].isinf())


def test_backward_is_the_transpose_and_relative():
    """<turn(x), y> = <x, back(y)>, and products of turned q and k depend on the distance alone."""
    from state_space_sequence_amd import m3
    q, k = draw(2, 1, 40, 4, 4, 64, torch.float32)
    freqs = m3.rotary_frequencies(64, scaling="linear", factor=3.0, device="cuda")
    for layout in ("half", "interleaved"):
        tq, _ = m3.rotary(q, None, freqs, layout=layout, scale=1.5)
        bk, _ = m3.rotary(k, None, freqs, layout=layout, scale=1.5, backward=True)
        a, b = (tq.double() * k.double()).sum(), (q.double() * bk.double()).sum()
        size = 1.5 * float((q.double().abs() * k.double().abs()).sum())
        assert abs(float(a - b)) <= 8 * E * size
        o = lambda n: torch.tensor([n], dtype=torch.int32).cuda()
        one = lambda n: [t.double() for t in m3.rotary(q, k, freqs, layout=layout, offsets=o(n))]
        (q1, k1), (q2, k2) = one(5), one(900005)
        p1, p2 = (q1[0, 30] * k1[0, 10]).sum(-1), (q2[0, 30] * k2[0, 10]).sum(-1)
        assert ((p1 - p2).abs() <= 16 * E * 64).all()


def test_gradients_against_differences():
    from state_space_sequence_amd import m3
    q, k = draw(4, 2, 7, 3, 1, 20, torch.float32)
    dq, dk = draw(5, 2, 7, 3, 1, 20, torch.float32)
    freqs = m3.rotary_frequencies(12, device="cuda")
    pos = torch.arange(7).expand(2, 7)
    gq, gk = m3.rotary(dq, dk, freqs, layout="interleaved", scale=0.7, backward=True)
    for x, d, g in ((q, dq, gq), (k, dk, gk)):
        way = torch.randn_like(x).double().cpu()
        loss = lambda t: float((reference(t, freqs, pos, "interleaved", 0.7)[0] * d.double().cpu()).sum())
        num = (loss(x.double().cpu() + 1e-3 * way) - loss(x.double().cpu() - 1e-3 * way)) / 2e-3
        terms = g.double().cpu() * way
        # the loss is linear: differences are exact but for 64-bit roundings
        assert abs(float(terms.sum()) - num) <= 4 * E * float(terms.abs().sum()) + 1e-9


def test_empty_calls():
    from state_space_sequence_amd import m3
    freqs = m3.rotary_frequencies(8, device="cuda")
    for b, L in ((0, 5), (3, 0)):
        q = torch.zeros(b, L, 2, 16, device="cuda")
        assert m3.rotary(q, q.clone(), freqs)[1].shape == (b, L, 2, 16)


def test_captured_and_on_another_stream():
    from state_space_sequence_amd import m3
    q, k = draw(8, 2, 100, 8, 2, 64, torch.bfloat16)
    freqs = m3.rotary_frequencies(32, device="cuda")
    off = torch.tensor([3, 1 << 20], dtype=torch.int32).cuda()
    call = lambda stream=None: list(m3.rotary(q, k, freqs, offsets=off, stream=stream))
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = call(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        q.copy_(torch.randn_like(q))
        off.add_(17)
        eager = call()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))


def test_frequencies():
    from state_space_sequence_amd import m3
    f = m3.rotary_frequencies(64)
    assert f.shape == (32,) and f.dtype == torch.float32 and float(f[0]) == 1.0
    assert math.isclose(float(f[16]), 10000.0 ** -0.5, rel_tol=1e-6)
    lin = m3.rotary_frequencies(64, scaling="linear", factor=4)
    assert torch.allclose(lin * 4, f, rtol=1e-6)
    ntk = m3.rotary_frequencies(64, scaling="base", factor=4)
    assert float(ntk[0]) == 1.0 and math.isclose(float(ntk[31]), float(lin[31]), rel_tol=1e-6)
    parts = m3.rotary_frequencies(64, scaling="parts", factor=4, trained_length=4096)
    assert (parts <= f * 1.0000001).all() and (parts >= lin * 0.9999999).all()
    assert float(parts[0]) == 1.0 and math.isclose(float(parts[31]), float(lin[31]), rel_tol=1e-6)
    # a pair of 2 turns in the trained length lies 1/31 of the way from 1 to 32
    i = min(range(32), key=lambda j: abs(4096 * float(f[j]) / (2 * math.pi) - 2))
    keep = (4096 * float(f[i]) / (2 * math.pi) - 1) / 31
    assert math.isclose(float(parts[i]), float(f[i]) * (keep + (1 - keep) / 4), rel_tol=1e-5)
