"""Calls at once on two streams, and tensors whose elements pass 32 bits, of the recurrence, the block norm and the
rotary positions: the same bits as calls by themselves, and as small calls on slices."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rec(m3, x, r, ld, **kw):
    y, h, s = m3.recurrence_fwd(x, r, ld, want_states=True, **kw)
    g = m3.recurrence_bwd(x, r, ld, y, dh_final=h, **kw)
    return [y, h, s] + [g[n] for n in sorted(g)]


def test_two_streams_at_once():
    """Chains of two calls share the card: each has its workspace, and both end."""
    from state_space_sequence_amd import m3
    torch.manual_seed(1)
    a = [torch.randn(2, 6000, 640, device="cuda").to(BF) for _ in range(2)]
    b = [torch.randn(1, 9000, 200, device="cuda") for _ in range(2)]
    lda, ldb = -torch.rand(640, device="cuda"), -torch.rand(200, device="cuda")
    wa, wb = rec(m3, *a, lda), rec(m3, *b, ldb)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s):
            ga = rec(m3, *a, lda)
        with torch.cuda.stream(t):
            gb = rec(m3, *b, ldb)
        got.append((ga, gb))
    torch.cuda.synchronize()
    for ga, gb in got:
        assert all(torch.equal(p, q) for p, q in zip(wa, ga))
        assert all(torch.equal(p, q) for p, q in zip(wb, gb))


def test_recurrence_of_more_than_2_to_31_elements():
    from state_space_sequence_amd import m3
    L, C, cut = 530_000, 4160, 529_920  # (a multiple of 64)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(1, L, C, device="cuda", dtype=BF, generator=gen)
    r = torch.randn(1, L, C, device="cuda", dtype=BF, generator=gen)
    ld = -torch.rand(C, device="cuda") - 0.05
    y, h, states = m3.recurrence_fwd(x, r, ld, want_states=True)
    tail = [t[:, cut:].contiguous() for t in (x, r)]
    ty, th = m3.recurrence_fwd(*tail, ld, h0=states[:, cut // 64].contiguous())
    # the same tokens from the same state, joined in another order: fp32 sums of some ten terms that count, each off by 2^-24
    assert ((h - th).abs() <= 2.0 ** -18 * (1 + th.abs())).all()
    assert ((y[:, cut:].float() - ty.float()).abs() <= 2.0 ** -7 * ty.float().abs() + 2.0 ** -18).all()
    del y
    g = m3.recurrence_bwd(x, r, ld, x, states=states, dh_final=h)
    tg = m3.recurrence_bwd(*tail, ld, tail[0], states=states[:, cut // 64:].contiguous(), dh_final=h)
    for n in ("x", "decay_gate"):
        a, b = g[n][:, cut:].float(), tg[n].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16).all(), n
    assert all(torch.isfinite(t).all() for t in g.values())


def test_block_norm_and_rotary_of_more_than_2_to_31_elements():
    from state_space_sequence_amd import m3
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, C = 540_000, 4096
    x = torch.randn(n, C, device="cuda", dtype=BF, generator=gen)
    R = torch.randn(n, C, device="cuda", dtype=BF, generator=gen)
    w = torch.rand(C, device="cuda")
    kw = dict(post_norm=True, post_weight=w, pre_weight=w)
    y, out = m3.block_norm_fwd(x, R, **kw)
    g = m3.block_norm_bwd(x, out, y, R, **kw)
    for s in (slice(0, 70), slice(300_000, 300_033), slice(n - 65, n)):
        sy, sout = m3.block_norm_fwd(x[s], R[s], **kw)
        sg = m3.block_norm_bwd(x[s], out[s], y[s], R[s], **kw)
        assert torch.equal(y[s], sy) and torch.equal(out[s], sout)
        assert torch.equal(g["x"][s], sg["x"]) and torch.equal(g["residual"][s], sg["residual"])
    del y, out, g, R
    q = x.view(1, n, 32, 128)
    freqs = m3.rotary_frequencies(128, device="cuda")
    for layout in ("half", "interleaved"):
        o, _ = m3.rotary(q, None, freqs, layout=layout)
        s = slice(n - 40, n)
        want, _ = m3.rotary(q[:, s].contiguous(), None, freqs, layout=layout, offsets=torch.tensor([n - 40], dtype=torch.int32).cuda())
        assert torch.equal(o[:, s], want)
