"""GPU parity of linear attention with a decay for each head (m3_linattn_fwd, _bwd,
_step) with its definition in 64 bits.

Bounds, elementwise, on sum = the sum of the absolute values of the terms of an output
(the same recurrence on absolute values):
  fp32 arithmetic: every term passes at most N + P + L roundings of 2^-24 in sums and
  products, and its decay a^n carries the rounding of n log a, below 200 * 2^-24 for
  every weight that matters (|n log a| <= 200); F32 = (N + P + L + 200) 2^-24.
  bf16 inputs: products of inputs are exact in fp32; scores and states enter the next
  product as two bf16 parts, each term off by at most 2^-16, and F32 as above.
  An output stored in bf16 is rounded by at most 2^-8 of itself."""
from __future__ import annotations

import pytest
import torch

from tests.linattn_reference import reference

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DECAYS = [-0.5, -0.01, 0.0, float("-inf"), -3.0, -1e-4, -40.0, -0.1]


def draw(seed, b, L, H, G, N, P, io, h0=False, lengths=None, back=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, to=io: torch.randn(*s, generator=g).to(to).cuda()
    d = dict(q=r(b, L, H, N), k=r(b, L, G, N), v=r(b, L, G, P),
             log_decay=torch.tensor([DECAYS[(h + seed) % len(DECAYS)] for h in range(H)]).cuda(),
             h0=r(b, H, P, N, to=torch.float32) if h0 else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda())
    if back:
        d.update(dy=r(b, L, H, P), dh_final=r(b, H, P, N, to=torch.float32) if h0 else None)
    return d


def factor(d, exact32):
    N, P, L = d["q"].shape[-1], d["v"].shape[-1], d["q"].shape[1]
    f = (N + P + L + 200) * 2.0 ** -24
    return f if exact32 or d["q"].dtype is torch.float32 else f + 2.0 ** -16


def check(name, got, want, size, f):
    e = (got.double().cpu() - want).abs()
    bound = HALF[got.dtype] * want.abs() + f * size
    worst = float((e / bound.clamp(min=1e-300)).max()) if e.numel() else 0.0
    print("  %s: %.3f of the bound" % (name, worst), flush=True)
    assert torch.isfinite(got).all() and bool((e <= bound).all()), (name, worst)


# (b, L, H, G, N, P, h0, lengths, nsegments)
CASES = [
    (1, 1, 1, 1, 1, 1, False, None, 0),
    (2, 1, 3, 3, 64, 64, True, None, 0),
    (1, 63, 2, 1, 64, 32, True, None, 0),
    (2, 64, 4, 2, 128, 64, False, None, 0),
    (1, 65, 2, 2, 128, 128, True, None, 0),
    (3, 130, 8, 4, 48, 80, True, [130, 0, 77], 0),
    (2, 33, 3, 1, 17, 65, True, [1, 32], 0),
    (1, 97, 2, 1, 130, 70, True, None, 0),
    (2, 150, 2, 2, 256, 256, True, [149, 128], 0),
    (1, 70, 2, 1, 255, 9, False, None, 0),
    (1, 700, 2, 1, 64, 64, True, None, 3),
    (3, 700, 2, 1, 72, 136, True, [640, 64, 0], 5),
    (2, 300, 8, 8, 256, 24, False, [300, 193], 2),
]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d-L%d-H%d.%d-N%d-P%d-s%d" % (c[:6] + c[8:]))
def test_forward(case, io):
    from state_space_sequence_amd import m3
    b, L, H, G, N, P, h0, lengths, nseg = case
    print("forward", case, io, flush=True)
    d = draw(L + N, b, L, H, G, N, P, io, h0, lengths)
    y, h = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=0.3, h0=d["h0"], lengths=d["lengths"],
                          nsegments=nseg)
    torch.cuda.synchronize()
    want, size = (reference(**d, scale=0.3, magnitude=m) for m in (False, True))
    check("y", y, want["y"], size["y"], factor(d, False))
    check("h", h, want["h"], size["h"], factor(d, True))


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d-L%d-H%d.%d-N%d-P%d-s%d" % (c[:6] + c[8:]))
def test_backward(case, io):
    from state_space_sequence_amd import m3
    b, L, H, G, N, P, h0, lengths, nseg = case
    print("backward", case, io, flush=True)
    d = draw(L + N + 1, b, L, H, G, N, P, io, h0, lengths, back=True)
    g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dy"], scale=0.3, h0=d["h0"], lengths=d["lengths"],
                       dh_final=d["dh_final"], nsegments=nseg)
    torch.cuda.synchronize()
    want, size = (reference(**d, scale=0.3, magnitude=m) for m in (False, True))
    for name in ("q", "k", "v"):
        check(name, g[name], want[name], size[name], factor(d, False))
    for name in ("log_decay", "h0"):
        check(name, g[name], want[name], size[name], factor(d, True))


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dims", [(1, 1, 1, 1, 1), (2, 4, 2, 64, 64), (3, 6, 2, 100, 37), (1, 2, 2, 256, 256),
                                  (40, 32, 8, 128, 64), (2, 3, 1, 33, 130), (300, 4, 4, 16, 24)])
def test_step(dims, io, state):
    from state_space_sequence_amd import m3
    b, H, G, N, P = dims
    d = draw(N, b, 1, H, G, N, P, io, h0=True)
    d["h0"] = d["h0"].to(state)
    h = d["h0"].clone()
    y = m3.linattn_step(d["q"][:, 0].contiguous(), d["k"][:, 0].contiguous(), d["v"][:, 0].contiguous(), d["log_decay"],
                        h, scale=0.3)
    torch.cuda.synchronize()
    want, size = (reference(**d, scale=0.3, magnitude=m) for m in (False, True))
    check("y", y[:, None], want["y"], size["y"], (N + 8) * 2.0 ** -24)
    # (the decay of a gone state, e^-40, and the product's and the sum's roundings)
    check("h", h, want["h"], size["h"], 64 * 2.0 ** -24)


def test_prompt_in_two_parts_and_steps():
    """A prompt, its continuation and single tokens from the states give what one call gives."""
    from state_space_sequence_amd import m3
    d = draw(5, 2, 150, 4, 2, 64, 64, torch.float32, h0=True)
    args = lambda a, b: [d[n][:, a:b].contiguous() for n in "qkv"] + [d["log_decay"]]
    y, h = m3.linattn_fwd(*args(0, 150), h0=d["h0"])
    y1, h1 = m3.linattn_fwd(*args(0, 77), h0=d["h0"])
    y2, h2 = m3.linattn_fwd(*args(77, 140), h0=h1)
    ys = [m3.linattn_step(*[d[n][:, t].contiguous() for n in "qkv"], d["log_decay"], h2) for t in range(140, 150)]
    got = torch.cat([y1, y2, torch.stack(ys, 1)], 1)
    torch.cuda.synchronize()
    size = reference(**d, scale=64 ** -0.5, magnitude=True)
    f = 2 * factor(d, True)  # both sides are off by at most one bound
    assert bool(((got - y).abs().cpu() <= f * size["y"]).all())
    assert bool(((h2 - h).abs().cpu() <= f * size["h"]).all())


def test_gradients_against_differences():
    """fp64 differences of the reference's loss agree with the kernel's gradients along random directions."""
    from state_space_sequence_amd import m3
    d = draw(8, 2, 40, 4, 2, 24, 16, torch.float32, h0=True, lengths=[40, 21], back=True)
    d["log_decay"] = torch.tensor([-0.5, -0.01, -0.2, -1.5]).cuda()
    g = m3.linattn_bwd(*(d[n] for n in ("q", "k", "v", "log_decay", "dy")), scale=0.3, h0=d["h0"],
                       lengths=d["lengths"], dh_final=d["dh_final"])
    fwd = {n: d[n].double().cpu() for n in ("q", "k", "v", "log_decay", "h0")}
    live = (torch.arange(40)[None] < d["lengths"].cpu()[:, None])[:, :, None, None]

    def loss(x):
        r = reference(**x, scale=0.3, lengths=d["lengths"])
        return float((r["y"] * d["dy"].double().cpu() * live).sum() + (r["h"] * d["dh_final"].double().cpu()).sum())

    gen = torch.Generator().manual_seed(1)
    for name in fwd:
        way = torch.randn(fwd[name].shape, generator=gen, dtype=torch.float64)
        eps = 1e-5
        num = (loss({**fwd, name: fwd[name] + eps * way}) - loss({**fwd, name: fwd[name] - eps * way})) / (2 * eps)
        terms = g[name].double().cpu() * way
        # differences in 64 bits: eps^2 of third derivatives and 1e-16 / eps of the loss; fp32 gradients
        assert abs(float(terms.sum()) - num) <= 1e-5 * float(terms.abs().sum()), name


def test_what_lies_behind_the_lengths_is_not_read():
    from state_space_sequence_amd import m3
    d = draw(3, 3, 100, 2, 1, 64, 64, torch.bfloat16, h0=True, lengths=[100, 33, 0], back=True)
    call = lambda x: (m3.linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], h0=x["h0"], lengths=x["lengths"]),
                      m3.linattn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dy"], h0=x["h0"], lengths=x["lengths"],
                                     dh_final=x["dh_final"]))
    (y, h), g = call(d)
    e = dict(d)
    for n in ("q", "k", "v", "dy"):
        e[n] = d[n].clone()
        e[n][1, 33:] = float("nan")
        e[n][2] = float("inf")
    (y2, h2), g2 = call(e)
    assert torch.equal(y, y2) and torch.equal(h, h2) and all(torch.equal(g[n], g2[n]) for n in g)
    assert not y[1, 33:].any() and not y[2].any() and torch.equal(h[2], d["h0"][2])
    for n in ("q", "k", "v"):
        assert not g[n][1, 33:].any() and not g[n][2].any()
    # lengths beyond the tensor, or negative, mean all and none of it
    f = dict(d, lengths=torch.tensor([1000, 33, -5], dtype=torch.int32).cuda())
    assert torch.equal(call(f)[0][0], y)


def test_empty_and_unwanted():
    from state_space_sequence_amd import m3
    d = draw(4, 2, 0, 2, 1, 32, 16, torch.float32, h0=True, back=True)
    y, h = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], h0=d["h0"])
    assert y.shape == (2, 0, 2, 16) and torch.equal(h, d["h0"])
    g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dy"], h0=d["h0"], dh_final=d["dh_final"])
    assert torch.equal(g["h0"], d["dh_final"]) and not g["log_decay"].any()
    e = draw(4, 0, 5, 2, 1, 32, 16, torch.float32, back=True)
    y, h = m3.linattn_fwd(e["q"], e["k"], e["v"], e["log_decay"])
    assert y.shape == (0, 5, 2, 16) and h.shape == (0, 2, 16, 32)
    assert not m3.linattn_bwd(e["q"], e["k"], e["v"], e["log_decay"], e["dy"])["log_decay"].any()
    f = draw(6, 2, 70, 2, 1, 32, 16, torch.float32, back=True)
    args = [f[n] for n in ("q", "k", "v", "log_decay")]
    y, h = m3.linattn_fwd(*args, want_state=False)
    assert h is None
    g = m3.linattn_bwd(*args, f["dy"])
    g2 = m3.linattn_bwd(*args, f["dy"], want_dh0=False, want_dlog_decay=False)
    assert set(g2) == {"q", "k", "v"} and all(torch.equal(g[n], g2[n]) for n in g2)


def test_captured_and_replayed():
    """A prompt, its gradients and a step in one graph, replayed with other inputs between."""
    from state_space_sequence_amd import m3
    d = draw(7, 1, 700, 2, 1, 64, 64, torch.bfloat16, h0=True, back=True)
    tok = [d[n][:, 0].contiguous() for n in "qkv"]

    def call(h):
        y, hf = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], h0=d["h0"], nsegments=3)
        g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dy"], h0=d["h0"], dh_final=d["dh_final"],
                           nsegments=3)
        h.copy_(hf)
        return [y, hf, m3.linattn_step(*tok, d["log_decay"], h), h] + [g[n] for n in sorted(g)]

    h = torch.empty(1, 2, 64, 64, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call(h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(h)
    for k in range(3):
        d["q"].copy_(torch.randn_like(d["q"]))
        d["dy"].mul_(0.5)
        eager = [t.clone() for t in call(torch.empty_like(h))]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(eager, out)), k


def test_on_another_stream():
    from state_space_sequence_amd import m3
    d = draw(9, 1, 700, 2, 1, 64, 64, torch.bfloat16)
    args = [d[n] for n in ("q", "k", "v", "log_decay")]
    y, h = m3.linattn_fwd(*args, nsegments=4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [m3.linattn_fwd(*args, nsegments=4, stream=s) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(y, a) and torch.equal(h, b) for a, b in outs)


def test_offsets_beyond_32_bits():
    """The last rows of tensors of more than 2^32 bytes (and 2^31 elements) are the right ones."""
    from state_space_sequence_amd import m3
    b, L, H, N, P = 1, 2 ** 19 + 65, 32, 128, 8
    torch.manual_seed(2)
    k, v = (torch.randn(b, L, 1, n, device="cuda").to(torch.bfloat16) for n in (N, P))
    q = torch.zeros(b, L, H, N, device="cuda", dtype=torch.bfloat16)
    q[:, -64:] = torch.randn(b, 64, H, N, device="cuda").to(torch.bfloat16)
    g = torch.full((H,), -1.0).cuda()  # tokens further than 200 back weigh less than e^-200
    y, h = m3.linattn_fwd(q, k, v, g, scale=0.3)
    torch.cuda.synchronize()
    sl = slice(L - 300, L)
    d = dict(q=q[:, sl], k=k[:, sl], v=v[:, sl], log_decay=g)
    want, size = (reference(**d, scale=0.3, magnitude=m) for m in (False, True))
    f = factor(d, False)
    check("y", y[:, -64:], want["y"][:, -64:], size["y"][:, -64:], f)
    check("h", h, want["h"], size["h"], factor(d, True))
    assert not y[:, :1000].any()


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dims", [(16, 70, 16, 4, 48, 72), (8, 40, 32, 32, 130, 64)])
def test_many_chains_of_unequal_sizes(dims, io):
    """Keys and values of different tiles on more workgroups than run at once."""
    from state_space_sequence_amd import m3
    b, L, H, G, N, P = dims
    d = draw(11, b, L, H, G, N, P, io, h0=True, lengths=[L - i % 3 for i in range(b)], back=True)
    want, size = (reference(**d, scale=0.3, magnitude=m) for m in (False, True))
    args, kw = (d["q"], d["k"], d["v"], d["log_decay"]), dict(scale=0.3, h0=d["h0"], lengths=d["lengths"])
    got = m3.linattn_bwd(*args, d["dy"], dh_final=d["dh_final"], **kw)
    torch.cuda.synchronize()
    for name in ("q", "k", "v", "h0"):
        check(name, got[name], want[name], size[name], factor(d, name == "h0"))


@pytest.mark.parametrize("nsegments", [1, 4])
def test_state_in_place(nsegments):
    """h_final may be h0 itself."""
    from state_space_sequence_amd import m3
    d = draw(12, 2, 600, 4, 2, 96, 80, torch.bfloat16, h0=True)
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    y, h = m3.linattn_fwd(*args, h0=d["h0"], nsegments=nsegments)
    h2 = d["h0"].clone()
    y2, same = m3.linattn_fwd(*args, h0=h2, h_final=h2, nsegments=nsegments)
    torch.cuda.synchronize()
    assert same is h2 and torch.equal(y, y2) and torch.equal(h, h2)


def test_most_heads_and_widest_rows():
    """65536 heads of 256 keys and values: the first and the last heads' rows, 2^25 and (gradients
    of shared keys, in fp32) 2^26 bytes apart, hold what a call of these heads alone gives."""
    from state_space_sequence_amd import m3
    H, L, D = 65536, 65, 256
    torch.manual_seed(3)
    k, v = (torch.randn(1, L, 1, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.zeros(1, L, H, D, device="cuda", dtype=torch.bfloat16)
    dy = torch.zeros(1, L, H, D, device="cuda", dtype=torch.bfloat16)
    some = [0, 1, H - 1]
    q[:, :, some] = torch.randn(1, L, 3, D, device="cuda").to(torch.bfloat16)
    dy[:, :, some] = torch.randn(1, L, 3, D, device="cuda").to(torch.bfloat16)
    ld = torch.full((H,), -0.1).cuda()
    y, _ = m3.linattn_fwd(q, k, v, ld, want_state=False)
    y2, _ = m3.linattn_fwd(q[:, :, some].contiguous(), k, v, ld[some], want_state=False)
    assert torch.equal(y[:, :, some], y2) and not y[:, :, 2:-1].any()
    del y
    got = m3.linattn_bwd(q, k, v, ld, dy, want_dh0=False, want_dlog_decay=False)
    want = m3.linattn_bwd(q[:, :, some].contiguous(), k, v, ld[some], dy[:, :, some].contiguous(), want_dh0=False,
                          want_dlog_decay=False)
    torch.cuda.synchronize()
    assert torch.equal(got["q"][:, :, some], want["q"]) and not got["q"][:, :, 2:-1].any()
    assert torch.equal(got["k"], want["k"]) and torch.equal(got["v"], want["v"])
