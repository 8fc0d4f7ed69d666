"""The operators as layers use them, forwards, backwards and token by token, against autograd over their definitions
in 64 bits on the CPU.

fp32 throughout: every operator passes its inputs' errors on, by a factor of at most a few (norms divide by deviations near 1,
states decay), and adds some 1e-6 of its values' size; ten in a row stay below 1e-4 of the norm of a tensor."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def near(got, want, tol=1e-4):
    want = want.detach()
    return float((got.double().cpu() - want).norm() / want.norm()) < tol


def rms(t, w, eps=1e-5):
    return t * (t * t).mean(-1, keepdim=True).add(eps).rsqrt() * w


def draws(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, k=1.0, m=0.0: (m + k * torch.randn(*s, generator=g)).cuda()


def leaf(t):
    return t.double().cpu().requires_grad_()


def recurrent_inputs():
    r = draws(1)
    b, L, C, D = 2, 150, 48, 32
    t = dict(stream=r(b, L, D), wp=r(D, k=0.1, m=1.0), wa=r(D, 3 * C, k=D ** -0.5), ld=-r(C).abs() - 0.05, wo=r(C, D, k=C ** -0.5),
             wz=r(D, D, k=D ** -0.5), post=r(D, k=0.1, m=1.0), scale=r(D, k=0.1, m=0.5), pre=r(D, k=0.1, m=1.0))
    return t, r(b, L, D), r(b, L, D), (b, L, C, D)


def recurrent_reference(t, dims):
    """The layer in 64 bits: (y, stream behind)."""
    b, L, C, D = dims
    u = rms(t["stream"], t["wp"])
    x, a, i = (u @ t["wa"]).split(C, -1)
    a = torch.exp(t["ld"] * torch.sigmoid(a))
    v = (1 - a * a).sqrt() * torch.sigmoid(i) * x
    h, hs = torch.zeros(b, C).double(), []
    for n in range(L):
        h = a[:, n] * h + v[:, n]
        hs.append(h)
    z = u @ t["wz"]
    o = rms(torch.stack(hs, 1) @ t["wo"], t["post"])
    R = 0.9 * t["stream"] + t["scale"] * torch.sigmoid(z) * o
    return rms(R, t["pre"]), R


def recurrent_layer(m3, t, dims, state=None):
    """The same by the operators; with a state one token, [b,D] in and out."""
    C = dims[2]
    u, _ = m3.block_norm_fwd(t["stream"], pre_weight=t["wp"], want_residual=False)
    x, a, i = ((u @ t["wa"]).split(C, -1))
    x, a, i = x.contiguous(), a.contiguous(), i.contiguous()
    kept = None
    if state is None:
        h, _, kept = m3.recurrence_fwd(x, a, t["ld"], input_gate=i, want_states=True)
    else:
        h = m3.recurrence_step(x, a, t["ld"], state, input_gate=i)
    o, z = h @ t["wo"], u @ t["wz"]
    y, R = m3.block_norm_fwd(o, t["stream"], z=z, activation="sigmoid", scale=t["scale"], post_norm=True, post_weight=t["post"],
                             pre_weight=t["pre"], residual_scale=0.9)
    return y, R, (u, x, a, i, kept, h, o, z)


def recurrent_backward(m3, t, saved, R, dy, dR):
    u, x, a, i, kept, h, o, z = saved
    g = m3.block_norm_bwd(o, R, dy, dR, z=z, activation="sigmoid", scale=t["scale"], post_norm=True, post_weight=t["post"],
                          pre_weight=t["pre"], residual_scale=0.9)
    out = {"post": g["post_weight"], "pre": g["pre_weight"], "scale": g["scale"]}
    flat = lambda q: q.reshape(-1, q.shape[-1])
    out["wo"], out["wz"] = flat(h).t() @ flat(g["x"]), flat(u).t() @ flat(g["z"])
    gr = m3.recurrence_bwd(x, a, t["ld"], g["x"] @ t["wo"].t().contiguous(), input_gate=i, states=kept)
    out["ld"] = gr["log_decay"]
    dxai = torch.cat([gr["x"], gr["decay_gate"], gr["input_gate"]], -1)
    out["wa"] = flat(u).t() @ flat(dxai)
    du = dxai @ t["wa"].t().contiguous() + g["z"] @ t["wz"].t().contiguous()
    first = m3.block_norm_bwd(t["stream"], t["stream"], du, g["residual"], pre_weight=t["wp"], want_dresidual=True)
    # (the first norm alone: its stream is its input, whose gradient is that of both uses)
    out["wp"], out["stream"] = first["pre_weight"], first["residual"]
    return out


def test_recurrent_layer():
    from state_space_sequence_amd import m3
    t, dy, dR, dims = recurrent_inputs()
    y, R, saved = recurrent_layer(m3, t, dims)
    got = recurrent_backward(m3, t, saved, R, dy, dR)
    torch.cuda.synchronize()
    ref = {n: leaf(v) for n, v in t.items()}
    ry, rR = recurrent_reference(ref, dims)
    ((ry * dy.double().cpu()).sum() + (rR * dR.double().cpu()).sum()).backward()
    assert near(y, ry) and near(R, rR)
    for n in ref:
        assert near(got[n], ref[n].grad), n


def test_recurrent_layer_token_by_token_and_captured():
    from state_space_sequence_amd import m3
    t, dy, dR, dims = recurrent_inputs()
    b, L, C, D = dims
    y, R, _ = recurrent_layer(m3, t, dims)
    state = torch.zeros(b, C, device="cuda")
    one = dict(t, stream=t["stream"][:, 0].contiguous())
    recurrent_layer(m3, one, dims, state)  # (library calls set up outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ty, tR, _ = recurrent_layer(m3, one, dims, state)
    state.zero_()
    for n in range(L):
        one["stream"].copy_(t["stream"][:, n])
        graph.replay()
        torch.cuda.synchronize()
        assert near(ty, y[:, n].double().cpu()) and near(tR, R[:, n].double().cpu()), n


def test_attention_layer_with_positions():
    """Rotary positions, linear attention, the gated norm of its heads, the norms around, and all the way back."""
    from state_space_sequence_amd import m3
    r = draws(2)
    b, L, H, G, N, P = 2, 90, 4, 2, 16, 8
    D = H * P
    ld = torch.tensor([-0.4, -0.1, -0.03, 0.0]).cuda()
    freqs = m3.rotary_frequencies(N, scaling="linear", factor=2.0, device="cuda")
    t = dict(q=r(b, L, H, N), k=r(b, L, G, N), v=r(b, L, G, P), z=r(b, L, D), stream=r(b, L, D), gw=r(D, k=0.1, m=1.0),
             gb=r(D, k=0.1), pre=r(D, k=0.1, m=1.0))
    dy, dR = r(b, L, D), r(b, L, D)
    q, k = m3.rotary(t["q"], t["k"], freqs, layout="interleaved")
    a, _ = m3.linattn_fwd(q, k, t["v"], ld)
    a = a.view(b, L, D)
    n = m3.group_norm_fwd(a, H, t["gw"], t["gb"], z=t["z"])
    y, R = m3.block_norm_fwd(n, t["stream"], pre_weight=t["pre"])
    g = m3.block_norm_bwd(n, R, dy, dR, pre_weight=t["pre"])
    gn = m3.group_norm_bwd(a, H, g["x"], t["gw"], t["gb"], z=t["z"])
    ga = m3.linattn_bwd(q, k, t["v"], ld, gn["x"].view(b, L, H, P))
    gq, gk = m3.rotary(ga["q"], ga["k"], freqs, layout="interleaved", backward=True)
    torch.cuda.synchronize()
    got = dict(q=gq, k=gk, v=ga["v"], z=gn["z"], stream=g["residual"], gw=gn["weight"], gb=gn["bias"], pre=g["pre_weight"])

    ref = {name: leaf(v) for name, v in t.items()}
    at = torch.arange(L).double()
    angle = at[:, None, None] * freqs.double().cpu()
    def turn(x):
        u, w = x[..., 0::2], x[..., 1::2]
        return torch.stack([u * angle.cos() - w * angle.sin(), u * angle.sin() + w * angle.cos()], -1).flatten(-2)
    q, k = turn(ref["q"]), turn(ref["k"]).repeat_interleave(H // G, 2)
    steps = (at[:, None] - at[None])
    decay = torch.where(steps >= 0, torch.exp(steps.clamp(min=0) * ld.double().cpu()[:, None, None]), torch.zeros(()).double())
    s = torch.einsum("blhn,bmhn->bhlm", q, k) * N ** -0.5 * decay
    a = torch.einsum("bhlm,bmhp->blhp", s, ref["v"].repeat_interleave(H // G, 2))
    u = (a - a.mean(-1, keepdim=True)) / (a.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
    o = (u.reshape(b, L, D) * ref["gw"] + ref["gb"]) * torch.nn.functional.silu(ref["z"])
    rR = ref["stream"] + o
    ry = rms(rR, ref["pre"])
    ((ry * dy.double().cpu()).sum() + (rR * dR.double().cpu()).sum()).backward()
    assert near(y, ry) and near(R, rR)
    for name in ref:
        # (a head's norm divides by its outputs' deviation, which is small for the first tokens)
        assert near(got[name], ref[name].grad, 1e-3), name
