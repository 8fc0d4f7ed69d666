"""Group norms over sequences whose partial sums a whole workgroup joins (more than 64 a group, and more than one a
thread), and calls whose tensors fit no cache, with the weights' gradients. Bounds as in the other tests of
this norm."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_norm import check, draw, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [False, True])
# partial sums of a group: 126, 512, 120 to 128 in pieces, 64 (and tensors that fit no cache)
@pytest.mark.parametrize("shape,groups,lengths", [((1, 1001, 1280), 32, [997]), ((1, 8192, 1024), 32, [8001]),
                                                  ((2, 300, 16384), 2, None), ((8, 4096, 1024), 16, None)])
def test_sequences(shape, groups, lengths, gate, io):
    from state_space_sequence_amd import m3
    print("joins", shape, groups, lengths, gate, io, flush=True)
    x, z, dy, w, b = draw(13, shape, io, gate, True)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    kw = dict(z=z, over="sequence", lengths=lens)
    y, g = m3.group_norm_fwd(x, groups, w, b, **kw), m3.group_norm_bwd(x, groups, dy, w, b, **kw)
    torch.cuda.synchronize()
    ref = reference(x, groups, w, b, z, "silu", "sequence", lengths, 1e-5, dy)
    check("y", y, ref["y"])
    for name in g:
        check(name, g[name], ref[name])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [False, True])
def test_weights_of_many_tokens(gate, io):
    """dw and db of 50000 tokens, whose tensors fit no cache."""
    from state_space_sequence_amd import m3
    n, C, G = 50000, 1024, 8
    x, z, dy, w, b = draw(14, (n, C), io, gate, True)
    g = m3.group_norm_bwd(x, G, dy, w, b, z=z)
    torch.cuda.synchronize()
    dw, db, sw, sb = (torch.zeros(C, dtype=torch.float64) for _ in range(4))
    for i in range(0, n, 10000):  # (the definition's sums are linear in the rows)
        some = lambda t: None if t is None else t[i:i + 10000].double()
        v, t, d = some(x).reshape(-1, G, C // G), some(z), some(dy)
        mu, r = v.mean(2, keepdim=True), 1 / torch.sqrt(v.var(2, correction=0, keepdim=True) + 1e-5)
        xh = ((v - mu) * r).reshape(-1, C)
        sh = (((v - mu).abs() + v.abs().amax(2, keepdim=True)) * r).reshape(-1, C)
        u, su = xh * w.double() + b.double(), sh * w.double().abs() + b.double().abs()
        t = u if t is None else t
        s = torch.sigmoid(t)
        du, sdu = (d * t * s, d.abs() * (t * s).abs()) if gate else (d * s * (1 + t * (1 - s)), d.abs() * (1.1 + 0.5 * su))
        dw += (du * xh).sum(0).cpu()
        db += du.sum(0).cpu()
        sw += (sdu * (sh + 1)).sum(0).cpu()
        sb += sdu.sum(0).cpu()
    check("weight", g["weight"], (dw, sw))
    check("bias", g["bias"], (db, sb))
