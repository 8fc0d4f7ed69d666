"""The buffers that the group norm's calls may write over: y over x or z, dx over x or dy, dz
over z, also where x and z are one tensor. The results are those of separate buffers, bit by bit."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("over,shape,groups", [("token", (2, 50, 64), 8), ("token", (70, 51), 3), ("sequence", (2, 300, 64), 8),
                                               ("sequence", (3, 33, 51), 3)])
def test_outputs_over_inputs(over, shape, groups, io):
    from state_space_sequence_amd import m3
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen)
    x, z, dy = (r(*shape).to(io).cuda() for _ in range(3))
    w, b = r(shape[-1]).cuda(), r(shape[-1]).cuda()
    fwd = lambda x, z, **kw: m3.group_norm_fwd(x, groups, w, b, z=z, over=over, **kw)
    bwd = lambda x, z, dy, **kw: m3.group_norm_bwd(x, groups, dy, w, b, z=z, over=over, **kw)
    y, g = fwd(x, z), bwd(x, z, dy)
    c = z.clone()
    assert torch.equal(fwd(x, c, y=c), y)
    for name in ("x", "dy"):
        t = {"x": x.clone(), "dy": dy.clone()}
        out = {k: torch.empty_like(g[k]) for k in g}
        out["x"] = t[name]
        got = bwd(t["x"], z, t["dy"], grads=out)
        assert all(torch.equal(got[k], g[k]) for k in g), name
    c = z.clone()
    got = bwd(x, c, dy, grads={"x": torch.empty_like(x), "z": c})
    assert torch.equal(got["x"], g["x"]) and torch.equal(got["z"], g["z"])
    # a gate that is x itself
    y, g = fwd(x, x), bwd(x, x, dy)
    c = x.clone()
    assert torch.equal(fwd(c, c, y=c), y)
    c = x.clone()
    got = bwd(c, c, dy, grads={"x": c, "z": torch.empty_like(x)})
    assert torch.equal(got["x"], g["x"]) and torch.equal(got["z"], g["z"])
    c = x.clone()
    got = bwd(c, c, dy, grads={"x": torch.empty_like(x), "z": c})
    assert torch.equal(got["x"], g["x"]) and torch.equal(got["z"], g["z"])
    for grads in ({"x": z, "z": torch.empty_like(x)}, {"x": torch.empty_like(x), "z": dy}, {"x": c, "z": c}):
        with pytest.raises(m3.M3Error):
            bwd(x, z, dy, grads=grads)
