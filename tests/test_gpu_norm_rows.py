"""Group norms whose gradients are summed by workgroups that take several rows each: many short
sequences, and tokens of groups wider than a workgroup's registers. Against the definition in 64 bits, with
the bounds of the other tests of this norm."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_norm import check, draw, reference

pytestmark = pytest.mark.gpu


# (over, shape, groups): several rows a workgroup; one and several pieces of a group; a last workgroup with fewer rows
ROWS = [("sequence", (2500, 5, 64), 4), ("sequence", (4099, 2, 8), 1), ("sequence", (2100, 3, 51), 3),
        ("sequence", (2051, 70, 40), 1), ("token", (1500, 4104), 1), ("token", (1031, 6000), 2)]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("over,shape,groups", ROWS)
def test_several_rows_a_workgroup(over, shape, groups, gate, io):
    from state_space_sequence_amd import m3
    print("rows", over, shape, groups, gate, io, flush=True)
    x, z, dy, w, b = draw(9, shape, io, gate, True)
    lengths = None
    if over == "sequence":
        lengths = (torch.arange(shape[0]) * 7 % (shape[1] + 1)).to(torch.int32)
        lengths[0], lengths[-1] = 0, shape[1]
        lengths = lengths.cuda()
    kw = dict(z=z, over=over, lengths=lengths)
    y, g = m3.group_norm_fwd(x, groups, w, b, **kw), m3.group_norm_bwd(x, groups, dy, w, b, **kw)
    torch.cuda.synchronize()
    ref = reference(x, groups, w, b, z, "silu", over, None if lengths is None else lengths.cpu(), 1e-5, dy)
    check("y", y, ref["y"])
    for name in g:
        check(name, g[name], ref[name])
    # without the weights' gradients the others are the same bits
    some = {"x": torch.empty_like(x), **({"z": torch.empty_like(x)} if gate else {})}
    m3.group_norm_bwd(x, groups, dy, w, b, grads=some, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(some[n], g[n]) for n in some)
