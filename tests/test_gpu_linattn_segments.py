"""Linear attention over many segments whose states survive: the split that the library picks
for long sequences on few chains, joins of more than eight segments, states of keys and values that no other
workgroup reads, and the decay's gradient over many chains. Bounds as in the other tests of
this operator; decays are near 1, so every segment's state reaches the last one."""
from __future__ import annotations

import pytest
import torch

from tests.linattn_reference import reference
from tests.test_gpu_linattn import check, draw, factor

pytestmark = pytest.mark.gpu

# (b, L, H, G, N, P, lengths, nsegments): 0 lets the library pick
CASES = [
    (1, 2400, 2, 2, 128, 64, None, 0),            # 19 segments of 2 chunks (bf16), 25 of 3 (fp32)
    (2, 2301, 2, 1, 64, 64, [2301, 1300], 0),
    (2, 1301, 4, 2, 72, 136, [1111, 1301], 17),   # two tiles of values, shared heads
    (3, 1100, 2, 2, 256, 24, [0, 1100, 65], 9),
]


def near_one(d):
    H = d["log_decay"].shape[0]
    d["log_decay"] = torch.tensor([0.0, -1e-4, -2e-3, -1e-5][:H]).cuda()
    return d


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d-L%d-H%d.%d-N%d-P%d" % c[:6])
def test_states_of_many_segments(case, io):
    from state_space_sequence_amd import m3
    b, L, H, G, N, P, lengths, nseg = case
    print("segments", case, io, flush=True)
    d = near_one(draw(L, b, L, H, G, N, P, io, True, lengths, back=True))
    kw = dict(scale=0.3, h0=d["h0"], lengths=d["lengths"], nsegments=nseg)
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    shape = m3.linattn_shape(d["q"], d["v"], nseg)
    segments = m3.linattn_workspace_bytes(shape) // (4 * b * H * N * P)
    assert segments >= 9, segments
    y, h = m3.linattn_fwd(*args, **kw)
    g = m3.linattn_bwd(*args, d["dy"], dh_final=d["dh_final"], **kw)
    torch.cuda.synchronize()
    want, size = (reference(**d, scale=0.3, magnitude=m) for m in (False, True))
    check("y", y, want["y"], size["y"], factor(d, False))
    check("h", h, want["h"], size["h"], factor(d, True))
    for name in ("q", "k", "v", "log_decay", "h0"):
        check(name, g[name], want[name], size[name], factor(d, name in ("log_decay", "h0")))


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dims", [(16, 70, 16, 4, 48, 72), (8, 40, 32, 32, 130, 64)])
def test_decay_gradient_of_many_chains(dims, io):
    from state_space_sequence_amd import m3
    b, L, H, G, N, P = dims
    d = draw(11, b, L, H, G, N, P, io, h0=True, lengths=[L - i % 3 for i in range(b)], back=True)
    want, size = (reference(**d, scale=0.3, magnitude=m) for m in (False, True))
    g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dy"], dh_final=d["dh_final"], scale=0.3, h0=d["h0"],
                       lengths=d["lengths"])
    torch.cuda.synchronize()
    check("log_decay", g["log_decay"], want["log_decay"], size["log_decay"], factor(d, True))
