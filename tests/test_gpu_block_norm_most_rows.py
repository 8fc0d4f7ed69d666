"""Block norm of 2^34 rows and more, of one channel, as small calls on slices of them have it, and their weight's gradient."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

N = (1 << 34) + 37
ENDS = (slice(0, 50), slice((1 << 33) - 21, (1 << 33) + 30), slice(N - 53, N))


def test_two_to_the_34_rows_of_one_channel():
    from state_space_sequence_amd import m3
    torch.manual_seed(1)
    w = torch.full((1,), 0.75, device="cuda")
    x = torch.empty(N, 1, device="cuda", dtype=torch.bfloat16).fill_(1.0)
    dy = torch.empty_like(x).fill_(0.5)
    for s in ENDS:
        x[s].normal_()
        dy[s].normal_()
    cut = [(x[s].clone(), dy[s].clone()) for s in ENDS]
    print("block norm rows", N, flush=True)
    # x is the stream too; the gradient of the norm before the next block, in the place of dy
    g = m3.block_norm_bwd(x, x, dy, pre_weight=w, grads={"x": dy, "pre_weight": torch.empty_like(w)})
    torch.cuda.synchronize()
    want = 0.5 * (N - sum(len(a) for a, _ in cut)) / 1.00001 ** 0.5
    for s, (a, b) in zip(ENDS, cut):
        t = m3.block_norm_bwd(a, a, b, pre_weight=w)
        assert torch.equal(dy[s], t["x"])
        a, b = a.double(), b.double()
        want += float((b * a * (a * a + 1e-5).rsqrt()).sum())
    # 256 roundings of 2^-24 of a thread's sum, 96 of a term and the join
    assert abs(float(g["pre_weight"]) - want) <= 352 * 2.0 ** -24 * want
    print("forward", flush=True)
    y, _ = m3.block_norm_fwd(x, pre_weight=w, y=x, want_residual=False)
    torch.cuda.synchronize()
    for s, (a, _) in zip(ENDS, cut):
        assert torch.equal(y[s], m3.block_norm_fwd(a, pre_weight=w, want_residual=False)[0])
