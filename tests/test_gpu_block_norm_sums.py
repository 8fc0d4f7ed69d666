"""Weights' gradients of the block norm over many narrow rows: what several threads of a workgroup sum, over 256 rows together,
is joined in 64 bits.

Whole numbers, so that every sum below is exact but for a join in fp32: of every `apart` rows (those that a workgroup takes
at a time) one is 2^21, one 1, one -2^21. A thread's rows are `apart` from each other, at most 65 of them: its sum is a whole
number of 7 bits times its value. Beside 65 * 2^21 fp32 has steps of 16."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

GROUPS = 768  # workgroups of a call whose rows are more


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,apart,passes", [(16, 16, 17), (60, 16, 17), (256, 4, 65)])
def test_rows_that_several_threads_sum(C, apart, passes, io):
    from state_space_sequence_amd import m3
    if io == torch.bfloat16:
        C *= 2  # (eight channels a lane in place of four)
    n = GROUPS * apart * passes
    print("block norm sums", n, C, io, flush=True)
    some = torch.zeros(apart, device="cuda")
    some[:3] = torch.tensor([2.0 ** 21, 1.0, -2.0 ** 21])
    x = some.repeat(n // apart)[:, None].expand(n, C).to(io).contiguous()
    one = torch.ones_like(x)
    g = m3.block_norm_bwd(x, one, None, one, scale=torch.ones(C, device="cuda"), pre_norm=False)
    assert (g["scale"] == n // apart).all(), g["scale"]
