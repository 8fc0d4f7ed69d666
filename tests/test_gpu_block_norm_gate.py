"""The gate of the block norm beside an fp32 stream, which takes its value as it is: against 64 bits.

Relative bound: the exponential is off by at most two steps (4 * 2^-24), 1 + e by half of one, the reciprocal by one, the product
with z by half of one: 8 * 2^-24. All else is multiplied by 1. In the gradients of bf16 blocks the exponential's
argument is rounded: |z| 2^-23 more."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = 8 * 2.0 ** -24


def values():
    """Every bf16 number of a size from 1/64 to 80, of both signs."""
    z = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    return z[(z.abs() >= 2.0 ** -6) & (z.abs() <= 80)]


def check(name, got, want, more=0.0):
    off = (got.double().cpu() - want).abs() / want.abs()
    print("  %s: off by %.2f * 2^-24" % (name, float(off.max()) * 2 ** 24), flush=True)
    assert (off <= BOUND + more).all(), name


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_the_gate_beside_an_fp32_stream(io, wide, act):
    from state_space_sequence_amd import m3
    z = values().to(io)
    if wide:  # rows that the registers do not hold
        z = torch.cat([z] * (1 + 16384 // len(z)))
    print("block norm gate", len(z), act, io, flush=True)
    v = z.double()
    want = torch.sigmoid(v) * (v if act == "silu" else 1)
    z = z[None].cuda()
    x, one = torch.ones_like(z), torch.ones(z.shape, device="cuda")
    kw = dict(z=z, activation=act, pre_norm=False)
    _, R = m3.block_norm_fwd(x, residual_dtype=torch.float32, **kw)
    check("R", R[0], want)
    g = m3.block_norm_bwd(x, R, None, one, scale=one[0], **kw)
    check("dscale", g["scale"], want, v.abs() * 2.0 ** -23 if io == torch.bfloat16 else 0.0)
