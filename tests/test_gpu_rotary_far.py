"""Angles of any size (GPU): at t turns the fraction of a turn is off by at
most 2^-25 + 2^-46 t, against exact decimal fractions."""
import decimal
import math

import pytest
import torch

from _ops_ref import turn

pytestmark = pytest.mark.gpu

PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.mark.parametrize("top", [0, 10, 30])
def test_angles_keep_their_fraction_of_a_turn(top):
    import frame_aligned_window_gb300 as fw
    g = torch.Generator().manual_seed(5 + top)
    dim, tokens, half = 64, 64, 32
    freq = torch.exp2(top * torch.rand(half, generator=g, dtype=torch.float64))
    freq = freq * torch.rand(half, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 1 << 24, (tokens, 1), generator=g).float()
    x = torch.randn((1, 1, tokens, dim), generator=g)
    rot = fw.wsattn_rotary_plan(dim, pair_axis=[0] * half, pair_freq=freq.tolist())
    got = fw.wsattn_rotary(rot, x.cuda(), pos.cuda()).cpu().double()
    fraction = torch.empty((tokens, half), dtype=torch.float64)
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        for i in range(tokens):
            for j in range(half):
                t = decimal.Decimal(float(pos[i, 0])) * decimal.Decimal(float(freq[j])) / (2 * PI)
                fraction[i, j] = float(t - t.to_integral_value())
    want = turn(x.double(), 2 * math.pi * fraction, True)
    turns = pos.double() * freq / (2 * math.pi)
    size = x.double().abs()[..., 0::2] + x.double().abs()[..., 1::2]
    # beside the angle: sine and cosine 2 ulp (2^-23 each), products and sum 2^-24 each
    tol = (2 * math.pi * (2.0 ** -25 + 2.0 ** -46 * turns) + 2.0 ** -21) * size
    assert ((got - want).abs() <= tol.repeat_interleave(2, -1)).all()
    assert turns.max() > 2.0 ** (18 + top)
