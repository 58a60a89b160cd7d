"""The sines and cosines of the rotation in 32 bits (GPU).

Rotating (1, 0) gives (cos, sin) with no other rounding (products with 1 and 0 are exact).  The angle is taken as
the remainder x to its nearest quarter turn, |x| <= 1/8, and in steps of 2^-24 the numbers are off by
- the angle: x to 32 bits 2^-28 turns, its dropped low half 2^-32: 0.39 + 0.03 radians, times at most 0.71;
- cos = 1 - 0.29: the square's rounding 0.29, its factor's 0.29, the constant's 0.15, higher terms 0.05, the result's
  half step 0.5: 1.6 with the angle;
- sin <= 0.71: 0.25 in the terms behind the first, the half step 0.5: less.
The frequency's rounding adds |pos| 2^-54 turns."""

import math

import pytest
import torch

from blockwise_long_context_b200 import binding as lvx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [100, 2 ** 20, 2 ** 31 - 1])
@pytest.mark.parametrize("inverse", [False, True])
def test_sines_and_cosines(most, inverse):
    S, n = 20000, 64
    g = torch.Generator().manual_seed(most)
    pos = torch.randint(-most, most + 1, (1, 1, S), generator=g).to(torch.int32).cuda()
    inv = (1e4 ** -(torch.arange(n, dtype=torch.float64) / n)).float().cuda()
    axis = torch.zeros(n, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, S, 1, 2 * n, device="cuda")
    x[..., :n] = 1
    y, _ = lvx.rope_axes(x, None, pos, inv, axis, inverse=inverse)
    angle = pos[0, 0].double()[:, None] * inv.double()
    want = torch.cat((angle.cos(), -angle.sin() if inverse else angle.sin()), -1)
    # (the 64-bit angle itself is off by half a step of its own)
    bound = 1.6 * 2.0 ** -24 + 2 * math.pi * most * 2.0 ** -54 + most * 2.0 ** -53
    assert float((y[0, :, 0].double() - want).abs().max()) <= bound
    # on the circle as well as its points are
    assert float(((y[0, :, 0, :n].double() ** 2 + y[0, :, 0, n:].double() ** 2) - 1).abs().max()) <= 4 * bound


def test_whole_quarter_turns():
    """A frequency of a quarter turn, as near as 32 bits have it: the four quadrants and their borders."""
    inv = torch.full((4,), math.pi / 2, device="cuda")
    pos = torch.arange(-40, 40, dtype=torch.int32, device="cuda").view(1, 1, 80)
    x = torch.zeros(1, 80, 1, 8, device="cuda")
    x[..., :4] = 1
    y, _ = lvx.rope_axes(x, None, pos, inv, torch.zeros(4, dtype=torch.int32, device="cuda"))
    angle = pos[0, 0].double()[:, None] * inv.double()
    want = torch.cat((angle.cos(), angle.sin()), -1)
    assert float((y[0, :, 0].double() - want).abs().max()) <= 1.6 * 2.0 ** -24 + 80 * 2.0 ** -53
