"""The codes of 8-bit AdamW states at every power of two that a block can have: values exactly on the borders
between two codes and next to them.

A value is scaled by 2^-e, which powf gives within 2^-24, and the product rounds once, 2^-24 more: its code is
the nearest to a value that is off by 2^-23, so no further from the value itself than the nearest one is, and twice that.
A root has two roundings more (the square's halves in it).
"""
import pytest
import torch

import convolution_implicit_gemm_amd as c3d

pytestmark = pytest.mark.gpu

B = c3d.ADAMW_BLOCK


def codes():
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def block(off):
    """The largest code, the 126 values halfway between two adjacent ones, times 1 + off, and 0."""
    c = codes()
    return torch.cat([c[126:], (c[:-1] + c[1:]) / 2 * (1 + off), torch.zeros(1, dtype=torch.float64)])


@pytest.mark.parametrize("count", [1, 7, 246])
@pytest.mark.parametrize("off", [0.0, 2.0 ** -20, -2.0 ** -20])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codes_are_nearest_at_every_power(dtype, off, count):
    # beta 0: m is the gradient, and v its square
    powers = torch.linspace(-126, 119, count).round().double() if count > 1 else torch.tensor([-16.0], dtype=torch.float64)
    sign = torch.ones((len(powers), B), dtype=torch.float64)
    sign[:, 2::3] = -1.0
    g = (sign * block(off)[None] * torch.exp2(powers)[:, None]).flatten().to(dtype).cuda()
    n = g.numel()
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda:0") for _ in range(2))
    ms, vs = (torch.zeros(len(powers), dtype=torch.uint8, device="cuda:0") for _ in range(2))
    w = torch.zeros(n, device="cuda:0")
    c3d.adamw_step(c3d.adamw_list(None, [g], [m], [v], master=[w], m_scale=[ms], v_scale=[vs]),
                   c3d.make_adamw_hyper(1e-3, beta1=0.0, beta2=0.0))
    y = g.double().cpu().view(-1, B) / torch.exp2(powers)[:, None]
    assert torch.equal(ms.cpu().double(), powers + 127)
    least = (y.abs()[:, :, None] - codes()).abs().amin(2)
    got = m.cpu().view(torch.float8_e4m3fn).view(-1, B).double()
    assert bool(((got - y).abs() <= least + 2 * 2.0 ** -23 * y.abs()).all())
    assert torch.equal(torch.signbit(got)[y != 0], torch.signbit(y)[y != 0])
    # squares below 2^-126 or above 2^128 are not the value's any more
    whole = (powers >= -53) & (powers <= 54)
    assert torch.equal(vs.cpu().double()[whole], powers[whole] + 127)
    got, y, least = v.cpu().view(torch.float8_e4m3fn).view(-1, B).double()[whole], y.abs()[whole], least[whole]
    away = (y > 0) & (y < 2.0 ** -9)  # never 0 for what is not 0
    assert bool((got[away] == 2.0 ** -9).all())
    assert bool(((got - y).abs() <= least + 2 * 2.0 ** -22 * y)[~away].all())
