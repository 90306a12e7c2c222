"""gelu in fp32 to the accuracy that its comment states (GPU).

Derived before the first run. Q evaluated in fp32 is 4.2e-7 off at most (step by step on
the CPU, 3 million points of [0, 14]). The exponential adds one unit in the last place,
1.2e-7, and the rounding of its correction, the product with it and that with z half of
one each, 6e-8: 7.2e-7 of gelu's value, of either sign of z. The slope is Phi(z) + z
phi(z) with the same errors in Phi and, without Q's, in phi, and two roundings: 7.2e-7 of
Phi and 4e-7 of |z| phi, which cancel near z = -0.75, so that only the sum bounds them.
"""

import math

import torch
import pytest

import backward_gate_up_amd as mlp
from tests._util import banner


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 70])  # the epilogue of a stream, and that of a tile
def test_gelu_in_fp32(T):
    banner(f"gelu fp32 T={T}")
    g = torch.Generator().manual_seed(1)
    z = torch.cat([torch.linspace(-12.5, 14, 200001), 26 * torch.rand(200000, generator=g) - 12.5, 0.5 * torch.randn(200000, generator=g),
                   torch.logspace(-8, 0, 999), -torch.logspace(-8, 0, 999)])
    z = z[: z.numel() // 8 * 8].cuda()
    w = torch.zeros(z.numel(), 8, device="cuda")
    w[:, 0] = z
    x = torch.zeros(T, 8, device="cuda")
    x[:, 0] = 1  # the layer's argument is z itself
    y, kept = mlp.linear_fwd(x, w, None, "gelu")
    assert torch.equal(kept[T - 1], z)
    d = z.double()
    cdf = 0.5 * torch.special.erfc(-d / math.sqrt(2))
    want = d * cdf
    assert ((y[T - 1].double() - want).abs() <= 7.2e-7 * want.abs()).all()
    density = d.abs() * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    dy = torch.zeros_like(y)
    dy[T - 1] = 1
    slope = mlp.linear_bwd(dy, x, w, kept, "gelu", (False, False, True))[2]
    want = cdf + d.sign() * density
    assert ((slope.double() - want).abs() <= 7.2e-7 * cdf + 4e-7 * density).all()
