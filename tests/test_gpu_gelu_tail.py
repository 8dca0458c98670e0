"""GELU far below zero, where its values are small: they and the slopes keep their digits."""
import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def arguments():
    """Every bf16 number from -12.5 to -2^-7 (the distribution function leaves fp32's normal numbers at -13)."""
    bits = torch.arange(0, 2 ** 15, dtype=torch.int32).to(torch.int16)
    v = bits.view(BF16)
    return -v[(v >= 2.0 ** -7) & (v <= 12.5)]


def cdf(z):
    """Phi(z) by the complementary error function: torch.special.ndtr, one half of 1 + erf, is 4e-6 off at -6.8 and
    zero from -8.3 on, also in 64 bits."""
    return 0.5 * torch.special.erfc(-z / 2 ** 0.5)


def relative(z):
    """Of Phi(z): the approximation as it is computed 4e-7; its exponential's argument is rounded three times
    (half of z^2 times that), the exponential and the reciprocal are good to a step each, a few products."""
    return 4e-7 + (1.5 * z.square() + 16) * ref.U32


@pytest.mark.parametrize("y_type", [torch.float32, BF16])
def test_values(y_type):
    z = arguments()
    y = torch.empty(1, len(z), dtype=y_type, device=DEV)
    coat.linear(torch.ones(1, 1, dtype=BF16, device=DEV), z[:, None].to(DEV), y, act=coat.ACT_GELU)
    want = (z.double() * cdf(z.double()))[None]
    ref.check("y", y, want, (relative(z.double()) + 2 * ref.U32) * want.abs())
    coat.linear(torch.ones(1, 1, dtype=BF16, device=DEV), -z[:, None].to(DEV), y, act=coat.ACT_GELU)
    want = (-z.double() * cdf(-z.double()))[None]
    ref.check("y", y, want, (relative(torch.zeros(1, dtype=torch.float64)) + 2 * ref.U32) * want.abs())


def test_slopes():
    """Through the bias gradient of one token, which is the slope in fp32."""
    z = arguments()
    z = z[z <= -1.0]
    one, w = torch.ones(1, 1, dtype=BF16, device=DEV), torch.ones(len(z), 1, dtype=BF16, device=DEV)
    db = torch.empty(len(z), device=DEV)
    coat.linear_backward(torch.ones(1, len(z), device=DEV), one, w, None, None, db, act=coat.ACT_GELU, z=z[None].to(DEV))
    zz = z.double()
    phi, density = cdf(zz), torch.exp(-zz.square() / 2) / (2 * torch.pi) ** 0.5
    want = phi + zz * density
    ref.check("slope", db, want, relative(zz) * (phi + zz.abs() * density))
