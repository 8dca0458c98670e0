"""Epilogues and backward passes whose products are made in tiles of 256 x 256: dropout, residual and
activation in them, gradients through an activation and from fp32."""
import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
P = 0.25
# y, dx and dw: large tiles for the first two, for the first and the last
SIZES = [(8100, 4090, 1600), (4090, 8190, 2003)]


def factors(m, n, rng, offset):
    """0 or 1 / (1 - p): the mask as ``dropout`` has it, which is tested against its definition."""
    f = torch.empty(m, n, device=DEV)
    coat.dropout(torch.ones(m, n, dtype=BF16, device=DEV), f, p=P, rng=rng, offset=offset)
    return (f > 0).double() / (1 - P)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("y_type,act", [(BF16, "silu"), (F32, "gelu")])
def test_dropout_and_residual(size, y_type, act):
    m, n, k = size
    x, w, b, r, rng = (t.to(DEV) for t in inputs(m, n, k, 5, y_type))
    y, z = torch.empty(m, n, dtype=y_type, device=DEV), torch.empty(m, n, dtype=BF16, device=DEV)
    coat.linear(x, w, y, bias=b, act=ref.ACTS[act], z=z, residual=r, scale=0.7071, p=P, rng=rng, offset=3)
    f = factors(m, n, rng, 3)
    for rows in (slice(0, 260), slice(m // 2, m // 2 + 130), slice(m - 70, m)):
        want, ey, wz, ez = ref.linear(ref.f64(x[rows]), ref.f64(w), ref.f64(b), act, f[rows].cpu(), 0.7071, ref.f64(r[rows]))
        ref.check("y", y[rows], want, ey)
        ref.check("z", z[rows], wz, ez)
        own = ref.factors(m, n, P, rng.cpu(), 3, rows.stop - 1, 1)
        assert torch.equal(own, f[rows.stop - 1:rows.stop].cpu())


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dy_type,act", [(F32, "gelu"), (BF16, "silu"), (F32, "none")])
def test_backward(size, dy_type, act):
    m, n, k = size
    x, w, _, _, rng = (t.to(DEV) if t is not None else None for t in inputs(m, n, k, 6, BF16, False, False))
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    dy = torch.randn(m, n, generator=g, device=DEV).to(dy_type)
    z = (2 * torch.randn(m, n, generator=g, device=DEV)).to(BF16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device=DEV)
    coat.linear_backward(dy, x, w, dx, dw, db, act=ref.ACTS[act], z=z if act != "none" else None, scale=0.7071, p=P, rng=rng, offset=-2)
    want = ref.linear_backward(dy.double(), x.double(), w.double(), z.double(), act, factors(m, n, rng, -2), 0.7071)
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
        ref.check(name, got, *(t.cpu() for t in want[name]))
        off = (got.double() - want[name][0]).norm() / want[name][0].norm()
        # dz and the gradient are each rounded to bf16, in the mean of squares by half a step over the root of 3;
        # dbias is held in fp32
        assert float(off) < (1e-4 if name == "dbias" else 1.1 * 2 ** 0.5 * ref.half_step(BF16) / 3 ** 0.5), (name, float(off))
