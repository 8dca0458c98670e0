"""Dropout without a stored mask against its definition on Python's own integers."""
import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def numbers(seed):
    return torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=gen(seed))


def test_generator_words():
    """The published generator's own vectors for a counter and key of zeros and of ones."""
    assert ref.philox_words(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 2 ** 64 - 1
    assert ref.philox_words(ones, ones, ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 9), (17, 63), (64, 64), (33, 255), (2, 1000), (300, 12), (257, 3)])
@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("y_type", [BF16, F32])
def test_dropout(rows, cols, x_type, y_type):
    rng = numbers(rows + cols)
    x = torch.randn(rows, cols, generator=gen(1)).to(x_type)
    r = (2 * torch.randn(rows, cols, generator=gen(2))).to(y_type)
    for p, scale, residual, offset in ((0.1, 1.0, True, 0), (0.5, 0.3, False, 7), (0.0, 2.0, True, 0), (0.9, 1.0, False, -11)):
        y = torch.full((rows, cols), 9.0, dtype=y_type, device=DEV)
        coat.dropout(x.to(DEV), y, p=p, rng=rng.to(DEV), offset=offset, residual=r.to(DEV) if residual else None, scale=scale)
        v = scale * ref.dropped(ref.factors(rows, cols, p, rng, offset), ref.f64(x))
        want = ref.f64(r) + v if residual else v
        ref.check("y", y, want, 4 * ref.U32 * (v.abs() + want.abs()))
        dx = torch.empty(rows, cols, dtype=y_type, device=DEV)
        coat.dropout_backward(x.to(DEV), dx, p=p, rng=rng.to(DEV), offset=offset, scale=scale)
        ref.check("dx", dx, v, 4 * ref.U32 * v.abs())


def test_probability_is_rounded_and_never_one():
    rng, x = numbers(3), torch.ones(16, 64, device=DEV)
    for p in (2.0 ** -18, 0.99999999, 65535.4 / 65536, 1 / 65536):
        p32 = float(torch.tensor(p, dtype=torch.float32))
        if p32 >= 1.0:
            continue
        y = torch.empty(16, 64, device=DEV)
        coat.dropout(x, y, p=p, rng=rng.to(DEV))
        want = ref.factors(16, 64, p32, rng) if p32 >= 2.0 ** -17 else torch.ones(16, 64, dtype=torch.float64)
        ref.check("y", y, want, 4 * ref.U32 * want)


def test_dropped_places_take_nothing_in_and_others_keep_what_they_hold():
    rng = numbers(5)
    f = ref.factors(9, 40, 0.5, rng)
    for bad in (float("nan"), float("inf")):
        x = torch.where(f > 0, 1.0, bad).float().to(DEV)
        y = torch.empty(9, 40, device=DEV)
        coat.dropout(x, y, p=0.5, rng=rng.to(DEV))
        assert torch.equal(y.cpu(), f.float())
        x = torch.where(f > 0, bad, 1.0).float().to(DEV)
        coat.dropout(x, y, p=0.5, rng=rng.to(DEV))
        assert (torch.isfinite(y.cpu()) == (f == 0)).all()


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (8, 8)])
def test_strides_and_gaps(pad, shift):
    rng, rows, cols = numbers(8), 37, 45
    x = torch.randn(rows, cols, generator=gen(3))
    for t in (BF16, F32):
        a = torch.full((shift + rows * (cols + pad),), float("nan"), dtype=t, device=DEV)
        b = a.clone()
        xa, yb = (v[shift:].view(rows, cols + pad)[:, :cols] for v in (a, b))
        xa.copy_(x)
        coat.dropout(xa, yb, p=0.3, rng=rng.to(DEV))
        v = ref.dropped(ref.factors(rows, cols, 0.3, rng), ref.f64(xa))
        ref.check("y", yb, v, 4 * ref.U32 * v.abs())
        assert torch.isnan(b[shift:].view(rows, cols + pad)[:, cols:]).all() and torch.isnan(b[:shift]).all()


def test_in_place():
    rng = numbers(9).to(DEV)
    x, r = (torch.randn(50, 70, generator=gen(i)).to(BF16).to(DEV) for i in (1, 2))
    y = torch.empty_like(x)
    coat.dropout(x, y, p=0.2, rng=rng, residual=r)
    a, b = x.clone(), r.clone()
    coat.dropout(a, a, p=0.2, rng=rng, residual=r)
    coat.dropout(x, b, p=0.2, rng=rng, residual=b)
    assert torch.equal(a, y) and torch.equal(b, y)


def test_the_mask_of_the_linear_layer_is_the_same():
    rng = numbers(10).to(DEV)
    x = torch.randn(40, 24, generator=gen(4)).to(BF16).to(DEV)
    eye = torch.eye(24, dtype=BF16, device=DEV)
    y, z = torch.empty(40, 24, device=DEV), torch.empty(40, 24, device=DEV)
    coat.linear(x, eye, y, p=0.3, rng=rng, offset=2)
    coat.dropout(x, z, p=0.3, rng=rng, offset=2)
    assert torch.equal(y, z)


def test_seeds_steps_and_offsets_differ_and_add_up():
    x = torch.ones(64, 128, device=DEV)

    def mask(seed, step, offset):
        y = torch.empty_like(x)
        coat.dropout(x, y, p=0.5, rng=torch.tensor([seed, step], device=DEV), offset=offset)
        return y > 0

    a = mask(1, 10, 0)
    assert torch.equal(a, mask(1, 7, 3)) and torch.equal(mask(1, -1, 1), mask(1, 0, 0))
    for other in (mask(2, 10, 0), mask(1, 11, 0), mask(1, 10, 1), mask(1 + 2 ** 32, 10, 0), mask(1, 10 + 2 ** 32, 0)):
        same = float((a == other).float().mean())
        assert 0.4 < same < 0.6
    share = float(mask(3, 0, 0).float().mean())  # 8192 draws: five deviations are 0.028
    assert abs(share - 0.5) < 0.028


def test_large_matrix():
    """More blocks of 8 columns than one launch has threads; rows in the middle and at the end."""
    rng, rows, cols = numbers(12), 70001, 1027
    x = torch.ones(rows, cols, dtype=BF16, device=DEV)
    coat.dropout(x, x, p=0.25, rng=rng.to(DEV))
    for r in (0, 4095, 35000, 70000):
        f = ref.factors(rows, cols, 0.25, rng, 0, r, 1)
        ref.check("y", x[r:r + 1], f, 4 * ref.U32 * f)
