"""The linear layer with its epilogue and its backward pass against plain 64-bit forms."""
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


def strided(t, ld=None, shift=0):
    """t on the GPU, rows ld apart, its first element `shift` elements behind a multiple of 256 bytes; the gaps are NaN."""
    if t is None:
        return None
    rows, cols = t.shape
    ld = cols if ld is None else ld
    flat = torch.full((shift + rows * ld + 64,), float("nan"), dtype=t.dtype, device=DEV)
    v = flat[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(t)
    return v


def inputs(m, n, k, seed, y_type, bias=True, residual=True):
    g = gen(seed)
    x = torch.randn(m, k, generator=g).to(BF16)
    w = (torch.randn(n, k, generator=g) / max(1, k) ** 0.5).to(BF16)
    b = (0.3 * torch.randn(n, generator=g)).to(BF16 if seed % 2 else F32) if bias else None
    r = (3 * torch.randn(m, n, generator=g)).to(y_type) if residual else None
    rng = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=g)
    return x, w, b, r, rng


def run_linear(m, n, k, act, p, y_type, seed, bias=True, residual=True, keep=True, pad=(0, 0, 0), shift=0, scale=0.7071, offset=5,
               sample=None):
    x, w, b, r, rng = inputs(m, n, k, seed, y_type, bias, residual)
    xd, wd = strided(x, k + pad[0], shift), strided(w, k + pad[1], shift)
    yd = strided(torch.zeros(m, n, dtype=y_type), n + pad[2], shift)
    zd = strided(torch.zeros(m, n, dtype=BF16), n + pad[2], shift) if keep else None
    rd = strided(r, n + pad[2], shift)
    coat.linear(xd, wd, yd, bias=b.to(DEV) if bias else None, act=ref.ACTS[act], z=zd, residual=rd, scale=scale, p=p, rng=rng.to(DEV),
                offset=offset)
    torch.cuda.synchronize()
    rows = slice(0, m) if sample is None else slice(*sample)
    f = ref.factors(m, n, p, rng, offset, rows.start, rows.stop - rows.start)
    y, ey, z, ez = ref.linear(ref.f64(x)[rows], ref.f64(w), ref.f64(b), act, f, scale, ref.f64(r)[rows] if residual else None)
    ref.check("y", yd[rows], y, ey)
    if keep:
        ref.check("z", zd[rows], z, ez)
    for t in (yd, zd):  # what lies between the rows is as it was
        if t is not None and pad[2]:
            whole = torch.as_strided(t, (m, n + pad[2]), (n + pad[2], 1), t.storage_offset())
            assert torch.isnan(whole[:, n:]).all()


SIZES = [(1, 1, 1), (1, 8, 16), (2, 3, 5), (1, 333, 520), (5, 77, 64), (16, 130, 129), (17, 40, 8), (31, 64, 200), (33, 129, 72),
         (64, 64, 64), (65, 66, 67), (100, 260, 136), (129, 257, 191), (257, 300, 328)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("y_type", [BF16, F32])
def test_linear_sizes(size, y_type):
    run_linear(*size, "gelu", 0.25, y_type, sum(size))


@pytest.mark.parametrize("act", list(ref.ACTS))
@pytest.mark.parametrize("m", [3, 70])
def test_linear_activations(act, m):
    for p in (0.0, 0.4):
        for bias, residual, keep in ((True, False, True), (False, True, False), (False, False, True)):
            run_linear(m, 72, 48, act, p, F32, 7 + m, bias, residual, keep)


@pytest.mark.parametrize("pad,shift", [((8, 8, 8), 0), ((1, 0, 3), 0), ((0, 5, 0), 0), ((0, 0, 0), 1), ((3, 8, 1), 4), ((8, 16, 0), 8)])
@pytest.mark.parametrize("m", [4, 40, 150])
def test_linear_strides_and_alignments(pad, shift, m):
    run_linear(m, 136, 96, "silu", 0.1, BF16, 11, pad=pad, shift=shift)


@pytest.mark.parametrize("size", [(300, 1100, 640), (700, 300, 2048), (130, 128, 5000), (24, 1000, 4100), (1, 2500, 3000)])
def test_linear_long(size):
    run_linear(*size, "silu", 0.0, F32, 3)


def test_linear_many_tiles():
    """More tiles than workgroups of one round, with a last row of tiles that is not full."""
    run_linear(4200, 4300, 96, "gelu_tanh", 0.1, BF16, 5, sample=(4100, 4140))
    run_linear(4200, 4300, 96, "relu", 0.0, F32, 6, sample=(0, 300))


@pytest.mark.parametrize("size,pad,shift", [((8100, 4090, 1600), (0, 0, 0), 0), ((4090, 8190, 2003), (0, 0, 1), 0), ((8192, 4096, 1536), (8, 0, 0), 8),
                                            ((4300, 12288, 1032), (0, 0, 0), 0)])
def test_large_tiles(size, pad, shift):
    """Sizes whose products are made in large tiles, several of them a workgroup, with edges and a short last step."""
    m, n, k = size
    run_linear(m, n, k, "gelu", 0.0, BF16, 5, pad=pad, shift=shift, sample=(m - 70, m))
    run_linear(m, n, k, "silu", 0.0, F32, 6, pad=pad, shift=shift, sample=(200, 300))
    x, w, _, _, _ = inputs(m, n, k, 7, BF16, False, False)
    dy = torch.randn(m, n, generator=gen(8)).to(BF16)
    dx, dw = torch.empty(m, k, dtype=BF16, device=DEV), torch.empty(n, k, dtype=BF16, device=DEV)
    db = torch.empty(n, device=DEV)
    coat.linear_backward(strided(dy, n + pad[0], shift), strided(x, k + pad[1], shift), strided(w, k + pad[1], shift), dx, dw, db, scale=0.5)
    D, X, W = (t.to(DEV).double() for t in (dy, x, w))
    for got, want, terms in ((dx, 0.5 * (D @ W), 0.5 * (D.abs() @ W.abs())),
                             (dw, 0.5 * (D.t().contiguous() @ X), 0.5 * (D.abs().t().contiguous() @ X.abs()))):
        depth = n if got is dx else m
        ref.check("gradient", got, want.cpu(), (ref.sum_error(terms, depth) + 4 * ref.U32 * terms).cpu())
    assert float((db.double() - 0.5 * D.sum(0)).abs().max()) < 1e-3


def test_rows_past_what_tiles_take():
    """Rows of 2^22 values and more."""
    m, n, k = 3, 5, (1 << 22) + 8
    g = gen(3)
    x, w = torch.randn(m, k, generator=g).to(BF16).to(DEV), torch.randn(n, k, generator=g).to(BF16).to(DEV)
    y = torch.empty(m, n, device=DEV)
    coat.linear(x, w, y)
    X, W = x.double(), w.double()
    # sums of 2^18 instructions of independent signs: the mean of squares, not the worst case
    assert float((y.double() - X @ W.t().contiguous()).abs().max()) < 1e-3 * k ** 0.5
    dy = torch.randn(m, n, generator=g).to(BF16).to(DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    coat.linear_backward(dy, x, w, dx, dw)
    D = dy.double()
    for got, want, mag in ((dx, D @ W, D.abs() @ W.abs()), (dw, D.t().contiguous() @ X, D.abs().t().contiguous() @ X.abs())):
        off = (got.double() - want).abs()
        assert bool((off <= 2.0 ** -8 * want.abs() + 1e-5 * mag + 1e-30).all())


def test_rows_far_apart():
    """Rows nearly 2^22 elements apart, over 2^31 elements in all: the same results as close together."""
    m, n, k, ld = 600, 200, 64, (1 << 22) - 8
    flat = torch.empty(m * ld, dtype=BF16, device=DEV)
    x = flat.view(m, ld)[:, :k]
    x.copy_(torch.randn(m, k, generator=gen(4)))
    close, w = x.contiguous(), torch.randn(n, k, generator=gen(5)).to(BF16).to(DEV)
    y, z = torch.empty(m, n, device=DEV), torch.empty(m, n, device=DEV)
    coat.linear(x, w, y)
    coat.linear(close, w, z)
    assert torch.equal(y, z)
    labels = torch.randint(0, n, (m,), generator=gen(6)).to(DEV)
    labels[::3] = -100
    out = []
    for t in (x, close):
        loss, lse = torch.empty(m, device=DEV), torch.empty(m, device=DEV)
        dx, dw = torch.empty_like(close), torch.empty_like(w)
        coat.linear_cross_entropy(t, w, labels, loss, lse)
        coat.linear_cross_entropy_backward(t, w, labels, lse, torch.ones(1, device=DEV), dx, dw)
        out.append((loss, lse, dx, dw))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_linear_extremes():
    """No columns of x, no rows, and what NaN and Inf reach."""
    x, w, b, r, rng = inputs(4, 24, 16, 1, F32)
    y = torch.full((4, 24), 7.0, device=DEV)
    coat.linear(torch.empty(4, 0, dtype=BF16, device=DEV), torch.empty(24, 0, dtype=BF16, device=DEV), y, bias=b.to(DEV))
    assert torch.equal(y.cpu(), b.float().expand(4, 24))
    coat.linear(torch.empty(0, 16, dtype=BF16, device=DEV), w.to(DEV), torch.empty(0, 24, device=DEV))
    coat.linear(x.to(DEV), torch.empty(0, 16, dtype=BF16, device=DEV), torch.empty(4, 0, device=DEV))
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    for act in ref.ACTS:
        coat.linear(x.to(DEV), w.to(DEV), y, bias=b.to(DEV), act=ref.ACTS[act])
        got = y.cpu()
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[3]).all() and torch.isnan(got[1]).all()
        assert not torch.isfinite(got[2])[w[:, 5] > 0].any()
        coat.linear(x.to(DEV), w.to(DEV), y, act=ref.ACTS[act], p=0.5, rng=rng.to(DEV))
        f = ref.factors(4, 24, 0.5, rng)
        assert (y.cpu()[1:3][f[1:3] == 0] == 0).all()  # dropped whatever it was


def test_linear_large_values():
    """Activations where an exponential over- or underflows."""
    z = torch.tensor([[-3e38, -1e20, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e20, 3e38]])
    one = torch.ones(1, 1, dtype=BF16, device=DEV)
    w = z.t().to(BF16).to(DEV)
    for act in ref.ACTS:
        y = torch.empty(1, 11, device=DEV)
        coat.linear(one, w, y, act=ref.ACTS[act])
        zz = w.double().cpu().t()
        want = ref.activation(zz, act) if act != "gelu_tanh" else zz * torch.sigmoid(torch.clamp(1.6 * zz ** 3, -1e4, 1e4))
        if act == "gelu_tanh":
            want[0, 4:7] = ref.activation(zz[:, 4:7], act)
        assert torch.isfinite(y[0, 1:-1]).all(), act
        ref.check(act, y[:, 1:-1], want[:, 1:-1], ref.ACT * zz[:, 1:-1].abs())
        dx = torch.empty(1, 1, dtype=BF16, device=DEV)
        dw = torch.empty(11, 1, dtype=BF16, device=DEV)
        coat.linear_backward(torch.ones(1, 11, device=DEV), one, w, dx, dw, act=ref.ACTS[act], z=w.t().contiguous())
        slope = {"none": [1.0] * 11}.get(act, [0.0] * 5 + [0.0 if act == "relu" else 0.5] + [1.0] * 5)
        assert torch.allclose(dw.cpu().float()[1:-1, 0], torch.tensor(slope)[1:-1], atol=0.004), act


@pytest.mark.parametrize("m", [1, 20, 300])
def test_linear_repeats_and_in_place_residual(m):
    x, w, b, r, rng = [t.to(DEV) for t in inputs(m, 200, 328, 2, BF16)]
    how = dict(bias=b, act=coat.ACT_SILU, p=0.3, rng=rng, scale=0.5)
    y0, y1, z0, z1 = (torch.empty(m, 200, dtype=BF16, device=DEV) for _ in range(4))
    coat.linear(x, w, y0, residual=r, z=z0, **how)
    coat.linear(x, w, y1, residual=r, z=z1, **how)
    assert torch.equal(y0, y1) and torch.equal(z0, z1)
    coat.linear(x, w, r, residual=r, **how)
    assert torch.equal(r, y0)


# ---------------------------------------------------------------- backward

def run_backward(m, n, k, act, p, dy_type, seed, bias=True, pad=(0, 0, 0), shift=0, scale=0.7071, offset=-3, bias_type=F32,
                 rows=None):
    x, w, _, _, rng = inputs(m, n, k, seed, BF16, False, False)
    g = gen(seed + 1)
    dy = torch.randn(m, n, generator=g).to(dy_type)
    z = (2 * torch.randn(m, n, generator=g)).to(BF16) if act != "none" else None
    dx, dw = strided(torch.zeros(m, k, dtype=BF16), k + pad[2], shift), strided(torch.zeros(n, k, dtype=BF16), k + pad[2], shift)
    db = torch.full((n,), 9.0, dtype=bias_type, device=DEV) if bias else None
    coat.linear_backward(strided(dy, n + pad[0], shift), strided(x, k + pad[1], shift), strided(w, k + pad[1], shift), dx, dw, db,
                         act=ref.ACTS[act], z=strided(z, n + pad[0], shift), scale=scale, p=p, rng=rng.to(DEV), offset=offset)
    torch.cuda.synchronize()
    want = ref.linear_backward(ref.f64(dy), ref.f64(x), ref.f64(w), ref.f64(z), act, ref.factors(m, n, p, rng, offset), scale)
    ref.check("dx", dx, *want["dx"])
    ref.check("dw", dw, *want["dw"])
    if bias:
        ref.check("dbias", db, *want["dbias"])
    if pad[2]:
        for t in (dx, dw):
            whole = torch.as_strided(t, (t.shape[0], k + pad[2]), (k + pad[2], 1), t.storage_offset())
            assert torch.isnan(whole[:, k:]).all()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dy_type", [BF16, F32])
def test_backward_sizes(size, dy_type):
    run_backward(*size, "silu", 0.25, dy_type, sum(size), bias_type=BF16 if dy_type == BF16 else F32)


@pytest.mark.parametrize("act", list(ref.ACTS))
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_backward_activations(act, p):
    for scale in (1.0, 0.3):
        for dy_type in (BF16, F32):
            run_backward(66, 72, 48, act, p, dy_type, 3, scale=scale)


@pytest.mark.parametrize("pad,shift", [((8, 8, 8), 0), ((1, 0, 3), 0), ((0, 5, 0), 0), ((0, 0, 0), 1), ((3, 8, 1), 4), ((8, 16, 0), 8)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_strides_and_alignments(pad, shift, act):
    for dy_type in (BF16, F32):
        run_backward(150, 136, 96, act, 0.0, dy_type, 11, pad=pad, shift=shift, scale=1.0)


@pytest.mark.parametrize("size", [(300, 1100, 640), (2100, 300, 200), (130, 5000, 128), (1, 1000, 640), (2500, 72, 40)])
def test_backward_long(size):
    run_backward(*size, "none", 0.0, BF16, 3, scale=1.0)
    run_backward(*size, "gelu", 0.0, F32, 4)


def test_backward_parts_alone():
    """Each gradient is the same, bit for bit, whichever others are asked for."""
    x, w, _, _, rng = [t.to(DEV) if t is not None else None for t in inputs(90, 72, 64, 2, BF16, False, False)]
    g = gen(9)
    dy, z = torch.randn(90, 72, generator=g).to(DEV), torch.randn(90, 72, generator=g).to(BF16).to(DEV)
    how = dict(act=coat.ACT_GELU, z=z, p=0.2, rng=rng, scale=2.0)
    new = lambda: (torch.empty(90, 64, dtype=BF16, device=DEV), torch.empty(72, 64, dtype=BF16, device=DEV), torch.empty(72, device=DEV))
    whole = new()
    coat.linear_backward(dy, x, w, *whole, **how)
    for i in range(3):
        one = new()
        coat.linear_backward(dy, x, w, *[t if j == i else None for j, t in enumerate(one)], **how)
        assert torch.equal(one[i], whole[i])


def test_backward_empty():
    x, w, _, _, _ = [t.to(DEV) if t is not None else None for t in inputs(4, 24, 16, 1, F32, False, False)]
    dx, dw, db = torch.ones(4, 16, dtype=BF16, device=DEV), torch.ones(24, 16, dtype=BF16, device=DEV), torch.ones(24, device=DEV)
    coat.linear_backward(torch.empty(0, 24, device=DEV), x[:0], w, dx[:0], dw, db)
    assert (dw == 0).all() and (db == 0).all() and (dx == 1).all()
    coat.linear_backward(torch.empty(4, 0, device=DEV), x, w[:0], dx, dw[:0], db[:0])
    assert (dx == 0).all()
    db.fill_(1.0)
    coat.linear_backward(torch.ones(4, 24, device=DEV), x[:, :0], w[:, :0], dx[:, :0], dw[:, :0], db)
    assert (db == 4).all()


def test_backward_dropped_places_take_nothing_in():
    x, w, _, _, rng = inputs(6, 24, 16, 1, F32, False, False)
    f = ref.factors(6, 24, 0.5, rng)
    dy, z = torch.ones(6, 24), torch.ones(6, 24)
    dy[f == 0], z[f == 0] = float("inf"), float("nan")
    dx, dw, db = torch.ones(6, 16, dtype=BF16, device=DEV), torch.ones(24, 16, dtype=BF16, device=DEV), torch.ones(24, device=DEV)
    coat.linear_backward(dy.to(DEV), x.to(DEV), w.to(DEV), dx, dw, db, act=coat.ACT_GELU, z=z.to(BF16).to(DEV), p=0.5, rng=rng.to(DEV))
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("size", [(1, 1, 1), (1, 2048, 72), (3, 40, 17), (32, 64, 200), (250, 8, 40), (2048, 1, 9), (20, 100, 1000)])
@pytest.mark.parametrize("dy_type,act", [(F32, "none"), (F32, "relu"), (BF16, "gelu"), (F32, "silu")])
@pytest.mark.parametrize("shift", [0, 1])
def test_few_values_are_not_rounded_on_the_way(size, dy_type, act, shift):
    """Up to 2048 values of dz: what the first bf16 term leaves counts, so that only the stored rounding is left."""
    m, n, k = size
    x, w, _, _, rng = inputs(m, n, k, 5, F32, False, False)
    g = gen(6)
    dy, z = torch.randn(m, n, generator=g).to(dy_type), (2 * torch.randn(m, n, generator=g)).to(BF16)
    f = ref.factors(m, n, 0.3, rng)
    want = ref.linear_backward(ref.f64(dy), ref.f64(x), ref.f64(w), ref.f64(z), act, f, 0.7, terms=2)
    dx, dw = torch.empty(m, k, dtype=BF16, device=DEV), torch.empty(n, k, dtype=BF16, device=DEV)
    how = dict(act=ref.ACTS[act], z=z.to(DEV) if act != "none" else None, p=0.3, rng=rng.to(DEV), scale=0.7)
    xs, ws, dys = strided(x, shift=shift), strided(w, shift=shift), strided(dy, shift=shift)
    coat.linear_backward(dys, xs, ws, dx, dw, **how)
    ref.check("dx", dx, *want["dx"])
    ref.check("dw", dw, *want["dw"])
    one = torch.empty_like(dw)
    coat.linear_backward(dys, xs, ws, None, one, **how)
    assert torch.equal(one, dw)


def test_gradients_of_zero_take_nothing_in():
    """dz is 0 where dy is, also beside a z that is not finite."""
    for m, n, k in ((6, 24, 16), (70, 72, 16)):
        x, w, _, _, _ = inputs(m, n, k, 1, F32, False, False)
        dy, z = torch.ones(m, n), torch.ones(m, n)
        dy[1], dy[2, 3], z[1], z[2, 3] = 0.0, -0.0, float("nan"), float("inf")
        want = ref.linear_backward(ref.f64(dy), ref.f64(x), ref.f64(w), torch.ones(m, n, dtype=torch.float64), "silu",
                                   torch.ones(m, n, dtype=torch.float64), 1.0)
        dx, dw, db = torch.ones(m, k, dtype=BF16, device=DEV), torch.ones(n, k, dtype=BF16, device=DEV), torch.ones(n, device=DEV)
        coat.linear_backward(dy.to(DEV), x.to(DEV), w.to(DEV), dx, dw, db, act=coat.ACT_SILU, z=z.to(BF16).to(DEV))
        for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
            ref.check(name, got, *want[name])


def test_infinite_operands_stay_infinite():
    g = gen(3)
    for m, n, k in ((6, 24, 16), (6, 24, 15), (70, 72, 16)):
        dy, x, w = torch.randn(m, n, generator=g), torch.randn(m, k, generator=g).to(BF16), torch.randn(n, k, generator=g).to(BF16)
        dy[1, 3], dy[2, 3] = 1.0, float("inf")
        x[0, 1], w[2, 3] = float("inf"), -float("inf")
        dx, dw = torch.empty(m, k, dtype=BF16, device=DEV), torch.empty(n, k, dtype=BF16, device=DEV)
        coat.linear_backward(dy.to(DEV), x.to(DEV), w.to(DEV), dx, dw)
        for got, want in ((dx, dy.double() @ w.double()), (dw, dy.double().t() @ x.double())):
            got = got.double().cpu()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)]) and torch.isinf(want).any()
            assert torch.equal(torch.isinf(got), torch.isinf(want))


def test_gradients_against_differences():
    """A step along a direction changes the loss sum(y c) by the gradients' product with it."""
    m, n, k = 40, 56, 32
    x, w, b, r, rng = inputs(m, n, k, 4, F32)
    c = torch.randn(m, n, generator=gen(8))
    for act in ("gelu", "silu", "gelu_tanh"):
        z = torch.empty(m, n, dtype=BF16, device=DEV)
        coat.linear(x.to(DEV), w.to(DEV), torch.empty(m, n, device=DEV), bias=b.to(DEV), act=ref.ACTS[act], z=z, p=0.2, rng=rng.to(DEV))
        dx, dw, db = (torch.empty(s, dtype=t, device=DEV) for s, t in (((m, k), BF16), ((n, k), BF16), ((n,), F32)))
        coat.linear_backward(c.to(DEV), x.to(DEV), w.to(DEV), dx, dw, db, act=ref.ACTS[act], z=z, p=0.2, rng=rng.to(DEV))
        f = ref.factors(m, n, 0.2, rng)
        loss = lambda xx, ww, bb: float((ref.linear(xx, ww, bb, act, f, 1.0, None)[0] * c.double()).sum())
        X, W, B = ref.f64(x), ref.f64(w), ref.f64(b)
        h = 1e-4
        for which, grad in ((0, dx), (1, dw), (2, db)):
            d = torch.randn(grad.shape, generator=gen(which), dtype=torch.float64)
            at = [X, W, B]
            up, down = list(at), list(at)
            up[which], down[which] = at[which] + h * d, at[which] - h * d
            want = (loss(*up) - loss(*down)) / (2 * h)
            got = float((grad.double().cpu() * d).sum())
            # z is stored in bf16 (a slope changes by at most 1.3 of its step), dz and the gradient are rounded
            # to it too: three half steps of each term, independent of each other
            size = float((grad.double().cpu() * d).norm()) + 1e-9
            assert abs(got - want) <= 40 * 2.0 ** -8 * size, (act, which, got, want, size)
