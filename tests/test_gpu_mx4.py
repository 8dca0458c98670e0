"""GPU tests of the 4-bit codec and product against 64-bit forms: codes, scale bytes and
values byte for byte, products within the error of their fp32 sums."""
import numpy as np
import pytest
import torch

import _ops64 as o

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SHAPES = [(1, 1), (1, 32), (1, 33), (3, 127), (5, 128), (2, 129), (7, 513), (33, 8), (129, 31), (130, 300), (257, 640),
          (1, 5120), (511, 65), (1029, 17), (37, 2731)]


@pytest.fixture(scope="module")
def coat():
    import fp8_optimizer_state_amd as c
    assert torch.cuda.is_available()
    c.lib()
    return c


def values(rows, cols, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.pow(2.0, torch.randint(-8, 9, (1, cols), generator=g).float())
    return x.to(dtype)


def guarded(rows, width):
    """A uint8 matrix with a row of 0xA5 before and after it in memory."""
    buf = torch.full(((rows + 2) * max(width, 1) + 32,), 0xA5, dtype=torch.uint8, device="cuda")
    off = (-(-max(width, 1) // 16)) * 16
    return buf, buf[off:off + rows * width].view(rows, width)


def untouched(buf, view):
    mask = torch.ones_like(buf, dtype=torch.bool)
    off = view.storage_offset()
    mask[off:off + view.numel()] = False
    return bool((buf[mask] == 0xA5).all())


def quantize(coat, x, along, down):
    rows, cols = x.shape
    got = {}
    if along:
        got["q"], got["s"] = guarded(rows, o.code_bytes(cols)), guarded(rows, o.scale_bytes(cols))
    if down:
        got["q_t"], got["s_t"] = guarded(cols, o.code_bytes(rows)), guarded(cols, o.scale_bytes(rows))
    coat.mx4_quantize(x, **{k: v[1] for k, v in got.items()})
    torch.cuda.synchronize()
    assert all(untouched(*v) for v in got.values())
    return {k: v[1].cpu().numpy() for k, v in got.items()}


def check_quantize(coat, x, along=True, down=True):
    got = quantize(coat, x, along, down)
    v = o.f64(x)
    if along:
        q, s = o.mx4_quantize(v)
        assert np.array_equal(got["s"], s) and np.array_equal(got["q"], q)
    if down:
        q, s = o.mx4_quantize(np.ascontiguousarray(v.T))
        assert np.array_equal(got["s_t"], s) and np.array_equal(got["q_t"], q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("way", ["rows", "cols", "both"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(coat, rows, cols, way, dtype):
    check_quantize(coat, values(rows, cols, rows + cols, TYPES[dtype]).cuda(), way != "cols", way != "rows")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,off", [(1, 0), (8, 0), (3, 1), (64, 5), (16, 8)])
def test_quantize_strided(coat, pad, off, dtype):
    """Columns cut out of a wider matrix, at any element offset."""
    rows, cols = 131, 261
    wide = values(rows, cols + pad + off, 3, TYPES[dtype]).cuda()
    x = wide[:, off:off + cols]
    assert x.stride(0) != cols
    check_quantize(coat, x)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_blocks(coat, dtype):
    t = TYPES[dtype]
    tiny = 2.0 ** -133 if dtype == "bf16" else 2.0 ** -149
    x = values(14, 128, 5, torch.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 5] = float("nan")
    x[3, 40] = float("inf")
    x[4, 127] = -float("inf")
    x[5] = tiny
    x[6] = -tiny * 3
    x[7, :32] = 2.0 ** -126
    x[7, 32:64] = 2.0 ** -127
    x[7, 64:96] = torch.linspace(0, 1, 32) * 2.0 ** -124
    x[8] = torch.finfo(t).max
    x[9] = torch.finfo(t).max * torch.linspace(-1, 1, 128)
    x[10, 0::2] = torch.finfo(t).max
    x[10, 1::2] = 1.0
    x[11] = torch.pow(2.0, torch.arange(128).float() - 64)
    x[12] = -torch.pow(2.0, torch.arange(128).float() - 64) * 1.984375
    x = x.to(t).cuda()
    check_quantize(coat, x)
    check_quantize(coat, x.t().contiguous())


def test_quantize_every_bf16_value(coat):
    """Every finite bf16 value, each in blocks whose largest value is 1 or 2 - 2^-7
    times the powers of two up to its own magnitude's, two and 12 above."""
    bits = torch.arange(1 << 16, dtype=torch.int32)
    v = bits.to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    rows = []
    for up in (0, 1, 2, 12):
        for lead in (1.0, 2 - 2.0 ** -7):
            top = torch.ldexp(torch.tensor(lead), torch.frexp(v.float().abs())[1] - 1 + up).to(torch.bfloat16)
            keep = torch.isfinite(top.float())
            b = torch.zeros(int(keep.sum()), 32, dtype=torch.bfloat16)
            b[:, 7] = v[keep]
            b[:, 20] = top[keep]
            rows.append(b)
    x = torch.cat(rows)
    x = x[:x.shape[0] // 512 * 512].reshape(-1, 512 * 32).cuda()
    print("blocks", x.numel() // 32, flush=True)
    check_quantize(coat, x, True, False)
    check_quantize(coat, x.t().contiguous(), False, True)


def test_quantize_fp32_rounding_borders(coat):
    """fp32 values at each rounding border and one step to either side, over many scales."""
    mids = (o.GRID[1:] + o.GRID[:-1]) / 2
    base = torch.tensor(np.concatenate([mids, o.GRID, [5.0, 5.5, 6.5, 7.0, 7.9999995]]), dtype=torch.float32)
    near = torch.cat([base, torch.nextafter(base, torch.tensor(99.0)), torch.nextafter(base, torch.tensor(-99.0))])
    near = torch.cat([near, -near])
    rows = []
    for e in list(range(-124, 120, 7)) + [-127, -126, -125]:
        b = torch.zeros(near.numel(), 32)
        b[:, 3] = torch.ldexp(near, torch.tensor(e))
        b[:, 31] = torch.ldexp(torch.tensor(4.0), torch.tensor(e))
        rows.append(b)
    x = torch.cat(rows).reshape(-1, 32).cuda()
    check_quantize(coat, x, True, False)
    check_quantize(coat, x.t().contiguous(), False, True)


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(coat, dtype):
    t = TYPES[dtype]
    q = torch.zeros(256, 64, dtype=torch.uint8)
    q[:, :] = torch.randint(0, 256, (256, 64), generator=torch.Generator().manual_seed(1))
    q[:, :8] = torch.tensor([(2 * i) | ((2 * i + 1) << 4) for i in range(8)], dtype=torch.uint8)
    s = torch.zeros(256, 16, dtype=torch.uint8)
    s[:, :4] = torch.arange(256, dtype=torch.uint8)[:, None]
    for cols in (128, 100, 17):
        x = torch.full((256, 128), 7.0, dtype=t, device="cuda")
        coat.mx4_dequantize(q.cuda(), s.cuda(), x[:, :cols])
        want = torch.from_numpy(o.mx4_values(q.numpy(), s.numpy(), cols)).to(t)
        got = x.cpu()
        assert torch.equal(got[:, :cols].isnan(), want.isnan())
        assert torch.equal(got[:, :cols].nan_to_num(), want.nan_to_num())
        signs = ~want.isnan()
        assert torch.equal(torch.signbit(got[:, :cols])[signs], torch.signbit(want)[signs])
        assert bool((got[:, cols:] == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_round_trip(coat, rows, cols, dtype):
    x = values(rows, cols, 11, TYPES[dtype]).cuda()
    q, s = coat.mx4_empty(rows, cols)
    coat.mx4_quantize(x, q, s)
    back = torch.full((rows, cols + 3), 5.0, dtype=TYPES[dtype], device="cuda")
    coat.mx4_dequantize(q, s, back[:, 1:1 + cols])
    want = torch.from_numpy(o.mx4_values(q.cpu().numpy(), s.cpu().numpy(), cols)).to(TYPES[dtype])
    assert torch.equal(back[:, 1:1 + cols].cpu(), want)
    assert bool((back[:, 0] == 5.0).all()) and bool((back[:, 1 + cols:] == 5.0).all())


# ---------------------------------------------------------------- product

PRODUCTS = [(1, 1, 1), (1, 32, 64), (2, 3, 129), (16, 16, 128), (17, 33, 500), (31, 64, 513), (33, 31, 640), (64, 65, 1024),
            (1, 257, 2731), (5, 700, 1000), (65, 130, 4097), (128, 128, 256), (129, 255, 384), (257, 256, 512), (300, 513, 2048),
            (256, 256, 1), (512, 768, 640), (2600, 1300, 1030), (1030, 4100, 520),
            (70, 200, 5000), (129, 300, 13824), (33, 5120, 2731), (64, 65, 6000), (333, 640, 4100), (4100, 4100, 300), (300, 300, 3000), (4090, 4950, 300)]


def operand(rows, k, seed):
    x = values(rows, k, seed, torch.float32)
    q, s = o.mx4_quantize(o.f64(x))
    return q, s


def product(coat, aq, as_, bq, bs, dtype, pad=0, **kw):
    m, n = aq.shape[0], bq.shape[0]
    y = torch.full((m, n + pad), 9.0, dtype=dtype, device="cuda")
    d = lambda t: torch.from_numpy(t).cuda()  # noqa: E731
    coat.mx4_matmul(d(aq), d(as_), d(bq), d(bs), y[:, :n], **kw)
    torch.cuda.synchronize()
    assert bool((y[:, n:] == 9.0).all())
    return y[:, :n]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(coat, m, n, k, dtype):
    aq, as_ = operand(m, k, 1)
    bq, bs = operand(n, k, 2)
    got = o.f64(product(coat, aq, as_, bq, bs, TYPES[dtype], pad=m % 3))
    want, mag = o.mx4_matmul(aq, as_, bq, bs, k)
    assert (np.abs(got - want) <= o.matmul_bound(want, mag, k, TYPES[dtype])).all()


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product_of_whole_numbers(coat, m, n, k):
    """Equal scales: every sum is exact in fp32, so every bit has to be right."""
    g = np.random.default_rng(m + n + k)
    aq, bq = (g.integers(0, 256, (r, o.code_bytes(k)), dtype=np.uint8) for r in (m, n))
    as_, bs = (np.full((r, o.scale_bytes(k)), 127, np.uint8) for r in (m, n))
    got = o.f64(product(coat, aq, as_, bq, bs, torch.float32))
    want, _ = o.mx4_matmul(aq, as_, bq, bs, o.code_bytes(k) * 2)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("m,n,k", [(20, 20000, 5000), (32, 4200, 14000)])
def test_product_of_few_rows_with_much(coat, m, n, k):
    """Few rows of A are not taken by themselves where B is large: the same bits as among more rows (exact sums)."""
    g = torch.Generator(device="cuda").manual_seed(k)
    aq, bq = (torch.randint(0, 256, (r, o.code_bytes(k)), dtype=torch.uint8, device="cuda", generator=g) for r in (200, n))
    as_, bs = (torch.full((r, o.scale_bytes(k)), 127, dtype=torch.uint8, device="cuda") for r in (200, n))
    few, many = torch.full((m + 1, n), 9.0, device="cuda"), torch.empty(200, n, device="cuda")
    coat.mx4_matmul(aq[:m], as_[:m], bq, bs, few[:m])
    coat.mx4_matmul(aq, as_, bq, bs, many)
    torch.cuda.synchronize()
    assert torch.equal(few[:m], many[:m]) and bool((few[m] == 9.0).all())


@pytest.mark.parametrize("m,n,k", [(3, 5, 640), (130, 260, 640)])
def test_product_takes_each_scale_at_its_block(coat, m, n, k):
    """One value a row, scales all different: a scale or a code at a wrong place shows."""
    g = np.random.default_rng(5)
    aq, bq = np.zeros((m, o.code_bytes(k)), np.uint8), np.zeros((n, o.code_bytes(k)), np.uint8)
    bq[:] = 0x22  # ones
    at = g.integers(0, k, m)
    aq[np.arange(m), at // 2] = np.where(at % 2, 0x50, 0x05)
    as_, bs = (g.integers(100, 150, (r, o.scale_bytes(k)), dtype=np.uint8) for r in (m, n))
    got = o.f64(product(coat, aq, as_, bq, bs, torch.float32))
    want, _ = o.mx4_matmul(aq, as_, bq, bs, k)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("m,n,k", [(3, 5, 640), (130, 260, 640), (260, 520, 1100)])
def test_product_with_nan_blocks(coat, m, n, k):
    """A block that held a NaN or Inf makes its row (or column) of y NaN, and nothing else."""
    aq, as_ = operand(m, k, 1)
    bq, bs = operand(n, k, 2)
    as_[1, 3] = 255
    bs[n - 1, o.code_bytes(k) * 2 // 32 - 1] = 255
    aq[1, 48:64] = 0
    got = o.f64(product(coat, aq, as_, bq, bs, torch.float32))
    want, mag = o.mx4_matmul(aq, as_, bq, bs, o.code_bytes(k) * 2)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= o.matmul_bound(want, mag, k, torch.float32)[ok]).all()


def test_product_of_extreme_scales(coat):
    """Products past fp32 are infinite, products under it vanish or are subnormal."""
    k = 128
    aq, bq = np.full((6, 64), 0x22, np.uint8), np.full((40, 64), 0x22, np.uint8)
    as_, bs = np.zeros((6, 16), np.uint8), np.zeros((40, 16), np.uint8)
    as_[:] = np.array([0, 1, 63, 127, 200, 254])[:, None]
    bs[:] = np.linspace(0, 254, 40).astype(np.uint8)[:, None]
    got = o.f64(product(coat, aq, as_, bq, bs, torch.float32))
    with np.errstate(over="ignore"):
        want = o.mx4_matmul(aq, as_, bq, bs, k)[0].astype(np.float32).astype(np.float64)
    normal = np.abs(want) >= 2.0 ** -126
    assert np.array_equal(got[normal], want[normal])
    assert (np.abs(got[~normal] - want[~normal]) <= 2.0 ** -126).all()


def test_product_without_terms(coat):
    q, s = coat.mx4_empty(5, 0)
    q2, s2 = coat.mx4_empty(7, 0)
    y = torch.full((5, 7), 3.0, device="cuda")
    coat.mx4_matmul(q, s, q2, s2, y)
    assert bool((y == 0).all())
    q, s = coat.mx4_empty(0, 64)
    q2, s2 = coat.mx4_empty(7, 64)
    coat.mx4_matmul(q, s, q2, s2, y[:0])
    coat.mx4_quantize(torch.empty(0, 64, device="cuda"), q, s)


def test_linear_layer_and_its_gradients(coat):
    """Y = X W^T, dX = dY W and dW = dY^T X through the row and column forms of one pass,
    against the products of the quantized values."""
    t, i, out = 333, 200, 145
    x, w, dy = (values(r, c, s, torch.bfloat16).cuda() for r, c, s in ((t, i, 1), (out, i, 2), (t, out, 3)))
    forms = {}
    for name, v in (("x", x), ("w", w), ("dy", dy)):
        forms[name], forms[name + "t"] = coat.mx4_empty(*v.shape), coat.mx4_empty(*v.shape[::-1])
        coat.mx4_quantize(v, *forms[name], *forms[name + "t"])
    for a, b, shape in (("x", "w", (t, out)), ("dy", "wt", (t, i)), ("dyt", "xt", (out, i))):
        y = torch.empty(*shape, device="cuda")
        coat.mx4_matmul(*forms[a], *forms[b], y)
        host = [f.cpu().numpy() for f in forms[a] + forms[b]]
        k = host[0].shape[1] * 2
        want, mag = o.mx4_matmul(*host, k)
        assert (np.abs(o.f64(y) - want) <= o.matmul_bound(want, mag, k, torch.float32)).all()


def unpacked(q):
    """The codes' values in fp32, on the GPU."""
    table = torch.tensor([v * s for s in (1, -1) for v in o.GRID], dtype=torch.float32, device="cuda")
    return table[torch.stack([q & 15, q >> 4], dim=2).view(q.shape[0], -1).int()]


def check_all_of_y(coat, m, n, k, pad, dtype):
    """Equal scales: every partial sum is a multiple of 1/4 under 36 k < 2^22, exact in fp32 in any
    order, so y has to be the sum rounded once. Every element, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    ops = []
    for rows in (m, n):
        q, s = coat.mx4_empty(rows, k)
        ops.append((q.random_(0, 256, generator=g), s.fill_(127)))
    y = torch.full((m, n + pad), 9.0, dtype=dtype, device="cuda")
    print("product", m, n, k, pad, dtype, flush=True)
    coat.mx4_matmul(*ops[0], *ops[1], y[:, :n])
    torch.cuda.synchronize()
    a, b = (unpacked(q) for q, _ in ops)
    assert a.shape[1] * 36 < 1 << 22
    want = torch.matmul(a, b.t().contiguous()).to(dtype)
    assert torch.equal(y[:, :n], want) and bool((y[:, n:] == 9.0).all())


# Large tiles in the state that most products run them in (the host driver of the launch
# shapes holds the same list): several tiles one after the other on a compute unit, whole
# ones, each over several groups of steps that end after one, two, three or four of them;
# rows of y that fill lines and rows that do not; edges among the whole tiles; and the
# last columns or rows in small tiles.
LARGE = [(8192, 8192, 1100, 0), (8192, 8192, 1280, 0), (8192, 8192, 1400, 3), (8192, 8192, 1536, 0), (8192, 8192, 300, 0),
         (16384, 4000, 1100, 0), (8000, 8300, 1100, 0), (4096, 5120, 5120, 0), (5120, 4096, 5120, 8), (2600, 13824, 5120, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,pad", LARGE)
def test_product_in_many_large_tiles(coat, m, n, k, pad, dtype):
    check_all_of_y(coat, m, n, k, pad, TYPES[dtype])


# one side within a small tile, the other over more of them than there are compute units
NARROW = [(128, 40000, 1100, 0), (100, 40000, 1280, 0), (64, 40001, 1400, 3), (40000, 128, 1536, 0), (70000, 33, 300, 0), (20, 128256, 5120, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,pad", NARROW)
def test_product_with_a_narrow_side(coat, m, n, k, pad, dtype):
    check_all_of_y(coat, m, n, k, pad, TYPES[dtype])
