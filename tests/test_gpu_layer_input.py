"""GPU tests of the layer-input operators run together: a training step through a block
border, 4-bit products and the FP8 AdamW step; streams, captured graphs, repeated calls
and matrices past 2^32 elements."""
import numpy as np
import pytest
import torch

import _ops64 as o

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module")
def coat():
    import fp8_optimizer_state_amd as c
    assert torch.cuda.is_available()
    c.lib()
    return c


def randn(*shape, seed, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def values(q, s, cols):
    return o.mx4_values(q.cpu().numpy(), s.cpu().numpy(), cols)


def close(got, want, err, dtype):
    bound = err + o.half_step(dtype) * (np.abs(want) + err) + 2.0 ** -133
    assert (np.abs(o.f64(got) - want) <= bound).all(), float(np.max(np.abs(o.f64(got) - want) / bound))


def test_training_step(coat):
    """border -> layer input in 4-bit form -> product with 4-bit weights; the gradients back
    through both products and the border into the FP8 AdamW step's bf16 gradients; the step's
    bf16 weights quantized again. Each stage against its 64-bit form on the kernels' inputs."""
    t, c, f = 200, 256, 320
    sizes = [f * c, c, c]  # a weight matrix, w_post, w_pre
    st = coat.ParamListState(sizes, 128)
    for i, n in enumerate(sizes):
        st.tensor(i).params.copy_(randn(n, seed=i, dtype=torch.float32, scale=0.02) + (1.0 if i else 0.0))
    st.params_bf16.copy_(st.params)
    zeros = [torch.zeros(n, device="cuda") for n in sizes]
    st.quantize_moments(zeros, zeros, fmt_m=0, fmt_v=1)
    w, w_post, w_pre = (st.tensor(i).params_bf16 for i in range(3))
    w = w.view(f, c)
    dw, dw_post, dw_pre = (st.tensor(i).grads for i in range(3))
    dw = dw.view(f, c)

    y, r, dz, d_out = (randn(*s, seed=10 + i) for i, s in enumerate(((t, c), (t, c), (t, f), (t, c))))
    gate = randn(4, c, seed=20)
    how = dict(w_post=w_post, w_pre=w_pre, gate=gate, rows_per_gate=50, scale=0.5, eps=EPS)
    r_out, h, z = torch.empty_like(r), torch.empty_like(r), torch.empty_like(dz)
    xq, wq, wtq, dzq, dztq, htq = (coat.mx4_empty(*s) for s in ((t, c), (f, c), (c, f), (t, f), (f, t), (c, t)))
    coat.block_norm(y, r, r_out, h, q=xq[0], q_scale=xq[1], fmt=coat.FMT_MX4, **how)
    coat.mx4_quantize(w, *wq, *wtq)
    coat.mx4_matmul(*xq, *wq, z)
    # backward: the gradient quantized both ways, the layer input down its columns
    coat.mx4_quantize(dz, *dzq, *dztq)
    coat.mx4_quantize(h, None, None, *htq)
    dh, dr, dy, dgate = torch.empty_like(h), torch.empty_like(r), torch.empty_like(y), torch.empty_like(gate)
    coat.mx4_matmul(*dzq, *wtq, dh)
    coat.mx4_matmul(*dztq, *htq, dw)
    coat.block_norm_backward(y, r_out, d_out, dh, dr, dy, dw_post=dw_post, dw_pre=dw_pre, dgate=dgate, **how)
    torch.cuda.synchronize()

    n64 = o.f64
    want, err = o.border(n64(y), n64(r), n64(w_post), n64(w_pre), n64(gate), 50, 0.5, EPS, True)
    close(r_out, want, o.U32 * err, BF)
    want = o.layer_input(n64(r_out), n64(w_pre), EPS)
    close(h, want, o.U32 * (o.SUM / 2 + 6) * np.abs(want), BF)
    for got, a, b, k in ((z, xq, wq, c), (dh, dzq, wtq, f), (dw, dztq, htq, t)):
        want, mag = o.mx4_matmul(*(v.cpu().numpy() for v in a + b), k)
        assert (np.abs(n64(got) - want) <= o.matmul_bound(want, mag, k, BF)).all()
    q, s = o.mx4_quantize(n64(h))
    assert np.array_equal(xq[0].cpu().numpy(), q) and np.array_equal(xq[1].cpu().numpy(), s)
    back = o.border_backward(n64(y), n64(r_out), n64(d_out), n64(dh), n64(w_post), n64(w_pre), n64(gate), 50, 0.5, EPS, True, 4)
    for name, got, steps in (("dr", dr, o.DR_STEPS), ("dy", dy, o.DY_STEPS), ("dw_post", dw_post, o.dw_steps(t)),
                             ("dw_pre", dw_pre, o.dw_steps(t)), ("dgate", dgate, o.dw_steps(t))):
        close(got, back[name][0], o.U32 * steps * back[name][1], BF)

    before = st.params.clone()
    st.step(fmt_m=0, fmt_v=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=1)
    coat.mx4_quantize(w, *wq)
    torch.cuda.synchronize()
    # the first step of Adam moves every weight with a gradient by about lr against its sign
    moved = n64(st.tensor(0).params - before[:f * c]) * np.sign(n64(dw).reshape(-1))
    strong = np.abs(n64(dw).reshape(-1)) > 1e-3
    assert strong.any() and np.allclose(moved[strong], -1e-3, rtol=1e-2)
    q, s = o.mx4_quantize(n64(w))
    assert np.array_equal(wq[0].cpu().numpy(), q) and np.array_equal(wq[1].cpu().numpy(), s)


class Together:
    """Every operator once, on buffers of its own; `run` may be captured."""

    def __init__(self, coat, t, c, f, seed, splits=True):
        self.coat, self.shape = coat, (t, c, f)
        self.y, self.r, self.dh, self.d_out = (randn(t, c, seed=seed + i) for i in range(4))
        self.w = randn(f, c, seed=seed + 5, scale=0.02)
        self.w_post, self.w_pre, self.gate = randn(c, seed=seed + 6), randn(c, seed=seed + 7), randn(1, c, seed=seed + 8)
        e = torch.empty
        self.out = dict(r_out=e(t, c, dtype=BF, device="cuda"), h=e(t, c, dtype=BF, device="cuda"),
                        dr=e(t, c, dtype=BF, device="cuda"), dy=e(t, c, dtype=BF, device="cuda"),
                        dw_post=e(c, device="cuda"), dw_pre=e(c, device="cuda"), dgate=e(1, c, device="cuda"),
                        z=e(t, f, device="cuda"), back=e(t, c, dtype=BF, device="cuda"))
        self.xq, self.xtq, self.wq = coat.mx4_empty(t, c), coat.mx4_empty(c, t), coat.mx4_empty(f, c)

    def run(self, stream=None):
        coat, q = self.coat, self.out
        how = dict(w_post=self.w_post, w_pre=self.w_pre, gate=self.gate, scale=0.5, eps=EPS, stream=stream)
        coat.block_norm(self.y, self.r, q["r_out"], q["h"], **how)
        coat.mx4_quantize(q["h"], *self.xq, *self.xtq, stream=stream)
        coat.mx4_quantize(self.w, *self.wq, stream=stream)
        coat.mx4_matmul(*self.xq, *self.wq, q["z"], stream=stream)
        coat.mx4_dequantize(*self.xq, q["back"], stream=stream)
        coat.block_norm_backward(self.y, q["r_out"], self.d_out, self.dh, q["dr"], q["dy"], dw_post=q["dw_post"],
                                 dw_pre=q["dw_pre"], dgate=q["dgate"], **how)

    def results(self):
        return {k: v.clone() for k, v in self.out.items()}

    def wipe(self):
        for v in self.out.values():
            v.zero_()


def same(a, b):
    return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


SIZES = [(1, 256, 300), (70, 1000, 300), (64, 8192, 300), (300, 520, 700)]


@pytest.mark.parametrize("t,c,f", SIZES)
def test_repeats_give_the_same_bits(coat, t, c, f):
    w = Together(coat, t, c, f, 1)
    w.run()
    first = w.results()
    for _ in range(3):
        w.wipe()
        w.run()
        assert same(first, w.results())


@pytest.mark.parametrize("t,c,f", SIZES)
def test_another_stream(coat, t, c, f):
    """On a stream passed in, and on one made current; two sets of buffers at once."""
    a, b = Together(coat, t, c, f, 1), Together(coat, t, c, f, 2)
    a.run()
    b.run()
    want_a, want_b = a.results(), b.results()
    a.wipe()
    b.wipe()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.run(s1)
        with torch.cuda.stream(s2):
            b.run()
    s1.synchronize()
    s2.synchronize()
    assert same(want_a, a.results()) and same(want_b, b.results())


@pytest.mark.parametrize("t,c,f", SIZES)
def test_captured_and_replayed(coat, t, c, f):
    """Captured into graphs, replayed with eager calls between; each replay against the
    eager result, for new inputs too. Two graphs, each with workspaces of its own."""
    a, b = Together(coat, t, c, f, 1), Together(coat, t, c, f, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run()
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for w in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w.run()
        graphs.append(g)
    for replay in range(4):
        for w in (a, b):
            w.y.copy_(randn(t, c, seed=100 + replay))
            w.run()
        want = [w.results() for w in (a, b)]
        for w in (a, b):
            w.wipe()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(want[0], a.results()) and same(want[1], b.results()), replay


def test_workspaces_of_the_caller(coat):
    """A caller's workspace is used and need not start cleared; one that is too small, of another
    type or missing in a slice is refused."""
    m, n, k = 64, 300, 8192
    aq, bq = coat.mx4_empty(m, k), coat.mx4_empty(n, k)
    coat.mx4_quantize(randn(m, k, seed=1), *aq)
    coat.mx4_quantize(randn(n, k, seed=2), *bq)
    need = coat.mx4_matmul_workspace_bytes(m, n, k)
    assert need > 0  # few tiles and a long k: the product is split
    y, y2 = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    coat.mx4_matmul(*aq, *bq, y)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    coat.mx4_matmul(*aq, *bq, y2, workspace=ws[:need])
    assert torch.equal(y, y2) and bool((ws[need:] == 0xFF).all())
    with pytest.raises(ValueError, match="workspace"):
        coat.mx4_matmul(*aq, *bq, y, workspace=ws[:need - 1])
    with pytest.raises(ValueError, match="workspace"):
        coat.mx4_matmul(*aq, *bq, y, workspace=ws.view(torch.int32))
    with pytest.raises(coat.CoatError):
        coat.mx4_matmul(*aq, *bq, y, workspace=ws[16:16 + need])  # off its alignment
    x, w = randn(300, 128, seed=3), torch.ones(128, dtype=BF, device="cuda")
    need = coat.block_norm_backward_workspace_bytes(300, 128)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    dr, dw, dw2 = torch.empty_like(x), torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
    coat.block_norm_backward(None, x, x, x, dr, w_pre=w, dw_pre=dw)
    coat.block_norm_backward(None, x, x, x, dr, w_pre=w, dw_pre=dw2, workspace=ws[:need])
    assert torch.equal(dw, dw2) and bool((ws[need:] == 0xFF).all())
    with pytest.raises(ValueError, match="workspace"):
        coat.block_norm_backward(None, x, x, x, dr, w_pre=w, dw_pre=dw, workspace=ws[:need - 1])


def test_refusals_on_the_gpu(coat):
    x = randn(8, 64, seed=1)
    q, s = coat.mx4_empty(8, 64)
    with pytest.raises(ValueError, match="shape"):
        coat.mx4_quantize(x, q[:, :32], s)
    with pytest.raises(ValueError, match="gaps"):
        coat.mx4_quantize(x.t(), *coat.mx4_empty(64, 8))
    with pytest.raises(ValueError, match="gaps"):
        coat.mx4_quantize(x[:1].expand(8, 64), q, s)
    with pytest.raises(ValueError, match="GPU"):
        coat.mx4_quantize(x, q.cpu(), s)
    with pytest.raises(ValueError, match="pair"):
        coat.mx4_quantize(x, q, None)
    with pytest.raises(ValueError, match="shape"):
        coat.mx4_matmul(q, s, q, s, torch.empty(8, 9, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        coat.block_norm(x.t().contiguous().t(), x, torch.empty_like(x), torch.empty_like(x))
    with pytest.raises(ValueError, match="uint8"):
        coat.mx4_dequantize(q.view(torch.int8), s, x)
    with pytest.raises(coat.CoatError):
        coat.block_norm(None, x, None, x.clone(), eps=0.0)
    with pytest.raises(ValueError, match="shape"):
        coat.block_norm(x, x, torch.empty_like(x), torch.empty_like(x), gate=torch.empty(2, 64, dtype=BF, device="cuda"), rows_per_gate=8)


# ---------------------------------------------------------------- large matrices

def test_codec_past_2_32_elements(coat):
    """Codes, scale bytes and values of rows about byte and element offsets 2^31 and 2^32."""
    rows, cols = (1 << 20) + 3, 4100
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for r0 in range(0, rows, 1 << 17):
        x[r0:r0 + (1 << 17)] = torch.randn(min(1 << 17, rows - r0), cols, generator=g, device="cuda").to(BF)
    q, s = coat.mx4_empty(rows, cols)
    qt, s_t = coat.mx4_empty(cols, rows)
    print("quantize", rows, cols, flush=True)
    coat.mx4_quantize(x, q, s, qt, s_t)
    picks = sorted({0, 1, rows - 1, rows - 2, *((1 << b) // cols + d for b in (31, 32) for d in (-1, 0, 1)),
                    *((1 << 31) // q.shape[1] + d for d in (-1, 0, 1)), *range(5, rows, 99991)})
    at = torch.tensor(picks, device="cuda")
    wq, ws = o.mx4_quantize(o.f64(x[at]))
    assert np.array_equal(q[at].cpu().numpy(), wq) and np.array_equal(s[at].cpu().numpy(), ws)
    for c in (0, 1, 2047, 2048, cols - 1):
        wq, ws = o.mx4_quantize(o.f64(x[:, c])[None])
        assert np.array_equal(qt[c:c + 1].cpu().numpy(), wq) and np.array_equal(s_t[c:c + 1].cpu().numpy(), ws)
    del qt, s_t
    back = torch.empty_like(x)
    coat.mx4_dequantize(q, s, back)
    want = torch.from_numpy(values(q[at], s[at], cols)).to(BF)
    assert torch.equal(back[at].cpu(), want)
    q2, s2 = coat.mx4_empty(rows, cols)
    coat.mx4_quantize(x, q2, s2)  # along the rows alone: another kernel
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_border_past_2_32_elements(coat):
    rows, cols = (1 << 20) + 3, 4100
    y, r = torch.empty(rows, cols, dtype=BF, device="cuda"), torch.empty(rows, cols, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    for r0 in range(0, rows, 1 << 17):
        for v in (y, r):
            v[r0:r0 + (1 << 17)] = torch.randn(min(1 << 17, rows - r0), cols, generator=g, device="cuda").to(BF)
    w_post, w_pre, gate = randn(cols, seed=1), randn(cols, seed=2), randn(1, cols, seed=3)
    how = dict(w_post=w_post, w_pre=w_pre, gate=gate, scale=0.5, eps=EPS)
    h = torch.empty_like(y)
    print("border", rows, cols, flush=True)
    keep = torch.tensor(sorted({0, rows - 1, *((1 << b) // cols + d for b in (31, 32) for d in (-1, 0, 1)), *range(7, rows, 99991)}),
                        device="cuda")
    ys, rs = y[keep], r[keep]
    ro, hs = torch.empty_like(ys), torch.empty_like(ys)
    coat.block_norm(ys, rs, ro, hs, **how)
    coat.block_norm(y, r, r, h, **how)
    assert torch.equal(r[keep], ro) and torch.equal(h[keep], hs)
    dr, dy = torch.empty_like(ys), torch.empty_like(ys)
    coat.block_norm_backward(ys, ro, None, hs, dr, dy, **how)
    dr2, dy2 = torch.empty_like(y), torch.empty_like(y)
    coat.block_norm_backward(y, r, None, h, dr2, dy2, **how)
    assert torch.equal(dr2[keep], dr) and torch.equal(dy2[keep], dy)


@pytest.mark.parametrize("m,n,k", [(1 << 20, 33, 8200), (33, 1 << 20, 8200), (70000, 70016, 130)])
def test_product_past_2_32_bytes(coat, m, n, k):
    """Operands or results past 2^32 bytes (or elements): sampled rows and columns in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    ops = []
    for rows in (m, n):
        q, s = coat.mx4_empty(rows, k)
        q.random_(0, 256, generator=g)
        s.random_(120, 134, generator=g)
        ops.append((q, s))
    y = torch.empty(m, n, dtype=BF, device="cuda")
    print("product", m, n, k, flush=True)
    coat.mx4_matmul(*ops[0], *ops[1], y)
    pick = lambda size: torch.tensor(sorted({0, 1, size - 1, size // 2, size // 3, (1 << 31) // ops[0][0].shape[1] % size,  # noqa: E731
                                             (1 << 31) // n % size, (1 << 32) // n % size, *range(3, size, max(1, size // 40))}), device="cuda")
    rows, cols = pick(m), pick(n)
    kp = ops[0][0].shape[1] * 2
    want, mag = o.mx4_matmul(*(v[rows].cpu().numpy() for v in ops[0]), *(v[cols].cpu().numpy() for v in ops[1]), kp)
    got = o.f64(y[rows][:, cols])
    assert (np.abs(got - want) <= o.matmul_bound(want, mag, kp, BF)).all()


def test_product_over_a_very_long_k(coat):
    """Rows longer than the tiled forms take."""
    m, n, k = 40, 33, (1 << 22) + 700
    g = torch.Generator(device="cuda").manual_seed(6)
    ops = []
    for rows in (m, n):
        q, s = coat.mx4_empty(rows, k)
        q.random_(0, 256, generator=g)
        s.fill_(127)
        ops.append((q, s))
    y = torch.empty(m, n, device="cuda")
    coat.mx4_matmul(*ops[0], *ops[1], y)
    kp = ops[0][0].shape[1] * 2
    sub = (0, 1, m - 1), (0, n - 1)
    want, mag = o.mx4_matmul(*(v[list(sub[0])].cpu().numpy() for v in ops[0]), *(v[list(sub[1])].cpu().numpy() for v in ops[1]), kp)
    got = o.f64(y)[np.ix_(*sub)]
    assert (np.abs(got - want) <= o.matmul_bound(want, mag, kp, torch.float32)).all()


def test_quantize_in_more_tiles_than_an_axis_of_a_grid(coat):
    """Over 2^24 tiles of 256 threads: one long column down the tiles, the same values as a row."""
    n = (1 << 29) + 600
    x = torch.empty(n, 1, dtype=BF, device="cuda")
    for at in range(0, n, 1 << 27):
        x[at:at + (1 << 27)] = randn(min(1 << 27, n - at), 1, seed=at + 1)
    got, want = coat.mx4_empty(1, n), coat.mx4_empty(1, n)
    for v in (*got, *want):
        v.fill_(0xA5)
    print("quantize", n, flush=True)
    coat.mx4_quantize(x, None, None, *got)
    coat.mx4_quantize(x.view(1, n), *want)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_product_in_more_workgroups_than_an_axis_of_a_grid(coat):
    """Over 2^24 workgroups of 256 threads (no terms: zeros) and over 2^26 of 64 (one row, one term)."""
    m = (1 << 30) + 70
    y = torch.full((m + 1, 1), 9.0, dtype=BF, device="cuda")
    print("product", m, 1, 0, flush=True)
    coat.mx4_matmul(*coat.mx4_empty(m, 0), *coat.mx4_empty(1, 0), y[:m])
    torch.cuda.synchronize()
    assert bool((y[:m] == 0).all()) and y[m].item() == 9.0
    n = (1 << 30) + 40
    y = y[:n].view(1, n).fill_(9.0)
    bq, bs = (v.zero_() for v in coat.mx4_empty(n, 1))
    bs[:, 0] = 127
    step = 1 << 27
    for at in range(0, n, step):  # each row's one code: its number and the eighth part of it, mod 16
        i = torch.arange(at, min(n, at + step), device="cuda")
        bq[at:at + step, 0] = ((i + i // 8) % 16).to(torch.uint8)
    aq, as_ = (v.zero_() for v in coat.mx4_empty(1, 1))
    aq[0, 0], as_[0, 0] = 5, 127  # 3
    print("product", 1, n, 1, flush=True)
    # the C call: the binding takes k as the codes hold it, 128, which so many rows are not few for
    assert coat.lib().coat_mx4_matmul(aq.data_ptr(), as_.data_ptr(), 1, bq.data_ptr(), bs.data_ptr(), n, 1, y.data_ptr(), n, 0,
                                      None, 0, torch.cuda.current_stream().cuda_stream) == coat.COAT_OK
    table = torch.tensor([v * s * 3 for s in (1, -1) for v in o.GRID], dtype=BF, device="cuda")
    for at in range(0, n, step):
        assert torch.equal(y[0, at:at + step], table[bq[at:at + step, 0].long()])
