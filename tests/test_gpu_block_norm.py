"""GPU tests of the norms at a block's border, forward and backward, against 64-bit
forms, within the roundings counted there; the stored forms of the layer input byte for
byte those that the codecs give for the bf16 layer input."""
import numpy as np
import pytest
import torch

import _ops64 as o

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF, "fp32": F32}
EPS = 1e-5
SHAPES = [(1, 1), (1, 8), (3, 17), (2, 64), (5, 127), (33, 512), (7, 520), (9, 1029), (4, 2731), (3, 4096), (5, 4104), (2, 5120),
          (3, 8200), (2, 13824), (1, 16384), (700, 40)]


@pytest.fixture(scope="module")
def coat():
    import fp8_optimizer_state_amd as c
    assert torch.cuda.is_available()
    c.lib()
    return c


def make(rows, cols, seed, stream=BF, params=BF, rpg=None, post=True, pre=True, gated=True, y=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rpg = rpg or max(rows, 1)
    groups = -(-rows // rpg)
    mag = torch.pow(4.0, torch.randint(-3, 4, (rows, 1), generator=g).float())
    t = dict(r=(rn(rows, cols) * mag).to(stream), w_pre=(1 + 0.2 * rn(cols)).to(params) if pre else None,
             dr_out=rn(rows, cols).to(stream), dh=rn(rows, cols).to(BF) if pre else None)
    t["y"] = (rn(rows, cols) * mag.flip(0)).to(BF) if y else None
    t["w_post"] = (1 + 0.2 * rn(cols)).to(params) if y and post else None
    t["gate"] = rn(groups, cols).to(params) if y and gated else None
    t = {k: v.cuda() if v is not None else None for k, v in t.items()}
    return t, dict(rows_per_gate=rpg, scale=0.75, eps=EPS, post=post and y)


def n64(t):
    return None if t is None else o.f64(t)


def within(got, want, err, dtype, what):
    """|got - want| <= err + half a step of the stored value."""
    got = o.f64(got)
    bound = err + o.half_step(dtype) * (np.abs(want) + err) + 2.0 ** -133
    worst = np.max(np.abs(got - want) / bound) if got.size else 0.0
    assert worst <= 1.0, (what, float(worst))


def forward(coat, t, how, quant=None, h=True):
    rows, cols = t["r"].shape
    r_out = torch.full_like(t["r"], 7.0) if t["y"] is not None else None
    ho = torch.full((rows, cols), 7.0, dtype=BF, device="cuda") if h else None
    coat.block_norm(t["y"], t["r"], r_out, ho, w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"], **how, **(quant or {}))
    torch.cuda.synchronize()
    return r_out, ho


def check_forward(coat, t, how):
    r_out, h = forward(coat, t, how)
    stream = t["r"].dtype
    want, err = o.border(n64(t["y"]), n64(t["r"]), n64(t["w_post"]), n64(t["w_pre"]), n64(t["gate"]), how["rows_per_gate"],
                         how["scale"], EPS, how["post"])
    if r_out is not None:
        within(r_out, want, o.U32 * err, stream, "r_out")
    kept = n64(r_out if r_out is not None else t["r"])  # h is defined by the stored stream
    want = o.layer_input(kept, n64(t["w_pre"]), EPS)
    within(h, want, o.U32 * (o.SUM / 2 + 6) * np.abs(want), BF, "h")
    return r_out, h


def backward(coat, t, how, r, grads=F32, **kw):
    rows, cols = t["r"].shape
    out = dict(dr=torch.full_like(t["r"], 7.0), dy=torch.full((rows, cols), 7.0, dtype=BF, device="cuda") if t["y"] is not None else None)
    for name, src in (("dw_post", t["w_post"]), ("dw_pre", t["w_pre"]), ("dgate", t["gate"])):
        out[name] = torch.full(src.shape, 7.0, dtype=grads, device="cuda") if src is not None else None
    coat.block_norm_backward(t["y"], r, t["dr_out"], t["dh"], w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"], **out, **how, **kw)
    torch.cuda.synchronize()
    return out


def check_backward(coat, t, how, grads=F32, **kw):
    rows = t["r"].shape[0]
    out = backward(coat, t, how, t["r"], grads, **kw)
    want = o.border_backward(n64(t["y"]), n64(t["r"]), n64(t["dr_out"]), n64(t["dh"]), n64(t["w_post"]), n64(t["w_pre"]),
                             n64(t["gate"]), how["rows_per_gate"], how["scale"], EPS, how["post"], -(-rows // how["rows_per_gate"]))
    steps = dict(dr=o.DR_STEPS, dy=o.DY_STEPS, dw_post=o.dw_steps(rows), dw_pre=o.dw_steps(rows), dgate=o.dw_steps(rows))
    for name, got in out.items():
        if got is not None:
            value, mag = want[name]
            within(got, value, o.U32 * steps[name] * mag, got.dtype, name)
    return out


@pytest.mark.parametrize("params", TYPES)
@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(coat, rows, cols, stream, params):
    check_forward(coat, *make(rows, cols, rows + cols, TYPES[stream], TYPES[params]))


@pytest.mark.parametrize("params", TYPES)
@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(coat, rows, cols, stream, params):
    check_backward(coat, *make(rows, cols, rows + cols, TYPES[stream], TYPES[params]))


PARTS = [dict(post=False), dict(pre=False), dict(gated=False), dict(y=False), dict(post=False, gated=False),
         dict(pre=False, gated=False), dict(pre=False, post=False)]


@pytest.mark.parametrize("parts", PARTS, ids=lambda p: "-".join("no_" + k for k in p))
@pytest.mark.parametrize("rows,cols", [(5, 1029), (130, 256)])
def test_parts_left_out(coat, rows, cols, parts):
    t, how = make(rows, cols, 3, **parts)
    if parts.get("pre", True):
        check_forward(coat, t, how)
    else:
        r_out, _ = forward(coat, t, how, h=False)
        want, err = o.border(n64(t["y"]), n64(t["r"]), n64(t["w_post"]), None, n64(t["gate"]), how["rows_per_gate"], how["scale"],
                             EPS, how["post"])
        within(r_out, want, o.U32 * err, BF, "r_out")
    check_backward(coat, t, how)


def test_norms_without_weights(coat):
    """post=True and a layer input, with weights of one."""
    t, how = make(9, 300, 4)
    t["w_post"] = t["w_pre"] = None
    check_forward(coat, t, how)
    out = check_backward(coat, t, how)
    assert out["dw_post"] is None and out["dw_pre"] is None


@pytest.mark.parametrize("grads", TYPES)
@pytest.mark.parametrize("rows,rpg", [(1, 1), (12, 1), (12, 5), (700, 1), (700, 2), (700, 3), (700, 699), (700, 700), (700, 4000),
                                      (1031, 257), (2100, 4), (2100, 5), (2100, 7), (2100, 1050), (1537, 1536), (5000, 3), (5000, 7),
                                      (5000, 301), (2600, 31)])
def test_gates_of_sequences(coat, rows, rpg, grads):
    """Tokens that share a gate row, in every way that rows are dealt to workgroups; a last gate row with fewer tokens."""
    t, how = make(rows, 72, rows + rpg, rpg=rpg)
    check_forward(coat, t, how)
    check_backward(coat, t, how, TYPES[grads])


@pytest.mark.parametrize("cols", [4099, 9000])
@pytest.mark.parametrize("rpg", [2, 3, 5, 31])
def test_gates_of_sequences_of_wide_rows(coat, rpg, cols):
    """Few workgroups of many threads: several gate rows, one, and parts of one to a workgroup."""
    t, how = make(600, cols, cols + rpg, rpg=rpg)
    check_backward(coat, t, how, BF)


def test_gate_for_all_by_default(coat):
    t, how = make(50, 64, 9)
    how["rows_per_gate"] = None
    a, b = forward(coat, t, how)
    how["rows_per_gate"] = 50
    c, d = forward(coat, t, how)
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("missing", ["dr_out", "dw_post", "dw_pre", "dgate"])
def test_gradients_left_out(coat, missing):
    t, how = make(40, 130, 6, rpg=7)
    if missing == "dr_out":
        t["dr_out"] = None
        check_backward(coat, t, how)
        return
    full = check_backward(coat, t, how)
    out = {k: torch.full_like(v, 5.0) for k, v in full.items()}
    dropped = out.pop(missing)
    coat.block_norm_backward(t["y"], t["r"], t["dr_out"], t["dh"], w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"], **out, **how)
    assert bool((dropped == 5.0).all())
    assert all(torch.equal(out[k], full[k]) for k in ("dr", "dy"))


def test_in_place(coat):
    """r_out may be r, and dr may be dr_out."""
    t, how = make(33, 1029, 7, stream=F32)
    r_out, h = forward(coat, t, how)
    r2, h2 = t["r"].clone(), torch.empty_like(h)
    coat.block_norm(t["y"], r2, r2, h2, w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"], **how)
    assert torch.equal(r2, r_out) and torch.equal(h2, h)
    out = backward(coat, t, how, t["r"])
    d2, dy2 = t["dr_out"].clone(), torch.empty_like(out["dy"])
    coat.block_norm_backward(t["y"], t["r"], d2, t["dh"], d2, dy2, w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"], **how)
    assert torch.equal(d2, out["dr"]) and torch.equal(dy2, out["dy"])


def test_no_rows(coat):
    t, how = make(0, 64, 1)
    forward(coat, t, how)
    out = backward(coat, t, how, t["r"])
    assert bool((out["dw_post"] == 0).all()) and bool((out["dw_pre"] == 0).all()) and out["dgate"].numel() == 0


def test_rows_without_values_and_infinities(coat):
    """A row of zeros stays zeros; a NaN or Inf stays within its row."""
    t, how = make(6, 520, 2, gated=False)
    t["y"][1] = 0.0
    t["r"][1] = 0.0
    t["y"][2, 5] = float("nan")
    t["r"][3, 519] = float("inf")
    r_out, h = forward(coat, t, how)
    assert bool((r_out[1] == 0).all()) and bool((h[1] == 0).all())
    assert bool(r_out[2].isnan().all()) and bool(h[2].isnan().all())
    assert bool(h[3].isnan()[519]) and bool((h[3, :519] == 0).all())
    keep = [0, 1, 4, 5]
    clean = {k: v[keep].contiguous() if k in ("y", "r", "dr_out", "dh") else v for k, v in t.items()}
    how4 = dict(how, rows_per_gate=4)
    r4, h4 = forward(coat, clean, how4)
    assert torch.equal(r_out[keep], r4) and torch.equal(h[keep], h4)
    out = backward(coat, t, how, t["r"])
    assert torch.equal(out["dr"][keep], backward(coat, clean, how4, clean["r"])["dr"])


@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("group", [16, 32, 64, 128, 256, 512])
def test_fp8_layer_input(coat, group, fmt, stream):
    for rows, cols in ((1, group), (3, group * 3), (5, max(5120, group)), (2, 8192 + 512)):
        t, how = make(rows, cols, group + rows, TYPES[stream])
        if rows == 5:
            t["y"][0] = 0.0
            t["r"][0] = 0.0
            t["y"][1, 100] = float("nan")
            t["w_pre"][7] = -0.0
        _, h = forward(coat, t, how)
        q = torch.full((rows, cols), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((rows, cols // group), 5.0, device="cuda")
        for keep in (True, False):
            _, h2 = forward(coat, t, how, dict(q=q, q_scale=s, group=group, fmt=fmt), h=keep)
            if keep:
                assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
            q2, s2 = torch.empty_like(q), torch.empty_like(s)
            coat.act_quantize(h, q2, s2, group=group, fmt=fmt)
            assert torch.equal(q, q2) and torch.equal(s.view(torch.int32), s2.view(torch.int32))


@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_4_bit_layer_input(coat, rows, cols, stream):
    t, how = make(rows, cols, 5, TYPES[stream])
    if rows > 1:
        t["y"][1, 0] = float("inf")
    _, h = forward(coat, t, how)
    a, b = coat.mx4_empty(rows, cols), coat.mx4_empty(rows, cols)
    for v in a:
        v.fill_(0xA5)
    coat.mx4_quantize(h, *b)
    forward(coat, t, how, dict(q=a[0], q_scale=a[1], fmt=coat.FMT_MX4), h=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_against_differences(coat):
    """Central differences of the 64-bit forward, in random directions, against the kernels' gradients."""
    rows, cols, rpg = 11, 48, 4
    t, how = make(rows, cols, 21, F32, F32, rpg=rpg)
    v = {k: n64(x) for k, x in t.items()}
    before, _ = o.border(v["y"], np.zeros_like(v["r"]), v["w_post"], None, v["gate"], rpg, how["scale"], EPS, True)
    stream = v["r"] - before  # the stream whose r' is r

    def total(y, r, w_post, w_pre, gate):
        out, _ = o.border(y, r, w_post, w_pre, gate, rpg, how["scale"], EPS, True)
        return (out * v["dr_out"]).sum() + (o.layer_input(out, w_pre, EPS) * v["dh"]).sum()

    out = backward(coat, t, how, t["r"])
    formula = o.border_backward(v["y"], v["r"], v["dr_out"], v["dh"], v["w_post"], v["w_pre"], v["gate"], rpg, how["scale"], EPS,
                                True, -(-rows // rpg))
    g = np.random.default_rng(1)
    at = dict(y=v["y"], r=stream, w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"])
    for name, grad in (("y", "dy"), ("r", "dr"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("gate", "dgate")):
        got = o.f64(out[grad])
        for _ in range(3):
            way = g.standard_normal(at[name].shape)
            # rows differ by 4^6 in size: the step is 1e-6 of the smallest row's values, and the five-point
            # formula's error its fourth power; the differences lose 1e-16 of the total over the step
            step = 1e-6 * np.abs(at[name]).min(axis=-1).max() if name in ("y", "r") else 1e-6
            f = [total(**dict(at, **{name: at[name] + k * step * way})) for k in (-2, -1, 1, 2)]
            want = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * step)
            size = np.abs(formula[grad][0] * way).sum()
            assert abs((formula[grad][0] * way).sum() - want) <= 1e-6 * (1 + size), name
            bound = 1e-6 * (1 + size) + (o.half_step(out[grad].dtype) + o.U32 * o.dw_steps(rows)) * np.abs(got * way).sum()
            assert abs((got * way).sum() - want) <= bound, name


def gradients_at(coat, t, how, eps):
    """check_backward with another eps, as fp32 holds it."""
    how = dict(how, eps=eps)
    eps = float(np.float32(eps))
    rows = t["r"].shape[0]
    out = backward(coat, t, how, t["r"])
    want = o.border_backward(n64(t["y"]), n64(t["r"]), n64(t["dr_out"]), n64(t["dh"]), n64(t["w_post"]), n64(t["w_pre"]),
                             n64(t["gate"]), how["rows_per_gate"], how["scale"], eps, how["post"], -(-rows // how["rows_per_gate"]))
    steps = dict(dr=o.DR_STEPS, dy=o.DY_STEPS, dw_post=o.dw_steps(rows), dw_pre=o.dw_steps(rows), dgate=o.dw_steps(rows))
    for name, got in out.items():
        within(got, want[name][0], o.U32 * steps[name] * want[name][1], got.dtype, name)


@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("cols", [5, 40, 1029, 4096, 9000])
@pytest.mark.parametrize("size", [1e-12, 1e8, 1e13, 1e14, 1e15, 1e16, 1e17])
def test_gradients_of_rows_of_any_size(coat, size, cols, stream):
    """Rows whose factor's cube leaves fp32's range (sums of squares up to 9e37 here, inside
    it): the projections on the rows keep their accuracy. dr_out is as large as they are."""
    t, how = make(6, cols, cols, TYPES[stream], F32, rpg=2)
    g = torch.Generator().manual_seed(cols + 1)
    for name, mag in (("r", size), ("y", size), ("dr_out", min(1.0, 1.0 / size))):
        t[name] = (torch.randn(6, cols, generator=g) * mag).to(t[name].dtype).cuda()
    check_forward(coat, t, how)
    gradients_at(coat, t, how, EPS)
    t["dr_out"] = None
    gradients_at(coat, t, how, EPS)


@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("eps", [1e-20, 1e-30, 2.0 ** -126])
def test_gradients_of_rows_of_zeros_with_a_small_eps(coat, eps, stream):
    """The factor of such a row is eps^-1/2, whose cube passes fp32; its gradient does not."""
    t, how = make(6, 520, 31, TYPES[stream], F32, rpg=2)
    t["r"][0] = 0.0
    t["y"][3] = 0.0
    t["r"][4] *= 1e-15 / t["r"][4].float().abs().max()
    gradients_at(coat, t, how, eps)


@pytest.mark.parametrize("cols", [40, 1029, 9000])
def test_gradient_of_an_output_that_is_not_normalised(coat, cols):
    """Without the post-norm dy = scale gate dr_out: an Inf or NaN in y shows in the gate's gradient alone."""
    t, how = make(6, cols, 17, post=False, pre=False, rpg=3)
    clean = backward(coat, t, how, t["r"])
    t["y"][1, 7] = float("inf")
    t["y"][4, cols - 1] = float("nan")
    out = backward(coat, t, how, t["r"])
    assert torch.equal(out["dr"], clean["dr"]) and torch.equal(out["dy"], clean["dy"])
    bad = torch.zeros_like(out["dgate"], dtype=torch.bool)
    bad[0, 7] = bad[1, cols - 1] = True
    assert torch.equal(out["dgate"][~bad], clean["dgate"][~bad]) and not bool(out["dgate"][bad].isfinite().any())


@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("cols", [40, 1029, 9000])
def test_an_infinity_in_y(coat, cols, stream):
    """Under the post-norm: NaN in its channel of r', r' = r in the row's others, NaN in all of h and dy;
    the weights' gradients NaN in that channel. Other rows and gate rows are those without it."""
    t, how = make(6, cols, 41, TYPES[stream], rpg=2)
    clean_r, clean_h = forward(coat, t, how)
    clean = backward(coat, t, how, t["r"])
    t["y"][3, 7] = -float("inf")
    r_out, h = forward(coat, t, how)
    keep, others = [0, 1, 2, 4, 5], torch.arange(cols, device="cuda") != 7
    assert torch.equal(r_out[keep], clean_r[keep]) and torch.equal(h[keep], clean_h[keep])
    assert bool(r_out[3, 7].isnan()) and torch.equal(r_out[3, others], t["r"][3, others]) and bool(h[3].isnan().all())
    out = backward(coat, t, how, t["r"])  # from a stream without it
    assert torch.equal(out["dr"], clean["dr"]) and torch.equal(out["dw_pre"], clean["dw_pre"])
    assert torch.equal(out["dy"][keep], clean["dy"][keep]) and bool(out["dy"][3].isnan().all())
    assert bool(out["dw_post"][7].isnan()) and bool(out["dw_post"][others].isfinite().all())
    assert torch.equal(out["dgate"][[0, 2]], clean["dgate"][[0, 2]])
    assert bool(out["dgate"][1, 7].isnan()) and bool(out["dgate"][1, others].isfinite().all())


@pytest.mark.parametrize("stream", TYPES)
@pytest.mark.parametrize("cols", [40, 1029, 9000])
def test_an_infinity_in_the_stream(coat, cols, stream):
    """NaN in its channel of h and 0 in the row's others; NaN in the row's dr and dy."""
    t, how = make(6, cols, 42, TYPES[stream], rpg=2)
    clean_r, clean_h = forward(coat, t, how)
    clean = backward(coat, t, how, t["r"])
    t["r"][3, cols - 1] = float("inf")
    r_out, h = forward(coat, t, how)
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(r_out[keep], clean_r[keep]) and torch.equal(h[keep], clean_h[keep])
    assert torch.equal(r_out[3, :-1], clean_r[3, :-1]) and bool(r_out[3, -1] == float("inf"))
    assert bool(h[3, -1].isnan()) and bool((h[3, :-1] == 0).all())
    out = backward(coat, t, how, t["r"])
    for name in ("dr", "dy"):
        assert torch.equal(out[name][keep], clean[name][keep]) and bool(out[name][3].isnan().all())
    assert bool(out["dw_pre"][-1].isnan()) and bool(out["dw_pre"][:-1].isfinite().all())
    assert bool(out["dw_post"].isnan().all())
    assert torch.equal(out["dgate"][[0, 2]], clean["dgate"][[0, 2]]) and bool(out["dgate"][1].isnan().all())


def test_rows_whose_squares_pass_fp32(coat):
    """Finite rows, in y and in the stream, over the documented limit: divided by infinity."""
    t, how = make(5, 1024, 43, F32, rpg=5)
    for name in ("y", "r"):
        t[name][1] = t[name][1].sign() * 1.2e18  # sum of squares 1.5e39
        t[name][2] = t[name][2].sign() * 4.5e17  # 2.1e38: inside
    r_out, h = forward(coat, t, how)
    assert torch.equal(r_out[1], t["r"][1]) and bool((h[1] == 0).all())
    want = o.layer_input(n64(r_out[2:3]), n64(t["w_pre"]), EPS)
    within(h[2:3], want, o.U32 * (o.SUM / 2 + 6) * np.abs(want), BF, "h")
    out = backward(coat, t, how, t["r"])
    assert torch.equal(out["dr"][1], t["dr_out"][1]) and bool((out["dy"][1] == 0).all())
    assert all(bool(v.isfinite().all()) for v in out.values())
