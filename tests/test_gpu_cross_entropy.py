"""The cross entropy of a vocabulary projection and its gradients against plain 64-bit forms."""
import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat
from test_gpu_linear import strided

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
IGNORE = -100


def inputs(tokens, vocab, cols, seed, ignored=0.3, lift=4.0):
    g = torch.Generator()
    g.manual_seed(seed)
    w = (torch.randn(vocab, cols, generator=g) / max(1, cols) ** 0.5).to(BF16)
    labels = torch.randint(0, vocab, (tokens,), generator=g)
    x = (torch.randn(tokens, cols, generator=g) + lift * torch.rand(tokens, 1, generator=g) * w[labels].float()).to(BF16)
    labels[torch.rand(tokens, generator=g) < ignored] = IGNORE
    dloss = torch.randn(tokens, generator=g)
    return x, w, labels, dloss


def run(x, w, labels, dloss, pad=(0, 0), shift=0, ignore=IGNORE, only=None, **kw):
    tokens, cols = x.shape
    vocab = w.shape[0]
    xd, wd, ld = strided(x, cols + pad[0], shift), strided(w, cols + pad[1], shift), labels.to(DEV)
    loss, lse = torch.full((tokens,), 9.0, device=DEV), torch.full((tokens,), 9.0, device=DEV)
    coat.linear_cross_entropy(xd, wd, ld, loss, lse, ignore_index=ignore, **kw)
    dx, dw = strided(torch.ones(tokens, cols, dtype=BF16), cols + pad[0], shift), strided(torch.ones(vocab, cols, dtype=BF16), cols + pad[1], shift)
    coat.linear_cross_entropy_backward(xd, wd, ld, lse, dloss.to(DEV), dx if only != "dw" else None, dw if only != "dx" else None,
                                       ignore_index=ignore)
    torch.cuda.synchronize()
    return loss, lse, dx, dw


def check(x, w, labels, dloss, ignore=IGNORE, **kw):
    loss, lse, dx, dw = run(x, w, labels, dloss, ignore=ignore, **kw)
    X, W = ref.f64(x), ref.f64(w)
    want, wlse, eloss, elog = ref.cross_entropy(X, W, labels, ignore)
    ref.check("loss", loss, want, eloss)
    ref.check("lse", lse, wlse, elog)
    grads = ref.cross_entropy_backward(X, W, labels, dloss.double(), ignore)
    ref.check("dx", dx, *grads["dx"])
    ref.check("dw", dw, *grads["dw"])
    out = labels == ignore
    assert (loss.cpu()[out] == 0).all() and (lse.cpu()[out] == 0).all() and (dx.cpu()[out] == 0).all()


SIZES = [(1, 1, 1), (1, 2, 8), (1, 300, 72), (3, 5, 7), (16, 33, 40), (17, 257, 64), (32, 100, 129), (33, 129, 96), (64, 31, 16), (65, 1000, 72),
         (130, 515, 200), (257, 700, 136), (300, 64, 64)]


@pytest.mark.parametrize("size", SIZES)
def test_sizes(size):
    check(*inputs(*size, sum(size)))
    x, w, labels, dloss = inputs(*size, sum(size) + 1, ignored=0.0)
    check(x, w, labels, torch.tensor([1.0 / 3]))


@pytest.mark.parametrize("pad,shift", [((8, 8), 0), ((1, 0), 0), ((0, 3), 0), ((0, 0), 1), ((8, 16), 8), ((5, 8), 4)])
@pytest.mark.parametrize("tokens", [5, 90])
def test_strides_and_alignments(pad, shift, tokens):
    check(*inputs(tokens, 300, 96, 3), pad=pad, shift=shift)


def by_norm(x, w, labels, dloss, got):
    """At sizes for 64 bits on the GPU: the losses to 1e-5, gradients to two roundings to bf16 of independent sign."""
    tokens = x.shape[0]
    X, W = x.to(DEV).double(), w.to(DEV).double()
    loss, lse, dx, dw = got
    kept = (labels != IGNORE).to(DEV)
    l = X @ W.t().contiguous()
    y = labels.clamp(min=0).to(DEV)
    want = torch.logsumexp(l, 1) - l.gather(1, y[:, None])[:, 0]
    assert float(((loss.double() - want) * kept).abs().max()) < 1e-5
    g = torch.softmax(l, 1)
    g[torch.arange(tokens, device=DEV), y] -= 1
    g = g * (dloss.to(DEV).double() * kept)[:, None]
    for out, exact in ((dx, g @ W), (dw, g.t().contiguous() @ X)):
        rows = exact.norm(dim=1) > 1e-3 * exact.norm(dim=1).max()
        off = (out.double() - exact).norm(dim=1) / exact.norm(dim=1)
        # a row's own rounding and that of g, each 2^-9 of its size at most in the mean of squares
        assert float(off[rows].max()) < 6 * 2.0 ** -9
        assert float((out.double() - exact).norm() / exact.norm()) < 2 * 2.0 ** -9


def test_pieces_of_the_vocabulary():
    """More tokens than one piece of the vocabulary holds gradients for: 2^27 numbers or 2048 columns."""
    x, w, labels, dloss = inputs(40000, 5000, 40, 4)
    by_norm(x, w, labels, dloss, run(x, w, labels, dloss))
    x, w, labels, dloss = inputs(70000, 4100, 24, 5)
    by_norm(x, w, labels, dloss, run(x, w, labels, dloss, pad=(1, 0)))


@pytest.mark.parametrize("size,pad", [((8100, 4090, 1600), (0, 0)), ((4100, 8190, 1500), (1, 3)), ((4097, 4097, 2500), (0, 4))])
def test_large_tiles(size, pad):
    x, w, labels, dloss = inputs(*size, 6, ignored=0.05)
    by_norm(x, w, labels, dloss, run(x, w, labels, dloss, pad=pad))


def test_long_rows_and_a_wide_vocabulary():
    check(*inputs(40, 9000, 24, 5, ignored=0.1))
    check(*inputs(70, 300, 2100, 6, ignored=0.1))
    check(*inputs(1, 5000, 1000, 7, ignored=0.0))
    check(*inputs(600, 1300, 328, 8, ignored=0.5))


@pytest.mark.parametrize("tokens", [1, 40, 200])
def test_every_token_left_out(tokens):
    x, w, labels, dloss = inputs(tokens, 77, 32, 6)
    labels[:] = IGNORE
    loss, lse, dx, dw = run(x, w, labels, dloss)
    assert (loss == 0).all() and (lse == 0).all() and (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("tokens", [6, 150])
def test_rows_left_out_may_hold_anything(tokens):
    x, w, labels, dloss = inputs(tokens, 300, 64, 7, ignored=0.5)
    labels[0], labels[-1] = IGNORE, IGNORE
    clean = run(x, w, labels, dloss)
    out = labels == IGNORE
    x2, d2 = x.clone(), dloss.clone()
    x2[out], d2[out] = float("nan"), float("inf")
    x2[0] = float("inf")
    for a, b in zip(clean, run(x2, w, labels, d2)):
        assert torch.equal(a, b)


def test_another_ignore_index():
    x, w, labels, dloss = inputs(50, 40, 32, 8, ignored=0.0)
    labels[::3] = 7
    check(x, w, labels, dloss, ignore=7)


@pytest.mark.parametrize("tokens", [4, 100])
def test_labels_outside_the_vocabulary_are_loud(tokens):
    x, w, labels, dloss = inputs(tokens, 64, 32, 9, ignored=0.0)
    clean = run(x, w, labels, dloss)
    for bad in (-1, 64, 2 ** 31, 2 ** 32 + 5, -2 ** 63, 2 ** 63 - 1):
        y = labels.clone()
        y[1] = bad
        loss, lse, dx, dw = run(x, w, y, dloss)
        assert torch.isnan(loss[1]) and torch.isnan(dx[1]).all() and torch.isnan(dw).all()
        keep = torch.arange(tokens) != 1
        assert torch.equal(loss.cpu()[keep], clean[0].cpu()[keep]) and torch.equal(dx.cpu()[keep], clean[2].cpu()[keep])
        assert torch.allclose(lse, clean[1], rtol=0, atol=1e-5)


def test_a_sure_token_keeps_its_digits():
    """Losses far under 1, whose lse - l[label] would lose them."""
    cols, vocab = 16, 40
    w = torch.zeros(vocab, cols, dtype=BF16)
    w[3, 0] = 1.0
    x = torch.zeros(5, cols, dtype=BF16)
    x[:, 0] = torch.tensor([4.0, 8.0, 16.0, 32.0, 64.0])
    labels = torch.full((5,), 3)
    loss = run(x, w, labels, torch.ones(5))[0].cpu().double()
    want = torch.log1p((vocab - 1) * torch.exp(-x[:, 0].double()))
    # an exponential of an argument up to 64, rounded to 64 * 2^-24, and a handful of steps
    assert ((loss - want).abs() <= want * (64 * 2 + 32) * ref.U32).all()


def test_large_and_infinite_logits():
    w = torch.tensor([[1.0], [2.0], [-1.0], [0.0]]).to(BF16)
    x = torch.tensor([[1e30], [-1e30], [3e38], [float("nan")]]).to(BF16)
    labels = torch.tensor([1, 2, 3, 0])
    loss, lse, dx, dw = run(x, w, labels, torch.ones(4))
    assert loss[0] == 0 and loss[1] == 0 and torch.isnan(loss[3])  # the label's logit is the largest by far
    assert float(lse[0]) == float(x[0, 0].double() * 2) and not torch.isfinite(loss[2])
    assert (dx[:2] == 0).all()
    loss = run(x[:1], w, torch.tensor([3]), torch.ones(1))[0]
    assert float(loss[0]) == float(x[0, 0].double() * 2)


@pytest.mark.parametrize("weights", [[0.0] * 20, [1e-38] * 20, [0.0, 3e30] + [1e-30] * 18, [-2.0] * 20])
def test_weights_of_the_losses(weights):
    x, w, labels, _ = inputs(20, 50, 24, 10, ignored=0.2)
    check(x, w, labels, torch.tensor(weights))


def test_an_infinite_weight_stays_in_its_row():
    x, w, labels, dloss = inputs(12, 50, 24, 11, ignored=0.0)
    clean = run(x, w, labels, dloss)
    top = int(dloss.abs().argmax())
    at = (top + 1) % 12
    d = dloss.clone()
    d[at] = float("inf")
    loss, lse, dx, dw = run(x, w, labels, d)
    keep = torch.arange(12) != at
    assert torch.equal(dx.cpu()[keep], clean[2].cpu()[keep]) and not torch.isfinite(dx[at]).any()


def test_one_gradient_alone_and_repeats():
    x, w, labels, dloss = inputs(200, 333, 72, 12)
    a, b = run(x, w, labels, dloss), run(x, w, labels, dloss)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    assert torch.equal(run(x, w, labels, dloss, only="dx")[2], a[2])
    assert torch.equal(run(x, w, labels, dloss, only="dw")[3], a[3])


def test_no_tokens():
    x, w, labels, _ = inputs(0, 30, 16, 13)
    none = torch.empty(0, device=DEV)
    dw = torch.ones(30, 16, dtype=BF16, device=DEV)
    dx = torch.empty(0, 16, dtype=BF16, device=DEV)
    coat.linear_cross_entropy(x.to(DEV), w.to(DEV), labels.to(DEV), none, none.clone())
    coat.linear_cross_entropy_backward(x.to(DEV), w.to(DEV), labels.to(DEV), none, torch.ones(1, device=DEV), dx, dw)
    assert (dw == 0).all()


def test_no_columns():
    x, w, labels, _ = inputs(5, 30, 0, 13)
    loss, lse = torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    coat.linear_cross_entropy(x.to(DEV), w.to(DEV), labels.clamp(min=0).to(DEV), loss, lse)
    assert torch.allclose(loss, torch.full((5,), 30.0, device=DEV).log()) and torch.allclose(lse, loss)


def test_many_tokens_left_out_here_and_there():
    """More labels than the workgroup that orders them takes in a turn."""
    x, w, labels, dloss = inputs(20000, 8, 8, 14, ignored=0.7)
    loss, lse, dx, dw = run(x, w, labels, dloss)
    l = x.double() @ w.double().t()
    kept = labels != IGNORE
    want = torch.logsumexp(l, 1) - l.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    assert ((loss.cpu().double() - torch.where(kept, want, torch.zeros_like(want))).abs() < 1e-5).all()
    g = ref.cross_entropy_backward(x.double(), w.double(), labels, dloss.double(), IGNORE)
    ref.check("dx", dx, *g["dx"])
    ref.check("dw", dw, *g["dw"])


@pytest.mark.parametrize("size", [(1, 2, 8), (1, 300, 72), (5, 1000, 100), (60, 33, 129), (16, 515, 200), (900, 2, 40)])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("ignored", [0.0, 0.4])
def test_few_tokens_are_not_rounded_on_the_way(size, shift, ignored):
    """Up to 16 tokens or 2048 logits: what the first bf16 term of a logit's gradient leaves counts too."""
    x, w, labels, dloss = inputs(*size, 21, ignored=ignored)
    _, _, dx, dw = run(x, w, labels, dloss, shift=shift)
    grads = ref.cross_entropy_backward(ref.f64(x), ref.f64(w), labels, dloss.double(), IGNORE, terms=2)
    ref.check("dx", dx, *grads["dx"])
    ref.check("dw", dw, *grads["dw"])


def test_gradients_against_differences():
    x, w, labels, dloss = inputs(30, 60, 24, 15)
    _, _, dx, dw = run(x, w, labels, dloss)
    X, W = ref.f64(x), ref.f64(w)
    total = lambda a, b: float((ref.cross_entropy(a, b, labels, IGNORE)[0] * dloss.double()).sum())
    g = torch.Generator()
    g.manual_seed(1)
    h = 1e-4
    for grad, which in ((dx, 0), (dw, 1)):
        d = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        want = (total(X + h * d, W) - total(X - h * d, W)) / (2 * h) if which == 0 else (total(X, W + h * d) - total(X, W - h * d)) / (2 * h)
        size = float((grad.double().cpu() * d).norm())
        # the gradient and g are each rounded to bf16: two half steps of each term, independent of each other
        assert abs(float((grad.double().cpu() * d).sum()) - want) <= 40 * 2.0 ** -8 * size


@pytest.mark.parametrize("tokens,terms", [(12, 2), (40, 1), (40, 2)])
def test_weights_far_apart(tokens, terms):
    """The largest weight on a token that counts, the others at 2^-100 of it (all digits kept), and so small that
    their ratio is no fp32 number (taken as zero, as documented)."""
    vocab = 50 if terms == 2 else 60
    x, w, labels, _ = inputs(tokens, vocab, 24, 17, ignored=0.0)
    top = 2.0 ** 40
    weights = torch.full((tokens,), top * 2.0 ** -100)
    weights[1] = -top
    _, _, dx, dw = run(x, w, labels, weights)
    X, W = ref.f64(x), ref.f64(w)
    grads = ref.cross_entropy_backward(X, W, labels, weights.double(), IGNORE, terms=terms)
    least = top * 2.0 ** -126  # what is under fp32's normal numbers before the factor
    ref.check("dx", dx, grads["dx"][0], grads["dx"][1] + least * W.abs().sum(0))
    ref.check("dw", dw, grads["dw"][0], grads["dw"][1] + least * X.abs().sum(0))
    weights = torch.full((tokens,), 1e-30)
    weights[1] = 3e30
    _, _, dx, dw = run(x, w, labels, weights)
    grads = ref.cross_entropy_backward(X, W, labels, weights.double(), IGNORE, terms=terms)
    ref.check("dx", dx[1:2], grads["dx"][0][1:2], grads["dx"][1][1:2])
    ref.check("dw", dw, *grads["dw"])
    want, error = (t[torch.arange(tokens) != 1] for t in grads["dx"])
    got = dx.double().cpu()[torch.arange(tokens) != 1]
    assert ((got - want).abs() <= want.abs() + error).all()  # the value or as little as zero


@pytest.mark.parametrize("tokens,ignored", [(3, 0.0), (16, 0.4)])
@pytest.mark.parametrize("shift", [0, 1])
def test_few_tokens_over_several_pieces(tokens, ignored, shift):
    """Second terms over a vocabulary of more than one piece (2^21 entries): their sums of dx lie in the workspace
    from piece to piece."""
    vocab, cols = (1 << 21) + 300, 8
    x, w, labels, dloss = inputs(tokens, vocab, cols, 22, ignored=ignored)
    labels[0] = vocab - 1
    if tokens > 3:
        labels[1], labels[2] = 0, (1 << 20) + 200
    loss, lse, dx, dw = run(x, w, labels, dloss, shift=shift)
    X, W = ref.f64(x), ref.f64(w)
    kept = labels != IGNORE
    at = labels.clamp(min=0)
    l = X @ W.t()
    want = torch.logsumexp(l, 1)
    # sums of 2^17 partial sums a thread at most, joined in a tree: the mean of squares, not the worst case
    assert float(((lse.cpu().double() - want) * kept).abs().max()) < 1e-5
    g = torch.exp(l - want[:, None])
    g[torch.arange(tokens), at] -= 1
    g = g * (dloss.double() * kept)[:, None]
    for out, exact in ((dx, g @ W), (dw, g.t() @ X)):
        off = (out.double().cpu() - exact).norm(dim=1)
        # the rounding that stores it: half a step of each element at most
        assert bool((off <= 1.1 * ref.half_step(BF16) * exact.norm(dim=1) + 1e-30).all())
    assert (dx.cpu()[~kept] == 0).all()
