"""Gradients against differences of the 64-bit loss along directions that lie half along the gradient, so that a
factor of a few percent in it shows, and to bounds that are counted from the roundings."""
import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
IGNORE = -100
# A rounding to bf16 is off by half a step of the value at most, evenly spread: in the mean of squares
# by that over the square root of 3.
ROUND = ref.half_step(BF16) / 3 ** 0.5


def direction(grad, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    noise = torch.randn(grad.shape, generator=g, dtype=torch.float64)
    return grad / grad.norm() + noise / noise.norm()


def along(f, at, which, d, h=1e-4):
    up, down = list(at), list(at)
    up[which], down[which] = at[which] + h * d, at[which] - h * d
    return (f(*up) - f(*down)) / (2 * h)


def agree(name, grad, d, want, squares):
    """squares: the sum of the squares of the terms that are rounded on the way, each taken once a rounding."""
    got = float((grad * d).sum())
    # independent roundings: five deviations, and 1e-5 for sums in fp32
    bound = 5 * ROUND * float(squares) ** 0.5 + 1e-5 * float((grad * d).abs().sum())
    assert abs(got - want) <= bound, (name, got, want, bound)
    for factor in (0.97, 1.03):
        assert abs(factor * got - want) > bound, (name, "a wrong factor would pass", factor, got, want, bound)


def linear_inputs(act, seed=4):
    m, n, k = 80, 112, 64
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn(m, k, generator=g).to(BF16)
    w = (torch.randn(n, k, generator=g) / k ** 0.5).to(BF16)
    b = 0.3 * torch.randn(n, generator=g)
    rng = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=g)
    return x, w, b, rng, torch.randn(m, n, generator=g)


def linear_agrees(act, p, x, w, b, rng, c, dx, dw, db):
    X, W, B, C = ref.f64(x), ref.f64(w), ref.f64(b), ref.f64(c)
    f = ref.factors(*c.shape, p, rng)
    at = [X, W, B]
    loss = lambda xx, ww, bb: float((ref.activation(xx @ ww.t() + bb, act) * f * C).sum())
    z = (X @ W.t() + B).requires_grad_()
    s = torch.autograd.grad(ref.activation(z, act).sum(), z, create_graph=True)[0]
    bend = torch.autograd.grad(s.sum(), z)[0] if s.requires_grad else torch.zeros_like(s)
    z, dz = z.detach(), C * f * s.detach()
    moved = C * f * bend.detach() * z   # what z as it is stored moves dz by, in units of z's rounding
    for which, (name, grad) in enumerate((("dx", dx), ("dw", dw), ("dbias", db))):
        grad = grad.double().cpu()
        d = direction(grad, which)
        # by what each value of dz enters the sum
        enters = d @ W.t() if name == "dx" else X @ d.t() if name == "dw" else d.expand_as(dz)
        squares = ((moved * enters) ** 2).sum()
        if name != "dbias":     # dz and the gradient are rounded to bf16, dbias is fp32
            squares = squares + ((dz * enters) ** 2).sum() + ((grad * d) ** 2).sum()
        agree((act, name), grad, d, along(loss, at, which, d), squares)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])  # a difference across relu's bend is not its slope
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_linear(act, p):
    x, w, b, rng, c = linear_inputs(act)
    m, n = c.shape
    z = torch.empty(m, n, dtype=BF16, device=DEV)
    how = dict(act=ref.ACTS[act], p=p, rng=rng.to(DEV))
    coat.linear(x.to(DEV), w.to(DEV), torch.empty(m, n, device=DEV), bias=b.to(DEV), z=z, **how)
    dx, dw, db = torch.empty(x.shape, dtype=BF16, device=DEV), torch.empty(w.shape, dtype=BF16, device=DEV), torch.empty(n, device=DEV)
    coat.linear_backward(c.to(DEV), x.to(DEV), w.to(DEV), dx, dw, db, z=z, **how)
    linear_agrees(act, p, x, w, b, rng, c, dx, dw, db)


def xent_inputs(tokens, vocab, cols, seed=15):
    g = torch.Generator()
    g.manual_seed(seed)
    w = (torch.randn(vocab, cols, generator=g) / cols ** 0.5).to(BF16)
    labels = torch.randint(0, vocab, (tokens,), generator=g)
    x = (torch.randn(tokens, cols, generator=g) + 3 * torch.rand(tokens, 1, generator=g) * w[labels].float()).to(BF16)
    labels[::5] = IGNORE
    return x, w, labels, torch.randn(tokens, generator=g)


def xent_agrees(x, w, labels, dloss, dx, dw):
    X, W, D = ref.f64(x), ref.f64(w), dloss.double()
    total = lambda a, b: float((ref.cross_entropy(a, b, labels, IGNORE)[0] * D).sum())
    kept = labels != IGNORE
    g = torch.softmax(X @ W.t(), 1)
    g[torch.arange(len(labels)), labels.clamp(min=0)] -= 1
    g = g * (D * kept)[:, None]
    for which, (name, grad) in enumerate((("dx", dx), ("dw", dw))):
        grad = grad.double().cpu()
        d = direction(grad, which)
        enters = d @ W.t() if which == 0 else X @ d.t()
        agree(name, grad, d, along(total, [X, W], which, d), ((g * enters) ** 2).sum() + ((grad * d) ** 2).sum())


@pytest.mark.parametrize("size", [(16, 90, 40), (60, 120, 48), (130, 515, 96)])
@pytest.mark.parametrize("with_loss", [False, True])
def test_cross_entropy(size, with_loss):
    x, w, labels, dloss = xent_inputs(*size)
    xd, wd, ld = x.to(DEV), w.to(DEV), labels.to(DEV)
    loss, lse = torch.empty(size[0], device=DEV), torch.empty(size[0], device=DEV)
    coat.linear_cross_entropy(xd, wd, ld, loss, lse)
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    coat.linear_cross_entropy_backward(xd, wd, ld, lse, dloss.to(DEV), dx, dw, loss=loss if with_loss else None)
    xent_agrees(x, w, labels, dloss, dx, dw)
