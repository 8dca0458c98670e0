"""Gradients of the cross entropy where the model is sure of the label: with the forward's loss they
keep the digits that the loss has."""
import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat
from test_gpu_linear import strided

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
IGNORE = -100


def run(x, w, labels, dloss, shift=0):
    tokens, cols = x.shape
    xd, wd, ld = strided(x, shift=shift), strided(w, shift=shift), labels.to(DEV)
    loss, lse = torch.empty(tokens, device=DEV), torch.empty(tokens, device=DEV)
    coat.linear_cross_entropy(xd, wd, ld, loss, lse, ignore_index=IGNORE)
    dx, dw = torch.ones(tokens, cols, dtype=BF16, device=DEV), torch.ones(w.shape[0], cols, dtype=BF16, device=DEV)
    coat.linear_cross_entropy_backward(xd, wd, ld, lse, dloss.to(DEV), dx, dw, loss=loss, ignore_index=IGNORE)
    torch.cuda.synchronize()
    return loss, lse, dx, dw


def sure(tokens, vocab, cols, seed, ignored=0.2):
    """Labels' logits far above the others: losses from about 1 down to far under the step of lse."""
    g = torch.Generator()
    g.manual_seed(seed)
    w = (torch.randn(vocab, cols, generator=g) / cols ** 0.5).to(BF16)
    labels = torch.randint(0, vocab, (tokens,), generator=g)
    x = (torch.randn(tokens, cols, generator=g) + torch.linspace(60, 5, tokens)[:, None] * w[labels].float()).to(BF16)
    labels[torch.rand(tokens, generator=g) < ignored] = IGNORE
    return x, w, labels, torch.randn(tokens, generator=g)


def exact(x, w, labels, dloss, device="cpu"):
    """(g, g without cancellation at the label, relative error of g's entries) in 64 bits."""
    x, w, labels = x.to(device).double(), w.to(device).double(), labels.to(device)
    kept = labels != IGNORE
    at = labels.clamp(min=0)[:, None]
    l = x @ w.t().contiguous()
    own = l.gather(1, at)
    others = l.scatter(1, at, float("-inf"))
    rest = torch.logsumexp(others, 1, keepdim=True)       # log sum of the others' exponentials
    lse = torch.logaddexp(rest, own)
    p = torch.exp(others - lse)
    g = p.scatter(1, at, -torch.exp(rest - lse))          # 1 - p of the label is the others' share
    weight = (dloss.to(device).double().expand(len(labels)) * kept)[:, None]
    # A logit's own error moves p and 1 - p by that much of themselves, twice where lse's logits and these
    # differ. lse and l are rounded, the exponentials' arguments (at most |l| + |lse|, and up to 2 |l| as the log
    # sum takes them) are rounded relative to their size and so are their products with log2 e.
    el = ref.sum_error(x.abs() @ w.abs().t().contiguous(), x.shape[1]).amax(1, keepdim=True)
    relative = 4 * el + ref.U32 * (64 + 8 * (l.abs().amax(1, keepdim=True) + lse.abs()))
    return weight * g, relative


def check(x, w, labels, dloss, got, terms):
    g, relative = exact(x, w, labels, dloss)
    own = g.gather(1, labels.clamp(min=0)[:, None])[:, 0] / dloss.double()
    assert float(own[labels != IGNORE].abs().min()) < 1e-8   # under the step of lse
    X, W = ref.f64(x), ref.f64(w)
    eg = g.abs() * (relative + ref.half_step(BF16) ** terms * (1 + relative)) + 2.0 ** -126
    for name, out, a, e, b in (("dx", got[2], g, eg, W.t()), ("dw", got[3], g.t(), eg.t(), X.t())):
        want, m = ref.product(a, b)
        ref.check(name, out, want, e @ b.abs().t() + ref.sum_error(m, a.shape[1], 128) + 4 * ref.U32 * m)


def test_a_sure_token_keeps_its_gradients_digits():
    """One column: dx is the label's own gradient, with nothing else in the sum."""
    vocab = 40
    w = torch.zeros(vocab, 16, dtype=BF16)
    w[3, 0] = 1.0
    x = torch.zeros(5, 16, dtype=BF16)
    x[:, 0] = torch.tensor([4.0, 8.0, 16.0, 32.0, 64.0])
    labels = torch.full((5,), 3)
    for dloss in (torch.ones(5), torch.tensor([1.0 / 3])):
        _, _, dx, dw = run(x, w, labels, dloss)
        z, d = x[:, 0].double(), dloss.double().expand(5)
        others = (vocab - 1) * torch.exp(-z)
        g = -others / (1 + others) * d
        # the loss is good to (64 * 2 + 32) steps; two bf16 terms, one rounding to bf16 stored
        near = (64 * 2 + 64) * ref.U32 + ref.half_step(BF16) ** 2 + ref.half_step(BF16)
        assert ((dx[:, 0].cpu().double() - g).abs() <= near * g.abs()).all()
        assert abs(float(dw[3, 0]) - float((g * z).sum())) <= near * float((g * z).sum().abs())
        other = float((torch.exp(-z) / (1 + others) * d * z).sum())
        assert ((dw[:, 0].cpu().double() - other).abs()[torch.arange(vocab) != 3] <= (near + 512 * ref.U32) * other).all()


@pytest.mark.parametrize("size,terms", [((1, 50, 64), 2), ((13, 1000, 96), 2), ((40, 30, 64), 2), ((60, 300, 96), 1), ((300, 1300, 136), 1),
                                        ((17, 9000, 40), 1)])
@pytest.mark.parametrize("shift", [0, 1])
def test_sure_tokens(size, terms, shift):
    x, w, labels, dloss = sure(*size, sum(size), ignored=0.0 if size[0] == 1 else 0.2)
    check(x, w, labels, dloss, run(x, w, labels, dloss, shift), terms)


@pytest.mark.parametrize("size", [(20000, 9000, 64), (8100, 4090, 1600), (4100, 8190, 328)])
def test_sure_tokens_in_pieces_and_large_tiles(size):
    """Every row of dx, however small, to the roundings of g and its own, in the mean of squares."""
    x, w, labels, dloss = sure(*size, 7)
    _, _, dx, dw = run(x, w, labels, dloss)
    g, relative = exact(x, w, labels, dloss, DEV)
    kept = (labels != IGNORE).to(DEV)
    W, X = w.to(DEV).double(), x.to(DEV).double()
    for out, a, b in ((dx, g, W), (dw, g.t().contiguous(), X)):
        want = a @ b
        size2 = (a.square() @ b.square()).sum(1).sqrt()   # of the terms, in the mean of squares
        off = (out.double() - want).norm(dim=1)
        worst = float(relative[kept].max())
        # each of g's entries is off by half a step at most and by its relative error, the sum by half a step stored
        bound = (4 * 2.0 ** -9 + 4 * worst) * size2 + 2.0 ** -9 * want.norm(dim=1) + 1e-30
        rows = kept if out is dx else torch.ones(len(want), dtype=torch.bool, device=DEV)
        assert bool((off <= bound)[rows].all()), float((off / bound)[rows].max())


def test_rows_left_out_and_labels_outside():
    """A loss that is not read where the token is left out; NaN for a label outside, in its own row."""
    x, w, labels, dloss = sure(50, 60, 32, 3)
    labels[0] = IGNORE
    clean = run(x, w, labels, dloss)
    xd, wd, ld = x.to(DEV), w.to(DEV), labels.to(DEV)
    loss = torch.where(ld == IGNORE, float("nan"), clean[0])
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    coat.linear_cross_entropy_backward(xd, wd, ld, clean[1], dloss.to(DEV), dx, dw, loss=loss, ignore_index=IGNORE)
    assert torch.equal(dx, clean[2]) and torch.equal(dw, clean[3])
    labels[5] = 60
    got = run(x, w, labels, dloss)
    keep = torch.arange(50) != 5
    assert torch.isnan(got[2][5]).all() and torch.equal(got[2].cpu()[keep], clean[2].cpu()[keep])


def test_large_and_infinite_logits():
    w = torch.tensor([[1.0], [2.0], [-1.0], [0.0]]).to(BF16)
    x = torch.tensor([[1e30], [-1e30], [float("nan")]]).to(BF16)
    _, _, dx, _ = run(x, w, torch.tensor([1, 2, 0]), torch.ones(3))
    assert (dx[:2] == 0).all() and torch.isnan(dx[2]).all()
    _, _, dx, _ = run(x[:1], w, torch.tensor([3]), torch.ones(1))   # all of it on another column: g is 1 there, -1 here
    assert float(dx[0, 0]) == 2.0


def test_captured_and_replayed():
    x, w, labels, dloss = (t.to(DEV) for t in sure(70, 300, 64, 5))
    loss, lse = torch.empty(70, device=DEV), torch.empty(70, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)

    def both():
        coat.linear_cross_entropy(x, w, labels, loss, lse)
        coat.linear_cross_entropy_backward(x, w, labels, lse, dloss, dx, dw, loss=loss)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (6, 7, 8):
        for t, new in zip((x, w, labels, dloss), sure(70, 300, 64, seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (loss, lse, dx, dw)]
        both()
        torch.cuda.synchronize()
        for a, b in zip(got, (loss, lse, dx, dw)):
            assert torch.equal(a, b)


def test_refusals():
    x, w, labels, dloss = (t.to(DEV) for t in sure(6, 30, 16, 5))
    lse = torch.zeros(6, device=DEV)
    for bad in (lse[:5], lse.double(), lse.cpu(), torch.zeros(12, device=DEV)[::2]):
        with pytest.raises(ValueError, match="loss"):
            coat.linear_cross_entropy_backward(x, w, labels, lse, dloss, torch.empty_like(x), loss=bad)
