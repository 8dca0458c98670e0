"""The training products run together, over the weights and gradients of the optimizer's
state: a training step against automatic differentiation in 64 bits, graphs, streams,
workspaces."""
import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
TOKENS, CHANNELS, HIDDEN, VOCAB = 72, 64, 160, 203
IGNORE = -100


class Model:
    """Embedding rows in, one block (norm, up projection with GELU, down projection with
    dropout onto the stream), norm, vocabulary projection and loss."""

    SIZES = [HIDDEN * CHANNELS, CHANNELS * HIDDEN, VOCAB * CHANNELS]
    SHAPES = [(HIDDEN, CHANNELS), (CHANNELS, HIDDEN), (VOCAB, CHANNELS)]

    def __init__(self, seed=0):
        g = torch.Generator()
        g.manual_seed(seed)
        self.state = coat.ParamListState(self.SIZES, 32)
        self.w, self.dw = [], []
        for i, shape in enumerate(self.SHAPES):
            t = self.state.tensor(i)
            t.params.copy_(torch.randn(t.params.numel(), generator=g) * shape[1] ** -0.5)
            t.params_bf16.copy_(t.params)
            self.w.append(t.params_bf16.view(shape))
            self.dw.append(t.grads.view(shape))
        self.b = (0.1 * torch.randn(HIDDEN, generator=g)).to(DEV)
        self.db = torch.empty(HIDDEN, device=DEV)
        self.r = torch.randn(TOKENS, CHANNELS, generator=g).to(BF16).to(DEV)
        self.labels = torch.randint(0, VOCAB, (TOKENS,), generator=g)
        self.labels[::7] = IGNORE
        self.labels = self.labels.to(DEV)
        self.rng = torch.randint(0, 2 ** 62, (2,), generator=g).to(DEV)
        new = lambda *s, t=BF16: torch.empty(*s, dtype=t, device=DEV)
        self.h, self.h2, self.dh, self.dh2 = (new(TOKENS, CHANNELS) for _ in range(4))
        self.a, self.z, self.da = (new(TOKENS, HIDDEN) for _ in range(3))
        self.r2, self.dr2, self.dr = (new(TOKENS, CHANNELS) for _ in range(3))
        self.loss, self.lse = new(TOKENS, t=F32), new(TOKENS, t=F32)
        self.dloss = torch.full((1,), 1.0 / int((self.labels != IGNORE).sum()), device=DEV)

    def forward(self):
        up, down, vocab = self.w
        coat.block_norm(None, self.r, None, self.h, eps=1e-5)
        coat.linear(self.h, up, self.a, bias=self.b, act=coat.ACT_GELU, z=self.z)
        coat.linear(self.a, down, self.r2, residual=self.r, p=0.2, rng=self.rng, offset=1, scale=0.7)
        coat.block_norm(None, self.r2, None, self.h2, eps=1e-5)
        coat.linear_cross_entropy(self.h2, vocab, self.labels, self.loss, self.lse)

    def backward(self):
        up, down, vocab = self.w
        coat.linear_cross_entropy_backward(self.h2, vocab, self.labels, self.lse, self.dloss, self.dh2, self.dw[2])
        coat.block_norm_backward(None, self.r2, None, self.dh2, self.dr2, eps=1e-5)
        coat.linear_backward(self.dr2, self.a, down, self.da, self.dw[1], p=0.2, rng=self.rng, offset=1, scale=0.7)
        coat.linear_backward(self.da, self.h, up, self.dh, self.dw[0], self.db, act=coat.ACT_GELU, z=self.z)
        coat.block_norm_backward(None, self.r, self.dr2, self.dh, self.dr, eps=1e-5)

    def step(self, n):
        self.state.step(fmt_m=coat.FMT_E4M3, fmt_v=coat.FMT_E5M2, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=n)

    def results(self):
        return [self.loss, self.lse, self.dr, self.db, *self.dw]


def test_training_step_against_automatic_differentiation():
    m = Model()
    m.forward()
    m.backward()
    leaf = [w.double().cpu().requires_grad_() for w in m.w] + [m.b.double().cpu().requires_grad_(), m.r.double().cpu().requires_grad_()]
    up, down, vocab, b, r = leaf
    norm = lambda t: t / (t.square().mean(1, True) + 1e-5).sqrt()
    a = ref.activation(norm(r) @ up.t() + b, "gelu")
    r2 = r + 0.7 * ref.factors(TOKENS, CHANNELS, 0.2, m.rng.cpu(), 1) * (a @ down.t())
    l = norm(r2) @ vocab.t()
    kept = m.labels.cpu() != IGNORE
    y = m.labels.cpu().clamp(min=0)
    loss = torch.where(kept, torch.logsumexp(l, 1) - l[torch.arange(TOKENS), y], torch.zeros(TOKENS, dtype=torch.float64))
    grads = torch.autograd.grad(loss.sum() / kept.sum(), leaf)
    # each of up to eight tensors on the way is rounded to bf16, 2^-9 of its size in the mean of squares
    near = lambda got, want: float((got.double().cpu() - want).norm() / want.norm()) < 8 * 2.0 ** -9
    assert near(m.loss, loss.detach())
    for got, want in zip((*m.dw, m.db, m.dr), grads):
        assert near(got, want)


def test_steps_run_and_repeat():
    """Two runs from the same state agree in every bit; the weights move."""
    out = []
    for _ in range(2):
        m = Model(3)
        first = [w.clone() for w in m.w]
        for n in range(1, 4):
            m.forward()
            m.backward()
            m.step(n)
            m.rng += 2
        out.append([t.clone() for t in (*m.results(), *m.w)])
        assert all(not torch.equal(a, b) for a, b in zip(first, m.w))
        assert all(torch.isfinite(t).all() for t in out[-1])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_captured_step():
    """A captured step replayed on new inputs, with random numbers that advance within the graph, against eager ones."""
    m, e = Model(5), Model(5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.forward()
        m.backward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward()
        m.backward()
        m.rng += 2
    m.rng.copy_(e.rng)
    g = torch.Generator()
    g.manual_seed(9)
    for i in range(4):
        r = torch.randn(TOKENS, CHANNELS, generator=g).to(BF16).to(DEV)
        y = torch.randint(0, VOCAB, (TOKENS,), generator=g)
        y[i::5] = IGNORE
        for x in (m, e):
            x.r.copy_(r)
            x.labels.copy_(y)
        graph.replay()
        e.forward()
        e.backward()
        e.rng += 2
        torch.cuda.synchronize()
        for a, b in zip(m.results(), e.results()):
            assert torch.equal(a, b), i
        torch.empty(1 << 20, device=DEV).normal_()  # other work between the replays
    assert torch.equal(m.rng, e.rng)


def test_two_graphs_with_workspaces_of_their_own():
    """Products with splits, whose partial sums lie in the workspace, in two graphs replayed at once."""
    x, w = (torch.randn(s, device=DEV).to(BF16) for s in ((100, 4096), (256, 4096)))
    need = coat.linear_workspace_bytes(100, 256, 4096)
    assert need > 0
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    want = torch.empty(100, 256, device=DEV)
    coat.linear(x, w, want)
    for s in streams:
        ws, y = torch.empty(need, dtype=torch.uint8, device=DEV), torch.empty(100, 256, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            coat.linear(x, w, y, workspace=ws)
        graphs.append(graph)
        outs.append((y, ws))
    for _ in range(5):
        for y, _ws in outs:
            y.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for y, _ws in outs:
            assert torch.equal(y, want)


def test_calls_on_two_streams_at_once():
    """The stream argument: work waits for that stream's, and each call's workspace is its own."""
    g = torch.Generator()
    g.manual_seed(2)
    x = torch.randn(300, 2048, generator=g).to(BF16).to(DEV)
    w = (torch.randn(500, 2048, generator=g) / 45).to(BF16).to(DEV)
    labels = torch.randint(0, 500, (300,), generator=g).to(DEV)
    rng = torch.tensor([1, 2], device=DEV)

    def run(stream):
        with torch.cuda.stream(stream):
            y = torch.empty(300, 500, device=DEV)
            loss, lse, dl = torch.empty(300, device=DEV), torch.empty(300, device=DEV), torch.ones(300, device=DEV)
            dx, dw, d = torch.empty_like(x), torch.empty_like(w), torch.empty_like(x)
        coat.linear(x, w, y, act=coat.ACT_SILU, p=0.1, rng=rng, stream=stream)
        coat.linear_cross_entropy(x, w, labels, loss, lse, stream=stream)
        coat.linear_cross_entropy_backward(x, w, labels, lse, dl, dx, dw, stream=stream)
        coat.dropout(x, d, p=0.5, rng=rng, stream=stream)
        return y, loss, lse, dx, dw, d

    want = run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [run(s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for out in got:
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_workspaces_given_by_the_caller():
    x, w, y = (torch.randn(s, device=DEV).to(BF16) for s in ((40, 33), (24, 33), (40, 24)))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    labels, loss, lse = torch.zeros(40, dtype=torch.int64, device=DEV), torch.empty(40, device=DEV), torch.empty(40, device=DEV)
    one = torch.ones(1, device=DEV)
    calls = [(coat.linear_workspace_bytes(40, 24, 33, False), lambda ws: coat.linear(x, w, y, workspace=ws)),
             (coat.linear_backward_workspace_bytes(40, 24, 33, False), lambda ws: coat.linear_backward(y, x, w, dx, dw, workspace=ws)),
             (coat.linear_cross_entropy_workspace_bytes(40, 24, 33, False),
              lambda ws: coat.linear_cross_entropy(x, w, labels, loss, lse, workspace=ws)),
             (coat.linear_cross_entropy_backward_workspace_bytes(40, 24, 33, False),
              lambda ws: coat.linear_cross_entropy_backward(x, w, labels, lse, one, dx, dw, workspace=ws))]
    for need, call in calls:
        assert need > 0
        guard = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        call(guard[:need])
        torch.cuda.synchronize()
        assert (guard[need:] == 0xA5).all()
        with pytest.raises(ValueError, match="workspace"):
            call(torch.empty(need - 1, dtype=torch.uint8, device=DEV))
        with pytest.raises(ValueError, match="workspace"):
            call(torch.empty(need, dtype=torch.int8, device=DEV))
        with pytest.raises(coat.CoatError):
            call(torch.empty(need + 256, dtype=torch.uint8, device=DEV)[8:])


def test_refusals_on_the_gpu():
    x, w, y = (torch.zeros(s, dtype=BF16, device=DEV) for s in ((4, 16), (8, 16), (4, 8)))
    rng = torch.zeros(2, dtype=torch.int64, device=DEV)
    bad = [lambda: coat.linear(x, w[:, :8], y), lambda: coat.linear(x, w, y[:, :4]), lambda: coat.linear(x.float(), w, y),
           lambda: coat.linear(x, w, y.half()), lambda: coat.linear(x, w, y, residual=y.float()), lambda: coat.linear(x, w, y, z=y.float()),
           lambda: coat.linear(x, w, y, p=0.5), lambda: coat.linear(x, w, y, p=0.5, rng=rng[:1]), lambda: coat.linear(x, w, y, act=9),
           lambda: coat.linear(x, w, y, bias=rng), lambda: coat.linear(x, w, y, bias=torch.zeros(7, device=DEV)),
           lambda: coat.linear(x, w.cpu(), y), lambda: coat.linear(x, w.t(), y), lambda: coat.linear_backward(y, x, w),
           lambda: coat.linear_backward(y, x, w, x, act=coat.ACT_SILU), lambda: coat.linear_backward(y, x, w, w),
           lambda: coat.dropout(x, y, p=0.1, rng=rng), lambda: coat.dropout(x, x, p=0.1), lambda: coat.dropout(x, x, p=1.0, rng=rng),
           lambda: coat.dropout(x, x, p=0.1, rng=rng.int()),
           lambda: coat.linear_cross_entropy(x, w, rng, rng, rng),
           lambda: coat.linear_cross_entropy(x, w[:0], torch.zeros(4, dtype=torch.int64, device=DEV), x[:, 0].float(), x[:, 0].float()),
           lambda: coat.linear_cross_entropy_backward(x, w, torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, device=DEV),
                                                      torch.zeros(3, device=DEV), x)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(coat.CoatError):
        coat.linear(x, w, y, scale=float("inf"))
