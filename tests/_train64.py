"""Plain 64-bit forms of the training products, written from their definitions, and
how far the kernels may be from them.

Rounding: a value stored in a type is off by at most finfo(type).eps / 2 of itself.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24  # half a step of fp32
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
# An activation's own error relative to |z|: the error function is off by 1.5e-7, the
# hardware's exponential and reciprocal by a step each, and a handful of roundings.
ACT = 4e-7
# The same of a slope, absolute: two such terms, the second times at most 1.2.
SLOPE = 1e-6


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().double().cpu()


def product(a, b):
    """a b^T and the sum of the magnitudes of its terms."""
    return a @ b.t(), a.abs() @ b.abs().t()


def sum_error(magnitude, k: int, joined: int = 64):
    """Largest error of a sum of k products held in fp32. A matrix instruction adds 16
    products: whatever its inner order, it is taken to lose at most four half steps of the
    magnitudes summed so far; up to `joined` partial sums are added after."""
    return 4 * U32 * (-(-k // 16) + joined) * magnitude


# ---------------------------------------------------------------- dropout

def philox_words(block: int, high: int, key: int):
    """Four words of Philox 4x32-10, on Python's own integers."""
    mask = 2 ** 32 - 1
    c = [block & mask, block >> 32 & mask, high & mask, high >> 32 & mask]
    k = [key & mask, key >> 32 & mask]
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [q >> 32 ^ c[1] ^ k[0], q & mask, p >> 32 ^ c[3] ^ k[1], p & mask]
        k = [(k[0] + 0x9E3779B9) & mask, (k[1] + 0xBB67AE85) & mask]
    return c


def factors(rows: int, cols: int, p: float, rng, offset: int = 0, row0: int = 0, nrows=None):
    """0 or 1 / (1 - p) for each element of rows row0 .. of the matrix, from the definition."""
    nrows = rows - row0 if nrows is None else nrows
    if p == 0:
        return torch.ones(nrows, cols, dtype=torch.float64)
    t = min(65535, int(math.floor(65536 * p + 0.5)))
    seed, step = (int(v) % 2 ** 64 for v in rng.tolist())
    high = (step + offset) % 2 ** 64
    blocks = -(-cols // 8)
    f = torch.zeros(nrows, blocks * 8, dtype=torch.float64)
    for r in range(nrows):
        for b in range(blocks):
            w = philox_words((row0 + r) * blocks + b, high, seed)
            for e in range(8):
                if (w[e // 2] >> (16 * (e % 2)) & 0xFFFF) >= t:
                    f[r, b * 8 + e] = 65536.0 / (65536 - t)
    return f[:, :cols]


def dropped(f, v):
    return torch.where(f > 0, v * f, torch.zeros_like(v))


# ---------------------------------------------------------------- linear layer

def activation(z, act: str):
    if act == "relu":
        return torch.where(z > 0, z, torch.where(z <= 0, torch.zeros_like(z), z))
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def activation_slope(z, act: str):
    if act == "relu":
        return (z > 0).double()
    if act == "none":
        return torch.ones_like(z)
    z = z.clone().requires_grad_()
    return torch.autograd.grad(activation(z, act).sum(), z)[0]


def linear(x, w, bias, act, f, scale, residual):
    """(y, its error before it is stored, z, its error before it is stored)."""
    z, mag = product(x, w)
    if bias is not None:
        z, mag = z + bias, mag + bias.abs()
    ez = sum_error(mag, x.shape[1]) + U32 * z.abs()
    a = activation(z, act)
    v = scale * dropped(f, a)
    y = v if residual is None else residual + v
    # every activation's slope is under 1.2
    ey = abs(scale) * dropped(f, 1.2 * ez + (0 if act == "none" else ACT) * z.abs()) + 6 * U32 * (v.abs() + y.abs())
    return y, ey, z, ez


def linear_backward(dy, x, w, z, act, f, scale, terms=1):
    """{name: (gradient, its error before it is stored)}; dz taken as `terms` values in bf16."""
    s = activation_slope(z, act) if act != "none" else torch.ones_like(dy)
    d = dropped(f, dy)
    dz = scale * d * s
    exact = abs(scale) * d.abs() * ((0 if act == "none" else SLOPE) + 6 * U32 * s.abs())
    edz = exact + half_step(torch.bfloat16) ** terms * (dz.abs() + exact)  # as the products take it
    m, n = dy.shape
    out = {}
    g, mag = product(dz, w.t())
    out["dx"] = g, edz @ w.abs() + sum_error(mag, n) + 4 * U32 * mag
    g, mag = product(dz.t(), x.t())
    out["dw"] = g, edz.t() @ x.abs() + sum_error(mag, m) + 4 * U32 * mag
    # a band's rows (8 to 64) are added at most 16 in a thread and joined in 2 more additions,
    # the bands (m / 8 at most) every fourth in a thread and joined in 2 more, and scaled
    out["dbias"] = dz.sum(0), exact.sum(0) + U32 * (24 + -(-m // 32)) * dz.abs().sum(0)
    return out


# ---------------------------------------------------------------- cross entropy

def cross_entropy(x, w, labels, ignore):
    """(loss, lse, error of the loss, error of lse); zeros where the label is ignored."""
    kept = labels != ignore
    at = torch.where(kept, labels, torch.zeros_like(labels))
    l, mag = product(torch.where(kept[:, None], x, torch.zeros_like(x)), w)
    lse = torch.logsumexp(l, 1)
    rows = torch.arange(len(at))
    loss = lse - l[rows, at]
    el = sum_error(mag, x.shape[1])
    top = el.max(1).values if l.shape[1] else el.sum(1)
    # an exponential's argument is rounded relative to its size (terms that count are
    # within 2 log(vocab) + 20 of the largest), its value by two steps, the sum by its depth
    own = U32 * (64 + 4 * (20 + 2 * math.log(max(2, l.shape[1]))) + 2 * lse.abs())
    zero = torch.zeros_like(loss)
    e = torch.where(kept, top + own, zero)
    return torch.where(kept, loss, zero), torch.where(kept, lse, zero), e + torch.where(kept, el[rows, at], zero), e


def cross_entropy_backward(x, w, labels, dloss, ignore, terms=1):
    """{name: (gradient, its error before it is stored)}; the logits' taken as `terms` values in bf16."""
    kept = labels != ignore
    at = torch.where(kept, labels, torch.zeros_like(labels))
    x = torch.where(kept[:, None], x, torch.zeros_like(x))
    l, mag = product(x, w)
    _, lse, _, elog = cross_entropy(x, w, labels, ignore)
    p = torch.softmax(l, 1)
    rows = torch.arange(len(at))
    weight = torch.where(kept, dloss.expand(len(at)), torch.zeros(len(at), dtype=torch.float64))[:, None]
    hot = torch.zeros_like(p)
    hot[rows, at] = 1.0
    g = weight * (p - hot)
    # lse as it is stored, and the logits computed again
    exact = weight.abs() * (p * (elog[:, None] + sum_error(mag, x.shape[1]) + U32 * (16 + 3 * (l.abs() + lse[:, None].abs())))
                            + 4 * U32 * hot)
    eg = exact + half_step(torch.bfloat16) ** terms * (g.abs() + exact)
    out = {}
    d, m = product(g, w.t())
    out["dx"] = d, eg @ w.abs() + sum_error(m, w.shape[0], 128) + 4 * U32 * m
    d, m = product(g.t(), x.t())
    out["dw"] = d, eg.t() @ x.abs() + sum_error(m, x.shape[0]) + 4 * U32 * m
    return out


def check(name: str, got, want, error, dtype=None):
    """got (stored in its type) is within `error` and its own rounding of want."""
    dtype = dtype or got.dtype
    tol = error + half_step(dtype) * (want.abs() + error) + 2.0 ** -133
    g = got.detach().double().cpu()
    off = (g - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), "%s: %d of %d, worst at %s: got %r, want %r, may be off by %r" % (
        name, int(bad.sum()), bad.numel(), tuple(int(i) for i in torch.nonzero(bad)[0]), float(g[bad][0]), float(want[bad][0]),
        float(tol[bad][0]))
