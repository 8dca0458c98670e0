"""Plain 64-bit forms of the layer-input operators, on the CPU, written from their
definitions: microscaled 4-bit floating point and the norms at a block's border.

Rounding: a value stored in a type is off by at most finfo(type).eps / 2 of itself.
"""
from __future__ import annotations

import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U32 = 2.0 ** -24  # half a step of fp32


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- 4-bit floating point

def code_bytes(k: int) -> int:
    return -(-k // 128) * 64


def scale_bytes(k: int) -> int:
    return -(-k // 512) * 16


def mx4_quantize(x: np.ndarray):
    """(q, s) of the rows of a 64-bit matrix, byte for byte, paddings included."""
    rows, cols = x.shape
    kp = code_bytes(cols) * 2
    b = np.zeros((rows, kp))
    b[:, :cols] = x
    b = b.reshape(rows, kp // 32, 32)
    mag = np.abs(b)
    bad = ~np.isfinite(mag).all(axis=2)
    top = np.where(bad, 0.0, np.where(np.isfinite(mag), mag, 0.0).max(axis=2))
    e = np.frexp(top)[1] - 1 - 2                       # floor(log2(top)) - 2
    e = np.where(top == 0, -127, np.maximum(e, -127))
    with np.errstate(invalid="ignore"):
        y = np.minimum(np.ldexp(mag, -e[:, :, None]), 6.0)
    y = np.where(bad[:, :, None], 0.0, y)
    # nearest of the grid by its distance, ties to the even code
    low = np.searchsorted(GRID, y, side="right") - 1
    high = np.minimum(low + 1, 7)
    dl, dh = y - GRID[low], GRID[high] - y
    code = np.where((dl < dh) | ((dl == dh) & (low % 2 == 0)), low, high)
    code = code + 8 * (np.signbit(b) & ~bad[:, :, None])
    code = code.reshape(rows, kp).astype(np.uint8)
    s = np.zeros((rows, scale_bytes(cols)), np.uint8)
    s[:, :kp // 32] = np.where(bad, 255, e + 127)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def mx4_values(q: np.ndarray, s: np.ndarray, cols: int) -> np.ndarray:
    """The 64-bit values that codes and scale bytes stand for."""
    c = np.stack([q & 15, q >> 4], axis=2).reshape(q.shape[0], -1)[:, :cols].astype(np.int64)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    b = np.repeat(s.astype(np.int64), 32, axis=1)[:, :cols]
    return np.where(b == 255, np.nan, np.ldexp(v, b - 127))


def mx4_matmul(aq, as_, bq, bs, k):
    """(product, sum of the magnitudes of its terms)."""
    a, b = mx4_values(aq, as_, k), mx4_values(bq, bs, k)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def matmul_bound(product, magnitude, k: int, dtype: torch.dtype):
    """Largest error of y. A matrix instruction adds 64 products to an fp32 sum: whatever
    its inner order, it is taken to lose at most four half steps of the magnitudes summed
    so far; there are ceil(k / 128) * 2 of them, and up to 64 partial sums to add after."""
    steps = -(-k // 128) * 2 + 64
    return 4 * U32 * steps * magnitude + half_step(dtype) * np.abs(product) + 2.0 ** -133


# ---------------------------------------------------------------- block border
#
# Errors are counted in half steps of fp32 (U32). A sum over the channels adds at
# most 16 values in a thread, 6 times across a wavefront and 16 wavefronts: 38
# roundings, and 1 in each term; the reciprocal root halves a relative error and
# adds about 2; the products that follow add one each.
SUM = 40


def norm(a, eps):
    return 1.0 / np.sqrt((a * a).mean(axis=1, keepdims=True) + eps)


def border(y, r, w_post, w_pre, gate, rpg, scale, eps, post):
    """(r', its error before it is stored in half steps of fp32) in 64 bits."""
    if y is None:
        return r, np.zeros_like(r)
    z = y
    if post:
        z = z * norm(y, eps) * (w_post if w_post is not None else 1.0)
    g = 1.0 if gate is None else gate[np.arange(r.shape[0]) // rpg]
    add = scale * g * z
    return r + add, np.abs(r) + (SUM / 2 + 8) * np.abs(add)


def layer_input(r, w_pre, eps):
    return r * norm(r, eps) * (w_pre if w_pre is not None else 1.0)


def border_backward(y, r, dr_out, dh, w_post, w_pre, gate, rpg, scale, eps, post, groups):
    """{name: (gradient, magnitude)}: the error is within U32 times the magnitude and the
    number of roundings given for it, before the result is stored."""
    out = {}
    ref = r if r is not None else dr_out
    rows, cols = ref.shape
    d = np.zeros((rows, cols)) if dr_out is None else dr_out.copy()
    dm = np.abs(d)
    if dh is not None:
        rho = norm(r, eps)
        w = w_pre if w_pre is not None else np.ones(cols)
        u = dh * w
        s2, s2m = (r * u).sum(1, keepdims=True), np.abs(r * u).sum(1, keepdims=True)
        d = d + rho * u - r * rho ** 3 * s2 / cols
        dm = dm + np.abs(rho * u) + np.abs(r) * rho ** 3 * s2m / cols
        out["dw_pre"] = (dh * r * rho).sum(0), np.abs(dh * r * rho).sum(0)
    out["dr"] = d, dm
    if y is not None:
        sig = norm(y, eps) if post else np.ones((rows, 1))
        yn = y * sig
        w = w_post if w_post is not None else np.ones(cols)
        at = np.arange(rows) // rpg
        g = np.ones((rows, cols)) if gate is None else gate[at]
        dz, dzm = scale * g * d, np.abs(scale * g) * dm
        zd, zdm = scale * w * yn * d, np.abs(scale * w * yn) * dm
        dg, dgm = np.zeros((groups, cols)), np.zeros((groups, cols))
        np.add.at(dg, at, zd)
        np.add.at(dgm, at, zdm)
        out["dgate"] = dg, dgm
        out["dw_post"] = (dz * yn).sum(0), (dzm * np.abs(yn)).sum(0)
        u, um = dz * w, dzm * np.abs(w)
        if post:
            out["dy"] = (sig * u - y * sig ** 3 * (y * u).sum(1, keepdims=True) / cols,
                         sig * um + np.abs(y) * sig ** 3 * (np.abs(y) * um).sum(1, keepdims=True) / cols)
        else:
            out["dy"] = dz, dzm
    return out


# roundings of a term of each result: a sum over the channels goes into dr (SUM and the
# reciprocal root's 1.5 SUM), a second one into dy; a sum over rows adds one a row at most
DR_STEPS = 3 * SUM
DY_STEPS = 6 * SUM


def dw_steps(rows: int) -> int:
    return DY_STEPS + min(rows, 64) + 600
