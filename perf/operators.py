"""Cases of the layer-input operators: what they compute, on what, and what they cost.

Two families, both on (tokens, channels) matrices with one row per token:

* The norms at a block's border. With y the block's output and r the residual stream,

      z  = w_post * y / sqrt(mean(y^2) + eps)         (z = y without the post-norm)
      r' = r + scale * gate * z                        (rounded to the stream's type)
      h  = w_pre * r' / sqrt(mean(r'^2) + eps)         (the next layer's input)

  gate is a matrix whose row t // rows_per_gate belongs to token t. h is returned in
  bf16, or stored as FP8 codes with an fp32 scale per group and read back. The
  backward pass takes the gradients of r' and h to those of r, y, w_post, w_pre and gate.

* Microscaled 4-bit floating point (E2M1 codes, one power-of-two scale per 32 values):
  quantisation of a matrix along its rows, its columns or both; reading back; and the
  product A B^T of two quantised matrices.

A quantised row of K values holds K rounded up to 128 of them (zeros at the end): 64 code
bytes per 128, the first value of a pair in the low half. Its scale bytes, one per 32
values, are padded with zeros to a multiple of 16.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 0), "e5m2": (torch.float8_e5m2, 57344.0, 1)}
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token through a block border while text is generated: latency alone
        dict(name="norm 1x5120", op="norm", tokens=1, cols=5120, res="bf16", rpg=1, post=True, fmt="bf16", group=0),
        # a training step's border on 16k tokens (Llama-2-13B width), the layer input stored in FP8
        dict(name="norm 16384x5120 e4m3", op="norm", tokens=16384, cols=5120, res="bf16", rpg=16384, post=True,
             fmt="e4m3", group=128),
        # the same border's backward pass, one gate per channel
        dict(name="norm-bwd 16384x5120", op="norm_bwd", tokens=16384, cols=5120, res="bf16", rpg=16384, post=True),
        # ragged: an odd width, an fp32 stream, gates of sequences that do not divide the tokens
        dict(name="norm-bwd 1031x2731", op="norm_bwd", tokens=1031, cols=2731, res="fp32", rpg=257, post=True),
        # one token's layer input before a 4-bit product
        dict(name="quantize 1x5120", op="quantize", rows=1, cols=5120, src="bf16", rowwise=True, colwise=False),
        # a down projection's input, along the channels for the product and along the tokens for its weight gradient
        dict(name="quantize 16384x13824 both", op="quantize", rows=16384, cols=13824, src="bf16", rowwise=True,
             colwise=True),
        # a small ragged matrix read back in fp32
        dict(name="dequantize 1029x2731", op="dequantize", rows=1029, cols=2731, out="fp32"),
        # a gate projection's weights exported to bf16
        dict(name="dequantize 13824x5120", op="dequantize", rows=13824, cols=5120, out="bf16"),
        # a gate projection for one token: the weights are read once
        dict(name="product 1x13824x5120", op="product", m=1, n=13824, k=5120, out="bf16"),
        # a short ragged prompt through a down projection
        dict(name="product 333x5120x13824", op="product", m=333, n=5120, k=13824, out="bf16"),
        # a gate projection over a training step's tokens
        dict(name="product 16384x13824x5120", op="product", m=16384, n=13824, k=5120, out="bf16"),
        # that projection's weight gradient over an odd number of tokens
        dict(name="product 13824x5120x8191", op="product", m=13824, n=5120, k=8191, out="fp32"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quantize", "dequantize", "product"])
    if op in ("norm", "norm_bwd"):
        tokens = _spread(rng, 1, 16384)
        cols = _spread(rng, 16, 8192)
        case = dict(op=op, tokens=tokens, cols=cols, res=rng.choice(["bf16", "fp32"]),
                    rpg=rng.choice([1, tokens, _spread(rng, 1, tokens)]), post=rng.random() < 0.7)
        if op == "norm":
            fmt = rng.choice(["bf16", "e4m3", "e5m2"])
            group = 0 if fmt == "bf16" else rng.choice([16, 32, 64, 128, 256, 512])
            if group:
                case["cols"] = max(group, cols // group * group)
            case.update(fmt=fmt, group=group)
        return case
    if op == "quantize":
        way = rng.choice(["rows", "cols", "both"])
        return dict(op=op, rows=_spread(rng, 1, 16384), cols=_spread(rng, 1, 13824), src=rng.choice(["bf16", "fp32"]),
                    rowwise=way != "cols", colwise=way != "rows")
    if op == "dequantize":
        return dict(op=op, rows=_spread(rng, 1, 16384), cols=_spread(rng, 1, 13824), out=rng.choice(["bf16", "fp32"]))
    return dict(op=op, m=_spread(rng, 1, 16384), n=_spread(rng, 1, 13824), k=_spread(rng, 1, 8192),
                out=rng.choice(["bf16", "fp32"]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, rows, cols):
    """Normal values times a scale per channel over four decades, one value in a thousand 50 times larger."""
    ch = torch.pow(10.0, torch.rand(cols, generator=g, device=DEV) * 4 - 3)
    x = _randn(g, rows, cols).mul_(ch)
    big = torch.randint(0, rows * cols, (rows * cols // 1000 + 1,), generator=g, device=DEV)
    x.view(-1)[big] *= 50.0
    return x


def _pad(k, unit):
    return (k + unit - 1) // unit * unit


def _quantized(g, rows, cols, weights):
    """Codes and scales of a random matrix, as a quantised layer input or weight matrix holds them."""
    x = _randn(g, rows, cols).mul_(0.02) if weights else _activations(g, rows, cols)
    q, s = _plain_quantize(x)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        t, c, res = case["tokens"], case["cols"], DTYPE[case["res"]]
        groups = -(-t // case["rpg"])
        st["y"] = _randn(g, t, c).to(torch.bfloat16)
        st["r"] = (_randn(g, t, c) * 3).to(res)
        st["w_post"] = (1 + 0.1 * _randn(g, c)).to(torch.bfloat16) if case["post"] else None
        st["w_pre"] = (1 + 0.1 * _randn(g, c)).to(torch.bfloat16)
        st["gate"] = (0.5 + 0.2 * _randn(g, groups, c)).to(torch.bfloat16)
        st["scale"] = 0.7071
        if op == "norm":
            st["r_out"] = torch.empty(t, c, dtype=res, device=DEV)
            st["h"] = torch.empty(t, c, dtype=torch.bfloat16, device=DEV)
            if case["group"]:
                st["q"] = torch.empty(t, c, dtype=torch.uint8, device=DEV)
                st["q_scale"] = torch.empty(t, c // case["group"], dtype=torch.float32, device=DEV)
        else:  # r is the stream after the border here
            st["d_out"] = _randn(g, t, c).to(res)
            st["dh"] = _randn(g, t, c).to(torch.bfloat16)
            st["dr"] = torch.empty(t, c, dtype=res, device=DEV)
            st["dy"] = torch.empty(t, c, dtype=torch.bfloat16, device=DEV)
            st["dw_post"] = torch.empty(c, dtype=torch.float32, device=DEV) if case["post"] else None
            st["dw_pre"] = torch.empty(c, dtype=torch.float32, device=DEV)
            st["dgate"] = torch.empty(groups, c, dtype=torch.float32, device=DEV)
    elif op == "quantize":
        r, c = case["rows"], case["cols"]
        st["x"] = _activations(g, r, c).to(DTYPE[case["src"]])
        if case["rowwise"]:
            st["q"] = torch.empty(r, _pad(c, 128) // 2, dtype=torch.uint8, device=DEV)
            st["s"] = torch.empty(r, _pad(c, 512) // 32, dtype=torch.uint8, device=DEV)
            st["v"] = torch.empty(r, c, dtype=torch.bfloat16, device=DEV)
        if case["colwise"]:
            st["q_t"] = torch.empty(c, _pad(r, 128) // 2, dtype=torch.uint8, device=DEV)
            st["s_t"] = torch.empty(c, _pad(r, 512) // 32, dtype=torch.uint8, device=DEV)
            st["v_t"] = torch.empty(c, r, dtype=torch.bfloat16, device=DEV)
    elif op == "dequantize":
        st["q"], st["s"] = _quantized(g, case["rows"], case["cols"], True)
        st["v"] = torch.empty(case["rows"], case["cols"], dtype=DTYPE[case["out"]], device=DEV)
    else:
        st["aq"], st["as"] = _quantized(g, case["m"], case["k"], False)
        st["bq"], st["bs"] = _quantized(g, case["n"], case["k"], True)
        st["out"] = torch.empty(case["m"], case["n"], dtype=DTYPE[case["out"]], device=DEV)
    return st


# ---------------------------------------------------------------- plain forms

def _plain_quantize(x):
    """E2M1 codes and E8M0 scales of x's rows: blocks of 32, the scale 2^(floor(log2 amax) - 2), values over 6 cut."""
    rows, cols = x.shape
    kp = _pad(cols, 128)
    b = torch.nn.functional.pad(x.float(), (0, kp - cols)).view(rows, kp // 32, 32)
    amax = b.abs().amax(dim=2)
    e = (torch.frexp(amax).exponent - 3).clamp_(min=-127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = torch.ldexp(b, -e.unsqueeze(2))
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(rows, kp)
    s = torch.nn.functional.pad(e + 127, (0, _pad(cols, 512) // 32 - kp // 32))
    return code[:, 0::2] | (code[:, 1::2] << 4), s.to(torch.uint8)


def _plain_values(q, s, cols):
    """The values that codes and scales stand for, in fp32."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), device=q.device)
    pairs = torch.stack((table[(q & 15).int()], table[(q >> 4).int()]), dim=2)
    v = pairs.view(q.shape[0], -1, 32)
    v = torch.ldexp(v, s[:, :v.shape[1]].int().unsqueeze(2) - 127)
    return v.reshape(q.shape[0], -1)[:, :cols]


def _plain_fp8(h, group, fmt):
    """h stored as FP8 codes with one fp32 scale per group, read back in bf16."""
    dt, top, _ = FP8[fmt]
    x = h.float().view(-1, group)
    s = x.abs().amax(dim=1, keepdim=True) / top
    code = (x / s).clamp(-top, top).to(dt)
    return (code.float() * s).to(torch.bfloat16).view(h.shape)


def _plain_norm(st):
    c = st["case"]
    z = st["y"].float()
    if c["post"]:
        z = z * torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS) * st["w_post"].float()
    gate = st["gate"].float().repeat_interleave(c["rpg"], dim=0)[:c["tokens"]]
    r = (st["r"].float() + st["scale"] * gate * z).to(st["r"].dtype)
    x = r.float()
    h = (x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * st["w_pre"].float()).to(torch.bfloat16)
    if c["group"]:
        h = _plain_fp8(h, c["group"], c["fmt"])
    return {"r": r, "h": h}


def _plain_norm_bwd(st):
    c = st["case"]
    t, n = c["tokens"], c["cols"]
    x, dh = st["r"].float(), st["dh"].float()
    rho = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    xn = x * rho
    u = dh * st["w_pre"].float()
    d = st["d_out"].float() + rho * (u - xn * (xn * u).mean(dim=1, keepdim=True))
    out = {"dw_pre": (dh * xn).sum(dim=0), "dr": d.to(st["r"].dtype)}
    yn = st["y"].float()
    if c["post"]:
        sig = torch.rsqrt((yn * yn).mean(dim=1, keepdim=True) + EPS)
        yn = yn * sig
        z = yn * st["w_post"].float()
    else:
        z = yn
    gate = st["gate"].float().repeat_interleave(c["rpg"], dim=0)[:t]
    dz = st["scale"] * gate * d
    zd = st["scale"] * z * d
    groups = st["gate"].shape[0]
    zd = torch.nn.functional.pad(zd, (0, 0, 0, groups * c["rpg"] - t))
    out["dgate"] = zd.view(groups, c["rpg"], n).sum(dim=1)
    if c["post"]:
        out["dw_post"] = (dz * yn).sum(dim=0)
        u = dz * st["w_post"].float()
        out["dy"] = (sig * (u - yn * (yn * u).mean(dim=1, keepdim=True))).to(torch.bfloat16)
    else:
        out["dy"] = dz.to(torch.bfloat16)
    return out


def _plain(st):
    c = st["case"]
    if c["op"] == "norm":
        return _plain_norm(st)
    if c["op"] == "norm_bwd":
        return _plain_norm_bwd(st)
    if c["op"] == "quantize":
        out = {}
        if c["rowwise"]:
            out["v"] = _plain_values(*_plain_quantize(st["x"]), c["cols"]).to(torch.bfloat16)
        if c["colwise"]:
            out["v_t"] = _plain_values(*_plain_quantize(st["x"].t()), c["rows"]).to(torch.bfloat16)
        return out
    if c["op"] == "dequantize":
        return {"v": _plain_values(st["q"], st["s"], c["cols"]).to(DTYPE[c["out"]])}
    a, b = _plain_values(st["aq"], st["as"], c["k"]), _plain_values(st["bq"], st["bs"], c["k"])
    return {"out": torch.matmul(a, b.t()).to(DTYPE[c["out"]])}


# ---------------------------------------------------------------- the framework's kernels

def _kernels(st):
    import fp8_optimizer_state_amd as coat

    c = st["case"]
    if c["op"] == "norm":
        how = dict(w_post=st["w_post"], w_pre=st["w_pre"], gate=st["gate"], rows_per_gate=c["rpg"], post=c["post"],
                   scale=st["scale"], eps=EPS)
        if c["group"]:
            fmt = FP8[c["fmt"]][2]
            coat.block_norm(st["y"], st["r"], st["r_out"], None, q=st["q"], q_scale=st["q_scale"], group=c["group"],
                            fmt=fmt, **how)
            coat.act_dequantize(st["q"], st["q_scale"], st["h"], group=c["group"], fmt=fmt)
        else:
            coat.block_norm(st["y"], st["r"], st["r_out"], st["h"], **how)
        return {"r": st["r_out"], "h": st["h"]}
    if c["op"] == "norm_bwd":
        coat.block_norm_backward(st["y"], st["r"], st["d_out"], st["dh"], st["dr"], st["dy"], w_post=st["w_post"],
                                 w_pre=st["w_pre"], gate=st["gate"], rows_per_gate=c["rpg"], post=c["post"],
                                 scale=st["scale"], eps=EPS, dw_post=st["dw_post"], dw_pre=st["dw_pre"],
                                 dgate=st["dgate"])
        out = {k: st[k] for k in ("dr", "dy", "dw_pre", "dgate")}
        if c["post"]:
            out["dw_post"] = st["dw_post"]
        return out
    if c["op"] == "quantize":
        coat.mx4_quantize(st["x"], st.get("q"), st.get("s"), st.get("q_t"), st.get("s_t"))
        out = {}
        if c["rowwise"]:
            coat.mx4_dequantize(st["q"], st["s"], st["v"])
            out["v"] = st["v"]
        if c["colwise"]:
            coat.mx4_dequantize(st["q_t"], st["s_t"], st["v_t"])
            out["v_t"] = st["v_t"]
        return out
    if c["op"] == "dequantize":
        coat.mx4_dequantize(st["q"], st["s"], st["v"])
        return {"v": st["v"]}
    coat.mx4_matmul(st["aq"], st["as"], st["bq"], st["bs"], st["out"])
    return {"out": st["out"]}


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------- cost

def _code_bytes(rows, cols):
    """Codes and scales of a quantised matrix: whole blocks of 32."""
    return rows * ((cols + 31) // 32) * 17


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        t, c = case["tokens"], case["cols"]
        res = 2 if case["res"] == "bf16" else 4
        groups = -(-t // case["rpg"])
        weights = (2 if case["post"] else 1) * c + groups * c
        if op == "norm":  # y, r in; r' and h out
            nbytes = t * c * (2 + res + res + 2) + 2 * weights
            if case["group"]:  # codes and scales written and read
                nbytes += 2 * t * (c + 4 * (c // case["group"]))
            return dict(bytes=nbytes, flops=12 * t * c)
        # y, r', their gradients' sources in; dr, dy and the gradients of the weights and gates out
        return dict(bytes=t * c * (2 + res + res + 2 + res + 2) + 2 * weights + 4 * weights, flops=30 * t * c)
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        nbytes = r * c * (2 if case["src"] == "bf16" else 4)
        if case["rowwise"]:
            nbytes += 2 * _code_bytes(r, c) + 2 * r * c
        if case["colwise"]:
            nbytes += 2 * _code_bytes(c, r) + 2 * r * c
        return dict(bytes=nbytes, flops=4 * r * c)
    if op == "dequantize":
        r, c = case["rows"], case["cols"]
        return dict(bytes=_code_bytes(r, c) + r * c * (2 if case["out"] == "bf16" else 4), flops=r * c)
    m, n, k = case["m"], case["n"], case["k"]
    return dict(bytes=_code_bytes(m, k) + _code_bytes(n, k) + m * n * (2 if case["out"] == "bf16" else 4),
                flops=2 * m * n * k)


# ---------------------------------------------------------------- 64 bits

def _exact_values(q, s, cols):
    """Each code's value from its bits: sign, two exponent bits with bias 1, one mantissa bit."""
    c = torch.stack((q.bitwise_and(15), q.bitwise_right_shift(4)), dim=-1).flatten(1).long()[:, :cols]
    expo, mant, sign = (c >> 1) & 3, c & 1, 1.0 - 2.0 * (c >> 3).double()
    mag = torch.where(expo == 0, 0.5 * mant.double(), (1.0 + 0.5 * mant.double()) * torch.exp2(expo.double() - 1.0))
    return sign * mag * torch.exp2(s.double() - 127.0).repeat_interleave(32, dim=1)[:, :cols]


def _exact_blocks(x):
    """x's rows rounded, block of 32 by block of 32, to the nearest grid value times the block's power of two."""
    rows, cols = x.shape
    n = -(-cols // 32)
    b = torch.zeros(rows, n * 32, dtype=torch.float64, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, n, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 2)
    v = (b / unit).abs().clamp(max=6.0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    return (torch.copysign(torch.round(v / step) * step, b) * unit).view(rows, -1)[:, :cols]


def _exact_norm(case, st):
    """The border in 64 bits; the stream and the layer input pass through the types they are stored in."""
    y, r, gate = st["y"].double(), st["r"].double(), st["gate"].double()
    at = torch.arange(case["tokens"], device=r.device) // case["rpg"]
    z = y
    if case["post"]:
        z = y / (y.square().mean(1, True) + EPS).sqrt() * st["w_post"].double()
    r = r + z * gate[at] * st["scale"]
    out = {"r": r}
    r = r.to(st["r"].dtype).double()
    h = r / (r.square().mean(1, True) + EPS).sqrt() * st["w_pre"].double()
    if case["group"]:
        dt, top, _ = FP8[case["fmt"]]
        g = h.to(torch.bfloat16).double().reshape(-1, case["group"])
        s = (g.abs().amax(1, True) / top).float().double()
        h = ((g / s).float().clamp(-top, top).to(dt).double() * s).reshape(h.shape)
    out["h"] = h
    return out


def _exact_norm_bwd(case, st):
    """Derivatives of sum(d_out * r') + sum(dh * h) by 64-bit automatic differentiation, at the stored stream."""
    leaf = {k: st[k].double().requires_grad_() for k in ("y", "gate", "w_pre") + (("w_post",) if case["post"] else ())}
    at = torch.arange(case["tokens"], device=st["r"].device) // case["rpg"]
    z = leaf["y"]
    if case["post"]:
        z = z / (z.square().mean(1, True) + EPS).sqrt() * leaf["w_post"]
    add = z * leaf["gate"][at] * st["scale"]
    r = (st["r"].double() - add.detach()).requires_grad_()  # the stream before the border
    s = r + add
    h = s / (s.square().mean(1, True) + EPS).sqrt() * leaf["w_pre"]
    total = (s * st["d_out"].double()).sum() + (h * st["dh"].double()).sum()
    names = ["y", "gate", "w_pre"] + (["w_post"] if case["post"] else [])
    got = torch.autograd.grad(total, [r] + [leaf[k] for k in names])
    return dict(zip(["dr"] + [{"y": "dy", "gate": "dgate", "w_pre": "dw_pre", "w_post": "dw_post"}[k] for k in names], got))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(case, st)
    if op == "norm_bwd":
        return _exact_norm_bwd(case, st)
    if op == "quantize":
        x = st["x"].double()
        out = {}
        if case["rowwise"]:
            out["v"] = _exact_blocks(x)
        if case["colwise"]:
            out["v_t"] = _exact_blocks(x.t())
        return out
    if op == "dequantize":
        return {"v": _exact_values(st["q"], st["s"], case["cols"])}
    a, b = _exact_values(st["aq"], st["as"], case["k"]), _exact_values(st["bq"], st["bs"], case["k"])
    return {"out": torch.matmul(a, b.t().contiguous())}
