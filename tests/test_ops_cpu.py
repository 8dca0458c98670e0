"""Refusals of the layer-input operators, before any device work (CPU only): through the
C ABI with addresses that are never read, and in the Python binding."""
import ctypes

import pytest
import torch

import fp8_optimizer_state_amd as coat

FAKE = 0x7F0000000000
OK, EINVAL, EALIGN = coat.COAT_OK, coat.COAT_EINVAL, coat.COAT_EALIGN
BIG = (1 << 31)


def test_sizes():
    L = coat.lib()
    for k, codes, scales in ((0, 0, 0), (1, 64, 16), (128, 64, 16), (129, 128, 16), (512, 256, 16), (513, 320, 32), (5120, 2560, 160)):
        assert L.coat_mx4_code_bytes(k) == coat.mx4_code_bytes(k) == codes
        assert L.coat_mx4_scale_bytes(k) == coat.mx4_scale_bytes(k) == scales
    q, s = coat.mx4_empty(3, 700, device="cpu")
    assert q.shape == (3, 384) and s.shape == (3, 32)


def test_quantize_arguments():
    f = coat.lib().coat_mx4_quantize

    def call(x=FAKE, rows=4, cols=64, ld=64, dtype=0, q=FAKE, s=FAKE, qt=None, st=None):
        return f(x, rows, cols, ld, dtype, q, s, qt, st, None)

    assert call(rows=-1) == call(cols=-1) == call(ld=63) == call(dtype=2) == call(dtype=-1) == EINVAL
    assert call(rows=BIG) == call(cols=BIG, ld=BIG) == call(rows=BIG - 1, ld=1 << 62) == EINVAL
    assert call(x=None) == call(q=None) == call(s=None) == call(qt=FAKE) == call(st=FAKE) == EINVAL
    assert call(q=None, s=None) == EINVAL
    assert call(x=FAKE + 1) == call(x=FAKE + 2, dtype=1) == call(q=FAKE + 8) == call(s=FAKE + 4) == EALIGN
    assert call(qt=FAKE + 8, st=FAKE) == call(qt=FAKE, st=FAKE + 1) == EALIGN
    assert call(rows=0, x=None) == call(cols=0, x=None) == OK


def test_dequantize_arguments():
    f = coat.lib().coat_mx4_dequantize

    def call(q=FAKE, s=FAKE, rows=4, cols=64, x=FAKE, ld=64, dtype=0):
        return f(q, s, rows, cols, x, ld, dtype, None)

    assert call(rows=-1) == call(cols=BIG, ld=BIG) == call(ld=3) == call(dtype=7) == EINVAL
    assert call(q=None) == call(s=None) == call(x=None) == EINVAL
    assert call(q=FAKE + 1) == call(s=FAKE + 8) == call(x=FAKE + 1) == call(x=FAKE + 2, dtype=1) == EALIGN
    assert call(rows=0, q=None) == OK


def test_matmul_arguments():
    L = coat.lib()

    def call(aq=FAKE, as_=FAKE, m=4, bq=FAKE, bs=FAKE, n=8, k=64, y=FAKE, ld=8, dtype=0, ws=None, nb=0):
        return L.coat_mx4_matmul(aq, as_, m, bq, bs, n, k, y, ld, dtype, ws, nb, None)

    assert call(m=-1) == call(n=-1, ld=0) == call(k=-1) == call(k=BIG) == call(ld=7) == call(dtype=3) == EINVAL
    assert call(aq=None) == call(as_=None) == call(bq=None) == call(bs=None) == call(y=None) == EINVAL
    assert call(aq=FAKE + 8) == call(as_=FAKE + 1) == call(bq=FAKE + 4) == call(bs=FAKE + 2) == call(y=FAKE + 1) == EALIGN
    assert call(y=FAKE + 2, dtype=1) == EALIGN
    assert call(m=0, aq=None) == call(n=0, y=None) == OK


def border(**kw):
    a = dict(rows=4, cols=64, rpg=4, eps=1e-5, scale=1.0, post=1, st=0, pt=0, gt=0)
    a.update(kw)
    return coat._Border(a["rows"], a["cols"], a["rpg"], a["eps"], a["scale"], a["post"], a["st"], a["pt"], a["gt"])


BAD_BORDERS = [dict(rows=-1), dict(rows=BIG), dict(cols=0), dict(cols=16385), dict(rpg=0), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("inf")), dict(scale=float("nan")), dict(post=2),
               dict(st=2), dict(pt=-1), dict(gt=5)]


def test_block_norm_arguments():
    f = coat.lib().coat_block_norm

    def call(b=None, y=FAKE, r=FAKE, wp=FAKE, wq=FAKE, g=FAKE, ro=FAKE, h=FAKE, q=None, s=None, group=0, fmt=0, **kw):
        return f(ctypes.byref(b or border(**kw)), y, r, wp, wq, g, ro, h, q, s, group, fmt, None)

    for bad in BAD_BORDERS:
        assert call(**bad) == EINVAL, bad
    assert f(None, FAKE, FAKE, None, None, None, FAKE, FAKE, None, None, 0, 0, None) == EINVAL
    assert call(r=None) == call(q=FAKE) == call(s=FAKE) == EINVAL
    for group, fmt in ((0, 0), (24, 0), (8, 0), (1024, 0), (128, 0), (32, 3), (32, 0x100), (16, 2), (64, 2)):
        assert call(q=FAKE, s=FAKE, group=group, fmt=fmt) == EINVAL, (group, fmt)  # 128 does not divide 64
    assert call(y=None) == call(y=None, wp=None) == call(y=None, wp=None, g=None) == EINVAL
    assert call(y=None, wp=None, g=None, ro=None, post=1) == EINVAL
    assert call(post=0) == EINVAL                                    # w_post without the post-norm
    assert call(h=None) == EINVAL                                    # w_pre without a layer input
    assert call(h=None, wq=None, ro=None) == EINVAL                  # nothing to write
    assert call(y=FAKE + 1) == call(r=FAKE + 1) == call(wp=FAKE + 1) == call(ro=FAKE + 1) == call(h=FAKE + 1) == EALIGN
    assert call(r=FAKE + 2, st=1) == call(g=FAKE + 2, pt=1) == EALIGN
    assert call(q=FAKE + 8, s=FAKE, group=32) == call(q=FAKE, s=FAKE + 2, group=32) == EALIGN
    assert call(q=FAKE, s=FAKE + 8, group=32, fmt=2) == EALIGN
    assert call(rows=0, y=FAKE, r=None) == OK


def test_block_norm_backward_arguments():
    L = coat.lib()
    need = L.coat_block_norm_backward_workspace_bytes(ctypes.byref(border()))
    assert need > 0 and need % 256 == 0
    assert need == coat.block_norm_backward_workspace_bytes(4, 64)
    assert L.coat_block_norm_backward_workspace_bytes(ctypes.byref(border(cols=0))) == 0

    def call(y=FAKE, r=FAKE, do=FAKE, dh=FAKE, wp=FAKE, wq=FAKE, g=FAKE, dr=FAKE, dy=FAKE, dwp=FAKE, dwq=FAKE, dg=FAKE, ws=FAKE,
             nb=need, **kw):
        return L.coat_block_norm_backward(ctypes.byref(border(**kw)), y, r, do, dh, wp, wq, g, dr, dy, dwp, dwq, dg, ws, nb, None)

    for bad in BAD_BORDERS:
        assert call(**bad) == EINVAL, bad
    assert call(y=None) == call(post=0) == call(dh=None) == call(dr=None) == call(dy=None) == call(r=None) == EINVAL
    assert call(wp=None) == call(wq=None) == call(g=None) == EINVAL  # a gradient of what is not there
    assert call(do=None, dh=None, wq=None, dwq=None) == EINVAL       # no gradient comes in
    assert call(ws=None) == call(nb=need - 1) == EINVAL
    assert call(ws=FAKE + 64) == call(dy=FAKE + 1) == call(dh=FAKE + 1) == call(do=FAKE + 1) == EALIGN
    assert call(dr=FAKE + 2, st=1) == call(wq=FAKE + 2, pt=1) == call(dg=FAKE + 2, gt=1) == EALIGN


def test_backward_workspace_is_enough_for_every_split():
    """The same bytes whether a gate gradient is asked for or not; they grow with neither rows nor gates without limit."""
    most = 0
    for rows in (1, 2, 511, 512, 513, 1024, 5000, 16384, 1 << 20):
        for rpg in (1, 2, 3, 7, 100, rows // 2 + 1, rows):
            most = max(most, coat.block_norm_backward_workspace_bytes(rows, 64, rpg))
    assert 0 < most <= 3 * 2 * 1024 * 64 * 4


# ---------------------------------------------------------------- the binding (tensors without a GPU)

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = coat.mx4_empty(4, 64, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        coat.mx4_quantize(x, q, s)
    with pytest.raises(ValueError, match="GPU"):
        coat.mx4_dequantize(q, s, x)
    with pytest.raises(ValueError, match="GPU"):
        coat.mx4_matmul(q, s, q, s, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="GPU"):
        coat.block_norm(None, x, None, x.clone())
    with pytest.raises(ValueError, match="GPU"):
        coat.block_norm_backward(None, x, None, x, x.clone())


def test_binding_refuses_shapes_and_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.float32)
    with pytest.raises(ValueError, match="one type"):
        coat.block_norm(x, x, x, x, w_post=w, w_pre=w.bfloat16())
    with pytest.raises(ValueError, match="one type"):
        coat.block_norm_backward(x, x, x, x, x, x, dw_post=w, dw_pre=w.bfloat16())
    with pytest.raises(ValueError, match="pair"):
        coat.block_norm(None, x, None, x, q=torch.zeros(4, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="divide"):
        coat.block_norm(None, x, None, x, q=torch.zeros(4, 64, dtype=torch.uint8), q_scale=w, group=48)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        coat.block_norm(None, x.half(), None, x)
    with pytest.raises(ValueError, match="rows_per_gate"):
        coat.block_norm(None, x, None, x, rows_per_gate=0)
    with pytest.raises(ValueError, match="matrix"):
        coat.block_norm(None, x[0], None, x[0])


def test_block_norm_refuses_a_subnormal_eps():
    """The factor of a row of zeros would be infinite, and its values NaN."""
    L = coat.lib()
    for eps in (2.0 ** -149, 1e-40, 1e-38, 2.0 ** -126 * (1 - 2.0 ** -23)):
        b = border(eps=eps)
        assert 0.0 < b.eps < 2.0 ** -126
        assert L.coat_block_norm(ctypes.byref(b), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, 0, 0, None) == EINVAL
        assert L.coat_block_norm_backward_workspace_bytes(ctypes.byref(b)) == 0
        assert L.coat_block_norm_backward(ctypes.byref(b), *[FAKE] * 13, 1 << 30, None) == EINVAL
    assert L.coat_block_norm_backward_workspace_bytes(ctypes.byref(border(eps=2.0 ** -126))) > 0


def test_binding_numbers_past_the_c_types():
    """A count that ctypes would cut to its low bits describes other memory than the binding has checked."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for rpg in (5, 2 ** 63, 2 ** 64 + 1):
        b, _, gate_shape = coat._border(x, None, None, x, rpg, 1.0, 1e-5, False, 0)
        assert (b.rows_per_gate, gate_shape) == (4, (1, 64))
        assert coat.block_norm_backward_workspace_bytes(4, 64, rpg) == coat.block_norm_backward_workspace_bytes(4, 64, 4)
    b, _, gate_shape = coat._border(x[:0], None, None, None, 2 ** 64 + 1, 1.0, 1e-5, False, 0)
    assert (b.rows_per_gate, gate_shape) == (1, (0, 64))
    q, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2)
    for fmt in (2 ** 32 + coat.FMT_MX4, 2 ** 32, -1, 3):
        with pytest.raises(ValueError, match="fmt"):
            coat.block_norm(None, x, None, x, q=q, q_scale=s, group=32, fmt=fmt)
