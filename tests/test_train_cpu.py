"""Refusals of the training products, before any device work (CPU only): through the C ABI
with addresses that are never read, and in the Python binding."""
import ctypes

import pytest
import torch

import _train64 as ref
import fp8_optimizer_state_amd as coat

FAKE = 0x7F0000000000
OK, EINVAL, EALIGN = coat.COAT_OK, coat.COAT_EINVAL, coat.COAT_EALIGN
BIG = 1 << 31
BIG_WS = 1 << 40
BF16 = torch.bfloat16


def epilogue(act=0, scale=1.0, p=0.0, offset=0, rng=None):
    return coat._Epilogue(act, scale, p, offset, rng)


BAD_EPILOGUES = [dict(act=-1), dict(act=5), dict(scale=float("nan")), dict(scale=float("inf")), dict(p=-0.1), dict(p=1.0),
                 dict(p=float("nan")), dict(p=0.5), dict(p=0.5, rng=FAKE, scale=3e38)]  # no random numbers; a factor past fp32


def test_constants_and_reference():
    assert (coat.ACT_NONE, coat.ACT_RELU, coat.ACT_GELU, coat.ACT_GELU_TANH, coat.ACT_SILU) == (0, 1, 2, 3, 4)
    assert list(ref.ACTS.values()) == [0, 1, 2, 3, 4]
    # the published generator's vectors
    assert ref.philox_words(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def test_linear_arguments():
    f = coat.lib().coat_linear

    def call(x=FAKE, m=4, k=16, ldx=16, w=FAKE, n=8, ldw=16, e=None, bias=None, bt=0, r=None, ldr=8, z=None, ldz=8, y=FAKE, ldy=8, yt=0,
             ws=FAKE, nb=BIG_WS, **kw):
        return f(x, m, k, ldx, w, n, ldw, ctypes.byref(e or epilogue(**kw)), bias, bt, r, ldr, z, ldz, y, ldy, yt, ws, nb, None)

    for bad in BAD_EPILOGUES:
        assert call(**bad) == EINVAL, bad
    assert f(FAKE, 4, 16, 16, FAKE, 8, 16, None, None, 0, None, 8, None, 8, FAKE, 8, 0, FAKE, BIG_WS, None) == EINVAL
    assert call(m=-1) == call(n=-1) == call(k=-1) == call(m=BIG) == call(n=BIG, ldy=BIG) == call(k=BIG, ldx=BIG, ldw=BIG) == EINVAL
    assert call(ldx=15) == call(ldw=15) == call(ldy=7) == call(z=FAKE, ldz=7) == call(r=FAKE, ldr=7) == call(m=BIG - 1, ldx=1 << 62) == EINVAL
    assert call(x=None) == call(w=None) == call(y=None) == call(bt=2) == call(yt=2) == EINVAL
    assert call(x=FAKE + 1) == call(w=FAKE + 1) == call(y=FAKE + 1) == call(z=FAKE + 1) == call(r=FAKE + 1) == call(bias=FAKE + 1) == EALIGN
    assert call(y=FAKE + 2, yt=1) == call(bias=FAKE + 2, bt=1) == call(p=0.5, rng=FAKE + 4) == EALIGN
    assert call(m=0, x=None, y=None) == call(n=0, w=None, y=None) == OK
    need = coat.linear_workspace_bytes(100, 8, 12, False)
    assert need > 0
    assert call(m=100, k=12, ws=None) == call(m=100, k=12, nb=need - 1) == EINVAL and call(m=100, k=12, ws=FAKE + 128) == EALIGN


def test_linear_backward_arguments():
    f = coat.lib().coat_linear_backward

    def call(dy=FAKE, lddy=8, dyt=0, x=FAKE, m=4, k=16, ldx=16, w=FAKE, n=8, ldw=16, e=None, z=None, ldz=8, dx=FAKE, lddx=16, dw=FAKE,
             lddw=16, db=FAKE, dbt=0, ws=FAKE, nb=BIG_WS, **kw):
        return f(dy, lddy, dyt, x, m, k, ldx, w, n, ldw, ctypes.byref(e or epilogue(**kw)), z, ldz, dx, lddx, dw, lddw, db, dbt, ws, nb, None)

    for bad in BAD_EPILOGUES:
        assert call(**bad) == EINVAL, bad
    assert call(m=-1) == call(n=BIG, lddy=BIG) == call(k=BIG, ldx=BIG, ldw=BIG, lddx=BIG, lddw=BIG) == EINVAL
    assert call(dy=None) == call(x=None) == call(w=None) == call(dx=None, dw=None, db=None) == call(dyt=3) == call(dbt=-1) == EINVAL
    assert call(act=2) == EINVAL                                           # an activation without z
    assert call(lddy=7) == call(ldx=15) == call(ldw=15) == call(lddx=15) == call(lddw=15) == call(z=FAKE, ldz=7) == EINVAL
    assert call(dy=FAKE + 1) == call(dy=FAKE + 2, dyt=1) == call(x=FAKE + 1) == call(w=FAKE + 1) == call(z=FAKE + 1) == EALIGN
    assert call(dx=FAKE + 1) == call(dw=FAKE + 1) == call(db=FAKE + 1) == call(db=FAKE + 2, dbt=1) == call(ws=FAKE + 64) == EALIGN
    need = coat.linear_backward_workspace_bytes(4, 8, 16)
    assert need > 0 and call(ws=None) == call(nb=need - 1) == EINVAL


def test_dropout_arguments():
    f = coat.lib().coat_dropout

    def call(x=FAKE, rows=4, cols=8, ldx=8, xt=0, r=None, ldr=8, scale=1.0, p=0.5, rng=FAKE, offset=0, y=FAKE, ldy=8, yt=0):
        return f(x, rows, cols, ldx, xt, r, ldr, scale, p, rng, offset, y, ldy, yt, None)

    assert call(rows=-1) == call(cols=BIG, ldx=BIG, ldy=BIG) == call(ldx=7) == call(ldy=7) == call(r=FAKE, ldr=7) == EINVAL
    assert call(x=None) == call(y=None) == call(rng=None) == call(xt=2) == call(yt=-1) == EINVAL
    assert call(p=1.0) == call(p=-1.0) == call(p=float("nan")) == call(scale=float("inf")) == call(scale=3e38) == EINVAL
    assert call(x=FAKE + 1) == call(x=FAKE + 2, xt=1) == call(y=FAKE + 1) == call(r=FAKE + 1) == call(rng=FAKE + 4) == EALIGN
    assert call(rows=0, x=None, y=None) == call(cols=0, x=None, y=None) == OK


def test_cross_entropy_arguments():
    f = coat.lib().coat_linear_cross_entropy

    def call(x=FAKE, t=4, k=16, ldx=16, w=FAKE, v=8, ldw=16, labels=FAKE, loss=FAKE, lse=FAKE, ws=FAKE, nb=BIG_WS):
        return f(x, t, k, ldx, w, v, ldw, labels, -100, loss, lse, ws, nb, None)

    assert call(t=-1) == call(t=BIG) == call(v=0) == call(v=BIG) == call(k=-1) == call(ldx=15) == call(ldw=15) == EINVAL
    assert call(x=None) == call(w=None) == call(labels=None) == call(loss=None) == call(lse=None) == EINVAL
    assert call(x=FAKE + 1) == call(w=FAKE + 1) == call(labels=FAKE + 4) == call(loss=FAKE + 2) == call(lse=FAKE + 2) == EALIGN
    need = coat.linear_cross_entropy_workspace_bytes(4, 8, 16)
    assert need > 0 and call(ws=None) == call(nb=need - 1) == EINVAL and call(ws=FAKE + 8) == EALIGN
    assert call(t=0, x=None, labels=None, loss=None, lse=None) == OK


def test_cross_entropy_backward_arguments():
    f = coat.lib().coat_linear_cross_entropy_backward

    def call(x=FAKE, t=4, k=16, ldx=16, w=FAKE, v=8, ldw=16, labels=FAKE, lse=FAKE, dl=FAKE, count=4, dx=FAKE, lddx=16, dw=FAKE, lddw=16,
             ws=FAKE, nb=BIG_WS):
        return f(x, t, k, ldx, w, v, ldw, labels, -100, lse, dl, count, dx, lddx, dw, lddw, ws, nb, None)

    assert call(t=-1, count=-1) == call(v=0) == call(ldx=15) == call(lddx=15) == call(lddw=15) == call(count=3) == call(count=0) == EINVAL
    assert call(x=None) == call(w=None) == call(labels=None) == call(lse=None) == call(dl=None) == call(dx=None, dw=None) == EINVAL
    assert call(dl=FAKE + 2) == call(dx=FAKE + 1) == call(dw=FAKE + 1) == call(lse=FAKE + 1) == call(ws=FAKE + 8) == EALIGN
    need = coat.linear_cross_entropy_backward_workspace_bytes(4, 8, 16)
    assert need > 0 and call(ws=None) == call(nb=need - 1) == EINVAL


def test_cross_entropy_backward_from_the_loss():
    f = coat.lib().coat_linear_cross_entropy_backward_loss

    def call(x=FAKE, t=4, lse=FAKE, loss=FAKE, dl=FAKE, ws=FAKE, nb=BIG_WS):
        return f(x, t, 16, 16, FAKE, 8, 16, FAKE, -100, lse, loss, dl, t, FAKE, 16, FAKE, 16, ws, nb, None)

    assert call(loss=FAKE + 2) == EALIGN and call(loss=FAKE + 2, lse=None) == call(loss=FAKE + 2, t=-1) == EINVAL
    need = coat.linear_cross_entropy_backward_workspace_bytes(4, 8, 16)
    assert call(nb=need - 1) == call(loss=None, nb=need - 1) == call(ws=None) == EINVAL


def test_workspaces():
    L = coat.lib()
    for name in ("coat_linear", "coat_linear_backward", "coat_linear_cross_entropy", "coat_linear_cross_entropy_backward"):
        f = getattr(L, name + "_workspace_bytes")
        for size in ((1, 1, 1), (1, 50257, 768), (1023, 50257, 768), (333, 5120, 13824), (16384, 13824, 5120), (70000, 4100, 24)):
            a, b = f(*size, 1), f(*size, 0)
            assert 0 <= a <= b and a % 256 == 0 and b % 256 == 0
        assert f(BIG, 8, 8, 1) == f(8, BIG, 8, 1) == f(8, 8, BIG, 1) == f(-1, 8, 8, 1) == 0
    # the loss's workspaces are far from the logits
    tokens, vocab, cols = 16384, 128256, 4096
    assert coat.linear_cross_entropy_workspace_bytes(tokens, vocab, cols) < tokens * vocab / 6
    assert coat.linear_cross_entropy_backward_workspace_bytes(tokens, vocab, cols) < tokens * vocab


# ---------------------------------------------------------------- the binding (tensors without a GPU)

def test_binding_refuses_cpu_tensors():
    x, w, y = torch.zeros(4, 16, dtype=BF16), torch.zeros(8, 16, dtype=BF16), torch.zeros(4, 8, dtype=BF16)
    labels, loss = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    for call in (lambda: coat.linear(x, w, y), lambda: coat.linear_backward(y, x, w, x.clone()), lambda: coat.dropout(x, x, p=0.0),
                 lambda: coat.dropout_backward(x, x, p=0.0), lambda: coat.linear_cross_entropy(x, w, labels, loss, loss),
                 lambda: coat.linear_cross_entropy_backward(x, w, labels, loss, loss, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_binding_refuses_random_numbers_that_are_not_there():
    for p in (-0.1, 1.0, 1.5, float("nan")):
        with pytest.raises(ValueError, match="p must be"):
            coat._random(p, None, 0, 0)
    with pytest.raises(ValueError, match="rng"):
        coat._random(0.5, None, 0, 0)
    with pytest.raises(ValueError, match="offset"):
        coat._random(0.0, None, 2 ** 63, 0)
    assert coat._random(0.0, None, 0, 0) is None
    for act in (-1, 5, 2 ** 32):
        with pytest.raises(ValueError, match="act"):
            coat._epilogue(act, 1.0, 0.0, None, 0, 0)
    with pytest.raises(ValueError, match="ignore_index"):
        coat._index64(-2 ** 63 - 1)


def test_binding_refuses_shapes():
    with pytest.raises(ValueError, match="matrix"):
        coat.linear(torch.zeros(16, dtype=BF16), torch.zeros(8, 16, dtype=BF16), torch.zeros(1, 8))
    with pytest.raises(ValueError, match="rows without gaps"):
        coat._row_stride(torch.zeros(4, 16)[:, ::2], "x")
    with pytest.raises(ValueError, match="rows without gaps"):
        coat._row_stride(torch.zeros(1, 16).expand(4, 16), "x")
