"""The full-precision operators' argument checks without a GPU: every case
below is refused (or a no-op) on the host, before any pointer is used."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)
FAKE2 = ctypes.c_void_p(0x8000000)
ODD = ctypes.c_void_p(0x10001)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def bl():
    import bit_linear_layers_b200 as m
    return m


def _ln(bl, x=FAKE, xt=1, ldx=None, w=FAKE, b=FAKE, y=FAKE2, yt=0, ldy=None, M=4, K=100, eps=1e-5):
    return bl.lib.bl_layer_norm(x, xt, K if ldx is None else ldx, w, b, y, yt, K if ldy is None else ldy, None, None,
                                M, K, eps, None)


def test_layer_norm_refusals(bl):
    assert _ln(bl, M=-1) == -1 and _ln(bl, K=0) == -1
    assert _ln(bl, M=1 << 31) == -2 and _ln(bl, K=1 << 31) == -2
    assert _ln(bl, M=(1 << 31) - 1, K=1 << 12) == -2      # 2^43 elements
    assert _ln(bl, ldx=99) == -1 and _ln(bl, ldy=99) == -1
    assert _ln(bl, ldx=1 << 50) == -2
    assert _ln(bl, xt=2) == -1 and _ln(bl, yt=-1) == -1
    for eps in (0.0, -1e-5, INF, NAN):
        assert _ln(bl, eps=eps) == -1
    assert _ln(bl, x=None) == -1 and _ln(bl, y=None) == -1
    assert _ln(bl, x=ODD) == -1 and _ln(bl, y=ODD) == -1 and _ln(bl, w=ODD) == -1 and _ln(bl, b=ODD) == -1
    assert _ln(bl, y=FAKE) == -1                            # in place, but of another type
    assert _ln(bl, y=FAKE, yt=1, ldy=128) == -1             # ... and of another pitch
    assert _ln(bl, M=0, x=None, y=None) == 0
    assert _ln(bl) == bl.BL_ERR_NO_DEVICE                   # valid: stops only at the device


def _lnb(bl, x=FAKE, xt=0, ldx=None, w=FAKE, mean=FAKE, rstd=FAKE, dy=FAKE, gt=0, lddy=None, dx=FAKE2, lddx=None,
         dw=FAKE2, db=FAKE, M=4, K=100, ws=FAKE, ws_bytes=1 << 30):
    return bl.lib.bl_layer_norm_backward(x, xt, K if ldx is None else ldx, w, mean, rstd, dy, gt,
                                         K if lddy is None else lddy, dx, K if lddx is None else lddx, dw, db, M, K, ws,
                                         ws_bytes, None)


def test_layer_norm_backward_refusals(bl):
    assert _lnb(bl, M=-1) == -1 and _lnb(bl, K=0) == -1 and _lnb(bl, xt=3) == -1 and _lnb(bl, gt=3) == -1
    assert _lnb(bl, ldx=99) == -1 and _lnb(bl, lddy=99) == -1 and _lnb(bl, lddx=99) == -1
    assert _lnb(bl, x=None) == -1 and _lnb(bl, dy=None) == -1 and _lnb(bl, mean=None) == -1 and _lnb(bl, rstd=None) == -1
    assert _lnb(bl, x=ODD) == -1 and _lnb(bl, dx=ODD) == -1 and _lnb(bl, dw=ODD) == -1 and _lnb(bl, mean=ODD) == -1
    assert _lnb(bl, dx=FAKE) == -1                          # dx over x
    assert _lnb(bl, dw=FAKE, db=FAKE) == -1                 # one buffer for both gradients
    need = bl.workspace_bytes(bl.BL_OP_LAYER_NORM_BACKWARD, 4, 0, 100)
    assert need > 0 and need % 256 == 0
    assert _lnb(bl, ws_bytes=need - 1) == -1 and _lnb(bl, ws=None) == -1
    assert _lnb(bl, ws_bytes=need) == bl.BL_ERR_NO_DEVICE
    assert _lnb(bl, dw=None, db=None, ws=None, ws_bytes=0) == bl.BL_ERR_NO_DEVICE  # dx alone needs none
    assert _lnb(bl, dx=None, dw=None, db=None, ws=None, ws_bytes=0) == 0           # nothing asked for
    assert _lnb(bl, M=0, x=None, dy=None, mean=None, rstd=None, dw=None, db=None, ws=None) == 0
    assert bl.workspace_bytes(bl.BL_OP_LAYER_NORM_BACKWARD, 0, 0, 100) == 0


def _emb(bl, ids=FAKE, it=1, table=FAKE, tt=0, y=FAKE2, yt=0, T=4, V=10, D=8):
    return bl.lib.bl_embedding(ids, it, table, tt, y, yt, T, V, D, 1.0, None)


def test_embedding_refusals(bl):
    assert _emb(bl, T=-1) == -1 and _emb(bl, V=0) == -1 and _emb(bl, D=0) == -1
    assert _emb(bl, T=1 << 31) == -2 and _emb(bl, V=1 << 31) == -2 and _emb(bl, V=1 << 30, D=1 << 10) == -2
    assert _emb(bl, it=2) == -1 and _emb(bl, tt=2) == -1 and _emb(bl, yt=2) == -1
    assert _emb(bl, ids=None) == -1 and _emb(bl, table=None) == -1 and _emb(bl, y=None) == -1
    assert _emb(bl, ids=ctypes.c_void_p(0x10004)) == -1    # 64-bit ids on a 4-byte boundary
    assert _emb(bl, it=0, ids=ctypes.c_void_p(0x10004)) == bl.BL_ERR_NO_DEVICE
    assert _emb(bl, y=ODD) == -1 and _emb(bl, table=ODD) == -1
    assert _emb(bl, T=0, ids=None, y=None) == 0


def _embb(bl, ids=FAKE, it=1, dy=FAKE, gt=0, d=FAKE2, tt=1, T=4, V=10, D=8, pad=-1, flags=0, ws=FAKE, ws_bytes=1 << 30):
    return bl.lib.bl_embedding_backward(ids, it, dy, gt, d, tt, T, V, D, 1.0, pad, flags, ws, ws_bytes, None)


def test_embedding_backward_refusals(bl):
    assert _embb(bl, T=-1) == -1 and _embb(bl, V=0) == -1 and _embb(bl, D=0) == -1
    assert _embb(bl, pad=10) == -1 and _embb(bl, flags=2) == -1
    assert _embb(bl, T=1 << 31) == -2 and _embb(bl, V=1 << 31) == -2 and _embb(bl, T=1 << 30, D=1 << 10) == -2
    assert _embb(bl, it=5) == -1 and _embb(bl, gt=5) == -1 and _embb(bl, tt=5) == -1
    assert _embb(bl, ids=None) == -1 and _embb(bl, dy=None) == -1 and _embb(bl, d=None) == -1
    assert _embb(bl, d=ODD) == -1 and _embb(bl, dy=ODD) == -1
    need = bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, 4, 10, 8)
    assert need > 0 and need % 256 == 0
    assert _embb(bl, ws_bytes=need - 1) == -1 and _embb(bl, ws=None) == -1
    for pad in (-1, -100, 0, 9):
        assert _embb(bl, pad=pad, ws_bytes=need) == bl.BL_ERR_NO_DEVICE
    assert _embb(bl, T=0, ids=None, dy=None, flags=1, ws=None) == 0
    assert bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, 0, 10, 8) == 0


def _clip(bl, rows, max_norm=1.0, stats=FAKE2, ws=FAKE, ws_bytes=1 << 20):
    t = (bl.GradTensor * max(len(rows), 1))(*rows)
    return bl.lib.bl_grad_clip(ctypes.byref(t), len(rows), max_norm, stats, ws, ws_bytes, None)


def test_grad_clip_refusals(bl):
    A, B = 0x100000, 0x200000
    ok = bl.BL_ERR_NO_DEVICE
    assert _clip(bl, [(A, A, 16, 1)]) == ok and _clip(bl, [(A, B, 16, 1)]) == ok and _clip(bl, [(A, None, 16, 1)]) == ok
    for m in (-1.0, NAN):
        assert _clip(bl, [(A, A, 16, 1)], max_norm=m) == -1
    assert _clip(bl, [(A, A, 16, 1)], max_norm=0.0) == ok and _clip(bl, [(A, A, 16, 1)], max_norm=INF) == ok
    assert _clip(bl, [(A, A, 16, 2)]) == -1 and _clip(bl, [(A, A, -1, 1)]) == -1 and _clip(bl, [(None, A, 4, 1)]) == -1
    assert _clip(bl, [(A + 2, A + 2, 16, 1)]) == -1 and _clip(bl, [(A + 2, A + 2, 16, 0)]) == ok
    assert _clip(bl, [(A, B + 1, 16, 0)]) == -1
    assert _clip(bl, [(A, A, 1 << 40, 1)]) == -2 and _clip(bl, [(A, None, 1 << 39, 1)] * 2) == -2
    assert _clip(bl, [(None, None, 0, 1), (A, A, 16, 1)]) == ok       # an empty tensor has no address
    # one tensor listed twice: scaled twice in place, or read while it is written
    assert _clip(bl, [(A, A, 16, 1), (A, A, 16, 1)]) == -1
    assert _clip(bl, [(A, A, 16, 1), (A, None, 16, 1)]) == -1
    assert _clip(bl, [(A, None, 16, 1), (A, None, 16, 1)]) == ok
    # an output over part of its own gradient, of another gradient, of another output
    assert _clip(bl, [(A, A + 16, 16, 1)]) == -1
    assert _clip(bl, [(A, B, 16, 1), (B + 60, None, 16, 1)]) == -1
    assert _clip(bl, [(A, B, 16, 1), (B + 64, None, 16, 1)]) == ok
    assert _clip(bl, [(A, B, 16, 1), (A + 64, B + 32, 16, 1)]) == -1
    assert _clip(bl, [(A, B, 16, 1)], stats=None) == -1 and _clip(bl, [(A, B, 16, 1)], ws=None) == -1
    need = bl.workspace_bytes(bl.BL_OP_GRAD_CLIP, 1, 0, 0)
    assert need > 0 and _clip(bl, [(A, B, 16, 1)], ws_bytes=need - 1) == -1
    assert bl.workspace_bytes(bl.BL_OP_GRAD_CLIP, 5000, 0, 0) > need


def test_the_binding_refuses_on_the_host(bl):
    import torch
    x = torch.zeros(2, 4)
    with pytest.raises(ValueError):
        bl.layer_norm(x)
    with pytest.raises(ValueError):
        bl.embedding(torch.zeros(2, dtype=torch.int64), x)
    with pytest.raises(ValueError):
        bl.embedding_backward(torch.zeros(2, dtype=torch.int64), x, 3)
    with pytest.raises(ValueError):
        bl.layer_norm_backward(x, None, x[:, 0], x[:, 0], x)
    with pytest.raises(ValueError):
        bl.grad_clip([], 1.0)
    with pytest.raises(ValueError):
        bl.grad_clip([x], 1.0)
