"""bl_layer_norm and bl_layer_norm_backward on the GPU against the fp64
statements of tests/train_ref.py, with the bounds derived there: every type
pair, widths around each power of two and odd ones, one row to many, row
pitches, unaligned views, absent weights, rows far from zero, constant rows,
NaN and infinities, other streams, graphs."""
import numpy as np
import pytest
import torch

import train_ref as R
from parity import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)]


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


def _inputs(M, K, xt, gt, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, K, generator=g) * (0.5 + torch.rand(K, generator=g)) + offset).to(xt)
    w, b = 1 + 0.2 * torch.randn(K, generator=g), 0.3 * torch.randn(K, generator=g)
    dy = torch.randn(M, K, generator=g).to(gt)
    return x, w, b, dy


def _pitched(t, extra, device="cuda"):
    """t as the left columns of a wider buffer."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), 7.0, dtype=t.dtype, device=device)
    buf[:, :t.shape[1]] = t.to(device)
    return buf[:, :t.shape[1]], buf


def _forward(bl, x, w, b, yt, **kw):
    y, mean, rstd = bl.layer_norm(x.cuda(), None if w is None else w.cuda(), None if b is None else b.cuda(),
                                  out_dtype=yt, stats=True, **kw)
    return y, mean, rstd


def _check_forward(y, mean, rstd, x, w, b, yt, what, eps=1e-5):
    x64 = R.f64(x)
    w64, b64 = (None if t is None else R.f64(t) for t in (w, b))
    ry, rm, rr, z = R.layer_norm(x64, w64, b64, eps)
    R.check(y, ry, R.layer_norm_bound(ry, z, w64, b64, yt), what + " y")
    g = R.gamma(x.shape[1])
    # the mean is the kept rounding of a sum of x; rstd is off by gamma + 3 u
    R.check(mean, rm, g * np.abs(x64).mean(1) + R.U * np.abs(rm) + 1e-40, what + " mean")
    R.check(rstd, rr, (g + 4 * R.U) * rr, what + " rstd")


def _check_backward(got, x, w, dy, what, eps=1e-5):
    x64, g64 = R.f64(x), R.f64(dy)
    w64 = None if w is None else R.f64(w)
    ref = R.layer_norm_backward(x64, w64, g64, eps)
    bounds = R.layer_norm_backward_bounds(x64, w64, g64, x.dtype, eps)
    for t, r, bd, name in zip(got, ref, bounds, ("dx", "dweight", "dbias")):
        R.check(t, r, bd, f"{what} {name}")


WIDTHS = [1, 2, 3, 7, 8, 31, 32, 33, 64, 100, 128, 255, 256, 257, 384, 768, 1000, 1001, 1024, 1032, 2047, 2048, 2056,
          4096, 5001, 5632, 8184, 8192, 8200, 11008, 16384, 20000]


@pytest.mark.parametrize("K", WIDTHS)
def test_widths(bl, K):
    M = 5 if K > 2048 else 37
    x, w, b, dy = _inputs(M, K, BF16, BF16, seed=K)
    y, mean, rstd = _forward(bl, x, w, b, BF16)
    _check_forward(y, mean, rstd, x, w, b, BF16, f"K={K}")
    _check_backward(bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda()), x, w, dy, f"K={K}")


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("M,K", [(1, 4096), (3, 129), (70, 1024), (333, 777), (1300, 256), (9, 12000), (2500, 2048)])
def test_types(bl, M, K, xt, yt):
    x, w, b, dy = _inputs(M, K, xt, yt, seed=M + K)
    y, mean, rstd = _forward(bl, x, w, b, yt)
    _check_forward(y, mean, rstd, x, w, b, yt, f"{xt}->{yt}")
    assert y.dtype == yt
    got = bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda())
    assert got[0].dtype == xt
    _check_backward(got, x, w, dy, f"{xt}->{yt}")


@pytest.mark.parametrize("M", [1, 2, 5, 147, 148, 149, 295, 297, 593, 1185, 4099])
def test_row_counts(bl, M):
    for K in (96, 1536):
        x, w, b, dy = _inputs(M, K, BF16, BF16, seed=M)
        y, mean, rstd = _forward(bl, x, w, b, BF16)
        _check_forward(y, mean, rstd, x, w, b, BF16, f"M={M}")
        _check_backward(bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda()), x, w, dy, f"M={M}")


@pytest.mark.parametrize("K", [301, 640, 701, 766, 1001, 1501, 1530, 2050, 2304, 3500, 4999, 5000, 6000, 7001])
@pytest.mark.parametrize("M", [1, 7, 150, 450, 1333])
def test_tiles_of_every_height(bl, M, K):
    """Few rows to many: the tiles of the gradient take one row to eight, the last one fewer."""
    x, w, b, dy = _inputs(M, K, BF16, BF16, seed=M * K)
    y, mean, rstd = _forward(bl, x, w, b, BF16)
    _check_forward(y, mean, rstd, x, w, b, BF16, f"{M}x{K}")
    _check_backward(bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda()), x, w, dy, f"{M}x{K}")


@pytest.mark.parametrize("K", [256, 1000, 4096, 9000])
def test_absent_weight_and_bias(bl, K):
    x, w, b, dy = _inputs(19, K, F32, BF16, seed=K)
    for ww, bb in ((None, None), (w, None), (None, b)):
        y, mean, rstd = _forward(bl, x, ww, bb, BF16)
        _check_forward(y, mean, rstd, x, ww, bb, BF16, "absent")
        _check_backward(bl.layer_norm_backward(x.cuda(), None if ww is None else ww.cuda(), mean, rstd, dy.cuda()), x, ww,
                        dy, "absent")


@pytest.mark.parametrize("K,extra,shift", [(256, 8, 0), (256, 3, 0), (1000, 24, 0), (777, 1, 0), (1024, 7, 1), (4096, 16, 1),
                                           (5001, 7, 3), (2048, 128, 8), (9000, 8, 0)])
@pytest.mark.parametrize("xt,yt", TYPES)
def test_pitches_and_unaligned_views(bl, K, extra, shift, xt, yt):
    """x, y, dy and dx as column slices of wider buffers; what lies around them keeps its values."""
    M = 23
    x, w, b, dy = _inputs(M, K, xt, yt, seed=K + extra)
    wide = K + extra + shift

    def slot(t, dtype):
        buf = torch.full((M, wide), 7.0, dtype=dtype, device="cuda")
        view = buf[:, shift:shift + K]
        if t is not None:
            view.copy_(t)
        return view, buf

    xv, _ = slot(x, xt)
    yv, ybuf = slot(None, yt)
    y, mean, rstd = bl.layer_norm(xv, w.cuda(), b.cuda(), out=yv, stats=True)
    _check_forward(y, mean, rstd, x, w, b, yt, "pitch")
    dyv, _ = slot(dy, yt)
    dxv, dxbuf = slot(None, xt)
    got = bl.layer_norm_backward(xv, w.cuda(), mean, rstd, dyv, dx=dxv)
    _check_backward(got, x, w, dy, "pitch")
    for buf in (ybuf, dxbuf):
        assert bool((buf[:, :shift] == 7).all()) and bool((buf[:, shift + K:] == 7).all())


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("offset", [1e3, -3e4])
def test_rows_far_from_zero(bl, xt, offset):
    """The deviations are far below the mean: the bounds hold without a term for the mean's size."""
    for K in (200, 2048, 10000):
        x, w, b, dy = _inputs(11, K, xt, F32, seed=1, offset=offset)
        y, mean, rstd = _forward(bl, x, w, b, F32)
        _check_forward(y, mean, rstd, x, w, b, F32, "far")
        _check_backward(bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda()), x, w, dy, "far")


def test_constant_rows(bl):
    for K in (1, 100, 1024, 5000):
        x = torch.tensor([[0.0], [1.0], [-3.140625], [1e4]]).repeat(1, K).to(F32)
        w, b = torch.full((K,), 2.0), torch.full((K,), 0.5)
        y, mean, rstd = _forward(bl, x, w, b, F32)
        _check_forward(y, mean, rstd, x, w, b, F32, "constant")
        dy = torch.randn(4, K, generator=torch.Generator().manual_seed(3))
        _check_backward(bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda()), x, w, dy, "constant")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_row_stays_alone(bl, bad):
    for K in (96, 1024, 4096, 9000):
        x, w, b, dy = _inputs(40, K, F32, BF16, seed=2)
        good, gm, gr = _forward(bl, x, w, b, BF16)
        gdx = bl.layer_norm_backward(x.cuda(), w.cuda(), gm, gr, dy.cuda())[0]
        x[17, K // 3] = bad
        y, mean, rstd = _forward(bl, x, w, b, BF16)
        dx, dw, db = bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda())
        keep = torch.arange(40) != 17
        assert bool(torch.isnan(y[17].float()).all()) and bool(torch.isnan(rstd[17]))
        assert torch.equal(y[keep], good[keep]) and torch.equal(mean[keep.cuda()], gm[keep.cuda()])
        assert bool(torch.isnan(dx[17]).all()) and torch.equal(dx[keep], gdx[keep])
        assert bool(torch.isnan(dw).all()) and bool(torch.isfinite(db).all())


def test_in_place(bl):
    for M, K, t in ((37, 1000, BF16), (5, 4096, F32), (600, 512, BF16), (3, 20001, F32)):
        x, w, b, _ = _inputs(M, K, t, t, seed=4)
        ref = bl.layer_norm(x.cuda(), w.cuda(), b.cuda())
        y = x.cuda()
        assert bl.layer_norm(y, w.cuda(), b.cuda(), out=y) is y
        assert torch.equal(y, ref)


def test_parts_of_the_gradient(bl):
    for K in (512, 777, 9000):
        x, w, b, dy = (t.cuda() for t in _inputs(300, K, BF16, BF16, seed=5))
        _, mean, rstd = bl.layer_norm(x, w, b, stats=True)
        dx, dw, db = bl.layer_norm_backward(x, w, mean, rstd, dy)
        dx1, n1, n2 = bl.layer_norm_backward(x, w, mean, rstd, dy, want_dw=False)
        n3, dw1, db1 = bl.layer_norm_backward(x, w, mean, rstd, dy, want_dx=False)
        assert n1 is None and n2 is None and n3 is None
        assert torch.equal(dx, dx1) and torch.equal(dw, dw1) and torch.equal(db, db1)


def test_no_rows(bl):
    x = torch.empty((0, 300), dtype=BF16, device="cuda")
    w = torch.ones(300, device="cuda")
    y, mean, rstd = bl.layer_norm(x, w, None, stats=True)
    assert y.shape == (0, 300) and mean.numel() == 0
    dw, db = torch.full((300,), 7.0, device="cuda"), torch.full((300,), 7.0, device="cuda")
    bl.layer_norm_backward(x, w, mean, rstd, x, dweight=dw, dbias=db)
    assert not bool(dw.any()) and not bool(db.any())


def test_results_repeat_and_guards(bl):
    for M, K in ((701, 640), (64, 4096), (33, 9001)):
        x, w, b, dy = (t.cuda() for t in _inputs(M, K, BF16, BF16, seed=6))
        y, buf, s = guarded_empty((M, K), BF16, "cuda")
        mean, mbuf, ms = guarded_empty((M,), F32, "cuda")
        bl.layer_norm(x, w, b, out=y, stats=True, mean=mean)
        _, _, rstd = bl.layer_norm(x, w, b, stats=True)
        assert guards_intact(buf, M * K, sentinel=s) and guards_intact(mbuf, M, sentinel=ms)
        runs = []
        for _ in range(3):
            dx, dbuf, s = guarded_empty((M, K), BF16, "cuda")
            dw, wbuf, sw = guarded_empty((K,), F32, "cuda")
            db, bbuf, sb = guarded_empty((K,), F32, "cuda")
            bl.layer_norm_backward(x, w, mean, rstd, dy, dx=dx, dweight=dw, dbias=db)
            assert guards_intact(dbuf, M * K, sentinel=s) and guards_intact(wbuf, K, sentinel=sw)
            assert guards_intact(bbuf, K, sentinel=sb)
            runs.append((dx.clone(), dw.clone(), db.clone()))
        assert all(torch.equal(a, c) for r in runs[1:] for a, c in zip(runs[0], r))


def test_two_streams_at_once(bl):
    """Two backward passes on two streams, each with a workspace of its own."""
    cases = [tuple(t.cuda() for t in _inputs(900, K, BF16, BF16, seed=K)) for K in (1024, 1536)]
    stats = [bl.layer_norm(x, w, b, stats=True)[1:] for x, w, b, _ in cases]
    ref = [bl.layer_norm_backward(x, w, *st, dy) for (x, w, _, dy), st in zip(cases, stats)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i, ((x, w, _, dy), st) in enumerate(zip(cases, stats)):
            with torch.cuda.stream(streams[i]):
                got[i].append(bl.layer_norm_backward(x, w, *st, dy))
    torch.cuda.synchronize()
    for r, runs in zip(ref, got):
        for g in runs:
            assert all(torch.equal(a, c) for a, c in zip(r, g))


def test_captured(bl):
    x, w, b, dy = (t.cuda() for t in _inputs(513, 2048, BF16, BF16, seed=8))
    ws = torch.empty(bl.workspace_bytes(bl.BL_OP_LAYER_NORM_BACKWARD, 513, 0, 2048), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(x), torch.empty(513, device="cuda"), torch.empty(513, device="cuda"), torch.empty_like(x),
           torch.empty(2048, device="cuda"), torch.empty(2048, device="cuda")]

    def step():
        bl.layer_norm(x, w, b, out=out[0], stats=True, mean=out[1], rstd=out[2])
        bl.layer_norm_backward(x, w, out[1], out[2], dy, dx=out[3], dweight=out[4], dbias=out[5], ws=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(_inputs(513, 2048, BF16, BF16, seed=9)[0])
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, out))


def test_gradient_against_differences(bl):
    """dx and dweight against central differences of the fp64 forward pass."""
    M, K = 3, 24
    x, w, b, dy = _inputs(M, K, F32, F32, seed=10)
    _, mean, rstd = _forward(bl, x, w, b, F32)
    dx, dw, db = (R.f64(t) for t in bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda()))
    x64, w64, b64, g64 = (R.f64(t) for t in (x, w, b, dy))
    bx, bw, bb = R.layer_norm_backward_bounds(x64, w64, g64, F32)

    def loss(x, w, b):
        return float((R.layer_norm(x, w, b)[0] * g64).sum())

    h = 1e-4  # the quotient's own error stays below 1e-6 (h^2 times a third derivative of at most 100)
    for i in range(M):
        for k in range(K):
            e = np.zeros((M, K))
            e[i, k] = h
            assert abs((loss(x64 + e, w64, b64) - loss(x64 - e, w64, b64)) / (2 * h) - dx[i, k]) < bx[i, k] + 1e-6
    for k in range(K):
        e = np.zeros(K)
        e[k] = h
        assert abs((loss(x64, w64 + e, b64) - loss(x64, w64 - e, b64)) / (2 * h) - dw[k]) < bw[k] + 1e-6
        assert abs((loss(x64, w64, b64 + e) - loss(x64, w64, b64 - e)) / (2 * h) - db[k]) < bb[k] + 1e-6


def test_refusals(bl):
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    s = torch.zeros(4, device="cuda")
    bad = [lambda: bl.layer_norm(x.half()), lambda: bl.layer_norm(x[0]), lambda: bl.layer_norm(x.t()),
           lambda: bl.layer_norm(x, w[:32]), lambda: bl.layer_norm(x, w.to(BF16)), lambda: bl.layer_norm(x, w.cpu()),
           lambda: bl.layer_norm(x, w, out=x[:2]), lambda: bl.layer_norm(x, w, out=x, out_dtype=F32),
           lambda: bl.layer_norm_backward(x, w, s[:2], s, x), lambda: bl.layer_norm_backward(x, w, s, s, x[:, :32]),
           lambda: bl.layer_norm_backward(x, w, s, s, x, dx=x.float())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bl.layer_norm(x, w, eps=0.0), lambda: bl.layer_norm_backward(x, w, s, s, x, dx=x)):
        with pytest.raises(bl.BitLinearError):
            call()


@pytest.mark.parametrize("K", [100, 512, 1001, 4096, 13056, 20000])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_mean_near_zero(bl, K, xt):
    """Eighths between -4 and 4: their sums are exact in any order, so the kept mean is off by the roundings of 1 / K
    and of the product alone, however coarse the values are."""
    x = (torch.randint(-32, 33, (37, K), generator=torch.Generator().manual_seed(K)) / 8.0).to(xt)
    mean = bl.layer_norm(x.cuda(), stats=True)[1]
    ref = R.f64(x).mean(1)
    assert (ref ** 2 < R.f64(x).var(1)).all()
    R.check(mean, ref, 2.01 * R.U * np.abs(ref), "mean")


@pytest.mark.parametrize("M,K", [(1, 8200), (5, 8194), (70, 8193), (300, 8448), (33, 16400)])
@pytest.mark.parametrize("xt,gt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_long_rows(bl, M, K, xt, gt):
    """The gradient in two readings: accesses of every size, fewer rows than a CTA has warps and more."""
    x, w, b, dy = _inputs(M, K, xt, gt, M + K)
    y, mean, rstd = _forward(bl, x, w, b, gt)
    _check_forward(y, mean, rstd, x, w, b, gt, f"{M}x{K}")
    _check_backward(bl.layer_norm_backward(x.cuda(), w.cuda(), mean, rstd, dy.cuda()), x, w, dy, f"{M}x{K}")
