"""Layer norm and its gradient of rows in such numbers that every slot of a warp's (CTA's) ring of staged rows is
filled again several times, against the fp64 formulas on the device. The bounds are those of tests/train_ref.py."""
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U, EPS = R.U, 1e-5


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


def _inside(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


# 60013 rows: a warp takes six or more even with eight CTAs of eight warps on each of 148 SMs, and the ring has three
# or four slots. 1030 columns: the gradient's tiles, whose CTAs come round as often. From 8192 columns on: one row per
# CTA at a time, and 32 columns per thread read one by one.
@pytest.mark.parametrize("K", [64, 250, 301, 511, 512, 1030, 8193, 11008, 16383])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_many_rows(bl, K, xt, yt):
    M = 60013 if K < 1000 else 15013 if K < 8000 else 1013
    g = torch.Generator("cuda").manual_seed(K)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = (randn(M, K) * (1.0 + randn(K).abs()) + randn(M, 1)).to(xt)
    w, b, dy = 1.0 + 0.1 * randn(K), 0.1 * randn(K), randn(M, K).to(yt)
    y, mean, rstd = bl.layer_norm(x, w, b, eps=EPS, out_dtype=yt, stats=True)
    dx, dw, db = bl.layer_norm_backward(x, w, mean, rstd, dy)

    x64, g64, w64 = x.double(), dy.double(), w.double()
    mu = x64.mean(1, keepdim=True)
    d = x64 - mu
    r64 = ((d * d).mean(1, keepdim=True) + EPS).rsqrt()
    z = d * r64
    gk, gr = R.gamma(K), R.gamma_rows(M)
    tz = (gk + 6 * U) * (1 + z.abs())
    ref = z * w64 + b.double()
    t = (tz + 2 * U * z.abs()) * w64.abs() + U * (b.double().abs() + ref.abs())
    _inside(y, ref, t + R.half_step(yt) * (ref.abs() + t) + 2.0 ** -140, "y")
    # the mean: the sum's roundings, or with the correction fewer, and the kept value's own; rstd as derived there
    _inside(mean, mu[:, 0], (gk + 2 * U) * x64.abs().mean(1) + U * mu[:, 0].abs(), "mean")
    _inside(rstd, r64[:, 0], (gk + 4 * U) * r64[:, 0], "rstd")

    gw = g64 * w64
    mg, mgz = gw.mean(1, keepdim=True), (gw * z).mean(1, keepdim=True)
    ref = r64 * (gw - mg - z * mgz)
    amg, amgz = gw.abs().mean(1, keepdim=True), (gw * z).abs().mean(1, keepdim=True)
    t_mgz = (gk + 3 * U) * amgz + (gw.abs() * tz).mean(1, keepdim=True)
    t = ((gk + 3 * U) * amg + z.abs() * t_mgz + tz * (amgz + t_mgz) + 4 * U * (gw.abs() + amg + z.abs() * amgz))
    t = r64 * t + (gk + 4 * U) * ref.abs()
    _inside(dx, ref, t + R.half_step(xt) * (ref.abs() + t) + 2.0 ** -140, "dx")
    ref = (g64 * z).sum(0)
    t = (g64.abs() * tz).sum(0) + (gr + 2 * U) * (g64.abs() * (z.abs() + tz)).sum(0)
    _inside(dw, ref, t + U * ref.abs(), "dweight")
    _inside(db, g64.sum(0), (gr + U) * g64.abs().sum(0), "dbias")
