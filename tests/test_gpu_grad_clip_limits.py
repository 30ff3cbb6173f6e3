"""bl_grad_clip where the largest norm is infinite (the norm is wanted, nothing is to be scaled): gradients that
hold an infinity keep their values, a NaN still shows."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("count", [2, 1000])  # one launch of each kernel, and two
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
def test_infinite_largest_norm_and_an_infinity(bl, dtype, count, bad):
    src = [torch.randn(33 + i % 7, generator=torch.Generator().manual_seed(i)).to(dtype).cuda() for i in range(count)]
    src[1][5] = bad
    ts, outs = [t.clone() for t in src], [torch.full_like(t, 7.0) for t in src]
    for out in (None, outs):
        n, c = bl.grad_clip(ts, float("inf"), out=out)
        assert torch.isinf(n) and float(n) > 0 and float(c) == 1.0
        assert all(torch.equal(a, b) for a, b in zip(src, ts if out is None else out))
    stats = torch.empty(2, device="cuda")
    assert torch.isinf(bl.grad_norm(ts, stats=stats)) and float(stats[1]) == 1.0


@pytest.mark.parametrize("max_norm", [0.0, 1.0, float("inf")])
def test_nan_beside_an_infinity(bl, max_norm):
    ts = [torch.randn(100, device="cuda"), torch.randn(9, device="cuda")]
    ts[0][3], ts[1][2] = float("inf"), float("nan")
    n, c = bl.grad_clip(ts, max_norm)
    assert torch.isnan(n) and torch.isnan(c) and all(bool(torch.isnan(t).all()) for t in ts)


@pytest.mark.parametrize("max_norm", [0.0, 1.0, 3e38])
def test_finite_largest_norm_and_an_infinity(bl, max_norm):
    ts = [torch.randn(100, device="cuda")]
    ts[0][3] = float("inf")
    n, c = bl.grad_clip(ts, max_norm)
    assert torch.isinf(n) and float(c) == 0.0 and int(torch.count_nonzero(ts[0])) == 1 and bool(torch.isnan(ts[0][3]))
