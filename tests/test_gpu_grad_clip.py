"""bl_grad_clip on the GPU against its definition in fp64, with the bounds of
tests/train_ref.py: one element to millions, many tensors (more than one
launch holds), unaligned views, both types, in place and into other buffers,
values far outside the range whose squares fp32 holds, NaN and infinities."""
import numpy as np
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _check(bl, tensors, max_norm, what, in_place=False):
    """The norm, the coefficient and every scaled tensor."""
    src = [t.clone() for t in tensors]
    refs = [R.f64(t) for t in src]
    norm, coef = R.grad_clip(refs, max_norm)
    if in_place:
        outs = tensors
        n, c = bl.grad_clip(tensors, max_norm)
    else:
        outs = [torch.full_like(t, 7.0) for t in tensors]
        n, c = bl.grad_clip(tensors, max_norm, out=outs)
        assert all(torch.equal(a, b) for a, b in zip(src, tensors)), f"{what}: the gradients changed"
    assert n.dtype == F32 and n.dim() == 0 and c.dim() == 0
    R.check(n, np.asarray(norm), np.asarray(R.NORM_REL * norm), what + " norm")
    R.check(c, np.asarray(coef), np.asarray(R.COEF_REL * coef), what + " coef")
    if coef == 1.0:
        assert float(c) == 1.0 and all(torch.equal(a, b) for a, b in zip(src, outs))
    for i, (o, r) in enumerate(zip(outs, refs)):
        rel = R.COEF_REL + R.U + R.half_step(o.dtype)
        R.check(o, r * coef, rel * np.abs(r * coef) + 2.0 ** -133, f"{what} tensor {i}")
    return n, c


SIZES = [[1], [2, 1], [3, 8, 4, 1], [255, 256, 257], [8191, 8192, 8193], [1 << 20], [100001, 7, 65536, 1],
         [12345] * 40, [0, 5, 0, 0, 9, 0], [16384 * 3 + 1, 16384]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sizes(bl, sizes, dtype):
    for max_norm in (0.7, 1e9):
        ts = [torch.randn(n, generator=_gen(n + i)).to(dtype).cuda() for i, n in enumerate(sizes)]
        _check(bl, ts, max_norm, f"{sizes[:3]}")
        _check(bl, ts, max_norm, f"{sizes[:3]} in place", in_place=True)


def test_types_mixed_and_outputs_left_out(bl):
    ts = [torch.randn(n, generator=_gen(n)).to(t).cuda() for n, t in ((1000, BF16), (333, F32), (4097, BF16), (1, F32))]
    _check(bl, ts, 1.0, "mixed")
    keep = [t.clone() for t in ts]
    out = torch.empty_like(ts[1])
    n, c = bl.grad_clip(ts, 1.0, out=[None, out, ts[2], None])
    norm, coef = R.grad_clip([R.f64(t) for t in keep], 1.0)
    R.check(n, np.asarray(norm), np.asarray(R.NORM_REL * norm), "norm")
    assert torch.equal(ts[0], keep[0]) and torch.equal(ts[1], keep[1]) and torch.equal(ts[3], keep[3])
    for o, r in ((out, keep[1]), (ts[2], keep[2])):
        ref = R.f64(r) * coef
        R.check(o, ref, (R.COEF_REL + R.U + R.half_step(o.dtype)) * np.abs(ref), "out")
    assert torch.equal(bl.grad_norm(keep), n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift,oshift", [(0, 0), (1, 1), (3, 3), (1, 0), (0, 5), (7, 2)])
def test_unaligned_views(bl, dtype, shift, oshift):
    """Gradients that are slices of a flat buffer, odd sizes; what lies around the outputs keeps its value."""
    sizes = [5, 1, 8200, 17, 33, 9001, 2]
    flat = torch.randn(shift + sum(sizes), generator=_gen(shift)).to(dtype).cuda()
    obuf = torch.full((oshift + sum(sizes) + 8,), 7.0, dtype=dtype, device="cuda")
    ts = list(flat[shift:].split(sizes))
    outs = list(obuf[oshift:oshift + sum(sizes)].split(sizes))
    norm, coef = R.grad_clip([R.f64(t) for t in ts], 2.0)
    n, c = bl.grad_clip(ts, 2.0, out=outs)
    R.check(n, np.asarray(norm), np.asarray(R.NORM_REL * norm), "norm")
    ref = R.f64(flat[shift:]) * coef
    R.check(obuf[oshift:oshift + sum(sizes)], ref, (R.COEF_REL + R.U + R.half_step(dtype)) * np.abs(ref) + 2.0 ** -133, "out")
    assert bool((obuf[:oshift] == 7).all()) and bool((obuf[oshift + sum(sizes):] == 7).all())
    # in place: every other tensor, the rest of the buffer untouched
    before = flat.clone()
    bl.grad_clip(ts[::2], 0.5)
    at = shift
    for i, k in enumerate(sizes):
        if i % 2:
            assert torch.equal(flat[at:at + k], before[at:at + k])
        at += k
    assert torch.equal(flat[:shift], before[:shift])


def test_more_tensors_than_a_launch_holds(bl):
    sizes = [int(s) for s in np.random.default_rng(0).integers(1, 300, 2500)]
    flat = torch.randn(sum(sizes), generator=_gen(1)).cuda()
    ts = list(flat.split(sizes))
    keep = flat.clone()
    n, c = bl.grad_clip(ts, 3.0)
    norm, coef = R.grad_clip([R.f64(keep)], 3.0)
    R.check(n, np.asarray(norm), np.asarray(R.NORM_REL * norm), "norm")
    ref = R.f64(keep) * coef
    R.check(flat, ref, (R.COEF_REL + 2 * R.U) * np.abs(ref), "out")


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-10, 1e10, 1e18, 1e25, 1e35])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_scale(bl, scale, dtype):
    ts = [(torch.randn(n, generator=_gen(n)) * scale).to(dtype).cuda() for n in (10, 5000)]
    _check(bl, ts, 1.0, f"{scale}")
    # the same with zeros, and a few values of another scale
    ts[1][::3] = 0
    ts[1][::50] *= 1e-8
    _check(bl, ts, scale, f"{scale} mixed")


def test_zeros_and_bounds(bl):
    ts = [torch.zeros(1000, device="cuda")]
    n, c = _check(bl, ts, 1.0, "zeros")
    assert float(n) == 0.0 and float(c) == 1.0
    ts = [torch.randn(1000, generator=_gen(1)).cuda()]
    n, c = bl.grad_clip(ts, 0.0)
    assert float(c) == 0.0 and not bool(ts[0].any()) and float(n) > 0
    ts = [torch.randn(1000, generator=_gen(1)).cuda()]
    keep = ts[0].clone()
    n, c = bl.grad_clip(ts, float("inf"))
    assert float(c) == 1.0 and torch.equal(ts[0], keep)
    # a norm above the largest float
    ts = [torch.full((1000,), 3e38, device="cuda")]
    n, c = bl.grad_clip(ts, 1.0)
    assert torch.isinf(n) and abs(float(c) * 3e38 * 1000 ** 0.5 - 1) < 1e-5


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_not_finite(bl, dtype):
    for bad, out in ((float("nan"), None), (float("inf"), 0.0), (float("-inf"), 0.0)):
        ts = [torch.randn(n, generator=_gen(n)).to(dtype).cuda() for n in (100, 9000)]
        ts[0][7] = bad
        n, c = bl.grad_clip(ts, 1.0)
        if out is None:
            assert torch.isnan(n) and torch.isnan(c) and all(bool(torch.isnan(t).all()) for t in ts)
        else:
            assert torch.isinf(n) and float(c) == 0.0
            assert not bool(ts[1].any()) and bool(torch.isnan(ts[0][7])) and int(torch.count_nonzero(ts[0])) == 1


def test_results_repeat_on_streams_and_in_a_graph(bl):
    sizes = [300001, 17, 65536, 4099]
    flat = torch.randn(sum(sizes), generator=_gen(3)).cuda()
    ts = list(flat.split(sizes))
    outs = [torch.empty_like(t) for t in ts]
    n, c = bl.grad_clip(ts, 1.0, out=outs)
    ref = torch.cat([o.clone() for o in outs])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams * 2:
        with torch.cuda.stream(s):
            o = [torch.empty_like(t) for t in ts]
            got.append((bl.grad_clip(ts, 1.0, out=o), o))
    torch.cuda.synchronize()
    for (n1, c1), o in got:
        assert torch.equal(n, n1) and torch.equal(c, c1) and torch.equal(torch.cat(o), ref)
    stats = torch.empty(2, device="cuda")
    ws = torch.empty(bl.workspace_bytes(bl.BL_OP_GRAD_CLIP, len(ts), 0, 0), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bl.grad_clip(ts, 1.0, out=outs, stats=stats, ws=ws)
    for k in (1.0, 3.0, 1e-6):
        flat.copy_(torch.randn(sum(sizes), generator=_gen(int(k * 10))) * k)
        g.replay()
        torch.cuda.synchronize()
        norm, coef = R.grad_clip([R.f64(flat)], 1.0)
        R.check(stats, np.asarray([norm, coef]), R.COEF_REL * np.asarray([norm, coef]), "graph")
        r = R.f64(flat) * coef
        R.check(torch.cat(outs), r, (R.COEF_REL + 2 * R.U) * np.abs(r), "graph out")


def test_refusals(bl):
    t = torch.randn(64, device="cuda")
    for call in (lambda: bl.grad_clip([t], 1.0, out=[]), lambda: bl.grad_clip([t.half()], 1.0), lambda: bl.grad_clip([t[::2]], 1.0),
                 lambda: bl.grad_clip([t], 1.0, out=[t[:32]]), lambda: bl.grad_clip([t], 1.0, out=[t.to(BF16)]),
                 lambda: bl.grad_clip([t, t.cpu()], 1.0), lambda: bl.grad_clip([t], 1.0, stats=t)):
        with pytest.raises(ValueError):
            call()
    keep = t.clone()
    for call in (lambda: bl.grad_clip([t, t], 1.0), lambda: bl.grad_clip([t[:40], t[30:]], 1.0), lambda: bl.grad_clip([t], -1.0),
                 lambda: bl.grad_clip([t[:32]], 1.0, out=[t[16:48]]),
                 lambda: bl.grad_clip([t], 1.0, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(bl.BitLinearError):
            call()
    assert torch.equal(t, keep)


@pytest.mark.parametrize("count", [3, 100, 1100])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_bytes(bl, dtype, count):
    """From 96 MB of gradients on: ragged slices of one buffer that begin anywhere, in place; what lies around them
    keeps its value."""
    n = (100 << 20) // (2 if dtype == BF16 else 4)
    cuts = np.sort(np.random.default_rng(count).integers(0, n, count - 1))
    sizes = np.diff(np.concatenate([[0], cuts, [n]])).tolist()
    flat = torch.randn(n + 12, generator=torch.Generator("cuda").manual_seed(count), device="cuda").to(dtype)
    flat[:3], flat[n + 3:] = 7.0, 7.0
    src = flat[3:n + 3].clone()
    norm, coef = bl.grad_clip(list(flat[3:n + 3].split(sizes)), 100.0)
    ref_norm = float(src.double().square_().sum().sqrt())
    ref_coef = 100.0 / (ref_norm + 1e-6)
    assert abs(float(norm) - ref_norm) <= R.NORM_REL * ref_norm and abs(float(coef) - ref_coef) <= R.COEF_REL * ref_coef
    ref = src.double().mul_(ref_coef)
    off = (flat[3:n + 3].double() - ref).abs_()
    assert bool((off <= (R.COEF_REL + R.U + R.half_step(dtype)) * ref.abs() + 2.0 ** -133).all())
    assert bool((flat[:3] == 7).all()) and bool((flat[n + 3:] == 7).all())
