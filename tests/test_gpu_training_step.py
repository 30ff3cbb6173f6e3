"""One training step of a small binarized trunk through the library's calls in
a row -- lookup, layer norm, FBI-linear, and back: straight-through gradients,
the norm's gradient, the table's, then one norm over all of them -- against
the same step in fp64, eagerly and captured into a graph."""
import numpy as np
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
T, V, D, N = 200, 384, 256, 384
SCALE, MAX_NORM = 16.0, 0.5


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


def _inputs(seed):
    g = torch.Generator().manual_seed(seed)
    s = {"ids": torch.randint(0, V, (T,), generator=g), "table": 0.05 * torch.randn(V, D, generator=g),
         "w": 1 + 0.1 * torch.randn(D, generator=g), "b": 0.1 * torch.randn(D, generator=g),
         "W": 0.02 * torch.randn(N, D, generator=g), "dy": (0.1 * torch.randn(T, N, generator=g)).to(BF16)}
    s["ids"][T - 50:] = 0  # padding
    return {k: v.cuda() for k, v in s.items()}


def _step(bl, s):
    packed, alpha = bl.bin_pack(s["W"], bl.BL_PACK_FBI)
    h = bl.embedding(s["ids"], s["table"], scale=SCALE)
    x, mean, rstd = bl.layer_norm(h, s["w"], s["b"], out_dtype=BF16, stats=True)
    y = bl.bin_linear_w1a16(x, packed, alpha)
    dx, dW, dalpha = bl.bin_linear_w1a16_backward(x, packed, alpha, s["dy"])
    dh, dw, db = bl.layer_norm_backward(h, s["w"], mean, rstd, dx)
    dE = bl.embedding_backward(s["ids"], dh, V, scale=SCALE, padding_id=0)
    grads = [dW, dalpha, dw, db, dE]
    raw = [g.clone() for g in grads]
    norm, coef = bl.grad_clip(grads, MAX_NORM)
    return {"h": h, "x": x, "y": y, "dx": dx, "dh": dh, "raw": raw, "grads": grads, "norm": norm, "coef": coef}


def _check(s, r):
    """Each call against fp64 on what the call before it gave."""
    w, b, h = R.f64(s["w"]), R.f64(s["b"]), R.f64(r["h"])
    ids = s["ids"].cpu().numpy()
    assert torch.equal(r["h"], s["table"][s["ids"]] * SCALE)
    ry, _, _, z = R.layer_norm(h, w, b)
    R.check(r["x"], ry, R.layer_norm_bound(ry, z, w, b, BF16), "x")
    dx = R.f64(r["dx"])
    ref, bounds = R.layer_norm_backward(h, w, dx), R.layer_norm_backward_bounds(h, w, dx, F32)
    R.check(r["dh"], ref[0], bounds[0], "dh")
    R.check(r["raw"][2], ref[1], bounds[1], "dweight")
    R.check(r["raw"][3], ref[2], bounds[2], "dbias")
    dh = R.f64(r["dh"])
    dE = R.embedding_backward(ids, dh, V, SCALE, 0)
    R.check(r["raw"][4], dE, R.embedding_backward_bound(ids, dh, V, dE, F32, SCALE, 0), "dtable")
    raw = [R.f64(t) for t in r["raw"]]
    norm, coef = R.grad_clip(raw, MAX_NORM)
    assert coef < 1.0
    R.check(r["norm"], np.asarray(norm), np.asarray(R.NORM_REL * norm), "norm")
    for g, t in zip(r["grads"], raw):
        R.check(g, t * coef, (R.COEF_REL + 2 * R.U) * np.abs(t * coef), "clipped")


def test_step(bl):
    s = _inputs(1)
    r = _step(bl, s)
    torch.cuda.synchronize()
    assert bl.device_error() == (0, 0)
    _check(s, r)
    again = _step(bl, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(r["grads"], again["grads"]))


def test_step_in_a_graph(bl):
    s = _inputs(2)
    _step(bl, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = _step(bl, s)
    for seed in (3, 4):
        for k, v in _inputs(seed).items():
            s[k].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert bl.device_error() == (0, 0)
        _check(s, r)


def test_calls_after_other_work_in_a_graph(bl):
    """Captured right behind copies, fills, a join of two streams and the library's other kernels: each call sees
    what was written before it."""
    g0 = torch.Generator().manual_seed(9)
    src = torch.randn(300, 256, generator=g0).cuda()
    w, b = torch.randn(256, generator=g0).cuda(), torch.randn(256, generator=g0).cuda()
    ids_src = torch.randint(0, 40, (300,), generator=g0).cuda()
    x, h, z = torch.empty_like(src), torch.empty_like(src), torch.empty(300, 256, dtype=BF16, device="cuda")
    ids = torch.empty_like(ids_src)
    W = (0.02 * torch.randn(384, 256, generator=g0)).cuda()

    def step():
        x.copy_(src)                                   # a copy
        y, mean, rstd = bl.layer_norm(x, w, b, stats=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            h.copy_(y)
            ids.copy_(ids_src)
        z.zero_()
        torch.cuda.current_stream().wait_stream(side)  # a join
        dE = bl.embedding_backward(ids, h, 40)
        e = bl.embedding(ids, dE)
        dx, dw, db = bl.layer_norm_backward(x, w, mean, rstd, e)
        packed, alpha = bl.bin_pack(W, bl.BL_PACK_FBI)
        bl.layer_norm(dx, None, None, out=z)
        # prefetches the packed weights before it waits
        out = bl.bin_linear_w1a16(z[:8], packed, alpha, flags=bl.BL_FLAG_OVERLAP_PREVIOUS)
        grads = [dE, dw, db]
        norm, coef = bl.grad_clip(grads, 0.1)
        return [y, e, dx, z, out, *grads, norm, coef]

    step()
    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        for t in (x, h):
            t.fill_(7.0)
        ids.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(ref, got))
    assert bl.device_error() == (0, 0)
