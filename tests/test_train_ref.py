"""The fp64 statements in tests/train_ref.py themselves (CPU): the layer
norm's gradient against central differences of its forward pass and hand-worked
values, the embedding gradient as the adjoint of the lookup, the bounds'
sensitivity to planted mistakes."""
import numpy as np
import pytest

import train_ref as R


@pytest.mark.parametrize("M,K,affine", [(1, 2, True), (3, 5, True), (4, 16, False), (2, 33, True)])
def test_layer_norm_gradient_against_differences(M, K, affine):
    rng = np.random.default_rng(M * K)
    x, dy = rng.normal(1.0, 2.0, (M, K)), rng.normal(size=(M, K))
    w, b = (rng.normal(1, 0.3, K), rng.normal(size=K)) if affine else (None, None)
    dx, dw, db = R.layer_norm_backward(x, w, dy)

    def loss(x, w, b):
        return float((R.layer_norm(x, w, b)[0] * dy).sum())

    h = 1e-5
    for i in range(M):
        for k in range(K):
            e = np.zeros_like(x)
            e[i, k] = h
            # the difference quotient is off by h^2 / 6 times the third derivative (below 1e3 here) and by the
            # loss's rounding over h
            assert abs((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h) - dx[i, k]) < 1e-6
    if affine:
        for k in range(K):
            e = np.zeros(K)
            e[k] = h
            assert abs((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h) - dw[k]) < 1e-7
            assert abs((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h) - db[k]) < 1e-7


def test_layer_norm_by_hand():
    # x = (1, 3): mean 2, variance 1; with eps = 3 the root is 2 and z = (-1/2, 1/2)
    y, mean, rstd, z = R.layer_norm(np.array([[1.0, 3.0]]), np.array([2.0, 4.0]), np.array([1.0, -1.0]), eps=3.0)
    assert mean[0] == 2.0 and rstd[0] == 0.5 and z.tolist() == [[-0.5, 0.5]] and y.tolist() == [[0.0, 1.0]]
    # dy = (1, 0), w = 1: g - mean g = (1/2, -1/2), mean(g z) = -1/4, z times it = (1/8, -1/8): dx = (3/16, -3/16)
    dx, dw, db = R.layer_norm_backward(np.array([[1.0, 3.0]]), None, np.array([[1.0, 0.0]]), eps=3.0)
    assert dx.tolist() == [[0.1875, -0.1875]] and dw.tolist() == [-0.5, 0.0] and db.tolist() == [1.0, 0.0]


def test_embedding_gradient_is_the_adjoint_of_the_lookup():
    rng = np.random.default_rng(0)
    V, D, T = 7, 4, 40
    ids = rng.integers(0, V, T)
    E, dy = rng.normal(size=(V, D)), rng.normal(size=(T, D))
    d = R.embedding_backward(ids, dy, V, scale=0.5)
    assert np.isclose((0.5 * E[ids] * dy).sum(), (d * E).sum(), rtol=1e-12)
    d = R.embedding_backward(ids, dy, V, scale=0.5, padding_id=int(ids[0]))
    assert not d[ids[0]].any()
    d = R.embedding_backward([-1, V, 2], dy[:3], V)
    assert np.array_equal(d[2], dy[2]) and np.abs(d).sum() == np.abs(dy[2]).sum()


def test_grad_clip_by_hand():
    norm, coef = R.grad_clip([np.array([3.0, 0.0]), np.array([4.0])], 1.0)
    assert norm == 5.0 and abs(coef - 1.0 / 5.000001) < 1e-15
    assert R.grad_clip([np.array([3.0]), np.array([4.0])], 6.0) == (5.0, 1.0)


@pytest.mark.parametrize("mistake", ["no mean g", "no mean gz", "unbiased variance", "eps outside", "no weight"])
def test_the_bounds_catch_a_mistake(mistake):
    rng = np.random.default_rng(5)
    M, K = 6, 96
    x, dy, w = rng.normal(0.3, 1.0, (M, K)), rng.normal(size=(M, K)), rng.normal(1, 0.2, K)
    y, mean, rstd, z = R.layer_norm(x, w, eps=1e-2)
    dx, _, _ = R.layer_norm_backward(x, w, dy, eps=1e-2)
    g = dy * w
    mg, mgz = g.mean(1, keepdims=True), (g * z).mean(1, keepdims=True)
    var = x.var(1, keepdims=True)
    r = rstd[:, None]
    wrong = {"no mean g": r * (g - z * mgz), "no mean gz": r * (g - mg),
             "no weight": r * (dy - dy.mean(1, keepdims=True) - z * (dy * z).mean(1, keepdims=True))}
    if mistake in wrong:
        import torch
        b, _, _ = R.layer_norm_backward_bounds(x, w, dy, torch.float32, eps=1e-2)
        assert (np.abs(wrong[mistake] - dx) > b).mean() > 0.5
    else:
        import torch
        b = R.layer_norm_bound(y, z, w, None, torch.float32)
        d = x - mean[:, None]
        bad = d / np.sqrt(var * K / (K - 1) + 1e-2) * w if mistake == "unbiased variance" else d / (np.sqrt(var) + 1e-2) * w
        assert (np.abs(bad - y) > b).mean() > 0.5
