"""fp64 statements (numpy) of the full-precision operators of a training step,
and the error bounds their GPU tests use.

u = 2^-24 is half an fp32 step, `half_step(t)` half a step of an output type
t, relative to the value (bf16 2^-8, fp32 2^-24).

Sums. A sum of K terms formed as serial runs of at most n terms that a tree
of at most 16 levels joins is off by at most (n + 16) u times the sum of the
absolute values. A row's sums run over at most max(K / 256, 32) terms per
thread, so gamma(K) = (max(K / 256, 32) + 16) u; sums over M rows over at
most M / 64 + 64 terms, so gamma_rows(M) = (M / 64 + 80) u.

Layer norm. d = x - c is off by u |d|, and the mean of the d by gamma mean|d|
<= gamma sigma, so z = (d - mean d) rstd is off by gamma + 3 u |z| from the
mean and the three roundings, and by |z| times the relative error of rstd:
the variance is off by gamma + 3 u relative, plus twice the product of the
mean's error and the mean, which the correction leaves below gamma, so rstd
by at most gamma + 3 u (half of twice that). Together
    tol_z = (gamma + 6 u) (1 + |z|).
y = z w + b adds two roundings and the output's own.

Gradient. With g = dy w, dx = rstd (g - mean g - z mean(g z)): mean g is off
by (gamma + u) mean|g|, mean(g z) by (gamma + 3 u) mean|g z| + mean(|g| tol_z);
the difference has three roundings of its largest parts, and rstd one more
and its own error (gamma + 3 u).
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def gamma(K: int) -> float:
    return (max(K / 256, 32) + 16) * U


def gamma_rows(M: int) -> float:
    return (M / 64 + 80) * U


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd, z)"""
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    z = d * rstd[:, None]
    y = z if w is None else z * w
    return (y if b is None else y + b), mean, rstd, z


def layer_norm_backward(x, w, dy, eps=1e-5):
    """(dx, dweight, dbias)"""
    _, _, rstd, z = layer_norm(x, eps=eps)
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - z * (g * z).mean(1, keepdims=True))
    return dx, (dy * z).sum(0), dy.sum(0)


def tol_z(z):
    return (gamma(z.shape[1]) + 6 * U) * (1 + np.abs(z))


def layer_norm_bound(y, z, w, b, dtype):
    t = tol_z(z) + 2 * U * np.abs(z)
    if w is not None:
        t = t * np.abs(w)
    if b is not None:
        t = t + U * (np.abs(b) + np.abs(y))
    return t + half_step(dtype) * (np.abs(y) + t) + 2.0 ** -140


def layer_norm_backward_bounds(x, w, dy, dtype, eps=1e-5):
    """(bound of dx, of dweight, of dbias)"""
    M, K = x.shape
    _, _, rstd, z = layer_norm(x, eps=eps)
    g = dy if w is None else dy * w
    dx, dw, db = layer_norm_backward(x, w, dy, eps)
    tz, gk = tol_z(z), gamma(K)
    mg, mgz = np.abs(g).mean(1, keepdims=True), np.abs(g * z).mean(1, keepdims=True)
    t_mgz = (gk + 3 * U) * mgz + (np.abs(g) * tz).mean(1, keepdims=True)
    t = (gk + 3 * U) * mg + np.abs(z) * t_mgz + tz * (mgz + t_mgz) + 4 * U * (np.abs(g) + mg + np.abs(z) * mgz)
    t = rstd[:, None] * t + (gk + 4 * U) * np.abs(dx)
    gr = gamma_rows(M)
    t_dw = (np.abs(dy) * tz).sum(0) + (gr + 2 * U) * (np.abs(dy) * (np.abs(z) + tz)).sum(0)
    return (t + half_step(dtype) * (np.abs(dx) + t) + 2.0 ** -140, t_dw + U * np.abs(dw) + 2.0 ** -140,
            (gr + U) * np.abs(dy).sum(0) + 2.0 ** -140)


def embedding_backward(ids, dy, V, scale=1.0, padding_id=None):
    d = np.zeros((V, dy.shape[-1]))
    for t, v in enumerate(ids):
        if 0 <= v < V and v != padding_id:
            d[v] += dy[t]
    return d * np.float64(np.float32(scale))


def embedding_backward_bound(ids, dy, V, ref, dtype, scale=1.0, padding_id=None, old=None):
    """n rows added in any order are off by n u times their absolute sum; the
    product with the scale and the sum with the old value add one rounding each."""
    n = np.bincount([v for v in ids if 0 <= v < V and v != padding_id], minlength=V)[:, None]
    s = embedding_backward(ids, np.abs(dy), V, abs(scale), padding_id)
    t = (n + 2) * U * s
    if old is not None:
        t = t + U * np.abs(ref)
    return t + half_step(dtype) * (np.abs(ref) + t) + 2.0 ** -140


def grad_clip(tensors, max_norm):
    """(norm, coef) of fp64 arrays"""
    norm = np.sqrt(sum(float((t * t).sum()) for t in tensors))
    return norm, min(1.0, max_norm / (norm + 1e-6))


# Squares are added eight at a time in fp32 (8 roundings and the squares' own), then in fp64: the sum of
# squares is off by 9 u, the norm by half of that and its rounding, the coefficient by one more, a product
# by one more and the output's.
NORM_REL = 6 * U
COEF_REL = 8 * U


def check(got: torch.Tensor, ref: np.ndarray, bound: np.ndarray, what: str):
    g = f64(got)
    assert g.shape == ref.shape, f"{what}: shape {g.shape}, not {ref.shape}"
    bad = ~(np.abs(g - ref) <= bound)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first at {i}: got {g[i]!r}, "
                             f"ref {ref[i]!r}, bound {bound[i]!r}")
