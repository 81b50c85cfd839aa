"""fp64 definitions (numpy) of the operators that a language model puts around
the recurrence: layer norm and the softmax cross entropy of an output
projection.  Tests only; shares nothing with the CUDA library."""
import numpy as np


def _np(x):
    return x.detach().to("cpu").double().numpy() if hasattr(x, "detach") else np.asarray(x, dtype=np.float64)


def layer_norm_fwd(x, w=None, b=None, eps=1e-5):
    """y, mean, rstd of rows x [..., D]."""
    x = _np(x)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if w is not None:
        y = y * _np(w)
    if b is not None:
        y = y + _np(b)
    return y, mean, rstd


def layer_norm_bwd(x, w, mean, rstd, dy):
    """dx, dw, db from the row statistics: with n the normalised row,
    dx = J^T (dy w) with the row's Jacobian J = rstd (I - 1 1^T / D - n n^T / D)."""
    x, mean, rstd, dy = _np(x), _np(mean), _np(rstd), _np(dy)
    n = (x - mean[..., None]) * rstd[..., None]
    a = dy * _np(w) if w is not None else dy
    D = x.shape[-1]
    dx = rstd[..., None] * (a - a.sum(-1, keepdims=True) / D - n * (a * n).sum(-1, keepdims=True) / D)
    rows = tuple(range(x.ndim - 1))
    return dx, (dy * n).sum(rows), dy.sum(rows)


def linear_ce_fwd(x, w, target):
    """loss [N], lse [N] of logits x w^T (x [N,D], w [V,D]); a negative target
    is not scored: its loss is 0."""
    x, w, t = _np(x), _np(w), np.asarray(target)
    z = x @ w.T
    m = z.max(1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(1))
    picked = z[np.arange(len(t)), np.maximum(t, 0)]
    return np.where(t < 0, 0.0, lse - picked), lse


def linear_ce_bwd(x, w, target, lse, dloss):
    """dx [N,D], dw [V,D] of sum_n dloss[n] loss[n], from the logits' lse."""
    x, w, t, lse, dloss = _np(x), _np(w), np.asarray(target), _np(lse), _np(dloss)
    g = np.exp(x @ w.T - lse[:, None])
    g[np.arange(len(t)), np.maximum(t, 0)] -= 1.0
    g = np.where((t < 0)[:, None], 0.0, g * dloss[:, None])
    return g @ w, g.T @ x
