"""fp64 definitions (numpy) of the gated delta rule, token by token, with its
gradients, and of the norm of query and key heads with the rotation by
position.  Tests only; shares nothing with the CUDA library."""
import numpy as np

from .lm import _np


def documents(B, T, segment_ids=None):
    """(row, first token, end) of every document, in row-major order."""
    if T == 0:
        return []
    out = []
    for b in range(B):
        cuts = [0]
        if segment_ids is not None:
            ids = np.asarray(segment_ids)[b]
            cuts += [t for t in range(1, T) if ids[t] != ids[t - 1]]
        out += [(b, s, e) for s, e in zip(cuts, cuts[1:] + [T])]
    return out


def _heads(x, H):
    return np.repeat(x, H // x.shape[2], axis=2)


def fwd(q, k, v, g, beta, scale, segment_ids=None, h0=None):
    """o [B,T,H,V], final states [n,H,K,V]."""
    q, k, v, g, beta = map(_np, (q, k, v, g, beta))
    B, T, H, V = v.shape
    q, k = _heads(q, H), _heads(k, H)
    docs = documents(B, T, segment_ids)
    o, last = np.zeros_like(v), np.zeros((len(docs), H, q.shape[3], V))
    for d, (b, s, e) in enumerate(docs):
        S = np.zeros((H, q.shape[3], V)) if h0 is None else _np(h0)[d].copy()
        for t in range(s, e):
            a = np.exp(g[b, t])[:, None, None]
            S = np.where(a == 0, 0.0, S) * a
            u = beta[b, t][:, None] * (v[b, t] - np.einsum("hkv,hk->hv", S, k[b, t]))
            S = S + k[b, t][:, :, None] * u[:, None]
            o[b, t] = scale * np.einsum("hkv,hk->hv", S, q[b, t])
        last[d] = S
    return o, last


def bwd(q, k, v, g, beta, do, scale, segment_ids=None, h0=None, dht=None):
    """dict of dq, dk, dv, dg, dbeta, dh0."""
    q, k, v, g, beta, do = map(_np, (q, k, v, g, beta, do))
    B, T, H, V = v.shape
    Hqk, K = q.shape[2:]
    q, k = _heads(q, H), _heads(k, H)
    docs = documents(B, T, segment_ids)
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    dh0 = np.zeros((len(docs), H, K, V))
    for d, (b, s, e) in enumerate(docs):
        S = np.zeros((H, K, V)) if h0 is None else _np(h0)[d].copy()
        kept = []
        for t in range(s, e):  # the decayed state before the token, the error of its prediction
            S = np.exp(g[b, t])[:, None, None] * S
            err = v[b, t] - np.einsum("hkv,hk->hv", S, k[b, t])
            kept.append((S, err))
            S = S + k[b, t][:, :, None] * (beta[b, t][:, None] * err)[:, None]
        dS = np.zeros((H, K, V)) if dht is None else _np(dht)[d].copy()
        for t in reversed(range(s, e)):
            P, err = kept[t - s]
            u = beta[b, t][:, None] * err
            S = P + k[b, t][:, :, None] * u[:, None]
            dq[b, t] = scale * np.einsum("hkv,hv->hk", S, do[b, t])
            dS = dS + scale * q[b, t][:, :, None] * do[b, t][:, None]
            du = np.einsum("hkv,hk->hv", dS, k[b, t])
            dk[b, t] = np.einsum("hkv,hv->hk", dS, u)
            db[b, t] = (du * err).sum(-1)
            dv[b, t] = beta[b, t][:, None] * du
            dk[b, t] -= np.einsum("hkv,hv->hk", P, dv[b, t])
            dS = dS - k[b, t][:, :, None] * dv[b, t][:, None]
            dg[b, t] = (dS * P).sum((1, 2))
            dS = np.exp(g[b, t])[:, None, None] * dS
        dh0[d] = dS
    group = lambda x: x.reshape(B, T, Hqk, H // Hqk, K).sum(3)  # noqa: E731
    return dict(dq=group(dq), dk=group(dk), dv=dv, dg=dg, dbeta=db, dh0=dh0)


def step(q, k, v, g, beta, state, idx, scale):
    """o and the slots idx of the pool after the tokens."""
    return fwd(q, k, v, g, beta, scale, None, _np(state)[np.asarray(idx)])


def _rotation(D, R, cos, sin, interleaved):
    """The D x D matrix of one position."""
    M = np.eye(D)
    for i in range(R):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R)
        M[a, a], M[a, b], M[b, a], M[b, b] = cos[i], -sin[i], sin[i], cos[i]
    return M


def _rotations(x, cos, sin, positions, interleaved):
    B, T, _, D = x.shape
    if cos is None:
        return np.broadcast_to(np.eye(D), (B, T, D, D))
    cos, sin = _np(cos), _np(sin)
    pos = np.broadcast_to(np.arange(T), (B, T)) if positions is None else np.asarray(positions)
    R = cos.shape[1]
    table = {p: _rotation(D, R, cos[p], sin[p], interleaved) if 0 <= p < len(cos) else np.eye(D)
             for p in np.unique(pos)}
    return np.stack([np.stack([table[p] for p in row]) for row in pos])


def head_norm_fwd(x, w=None, cos=None, sin=None, positions=None, eps=1e-6, norm="rms", interleaved=False):
    x = _np(x)
    m = (x ** 2).mean(-1, keepdims=True) if norm == "rms" else (x ** 2).sum(-1, keepdims=True)
    n = x / np.sqrt(m + eps) * (1.0 if w is None else _np(w))
    return np.einsum("btij,bthj->bthi", _rotations(x, cos, sin, positions, interleaved), n)


def head_norm_bwd(x, dy, w=None, cos=None, sin=None, positions=None, eps=1e-6, norm="rms", interleaved=False):
    """dx, dw: through the row's Jacobian r (I - n n^T / c), n = x r, c = D (rms) or 1 (l2)."""
    x, dy = _np(x), _np(dy)
    c = x.shape[-1] if norm == "rms" else 1
    r = 1 / np.sqrt((x ** 2).sum(-1, keepdims=True) / c + eps)
    n = x * r
    d = np.einsum("btij,bthi->bthj", _rotations(x, cos, sin, positions, interleaved), dy)
    a = d if w is None else d * _np(w)
    return r * (a - n * (a * n).sum(-1, keepdims=True) / c), (d * n).sum((0, 1, 2))
