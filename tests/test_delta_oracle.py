"""Pins of the fp64 definitions in oracle/delta.py (CPU): closed forms, central
finite differences of every gradient, the recurrence's own identities."""
import numpy as np
import pytest

import oracle
from oracle import delta


def rng(seed):
    return np.random.default_rng(seed)


def problem(seed, B=1, T=6, H=2, Hqk=1, K=4, V=3):
    r = rng(seed)
    q, k, v = r.normal(size=(B, T, Hqk, K)), r.normal(size=(B, T, Hqk, K)), r.normal(size=(B, T, H, V))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return q, k, v, -np.abs(r.normal(size=(B, T, H))) / 3, 1 / (1 + np.exp(-r.normal(size=(B, T, H))))


def fd(f, x, eps=1e-6):
    """Central differences of the scalar f over every element of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = f()
        x[i] = keep - eps
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * eps)
    return g


def test_orthogonal_keys_are_plain_gated_attention():
    """Keys that never meet again leave nothing to correct: with beta = 1 the rule is the SSD recurrence."""
    r = rng(0)
    T = 5
    k = np.eye(8)[None, :T, None]
    q, v, g = r.normal(size=(1, T, 1, 8)), r.normal(size=(1, T, 3, 4)), -np.abs(r.normal(size=(1, T, 3)))
    o, S = delta.fwd(q, k, v, g, np.ones((1, T, 3)), 0.5)
    ro, rS = oracle.fwd(q, k, v, g, 0.5)
    assert np.allclose(o, ro) and np.allclose(S, rS)


def test_a_key_written_with_beta_one_reads_its_value_back():
    q, k, v, g, b = problem(1, T=4)
    o, _ = delta.fwd(k, k, v, g, np.ones_like(b), 1.0, h0=rng(2).normal(size=(1, 2, 4, 3)))
    assert np.allclose(o, v)


@pytest.mark.parametrize("seg", [None, [[3, 3, 7, 7, 7, 3]]])
def test_gradients_are_differences(seg):
    q, k, v, g, b = problem(3)
    n = len(delta.documents(1, 6, seg))
    r = rng(4)
    h0, do, dht = r.normal(size=(n, 2, 4, 3)), r.normal(size=v.shape), r.normal(size=(n, 2, 4, 3))

    def loss():
        o, S = delta.fwd(q, k, v, g, b, 0.7, seg, h0)
        return (o * do).sum() + (S * dht).sum()

    got = delta.bwd(q, k, v, g, b, do, 0.7, seg, h0, dht)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", b), ("dh0", h0)):
        assert np.allclose(got[name], fd(loss, x), rtol=1e-6, atol=1e-7), name


def test_documents_are_independent():
    q, k, v, g, b = problem(5, T=7)
    seg = np.array([[0, 0, 1, 1, 1, 0, 0]])
    o, S = delta.fwd(q, k, v, g, b, 1.0, seg)
    for d, (s, e) in enumerate([(0, 2), (2, 5), (5, 7)]):
        ro, rS = delta.fwd(*(x[:, s:e] for x in (q, k, v, g, b)), 1.0)
        assert np.allclose(o[:, s:e], ro) and np.allclose(S[d], rS[0])


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm(norm, interleaved):
    r = rng(6)
    x, w, dy = r.normal(size=(2, 3, 2, 6)), r.normal(size=6), r.normal(size=(2, 3, 2, 6))
    angle = r.normal(size=(9, 2))
    pos = np.array([[0, 1, 2], [8, 3, 3]])
    args = (np.cos(angle), np.sin(angle), pos, 1e-3, norm, interleaved)
    y = delta.head_norm_fwd(x, w, *args)
    # a rotation keeps a row's length, and the pairs past 2 R channels as they were
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) * (6 if norm == "l2" else 1) + 1e-3) * w
    assert np.allclose((y ** 2).sum(-1), (n ** 2).sum(-1)) and np.allclose(y[..., 4:], n[..., 4:])
    i, j = (0, 1) if interleaved else (0, 2)
    z = (n[..., i] + 1j * n[..., j]) * np.exp(1j * angle[pos, 0])[:, :, None]
    assert np.allclose(y[..., i], z.real) and np.allclose(y[..., j], z.imag)
    loss = lambda: (delta.head_norm_fwd(x, w, *args) * dy).sum()
    dx, dw = delta.head_norm_bwd(x, dy, w, *args)
    assert np.allclose(dx, fd(loss, x), atol=1e-7) and np.allclose(dw, fd(loss, w), atol=1e-7)
