"""GPU parity of qk_norm_fwd / qk_norm_bwd with the fp64 definitions, and the
layer that they and the delta rule make together.

fp32 outputs: a sum of up to 256 squares (8 in sequence, then a tree), the reciprocal
root (2 ulp) and six more roundings: 2^-24 (8 + 5 + 2 + 6) < 2^-19 of the row's
largest value.  bf16 outputs: half an ulp (2^-9 to 2^-8 of the element) more.  dw sums
up to 10^4 rows in fp32, at most 64 in sequence: 2^-17 of the largest of the sums
of the terms' sizes."""
import numpy as np
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
from oracle import delta

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL = 2.0 ** -19
ULP = {BF: 2.0 ** -8, F32: 0.0}


def rows_close(a, b):
    """Element by element, relative to the row's largest value."""
    x = a.detach().to("cpu", torch.float64).numpy()
    top = np.abs(b).max(-1, keepdims=True) if b.size else b
    return bool((np.abs(x - b) <= TOL * top + ULP[a.dtype] * np.abs(b) + 1e-30).all())


def make(B, T, Hq, Hk, D, R, dtype, seed, fused=False, P=50):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = dict(q=(2 * r(B, T, Hq, D)).to(dtype), k=(2 * r(B, T, Hk, D)).to(dtype), dq=r(B, T, Hq, D).to(dtype),
             dk=r(B, T, Hk, D).to(dtype), wq=1 + 0.3 * r(D), wk=1 + 0.3 * r(D))
    dev = {n: t.cuda() for n, t in x.items()}
    if fused:
        p = torch.cat([x["q"].flatten(2), x["k"].flatten(2), r(B, T, 8 * Hk).to(dtype)], 2).cuda()
        q, k, _ = p.split([Hq * D, Hk * D, 8 * Hk], 2)
        dev["q"], dev["k"] = q.unflatten(2, (Hq, D)), k.unflatten(2, (Hk, D))
    angle = 3 * r(P, R)
    turn = dict(cos=angle.cos(), sin=angle.sin(), positions=torch.randint(0, P, (B, T), generator=g).to(torch.int32))
    if not R:
        turn = dict(cos=None, sin=None, positions=None)
    return x, dev, turn


def cuda(d):
    return {n: None if t is None else t.cuda() for n, t in d.items()}


CASES = [
    # B, T, Hq, Hk, D, R, dtype, fused, norm, interleaved
    (1, 1, 16, 16, 128, 64, BF, True, "rms", False),
    (2, 7, 4, 2, 128, 64, BF, False, "l2", True),
    (3, 5, 3, 1, 64, 32, BF, True, "rms", True),
    (2, 3, 5, 2, 256, 128, BF, False, "rms", False),
    (2, 3, 5, 3, 256, 64, F32, True, "l2", False),
    (1, 9, 2, 2, 128, 0, BF, False, "l2", False),
    (1, 40, 6, 2, 72, 24, F32, False, "l2", False),
    (1, 40, 6, 2, 72, 20, F32, False, "rms", True),
    (1, 40, 6, 2, 72, 20, F32, False, "rms", False),
    (2, 11, 3, 2, 41, 20, F32, True, "rms", False),
    (2, 11, 3, 2, 41, 20, BF, True, "rms", True),
    (1, 6, 2, 1, 8, 4, BF, False, "l2", True),
    (1, 6, 2, 1, 8, 4, BF, False, "rms", False),
    (1, 6, 1, 1, 1, 0, F32, False, "rms", False),
    (1, 3, 2, 1, 255, 127, F32, False, "rms", True),
    (2, 700, 8, 2, 128, 32, BF, True, "rms", False),
    (5, 611, 2, 1, 64, 16, F32, False, "l2", False),
]


@pytest.mark.parametrize("B,T,Hq,Hk,D,R,dtype,fused,norm,inter", CASES)
def test_against_the_definition(cuda_ok, B, T, Hq, Hk, D, R, dtype, fused, norm, inter):
    x, dev, turn = make(B, T, Hq, Hk, D, R, dtype, B + T + D + R, fused)
    kw = dict(eps=1e-3, norm=norm, interleaved=inter)
    outs = tuple(torch.full(x[n].shape, float("nan"), dtype=dtype, device="cuda") for n in ("q", "k"))
    got = glc.qk_norm_fwd(dev["q"], dev["k"], dev["wq"], dev["wk"], **cuda(turn), **kw, outs=outs)
    for y, n in zip(got, "qk"):
        assert rows_close(y, delta.head_norm_fwd(x[n], x["w" + n], **turn, **kw)), n
    dq, dk, dwq, dwk = glc.qk_norm_bwd(dev["q"], dev["k"], dev["dq"], dev["dk"], dev["wq"], dev["wk"], **cuda(turn), **kw)
    for d, dw, n in ((dq, dwq, "q"), (dk, dwk, "k")):
        rd, rw = delta.head_norm_bwd(x[n], x["d" + n], x["w" + n], **turn, **kw)
        # the subtracted part is at most as large as the gradient that it is subtracted from
        scale = np.abs(rd).max(-1, keepdims=True)
        r = 1 / np.sqrt((x[n].double().numpy() ** 2).sum(-1, keepdims=True) / (D if norm == "rms" else 1) + 1e-3)
        scale = np.maximum(scale, r * np.abs(x["d" + n].double().numpy()).max(-1, keepdims=True) * 2)
        a = d.detach().double().cpu().numpy()
        assert (np.abs(a - rd) <= 2 * TOL * scale + ULP[dtype] * np.abs(rd)).all(), "d" + n
        size = np.abs(delta.head_norm_fwd(x[n], None, eps=1e-3, norm=norm)).max() * np.abs(x["d" + n].double().numpy()).sum(
            (0, 1, 2)).max()
        assert (np.abs(dw.double().cpu().numpy() - rw) <= 2.0 ** -17 * size).all(), "dw" + n
    again = glc.qk_norm_bwd(dev["q"], dev["k"], dev["dq"], dev["dk"], dev["wq"], dev["wk"], **cuda(turn), **kw)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again))
    glc.get_device_error()


def test_no_weights_and_positions_in_order(cuda_ok):
    x, dev, turn = make(2, 9, 3, 3, 64, 32, BF, 1)
    got = glc.qk_norm_fwd(dev["q"], dev["k"], cos=turn["cos"].cuda(), sin=turn["sin"].cuda())
    for y, n in zip(got, "qk"):
        assert rows_close(y, delta.head_norm_fwd(x[n], None, turn["cos"], turn["sin"]))
    plain = glc.qk_norm_bwd(dev["q"], dev["k"], dev["dq"], dev["dk"])
    ones = glc.qk_norm_bwd(dev["q"], dev["k"], dev["dq"], dev["dk"], torch.ones(64, device="cuda"),
                           torch.ones(64, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(plain, ones))


@pytest.mark.parametrize("D", [64, 50])
def test_a_position_outside_the_tables(cuda_ok, D):
    x, dev, turn = make(1, 6, 2, 2, D, 8, F32, 2)
    turn["positions"][0, 1], turn["positions"][0, 4] = 50, -1
    y, _ = glc.qk_norm_fwd(dev["q"], dev["k"], **cuda(turn))
    with pytest.raises(glc.GlacoreError) as e:
        glc.get_device_error()
    assert e.value.status == glc.ERR_INDEX
    assert rows_close(y, delta.head_norm_fwd(x["q"], None, **turn))  # those tokens are not rotated
    glc.qk_norm_bwd(dev["q"], dev["k"], dev["dq"], dev["dk"], **cuda(turn))
    with pytest.raises(glc.GlacoreError):
        glc.get_device_error()


def test_rows_of_zeros_and_infinities(cuda_ok):
    x, dev, _ = make(1, 4, 2, 2, 64, 0, F32, 3)
    dev["q"][0, 1] = 0
    dev["q"][0, 2, 0, 5] = float("inf")
    y, _ = glc.qk_norm_fwd(dev["q"], dev["k"], eps=1e-6, norm="l2")
    ref, _ = glc.qk_norm_fwd(x["q"].cuda(), dev["k"], eps=1e-6, norm="l2")
    assert torch.all(y[0, 1] == 0) and torch.isnan(y[0, 2, 0, 5])
    assert torch.equal(y[0, [0, 3]], ref[0, [0, 3]]) and torch.equal(y[0, 2, 1], ref[0, 2, 1])


def test_captured_and_replayed(cuda_ok):
    def fresh(seed):
        _, dev, turn = make(3, 50, 4, 2, 128, 32, BF, seed)
        return dict(dev, **cuda(turn))

    def call(s):
        t = (s["wq"], s["wk"], s["cos"], s["sin"], s["positions"])
        return *glc.qk_norm_fwd(s["q"], s["k"], *t), *glc.qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], *t)

    state = fresh(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(state)
    for seed in (2, 3):
        values = fresh(seed)
        for n, v in values.items():
            state[n].copy_(v)
        graph.replay()
        want = call({n: v.clone() for n, v in values.items()})
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals(cuda_ok):
    z = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)
    q, k, cs, pos = z(2, 3, 4, 16), z(2, 3, 2, 16), z(9, 8), z(2, 3, dtype=torch.int32)
    glc.qk_norm_fwd(q, k, cos=cs, sin=cs, positions=pos)
    bad = [dict(cos=cs), dict(sin=cs), dict(positions=pos), dict(cos=cs, sin=cs[:4]), dict(cos=z(9, 9), sin=z(9, 9)),
           dict(cos=z(2, 8), sin=z(2, 8)), dict(cos=cs, sin=cs, positions=pos[:1]), dict(wq=z(15)), dict(wk=z(2, 16)),
           dict(norm="max"), dict(wq=z(16).cpu()), dict(cos=cs.cpu(), sin=cs)]
    for kw in bad:
        with pytest.raises(ValueError):
            glc.qk_norm_fwd(q, k, **kw)
        with pytest.raises(ValueError):
            glc.qk_norm_bwd(q, k, q, k, **kw)
    for kw in (dict(cos=cs, sin=cs, positions=pos.long()), dict(wq=z(16, dtype=BF))):
        with pytest.raises(TypeError):
            glc.qk_norm_fwd(q, k, **kw)
    for a, b in ((q[0], k[0]), (q, k[:1]), (q, k[..., :8])):
        with pytest.raises(ValueError):
            glc.qk_norm_fwd(a, b)
    with pytest.raises(ValueError):
        glc.qk_norm_bwd(q, k, k, q)
    with pytest.raises(TypeError):
        glc.qk_norm_bwd(q, k, q.bfloat16(), k)
    with pytest.raises(glc.GlacoreError):
        glc.qk_norm_fwd(z(1, 1, 1, 264), z(1, 1, 1, 264))
    with pytest.raises(glc.GlacoreError):
        glc.qk_norm_fwd(q, k, eps=-1.0)
    with pytest.raises(ValueError):
        glc.qk_norm_fwd(q, k, outs=(q, q))
    empty = glc.qk_norm_bwd(q[:, :0], k[:, :0], q[:, :0], k[:, :0])
    assert empty[0].numel() == 0 and torch.all(empty[2] == 0) and torch.all(empty[3] == 0)


@pytest.mark.parametrize("dtype,D,V", [(BF, 128, 128), (BF, 64, 64), (F32, 24, 40)])
def test_a_layer_of_both(cuda_ok, dtype, D, V):
    """Queries and keys of one projection normalised and rotated, the delta rule over a prompt, its tokens one at
    a time, and the gradients down to the projection: against the same chain in 64 bits.  Rounded intermediates (q
    and k in the operands' type) are handed from one definition to the next, as the library hands them on; what
    the next call makes of another rounding of a gradient is within 2^-7 of its size in bf16."""
    B, T, Hq, H, R = 2, 150, 2, 4, D // 4
    x, dev, _ = make(B, T, Hq, Hq, D, 0, dtype, 5, fused=True)
    g = torch.Generator("cpu")
    g.manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g)
    v, gate, beta, do = r(B, T, H, V).to(dtype), -r(B, T, H).abs() / 4, r(B, T, H).sigmoid(), r(B, T, H, V).to(dtype)
    angle = torch.arange(T)[:, None] * 10.0 ** -torch.arange(R)
    cos, sin = angle.cos(), angle.sin()
    cv, cg, cb, cdo, cc, cs = (t.cuda() for t in (v, gate, beta, do, cos, sin))
    qn, kn = glc.qk_norm_fwd(dev["q"], dev["k"], cos=cc, sin=cs, norm="l2")
    o, _ = glc.delta_fwd(qn, kn, cv, cg, cb)
    ro, _ = delta.fwd(qn, kn, v, gate, beta, D ** -0.5)
    size = np.abs(ro).max()
    got = o.double().cpu().numpy()
    assert (np.abs(got - ro) <= 2.0 ** -14 * size + ULP[dtype] * np.abs(ro)).all()
    # the last tokens one at a time, from the state of those before
    cut = T - 4
    _, pool = glc.delta_fwd(qn[:, :cut], kn[:, :cut], cv[:, :cut], cg[:, :cut], cb[:, :cut], output_final_state=True)
    for t in range(cut, T):
        pos = torch.full((B, 1), t, dtype=torch.int32, device="cuda")
        q1, k1 = glc.qk_norm_fwd(dev["q"][:, t:t + 1], dev["k"][:, t:t + 1], cos=cc, sin=cs, positions=pos, norm="l2")
        assert torch.equal(q1, qn[:, t:t + 1]) and torch.equal(k1, kn[:, t:t + 1])
        o1 = glc.delta_step(q1, k1, cv[:, t:t + 1], cg[:, t:t + 1], cb[:, t:t + 1], pool)
        a = o1.double().cpu().numpy()
        assert (np.abs(a - ro[:, t:t + 1]) <= 2.0 ** -14 * size + ULP[dtype] * np.abs(ro[:, t:t + 1])).all()
    dqn, dkn, *_ = glc.delta_bwd(qn, kn, cv, cg, cb, cdo)
    dq, dk, _, _ = glc.qk_norm_bwd(dev["q"], dev["k"], dqn, dkn, cos=cc, sin=cs, norm="l2")
    want = delta.bwd(qn, kn, v, gate, beta, do, D ** -0.5)
    for a, n, d in ((dq, "q", want["dq"]), (dk, "k", want["dk"])):
        rd, _ = delta.head_norm_bwd(x[n], d, None, cos, sin, norm="l2")
        a = a.double().cpu().numpy()
        tol = 2.0 ** -7 if dtype == BF else 2.0 ** -12
        assert np.linalg.norm(a - rd) <= tol * np.linalg.norm(rd)
