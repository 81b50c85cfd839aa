"""The gated delta rule beside infinities and NaN in places that its results do not depend on."""
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def operands(B, T, H, Hqk, K, V, dtype, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    norm = torch.nn.functional.normalize
    q, k = (norm(r(B, T, Hqk, K), dim=-1).to(dtype) for _ in range(2))
    return dict(q=q, k=k, v=r(B, T, H, V).to(dtype), g=-r(B, T, H).abs() / 4, beta=r(B, T, H).sigmoid(),
                do=r(B, T, H, V).to(dtype))


def forward(x, seg, n):
    return glc.delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 1.0, seg, None, True, n_seqs=n, poison=True)


def backward(x, seg, n):
    return glc.delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], 1.0, seg, n_seqs=n, poison=True)[:5]


@pytest.mark.parametrize("last", [1, 6, 17, 48, 63])
@pytest.mark.parametrize("B,T,H,Hqk,K,V,docs,dtype", [
    (6, 64, 4, 2, 128, 128, 0, BF),      # rows of one and a part chunk
    (4, 512, 16, 16, 128, 128, 0, BF),   # tiles made while the chains walk
    (2, 64, 4, 4, 128, 64, 5, BF),       # documents that end inside a row
    (3, 128, 3, 1, 72, 41, 0, BF),       # padded copies
    (3, 64, 2, 2, 24, 40, 3, F32)])
def test_a_short_last_chunk_beside_infinities(cuda_ok, B, T, H, Hqk, K, V, docs, dtype, last):
    """Every other row or document holds infinities and NaN in every operand: bit for bit the others' outputs, states
    and gradients are what they are beside finite values, every time."""
    each = T + last  # tokens of a document
    T = each * max(docs, 1)
    x = operands(B, T, H, Hqk, K, V, dtype, last + K)
    n = B * max(docs, 1)
    doc = (torch.arange(B * T, device="cuda") // each).view(B, T)
    seg = doc.int() if docs else None
    want_o, want_s = forward(x, seg, n)
    want = (want_o, *backward(x, seg, n))
    bad = doc % 2 == 1
    for name, t in x.items():
        t[bad] = INF if name in ("v", "beta") else NAN
        if name in ("q", "do"):
            t[bad & (torch.arange(T, device="cuda") % 3 == 0)] = -INF
    good = ~bad
    for _ in range(40):
        o, s = forward(x, seg, n)
        for a, b in zip((o, *backward(x, seg, n)), want):
            assert torch.equal(a[good], b[good])
        assert torch.equal(s[::2], want_s[::2])
    glc.get_device_error()


PATHS = [
    # B, T, H, Hqk, K, V, dtype, documents of a row, the forward's last launch
    (2, 200, 4, 2, 128, 128, BF, 1, "delta_chain"),
    (4, 576, 16, 16, 128, 64, BF, 1, "delta_overlap"),
    (2, 300, 2, 2, 64, 128, BF, 2, "delta_chain"),
    (2, 200, 4, 1, 72, 41, BF, 1, "delta_unpad"),
    (2, 48, 2, 2, 128, 128, BF, 1, "delta_scan"),
    (2, 130, 2, 1, 200, 136, BF, 1, "delta_scan"),
    (2, 133, 4, 2, 24, 40, F32, 1, "delta_scan")]


@pytest.mark.parametrize("name", ["g", "beta"])
@pytest.mark.parametrize("where", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("B,T,H,Hqk,K,V,dtype,docs,last", PATHS)
def test_nan_in_a_gate_or_a_writing_strength(cuda_ok, B, T, H, Hqk, K, V, dtype, docs, last, where, name):
    """Of one token and head: NaN from it on in that head of the document, in the gradients of all that it enters, and
    nowhere else but in the same chunk of 64 tokens; on every path."""
    x = operands(B, T, H, Hqk, K, V, dtype, 3)
    end = T // docs  # of the document, from token 0
    at = int(where * (end - 1))
    seg = (torch.arange(T, device="cuda") // end).clamp(max=docs - 1).int().expand(B, T).contiguous() if docs > 1 else None
    o0, s0 = forward(x, seg, B * docs)
    grads0 = backward(x, seg, B * docs)
    x[name][0, at, 0] = NAN
    with glc.LaunchTimer(8) as t:
        o, s = forward(x, seg, B * docs)
    assert t.labels[-1] == last
    before, after = at // 64 * 64, min(end, at // 64 * 64 + 64)  # its chunk
    nan = lambda a: bool(torch.isnan(a).all())

    def rest(a, b, heads=1):  # rows, documents and heads that the value does not enter
        assert torch.equal(a[1:], b[1:]) and torch.equal(a[0, end:], b[0, end:])
        assert torch.equal(a[0, :, heads:], b[0, :, heads:])

    assert nan(o[0, at:end, 0]) and nan(s[0, 0]) and torch.equal(o[0, :before, 0], o0[0, :before, 0])
    rest(o, o0)
    assert torch.equal(s[1:], s0[1:]) and torch.equal(s[0, 1:], s0[0, 1:])
    dq, dk, dv, dg, dbeta = got = backward(x, seg, B * docs)
    for a, b in zip(got, grads0):
        rest(a, b)
    assert nan(dq[0, at:end, 0]) and torch.equal(dq[0, :before, 0], grads0[0][0, :before, 0])
    assert nan(dv[0, :at + (name == "beta"), 0]) and torch.equal(dv[0, after:end, 0], grads0[2][0, after:end, 0])
    assert nan(dk[0, :end, 0]) and nan(dg[0, :end, 0])
    others = [i for i in range(end) if name == "g" or i != at]  # b_t's own gradient is of what it is multiplied with
    assert nan(dbeta[0, others, 0])
    glc.get_device_error()


@pytest.mark.parametrize("dtype,K,V,T", [(BF, 128, 128, 1), (F32, 40, 24, 5)])
@pytest.mark.parametrize("name", ["g", "beta"])
def test_nan_in_a_step(cuda_ok, dtype, K, V, T, name):
    x = operands(3, T, 2, 2, K, V, dtype, 4)
    x[name][1, T // 2, 1] = NAN
    pool = torch.randn(3, 2, K, V, device="cuda")
    o = glc.delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], pool, poison=False)
    bad = torch.zeros(3, T, 2, dtype=torch.bool, device="cuda")
    bad[1, T // 2:, 1] = True
    assert torch.equal(torch.isnan(o), bad[..., None].expand_as(o))
    assert torch.equal(torch.isnan(pool), bad.any(1)[..., None, None].expand_as(pool))


@pytest.mark.parametrize("B,T,H,Hqk,K,V,dtype,docs,last", PATHS)
def test_how_far_an_infinity_reaches(cuda_ok, B, T, H, Hqk, K, V, dtype, docs, last):
    """One in a token's v: the tokens behind it, and of those before it at most its chunk of 64 (token by token: none)."""
    x = operands(B, T, H, Hqk, K, V, dtype, 5)
    end = T // docs
    at = int(0.4 * (end - 1))
    seg = (torch.arange(T, device="cuda") // end).clamp(max=docs - 1).int().expand(B, T).contiguous() if docs > 1 else None
    want, states = forward(x, seg, B * docs)
    x["v"][0, at, 0, V // 2] = INF
    o, s = forward(x, seg, B * docs)
    clean = torch.ones(B, T, H, dtype=torch.bool, device="cuda")
    clean[0, at if last == "delta_scan" else at // 64 * 64:end, 0] = False
    assert torch.equal(o[clean], want[clean])
    assert not torch.isfinite(o[0, at:end, 0, V // 2]).any()
    assert torch.equal(s[1:], states[1:]) and torch.equal(s[0, 1:], states[0, 1:])
    columns = [c for c in range(V) if c != V // 2]  # they do not see each other
    assert torch.equal(o[..., columns], want[..., columns]) and torch.equal(s[..., columns], states[..., columns])
    glc.get_device_error()
