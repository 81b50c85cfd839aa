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
