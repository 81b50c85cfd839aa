"""GPU parity of linear_ce_fwd / linear_ce_bwd against the fp64 definition
(oracle/lm.py; for the larger cases the same formulas in torch float64).

Tolerances.  Logits: D bf16 products are exact and summed in fp32, 16 at a
time; a truncated running sum over D / 16 <= 160 steps is within
160 * 2^-23 = 2e-5 of the largest partial sum, so lse and loss are held to
2e-5 of the largest logit (+ 1).  fp32 operands lose nothing to their split and
their sums restart every 256 products: the same bound.
Gradients, element by element: bf16 rounds each G to within 2^-8 of itself and
the result once more, 2^-8 sum |G| |w| + 2^-8 |b|, plus 2e-5 S for the
exponent's error at logits up to 20, where S is the sum of the magnitudes of
the terms, (p + [v = target]) |dloss| |w|: an error of the exponent is one of p,
also where p - 1 cancels.  fp32: a chunk of 16 truncated steps (2e-6), up to
160 rounded sums of chunks (1e-5 at most), the exponent's error (1e-6 of a
logit of up to 20): 3e-5 S."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
from oracle import lm

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -8


def data(N, D, V, dtype, seed, skip=0.1):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    w = (2 * D ** -0.5 * torch.randn(V, D, generator=g)).to(dtype)
    t = torch.randint(0, V, (N,), generator=g)
    x = (torch.randn(N, D, generator=g) + 2 * torch.rand(N, 1, generator=g) * w[t].float()).to(dtype)
    t = torch.where(torch.rand(N, generator=g) < skip, -100, t)
    return x, w, t, torch.randn(N, generator=g)


def check_fwd(x, w, t, got):
    xd, wd = x.cuda().double(), w.cuda().double()
    z = xd @ wd.T
    top = float(z.abs().max()) + 1
    lse = torch.logsumexp(z, 1)
    tc = t.cuda()
    loss = torch.where(tc < 0, 0.0, lse - z.gather(1, tc.clamp(min=0)[:, None])[:, 0])
    assert float((got[1].double() - lse).abs().max()) <= 2e-5 * top
    assert float((got[0].double() - loss).abs().max()) <= 2e-5 * top
    assert torch.all(got[0][tc < 0] == 0)
    return lse.float()


def check_bwd(x, w, t, lse, dl, got):
    dx, dw = got
    assert dx.dtype == x.dtype and dw.dtype == w.dtype and dx.shape == x.shape and dw.shape == w.shape
    xd, wd, tc = x.cuda().double(), w.cuda().double(), t.cuda()
    p = (xd @ wd.T - lse.cuda().double()[:, None]).exp()
    hit = torch.zeros_like(p)
    hit[torch.arange(len(tc)), tc.clamp(min=0)] = 1
    scale = torch.where(tc < 0, 0.0, dl.cuda().double())[:, None]
    G, terms = (p - hit) * scale, (p + hit) * scale.abs()
    del p, hit
    for a, ref, size, S in ((dx, G @ wd, G.abs() @ wd.abs(), terms @ wd.abs()),
                            (dw, G.T @ xd, G.abs().T @ xd.abs(), terms.T @ xd.abs())):
        tol = ULP * size + 2e-5 * S + ULP * ref.abs() if x.dtype == torch.bfloat16 else 3e-5 * S
        assert bool(((a.double() - ref).abs() <= tol + 1e-30).all())
    assert torch.all(dx[tc < 0] == 0)


CASES = [
    # N, D, V, dtype
    (1, 8, 1, torch.bfloat16), (1, 64, 300, torch.bfloat16), (3, 32, 100, torch.bfloat16),
    (300, 64, 257, torch.bfloat16), (256, 256, 512, torch.bfloat16), (1000, 520, 1003, torch.bfloat16),
    (129, 1000, 5000, torch.bfloat16), (2, 2048, 999, torch.bfloat16), (50, 33, 77, torch.bfloat16),
    (7, 1, 5, torch.bfloat16), (600, 200, 20000, torch.bfloat16), (64, 512, 30011, torch.bfloat16),
    (1, 8, 1, torch.float32), (5, 64, 100, torch.float32), (130, 77, 129, torch.float32),
    (256, 256, 384, torch.float32), (301, 520, 2000, torch.float32), (2, 1030, 700, torch.float32),
    (40, 16, 20011, torch.float32),
    # many tokens, little else: dw's sum over the tokens is cut
    (4655, 48, 423, torch.bfloat16), (3001, 33, 300, torch.bfloat16), (2600, 40, 301, torch.float32),
]


@pytest.mark.parametrize("N,D,V,dtype", CASES)
def test_against_definition(cuda_ok, N, D, V, dtype):
    x, w, t, dl = data(N, D, V, dtype, N + D + V)
    c = [a.cuda() for a in (x, w, t)]
    got = glc.linear_ce_fwd(*c)
    lse = check_fwd(x, w, t, got)
    if N * V <= 300000:  # the definition by another hand
        loss, ref = lm.linear_ce_fwd(x, w, t)
        assert np.abs(got[0].cpu().numpy() - loss).max() <= 2e-5 * (np.abs((x.double() @ w.double().T).numpy()).max() + 1)
    grads = glc.linear_ce_bwd(*c, lse, dl.cuda())
    check_bwd(x, w, t, lse, dl, grads)
    again = glc.linear_ce_bwd(*c, lse, dl.cuda())
    assert torch.equal(grads[0], again[0]) and torch.equal(grads[1], again[1])  # a fixed order of sums
    assert torch.equal(got[0], glc.linear_ce_fwd(*c)[0])
    glc.get_device_error()


@pytest.mark.parametrize("dtype,N", [(torch.bfloat16, 70001), (torch.float32, 22000)])
def test_a_vocabulary_in_several_pieces(cuda_ok, dtype, N):
    """So many tokens that G's workspace holds 2048 columns at a time: 3 pieces,
    the last one ragged; dx is summed over them."""
    x, w, t, dl = data(N, 24, 4500, dtype, 5)
    need = glc.load().linear_ce_bwd_workspace_size(N, 24, 4500, glc._dtype_code(x))
    parts = 3 if dtype == torch.float32 else 1
    assert need < parts * 2 * N * 4500  # not the whole of G
    c = [a.cuda() for a in (x, w, t)]
    lse = check_fwd(x, w, t, glc.linear_ce_fwd(*c))
    check_bwd(x, w, t, lse, dl, glc.linear_ce_bwd(*c, lse, dl.cuda()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_is_the_difference_of_the_loss(cuda_ok, dtype):
    """Directional central differences of the loss itself: the loss is within
    2e-5 * 20 and the step 0.05, so the quotient is within 1e-2 plus the third
    derivative's share; the gradient's own rounding is far below."""
    x, w, t, _ = data(40, 64, 200, torch.float32, 6, skip=0.2)
    x, w = x.to(dtype).float(), w.to(dtype).float()
    g = torch.Generator("cpu")
    g.manual_seed(1)
    ux, uw = torch.randn(40, 64, generator=g) / 64, torch.randn(200, 64, generator=g) / 64
    f = lambda e: float(glc.linear_ce_fwd((x + e * ux).cuda(), (w + e * uw).cuda(), t.cuda())[0].double().sum())
    c = [x.to(dtype).cuda(), w.to(dtype).cuda(), t.cuda()]
    _, lse = glc.linear_ce_fwd(*c)
    dx, dw = glc.linear_ce_bwd(*c, lse, torch.ones(40, device="cuda"))
    slope = float((dx.double().cpu() * ux).sum() + (dw.double().cpu() * uw).sum())
    assert abs((f(0.05) - f(-0.05)) / 0.1 - slope) <= 1e-2 * (1 + abs(slope))


def test_no_token_scored(cuda_ok):
    x, w, _, dl = data(20, 64, 300, torch.bfloat16, 7)
    t = torch.full((20,), -1)
    loss, lse = glc.linear_ce_fwd(x.cuda(), w.cuda(), t.cuda())
    dx, dw = glc.linear_ce_bwd(x.cuda(), w.cuda(), t.cuda(), lse, torch.full((20,), float("nan"), device="cuda"))
    assert torch.all(loss == 0) and torch.isfinite(lse).all() and torch.all(dx == 0) and torch.all(dw == 0)


def test_no_tokens(cuda_ok):
    w = torch.ones(30, 16, device="cuda", dtype=torch.bfloat16)
    x, t = w[:0], torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = glc.linear_ce_fwd(x, w, t)
    dx, dw = glc.linear_ce_bwd(x, w, t, lse, loss)
    assert loss.shape == (0,) and dx.shape == (0, 16) and torch.all(dw == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_logits(cuda_ok, dtype):
    """Logits of +-30000: the softmax is one token, nothing overflows."""
    V, D = 500, 64
    w = torch.zeros(V, D)
    w[:, 0] = torch.linspace(-300, 300, V)
    x = torch.zeros(3, D)
    x[:, 0] = torch.tensor([100.0, -100.0, 0.0])
    x, w, t = x.to(dtype), w.to(dtype), torch.tensor([V - 1, V - 1, 3])
    c = [a.cuda() for a in (x, w, t)]
    lse = check_fwd(x, w, t, glc.linear_ce_fwd(*c))
    check_bwd(x, w, t, lse, torch.ones(3), glc.linear_ce_bwd(*c, lse, torch.ones(3, device="cuda")))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first,count", [(0, 64), (64, 64), (300, 1), (0, 500)])
def test_a_nan_among_the_logits_is_not_lost(cuda_ok, dtype, first, count):
    """Also where it is all that an epilogue has seen of a row so far."""
    x, w, t, _ = data(40, 64, 500, dtype, 11, skip=0)
    w[first:first + count] = float("nan")
    loss, lse = glc.linear_ce_fwd(x.cuda(), w.cuda(), t.cuda())
    assert torch.isnan(loss).all() and torch.isnan(lse).all()


def test_target_out_of_range_is_reported(cuda_ok):
    x, w, t, dl = data(20, 64, 300, torch.bfloat16, 8, skip=0)
    t[4] = 300
    c = [a.cuda() for a in (x, w, t)]
    loss, lse = glc.linear_ce_fwd(*c)
    with pytest.raises(glc.GlacoreError) as e:
        glc.get_device_error()
    assert e.value.status == glc.ERR_INDEX and loss[4] == 0
    dx, dw = glc.linear_ce_bwd(*c, lse, dl.cuda())
    with pytest.raises(glc.GlacoreError):
        glc.get_device_error()
    skipped = t.clone()
    skipped[4] = -1
    check_bwd(x, w, skipped, lse, dl, (dx, dw))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_misaligned_x_and_other_stream(cuda_ok, dtype):
    x, w, t, dl = data(33, 64, 200, dtype, 9)
    wide = torch.zeros(33, 80, dtype=dtype, device="cuda")
    wide[:, 8:72] = x.cuda()
    off = torch.zeros(33, 72, dtype=dtype, device="cuda")  # a row stride, and rows that start off 16 bytes
    off[:, 1:65] = x.cuda()
    odd = torch.zeros(33 * 64 + 1, dtype=dtype, device="cuda")[1:].view(33, 64)
    odd.copy_(x)
    lse = check_fwd(x, w, t, glc.linear_ce_fwd(x.cuda(), w.cuda(), t.cuda()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for v in (wide[:, 8:72], off[:, 1:65], odd):
        with torch.cuda.stream(side):
            got = glc.linear_ce_fwd(v, w.cuda(), t.cuda())
            grads = glc.linear_ce_bwd(v, w.cuda(), t.cuda(), lse, dl.cuda())
        side.synchronize()
        check_fwd(x, w, t, got)
        check_bwd(x, w, t, lse, dl, grads)


def test_refusals(cuda_ok):
    x = torch.zeros(4, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(9, 16, device="cuda", dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    loss, lse = glc.linear_ce_fwd(x, w, t)
    for bad in ((x, w.float(), t), (x, w[:, :8], t), (x, w, t[:3]), (x.view(2, 2, 16), w, t), (x.cpu(), w, t)):
        with pytest.raises(ValueError):
            glc.linear_ce_fwd(*bad)
    with pytest.raises(TypeError):
        glc.linear_ce_fwd(x, w, t.int())
    with pytest.raises(TypeError):
        glc.linear_ce_fwd(x.half(), w.half(), t)
    with pytest.raises(ValueError):
        glc.linear_ce_bwd(x, w, t, lse[:2], lse)
    lib, st = glc.load(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    need = lib.linear_ce_fwd_workspace_size(4, 16, 9, glc.BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    P = glc._ptr
    call = lambda x=P(x), w=P(w), t=P(t), N=4, D=16, V=9, xs=0, dt=glc.BF16, l=P(loss), s=P(lse), k=P(ws), n=need: \
        lib.linear_ce_fwd(x, w, t, N, D, V, xs, dt, l, s, k, n, st)
    assert call() == glc.OK
    for kw in (dict(x=None), dict(w=None), dict(t=None), dict(N=-1), dict(D=0), dict(V=0), dict(xs=8), dict(xs=20),
               dict(dt=5), dict(l=None), dict(s=None), dict(x=ctypes.c_void_p(x.data_ptr() + 2))):
        assert call(**kw) == glc.ERR_INVALID_ARG, kw
    for kw in (dict(k=None), dict(n=need - 1), dict(k=ctypes.c_void_p(ws.data_ptr() + 16))):
        assert call(**kw) == glc.ERR_WORKSPACE, kw
    torch.cuda.synchronize()
    glc.get_device_error()
