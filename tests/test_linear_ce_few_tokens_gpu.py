"""The loss and the gradient of a handful of tokens, where no other token's error
averages one out, against 64 bits.

Tolerances, element by element, with S = sum |G| |w| (dx) or sum |G| |x| (dw) of
the definition's own G = (p - [v = target]) dloss: the entry at the target keeps
its accuracy where p is near 1, so S has no p + 1 in it.  bf16: a logit's sum in
the tensor core is within 2e-5 of the largest logit (up to 20 here), so G is
within 4e-4 of itself; two bf16 parts of it leave 2^-16; the result is rounded
once, 2^-8 of itself.  One bf16 for G, or p - 1 from a logit with that error, is
well outside.  fp32: sums restart every 64 products, four truncated steps of
the large parts (4 * 2^-23 of a chunk's sum) and then up to 33 rounded sums
(33 * 2^-24): 2.5e-6 of a logit of up to 20 in G, 5e-5, and the same 2.5e-6 once
more in the products."""
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu


def data(N, D, V, dtype, seed, pull):
    """Tokens whose target's logit is `pull` above its noise."""
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    w = (2 * D ** -0.5 * torch.randn(V, D, generator=g)).to(dtype)
    t = torch.randint(0, V, (N,), generator=g)
    near = w[t].float()
    x = torch.randn(N, D, generator=g) + pull * near / near.square().sum(1, keepdim=True)
    dl = (0.5 + torch.rand(N, generator=g)) * torch.where(torch.rand(N, generator=g) < 0.5, -1.0, 1.0)
    return [a.cuda() for a in (x.to(dtype), w, t, dl)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,D,V", [(1, 1072, 17911), (1, 1392, 142), (2, 112, 235), (3, 33, 300), (5, 32, 661),
                                   (16, 520, 2000), (63, 64, 1003), (64, 2100, 500)])
@pytest.mark.parametrize("pull", [0.0, 7.0, 14.0])
def test_gradients_of_few_tokens(cuda_ok, N, D, V, dtype, pull):
    x, w, t, dl = data(N, D, V, dtype, N + D + V, pull)
    if N > 2:
        t[1] = -100
    xd, wd = x.double(), w.double()
    z = xd @ wd.T
    assert float(z.abs().max()) < 30  # 20 and some noise: the tolerances above
    lse = torch.logsumexp(z, 1).float()
    dx, dw = glc.linear_ce_bwd(x, w, t, lse, dl)
    hit = torch.zeros_like(z)
    hit[torch.arange(N), t.clamp(min=0)] = 1
    # p - 1 without cancellation: expm1 at the target
    G = torch.where(hit > 0, torch.expm1(z - lse.double()[:, None]), (z - lse.double()[:, None]).exp())
    G = G * torch.where(t < 0, 0.0, dl.double())[:, None]
    for got, ref, S in ((dx, G @ wd, G.abs() @ wd.abs()), (dw, G.T @ xd, G.abs().T @ xd.abs())):
        if dtype == torch.bfloat16:
            tol = 2.0 ** -8 * (1 + 2.0 ** -8) * ref.abs() + (4e-4 + 2.0 ** -16) * S
        else:
            tol = 5.25e-5 * S
        assert bool(((got.double() - ref).abs() <= tol + 1e-30).all())
    assert torch.all(dx[t < 0] == 0)
    again = glc.linear_ce_bwd(x, w, t, lse, dl)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,D,V", [(1, 1072, 17911), (1, 80, 1618), (2, 1384, 143), (3, 33, 300), (2, 888, 1050),
                                   (16, 520, 2000), (40, 64, 1003), (64, 2100, 500)])
@pytest.mark.parametrize("pull", [0.0, 7.0, 14.0])
def test_losses_of_few_tokens(cuda_ok, N, D, V, dtype, pull):
    """An error of the logits moves the loss by (1 - p) of itself: the target's own
    logit is within 2^-24 of itself, the others' sums are chunks of 32 truncated
    steps, 32 * 2^-23 of the largest logit, joined by up to 5 rounded ones.  With
    the exponentials' own 3e-6 that is (1 - p) (5e-6 top + 3e-6), and a few
    roundings of the loss itself."""
    x, w, t, _ = data(N, D, V, dtype, N + D + V, pull)
    if N > 2:
        t[1] = -100
    loss, lse = glc.linear_ce_fwd(x, w, t)
    z = x.double() @ w.double().T
    top = z.abs().amax(1)
    at = t.clamp(min=0)[:, None]
    zt = z.gather(1, at)[:, 0]
    others = torch.logsumexp(z.scatter(1, at, -float("inf")), 1)
    want = torch.where(t < 0, 0.0, torch.nn.functional.softplus(others - zt, threshold=1000))
    rest = torch.sigmoid(others - zt)  # 1 - p
    assert bool(((loss.double() - want).abs() <= rest * (5e-6 * top + 3e-6) + 2.0 ** -22 * want).all())
    exact = torch.logsumexp(z, 1)
    share = torch.where(t < 0, 1.0, rest)
    assert bool(((lse.double() - exact).abs() <= share * (5e-6 * top + 3e-6) + 2.0 ** -22 * (1 + top)).all())
    assert torch.all(loss[t < 0] == 0)
