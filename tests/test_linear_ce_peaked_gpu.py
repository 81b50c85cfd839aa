"""Losses of tokens whose softmax is nearly one token, at logits of any size.

Every row n of x holds one value c_n, in a column of its own in which w is 1 at
the target and -1 elsewhere: the logits are c_n and -c_n exactly (one product
each), and in closed form  loss = log1p((V - 1) e^(-2 c)),  lse = c + loss.

Tolerances.  The sum of exponentials is 1 at the largest logit plus terms of
e^(-2c), each within 2e-6 of itself (an exponent of up to 104 rounded to fp32,
104 * 2^-24 = 6e-6 of a term that small, and less for larger ones; sums of up
to 100 terms in a row, 6e-6): 2e-5 of the loss.  The sum is rounded at the size
of 1 a few times (2^-22), and lse once more at its own size (2^-24)."""
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu

N, V = 48, 1003


def peaked(dtype, D=64):
    """x, w, target, c: one target for each row, spread over the vocabulary."""
    t = torch.arange(N) * 911 % V
    w = torch.full((V, D), -1.0)
    w[t, torch.arange(N)] = 1.0
    c = torch.logspace(-0.3, 4.5, N).to(dtype).double()  # 0.5 .. 31600
    x = torch.zeros(N, D, dtype=torch.float64)
    x[torch.arange(N), torch.arange(N)] = c
    return x.to(dtype).cuda(), w.to(dtype).cuda(), t.cuda(), c.cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_loss_of_a_foreseen_token(cuda_ok, dtype):
    x, w, t, c = peaked(dtype)
    loss, lse = glc.linear_ce_fwd(x, w, t)
    want = torch.log1p((V - 1) * torch.exp(-2 * c))
    assert torch.all(loss >= 0)
    assert torch.all(loss[c > 100] == 0)  # nothing beside the target
    assert bool(((loss.double() - want).abs() <= 2e-5 * want + 2.0 ** -22).all())
    assert bool(((lse.double() - c - want).abs() <= 2e-5 * want + 2.0 ** -22 + 2.0 ** -24 * lse.double().abs()).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_from_the_forwards_own_lse(cuda_ok, dtype):
    """p of a row sums to 1, so G sums to 0: in a column in which all of w is -1,
    dx is minus that sum.  lse is rounded at its own size (2^-24 of it is the same
    share of p), the two bf16 parts of G leave 2^-16 of each, and the sum of V / 16
    truncated steps 63 * 2^-23 of sum |G| <= 2."""
    x, w, t, c = peaked(dtype)
    _, lse = glc.linear_ce_fwd(x, w, t)
    dx, _ = glc.linear_ce_bwd(x, w, t, lse, torch.ones(N, device="cuda"))
    bound = 2.0 ** -24 * lse.double().abs() + 2e-5 + 2 * (2.0 ** -16 + 63 * 2.0 ** -23)
    assert bool((dx[:, N:].double().abs() <= bound[:, None]).all())
