"""Layer norm gradients of rows far off centre, against oracle/lm.py from the same
row statistics.

dx = r (a - mean(a) - n mean(a n)) with n = (x - m) r: the difference x - m is one
rounding of itself, so every term keeps its own accuracy however large m is.  A
row's sums run over at most 64 values in sequence, then a tree: 80 * 2^-24 of the
sum of magnitudes covers them and the roundings of the terms.  Element by element
that is 80 * 2^-24 r (|a| + mean|a| + |n| mean|a n|), plus the rounding of dx's
own type, 2^-8 of it for bf16."""
import numpy as np
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
from oracle import lm

pytestmark = pytest.mark.gpu

CASES = [(torch.float32, off, D) for off in (0.0, 30.0, 1000.0, 30000.0) for D in (8, 64, 512, 1111, 2048, 8192, 9000)]
CASES += [(torch.bfloat16, off, D) for off in (0.0, 30.0, 300.0) for D in (64, 1334, 1335, 2048)]


@pytest.mark.parametrize("dtype,off,D", CASES)
def test_dx_of_rows_far_off_centre(cuda_ok, dtype, off, D):
    g = torch.Generator("cpu")
    g.manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=g)
    rows = 37
    x = (r(rows, D) + off * torch.where(r(rows, 1) < 0, -1.0, 1.0)).to(dtype)
    mean = x.double().mean(1)
    std = ((x.double() - mean[:, None]) ** 2).mean(1).add(1e-5).sqrt()
    n = (x.double() - mean[:, None]) / std[:, None]
    dy, w = (r(rows, D) + n).to(dtype), 1 + 0.5 * r(D)  # a part of dy goes with the normalised row
    mean, rstd = mean.float(), (1 / std).float()
    got = glc.layer_norm_bwd(x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), dy.cuda())
    want = lm.layer_norm_bwd(x, w, mean, rstd, dy)
    f = lambda t: t.double().numpy()
    rr = f(rstd)[:, None]
    nn, a = (f(x) - f(mean)[:, None]) * rr, f(dy) * f(w)
    avg = lambda v: np.abs(v).mean(1, keepdims=True)
    tol = 80 * 2.0 ** -24 * rr * (np.abs(a) + avg(a) + np.abs(nn) * avg(a * nn))
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want[0])
    assert bool((np.abs(f(got[0].cpu()) - want[0]) <= tol).all())
