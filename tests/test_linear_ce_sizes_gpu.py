"""linear_ce where both gradients take several rounds of the pairs of CTAs, on both
sides of the number of tokens up to which they are treated apart, and with one
token scored among many; and how far its long sums may drift."""
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
from test_linear_ce_gpu import check_bwd, check_fwd, data

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,D,V,dtype", [
    (3000, 2048, 12000, torch.bfloat16), (2100, 1000, 9000, torch.float32),
    (63, 256, 700, torch.bfloat16), (64, 256, 700, torch.bfloat16), (65, 256, 700, torch.bfloat16),
    (64, 31, 20000, torch.bfloat16), (64, 31, 2000, torch.float32), (65, 31, 2000, torch.float32),
    # few tokens of a vocabulary in two pieces, the last one ragged
    (64, 16, 2200001, torch.bfloat16), (64, 16, 1500001, torch.float32),
    (17, 4100, 257, torch.bfloat16), (33, 8, 1, torch.bfloat16), (33, 8, 1, torch.float32),
])
def test_against_definition(cuda_ok, N, D, V, dtype):
    x, w, t, dl = data(N, D, V, dtype, N + D + V)
    c = [a.cuda() for a in (x, w, t)]
    got = glc.linear_ce_fwd(*c)
    lse = check_fwd(x, w, t, got)
    grads = glc.linear_ce_bwd(*c, lse, dl.cuda())
    check_bwd(x, w, t, lse, dl, grads)
    again = glc.linear_ce_bwd(*c, lse, dl.cuda())
    assert torch.equal(grads[0], again[0]) and torch.equal(grads[1], again[1])
    # and from the forward's own lse, which is within 2^-20 of its size
    check_bwd(x, w, t, got[1], dl, glc.linear_ce_bwd(*c, got[1], dl.cuda()))
    glc.get_device_error()


@pytest.mark.parametrize("N", [40, 400])
def test_one_token_scored(cuda_ok, N):
    x, w, t, dl = data(N, 96, 500, torch.bfloat16, 12, skip=0)
    t[torch.arange(N) != 11] = -1
    c = [a.cuda() for a in (x, w, t)]
    lse = check_fwd(x, w, t, glc.linear_ce_fwd(*c))
    check_bwd(x, w, t, lse, dl, glc.linear_ce_bwd(*c, lse, dl.cuda()))


@pytest.mark.parametrize("dtype,bound", [(torch.bfloat16, 1.25e-6), (torch.float32, 1.1e-6)])
def test_long_sums_do_not_drift(cuda_ok, dtype, bound):
    """All products positive: a logit's sum grows steadily and the tensor core's
    truncation has one sign.  bf16: sums restart every 512 products, 32 steps of
    16; step k of a restart loses half a unit of the last place of k / 32 of the
    chunk on average, 16.5 * 2^-24 = 1e-6 of it in all, and 4 rounded sums of chunks
    4 * 2^-24 more.  (One sum over all 2048 would lose four times that.)  fp32:
    restarts every 4 steps, 2.5 * 2^-24, and 32 rounded sums whose parts grow
    likewise, 16 * 2^-24 at most.  Mean over the tokens, of lse's size."""
    g = torch.Generator("cuda")
    g.manual_seed(3)
    x = torch.rand(100, 2048, generator=g, device="cuda").to(dtype)
    w = (torch.rand(600, 2048, generator=g, device="cuda") / 64).to(dtype)
    t = torch.randint(0, 600, (100,), generator=g, device="cuda")
    _, lse = glc.linear_ce_fwd(x, w, t)
    want = torch.logsumexp(x.double() @ w.double().T, 1)
    assert float(((lse.double() - want).abs() / want).mean()) <= bound
