"""GPU parity of layer_norm_fwd / layer_norm_bwd against oracle/lm.py.

The kernels compute in fp32 from exact input values and round once.  fp32
results, max|a-b| / max|b|: a row sum of up to 20000 values runs over at most
64 values in sequence, then a tree, so its error is below 80 * 2^-24 = 5e-6 of
the sum of magnitudes; a handful of further roundings: 2e-5.  A bf16 value is
within half an ulp, at most 2^-8 of itself (8 significant bits), of such a
result, element by element.  Weight gradients add rows of either sign, so their
error, relative to sums of magnitudes as above, is up to sqrt(rows) larger
relative to the result: 1e-4 for up to 8192 rows."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
from oracle import lm

pytestmark = pytest.mark.gpu

TOL, TOL_STATS, TOL_DW = 2e-5, 2e-5, 1e-4
ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def rel(a, b):
    a = a.detach().to("cpu", torch.float64).numpy()
    return float(np.abs(a - b).max() / max(np.abs(b).max(), 1e-30)) if b.size else 0.0


def close(a, b, scale=None):
    """Every element within the fp32 tolerance (of the largest value, or of
    `scale`) plus the rounding of its own type."""
    tol = TOL * (np.abs(b).max() if scale is None else scale) + ULP[a.dtype] * np.abs(b)
    return bool((np.abs(a.detach().to("cpu", torch.float64).numpy() - b) <= tol).all())


def data(rows, D, dtype, seed):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (r(rows, D) * (1 + r(D).abs()) + 0.3 * r(D)).to(dtype)
    return x, r(rows, D).to(dtype), 1 + 0.5 * r(D), r(D)


CASES = [
    # rows, D, dtype: rows shared by a warp, rows of one warp, of several warps, longer than registers hold
    (1, 1, torch.float32), (3, 2, torch.bfloat16), (33, 8, torch.bfloat16), (7, 24, torch.bfloat16),
    (1000, 64, torch.float32), (5, 100, torch.float32), (130, 256, torch.bfloat16), (1, 2048, torch.bfloat16),
    (8192, 2048, torch.bfloat16), (5000, 2048, torch.float32), (77, 1111, torch.float32),
    (2000, 1111, torch.bfloat16), (9, 4095, torch.bfloat16), (650, 4096, torch.float32), (3, 8192, torch.bfloat16),
    (40, 8191, torch.float32), (5, 8193, torch.float32), (70, 20000, torch.bfloat16), (2, 20001, torch.float32),
    # rows on 4-byte addresses, and between them
    (33, 30, torch.bfloat16), (400, 1334, torch.bfloat16), (3, 4098, torch.bfloat16), (7, 8190, torch.bfloat16),
    (31, 4097, torch.bfloat16), (700, 8191, torch.bfloat16), (600, 1024, torch.float32), (2500, 17, torch.bfloat16),
]


@pytest.mark.parametrize("rows,D,dtype", CASES)
def test_against_oracle(cuda_ok, rows, D, dtype):
    x, dy, w, b = data(rows, D, dtype, rows + D)
    y, mean, rstd = glc.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), 1e-3)
    ry, rmean, rrstd = lm.layer_norm_fwd(x, w, b, 1e-3)
    assert mean.shape == rstd.shape == (rows,)
    assert np.abs(mean.cpu().double().numpy() - rmean).max() <= TOL_STATS * np.abs(x.double().numpy()).max()
    assert close(y, ry) and rel(rstd, rrstd) <= TOL_STATS
    dx, dw, db = glc.layer_norm_bwd(x.cuda(), w.cuda(), mean, rstd, dy.cuda())
    rdx, rdw, rdb = lm.layer_norm_bwd(x, w, mean, rstd, dy)
    # with D = 1 or 2 the exact dx is (nearly) zero: measured against its terms
    scale = max(np.abs(rdx).max(), (np.abs(dy.double().numpy() * w.double().numpy()) * rrstd[:, None]).max())
    assert close(dx, rdx, scale)
    assert rel(dw, rdw) <= TOL_DW and rel(db, rdb) <= TOL_DW
    again = glc.layer_norm_bwd(x.cuda(), w.cuda(), mean, rstd, dy.cuda())
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))  # a fixed order of sums


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_without_weights(cuda_ok, dtype):
    x, dy, _, _ = data(50, 72, dtype, 5)
    y, mean, rstd = glc.layer_norm_fwd(x.cuda())
    ry, _, _ = lm.layer_norm_fwd(x)
    assert close(y, ry)
    got = glc.layer_norm_bwd(x.cuda(), None, mean, rstd, dy.cuda())
    want = lm.layer_norm_bwd(x, None, mean, rstd, dy)
    assert close(got[0], want[0]) and rel(got[1], want[1]) <= TOL_DW and rel(got[2], want[2]) <= TOL_DW


@pytest.mark.parametrize("stride,offset", [(128, 0), (136, 8), (131, 0), (128, 3), (130, 0), (130, 2), (130, 1)])
def test_strided_and_misaligned_rows(cuda_ok, stride, offset):
    """x and dy as columns of a wider tensor: 16-byte aligned, or not."""
    wide, wide_dy, w, b = data(40, 160, torch.bfloat16, 6)
    flat, flat_dy = wide.reshape(-1).cuda(), wide_dy.reshape(-1).cuda()
    x = flat[offset:].as_strided((40, 64), (stride, 1))
    dy = flat_dy[offset:].as_strided((40, 64), (stride, 1))
    w, b = w[:64].cuda(), b[:64].cuda()
    y, mean, rstd = glc.layer_norm_fwd(x, w, b)
    assert close(y, lm.layer_norm_fwd(x, w, b)[0])
    got, want = glc.layer_norm_bwd(x, w, mean, rstd, dy), lm.layer_norm_bwd(x, w, mean, rstd, dy)
    assert close(got[0], want[0]) and rel(got[1], want[1]) <= TOL_DW and rel(got[2], want[2]) <= TOL_DW


def test_far_off_centre_rows_keep_their_deviation(cuda_ok):
    """mean = 1000 times the deviation: the deviation is taken from the mean,
    not as a difference of two large sums."""
    g = torch.Generator("cpu")
    g.manual_seed(8)
    x = torch.randn(20, 512, generator=g) + 1000
    y, _, _ = glc.layer_norm_fwd(x.cuda(), eps=0.0)
    # x - mean is exact to 2^-24 * 1000 = 6e-5 of a deviation of 1
    assert rel(y, lm.layer_norm_fwd(x, eps=0.0)[0]) <= 2e-4


def test_a_bad_row_stays_alone(cuda_ok):
    x, _, w, b = data(6, 64, torch.float32, 9)
    x[2, 5], x[4, 0] = float("nan"), float("inf")
    y, _, _ = glc.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    good = [0, 1, 3, 5]
    assert torch.isfinite(y[good]).all() and torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    assert close(y[good], lm.layer_norm_fwd(x[good], w, b)[0])


def test_no_rows_and_leading_axes(cuda_ok):
    w = torch.ones(16, device="cuda")
    y, mean, rstd = glc.layer_norm_fwd(torch.zeros(0, 16, device="cuda"), w, w)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = glc.layer_norm_bwd(y, w, mean, rstd, y)
    assert dx.shape == (0, 16) and torch.all(dw == 0) and torch.all(db == 0)
    x = torch.randn(2, 3, 4, 16, device="cuda")
    y, mean, rstd = glc.layer_norm_fwd(x, w)
    assert y.shape == x.shape and mean.shape == (2, 3, 4)
    assert close(y, lm.layer_norm_fwd(x, w)[0])


def test_refusals(cuda_ok):
    x = torch.zeros(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    with pytest.raises(ValueError):
        glc.layer_norm_fwd(x.cpu())
    with pytest.raises(ValueError):
        glc.layer_norm_fwd(x, torch.ones(8, device="cuda"))
    with pytest.raises(TypeError):
        glc.layer_norm_fwd(x.half(), w)
    with pytest.raises(TypeError):
        glc.layer_norm_fwd(x, w.bfloat16())
    with pytest.raises(glc.GlacoreError):
        glc.layer_norm_fwd(x, w, None, -1.0)
    _, mean, rstd = glc.layer_norm_fwd(x, w)
    with pytest.raises(ValueError):
        glc.layer_norm_bwd(x, w, mean, rstd, x[:2])
    lib, st = glc.load(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    dx, dw = torch.empty_like(x), torch.empty(2, 16, device="cuda")
    need = lib.layer_norm_bwd_workspace_size(4, 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    args = [glc._ptr(t) for t in (x, w, mean, rstd, x)]
    outs = [glc._ptr(dx), glc._ptr(dw[0]), glc._ptr(dw[1])]
    assert lib.layer_norm_bwd(*args, 4, 16, 0, 0, glc.F32, *outs, glc._ptr(ws), need - 1, st) == glc.ERR_WORKSPACE
    assert lib.layer_norm_bwd(*args, 4, 16, 8, 0, glc.F32, *outs, glc._ptr(ws), need, st) == glc.ERR_INVALID_ARG
    assert lib.layer_norm_bwd(*args, 4, 0, 0, 0, glc.F32, *outs, glc._ptr(ws), need, st) == glc.ERR_INVALID_ARG
    assert lib.layer_norm_bwd(*args, 4, 16, 0, 0, 7, *outs, glc._ptr(ws), need, st) == glc.ERR_INVALID_ARG
    assert lib.layer_norm_bwd(*args, 4, 16, 0, 0, glc.F32, *outs, glc._ptr(ws), need, st) == glc.OK
