"""Host-side checks of the layer norm, the step and the linear cross entropy
that need no GPU: bad arguments are refused before any launch, workspaces are
sized as documented."""
import ctypes

import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

A = ctypes.c_void_p(4096)  # an aligned address that no refused call touches
NULL = None


def norm_bwd(lib, x=A, w=A, mean=A, rstd=A, dy=A, rows=4, D=16, xs=0, ys=0, dt=glc.BF16, dx=A, dw=A, db=A, ws=A,
             n=1 << 30):
    return lib.layer_norm_bwd(x, w, mean, rstd, dy, rows, D, xs, ys, dt, dx, dw, db, ws, n, NULL)


def norm_fwd(lib, x=A, w=A, b=A, rows=4, D=16, xs=0, dt=glc.BF16, eps=1e-5, y=A, mean=A, rstd=A):
    return lib.layer_norm_fwd(x, w, b, rows, D, xs, dt, eps, y, mean, rstd, NULL)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(D=0), dict(D=1 << 31), dict(xs=8), dict(dt=3), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(x=NULL), dict(y=NULL), dict(mean=NULL), dict(rstd=NULL)])
def test_norm_fwd_refusals(kw):
    assert norm_fwd(glc.load(), **kw) == glc.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(D=0), dict(xs=8), dict(ys=15), dict(dt=-1), dict(x=NULL),
                                dict(mean=NULL), dict(rstd=NULL), dict(dy=NULL), dict(dx=NULL), dict(dw=NULL),
                                dict(db=NULL)])
def test_norm_bwd_refusals(kw):
    assert norm_bwd(glc.load(), **kw) == glc.ERR_INVALID_ARG


def test_norm_workspace():
    lib = glc.load()
    for rows, D in ((1, 1), (5000, 2048), (3, 20000)):
        need = lib.layer_norm_bwd_workspace_size(rows, D)
        assert need >= 2 * D * 4 and need % (2 * D * 4) == 0
        assert norm_bwd(lib, rows=rows, D=D, n=need - 1) == glc.ERR_WORKSPACE
        assert norm_bwd(lib, rows=rows, D=D, ws=NULL) == glc.ERR_WORKSPACE
        assert norm_bwd(lib, rows=rows, D=D, ws=ctypes.c_void_p(4096 + 16)) == glc.ERR_WORKSPACE
    assert lib.layer_norm_bwd_workspace_size(4, 0) == 0


def step_problem(**over):
    p = glc.Problem(B=3, T=1, H=4, Hqk=2, K=16, V=8, dtype=glc.F32, chunk_size=0, scale=1.0, reserved0=0, q=256, k=512,
                    v=768, g=1024, segment_ids=None, n_seqs=3, initial_state=None, workspace=None, workspace_bytes=0)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,kw", [
    (dict(B=0), {}), (dict(T=-1), {}), (dict(K=257), {}), (dict(V=0), {}), (dict(Hqk=3), {}), (dict(dtype=4), {}),
    (dict(q=None), {}), (dict(g=None), {}), (dict(scale=float("nan")), {}), (dict(q_stride=8), {}), (dict(n_seqs=2), {}),
    (dict(chunk_size=16), {}), (dict(segment_ids=4096), {}), (dict(initial_state=4096), {}),
    ({}, dict(state=NULL)), ({}, dict(o=NULL)), ({}, dict(n_slots=-1)), ({}, dict(n_slots=2, idx=NULL)),
    ({}, dict(state=ctypes.c_void_p(4097))), ({}, dict(idx=ctypes.c_void_p(4098))),
])
@pytest.mark.parametrize("name", ["gla_step", "ssd_step"])
def test_step_refusals(name, over, kw):
    p = step_problem(**over)
    a = dict(state=A, n_slots=9, idx=A, o=A) | kw
    assert getattr(glc.load(), name)(ctypes.byref(p), a["state"], a["n_slots"], a["idx"], a["o"],
                                     NULL) == glc.ERR_INVALID_ARG


def test_step_without_tokens_is_a_no_op():
    p = step_problem(T=0, n_seqs=0, q=None, k=None, v=None, g=None)
    assert glc.load().gla_step(ctypes.byref(p), NULL, 9, NULL, NULL, NULL) == glc.OK


def test_packed_problem_matches_the_structure():
    """The binding's packed form of glacore_problem, field by field."""
    fields = [3, 1, 4, 2, 16, 8, glc.F32, 0, 0.5, 0, 256, 512, 768, 1024, 0, 3, 0, 0, 0, 64, 72, 80]
    p = glc.Problem.from_buffer_copy(glc._PACK.pack(*fields))
    got = [getattr(p, n) or 0 for n, _ in glc.Problem._fields_]
    assert got == fields


def ce_fwd(lib, x=A, w=A, t=A, N=4, D=16, V=9, xs=0, dt=glc.BF16, loss=A, lse=A, ws=A, n=1 << 40):
    return lib.linear_ce_fwd(x, w, t, N, D, V, xs, dt, loss, lse, ws, n, NULL)


def ce_bwd(lib, x=A, w=A, t=A, lse=A, dl=A, N=4, D=16, V=9, xs=0, dt=glc.BF16, dx=A, dw=A, ws=A, n=1 << 40):
    return lib.linear_ce_bwd(x, w, t, lse, dl, N, D, V, xs, dt, dx, dw, ws, n, NULL)


COMMON = [dict(N=-1), dict(N=(1 << 30) + 1), dict(D=0), dict(D=1 << 22), dict(V=0), dict(V=(1 << 30) + 1), dict(xs=8),
          dict(xs=20), dict(dt=2), dict(x=NULL), dict(w=NULL), dict(t=NULL), dict(x=ctypes.c_void_p(4098)),
          dict(w=ctypes.c_void_p(4104)), dict(lse=NULL)]


@pytest.mark.parametrize("kw", COMMON + [dict(loss=NULL)])
def test_ce_fwd_refusals(kw):
    assert ce_fwd(glc.load(), **kw) == glc.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON + [dict(dl=NULL), dict(dx=NULL), dict(dw=NULL), dict(dx=ctypes.c_void_p(4100)),
                                         dict(dw=ctypes.c_void_p(4100))])
def test_ce_bwd_refusals(kw):
    assert ce_bwd(glc.load(), **kw) == glc.ERR_INVALID_ARG


@pytest.mark.parametrize("N,D,V,dt", [(1, 1, 1, glc.BF16), (16, 2048, 32000, glc.BF16), (100, 24, 777, glc.F32)])
def test_ce_workspaces(N, D, V, dt):
    lib = glc.load()
    for name, call in (("linear_ce_fwd", ce_fwd), ("linear_ce_bwd", ce_bwd)):
        need = getattr(lib, name + "_workspace_size")(N, D, V, dt)
        assert need > 0
        kw = dict(N=N, D=D, V=V, dt=dt)
        assert call(lib, n=need - 1, **kw) == glc.ERR_WORKSPACE
        assert call(lib, ws=NULL, **kw) == glc.ERR_WORKSPACE
        assert call(lib, ws=ctypes.c_void_p(4096 + 128), **kw) == glc.ERR_WORKSPACE
        assert getattr(lib, name + "_workspace_size")(N, 0, V, dt) == 0
        assert getattr(lib, name + "_workspace_size")(0, D, V, dt) == 0


def test_ce_workspace_is_bounded_by_a_piece_of_the_vocabulary():
    """Twice the vocabulary: no more workspace once G is cut into pieces (512
    MB of it at a time), beside the cuts of a gradient's sum (512 MB at most)."""
    lib = glc.load()
    N, D = 1 << 16, 512
    one, two = (lib.linear_ce_bwd_workspace_size(N, D, V, glc.BF16) for V in (1 << 16, 1 << 17))
    logits = 2 * N * (1 << 17)
    assert two <= one + (1 << 20) and two < logits // 4


def test_ce_forward_without_tokens_is_a_no_op():
    assert ce_fwd(glc.load(), N=0, x=NULL, w=NULL, t=NULL, loss=NULL, lse=NULL, ws=NULL, n=0) == glc.OK


def test_binding_refuses_cpu_tensors():
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        glc.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        glc.linear_ce_fwd(x, x, t)
    q = torch.zeros(1, 1, 1, 8)
    with pytest.raises(ValueError):
        glc.gla_step(q, q, q, q, torch.zeros(1, 1, 8, 8))


def off(n):
    return ctypes.c_void_p(4096 + n)


def test_pointers_between_elements_are_refused():
    lib = glc.load()
    for kw in (dict(x=off(1)), dict(y=off(1)), dict(w=off(2)), dict(b=off(2)), dict(mean=off(2)), dict(rstd=off(2)),
               dict(x=off(2), dt=glc.F32), dict(y=off(2), dt=glc.F32)):
        assert norm_fwd(lib, **kw) == glc.ERR_INVALID_ARG, kw
    for kw in (dict(x=off(1)), dict(dy=off(1)), dict(dx=off(1)), dict(w=off(2)), dict(mean=off(2)), dict(rstd=off(2)),
               dict(dw=off(2)), dict(db=off(2)), dict(dy=off(2), dt=glc.F32)):
        assert norm_bwd(lib, **kw) == glc.ERR_INVALID_ARG, kw
    for kw in (dict(t=off(4)), dict(lse=off(2))):
        assert ce_fwd(lib, **kw) == glc.ERR_INVALID_ARG, kw
        assert ce_bwd(lib, **kw) == glc.ERR_INVALID_ARG, kw
    assert ce_fwd(lib, loss=off(2)) == ce_bwd(lib, dl=off(2)) == glc.ERR_INVALID_ARG
    for over, o in ((dict(q=4098), A), (dict(g=4098), A), (dict(v=4097, dtype=glc.BF16), A), ({}, off(2)),
                    (dict(dtype=glc.BF16), off(1))):
        for call in (lib.gla_step, lib.ssd_step):
            assert call(ctypes.byref(step_problem(**over)), A, 9, A, o, NULL) == glc.ERR_INVALID_ARG, over
