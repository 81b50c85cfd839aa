"""Host-side checks of the gated delta rule and the head norm that need no GPU:
bad arguments are refused before any launch, workspaces are sized as documented."""
import ctypes

import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

A = ctypes.c_void_p(4096)  # an aligned address that no refused call touches
ODD = ctypes.c_void_p(4097)
NULL = None


def problem(**over):
    p = glc.Problem(B=3, T=100, H=4, Hqk=2, K=16, V=8, dtype=glc.F32, chunk_size=0, scale=1.0, reserved0=0, q=256, k=512,
                    v=768, g=1024, segment_ids=None, n_seqs=3, initial_state=None, workspace=4096,
                    workspace_bytes=1 << 40)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def fwd(p, beta=A, o=A, ht=A):
    return glc.load().delta_fwd(ctypes.byref(p), beta, o, ht, NULL)


def bwd(p, beta=A, do=A, dht=A, dq=A, dk=A, dv=A, dg=A, db=A, dh0=A):
    return glc.load().delta_bwd(ctypes.byref(p), beta, do, dht, dq, dk, dv, dg, db, dh0, NULL)


def step(p, beta=A, state=A, n_slots=9, idx=A, o=A):
    return glc.load().delta_step(ctypes.byref(p), beta, state, n_slots, idx, o, NULL)


BAD = [dict(B=0), dict(T=-1), dict(K=257), dict(V=0), dict(Hqk=3), dict(dtype=4), dict(q=None), dict(g=None),
       dict(scale=float("nan")), dict(q_stride=8), dict(v_stride=31), dict(n_seqs=2), dict(reserved0=1), dict(g=1026),
       dict(q=257), dict(v=770), dict(initial_state=4098)]


@pytest.mark.parametrize("over", BAD)
def test_refusals(over):
    assert fwd(problem(**over)) == glc.ERR_INVALID_ARG
    assert bwd(problem(**over)) == glc.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(beta=NULL), dict(o=NULL), dict(beta=ODD), dict(o=ODD), dict(ht=ODD)])
def test_fwd_pointers(kw):
    assert fwd(problem(), **kw) == glc.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["beta", "do", "dq", "dk", "dv", "dg", "db"])
@pytest.mark.parametrize("at", [NULL, ODD])
def test_bwd_pointers(name, at):
    assert bwd(problem(), **{name: at}) == glc.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["dht", "dh0"])
def test_bwd_state_alignment(name):
    assert bwd(problem(), **{name: ODD}) == glc.ERR_INVALID_ARG


@pytest.mark.parametrize("chunk", [16, 32, 128])
def test_other_chunk_lengths(chunk):
    assert fwd(problem(chunk_size=chunk)) == glc.ERR_UNSUPPORTED
    assert bwd(problem(chunk_size=chunk)) == glc.ERR_UNSUPPORTED
    assert glc.load().delta_bwd_workspace_size(ctypes.byref(problem(chunk_size=chunk))) == 0


@pytest.mark.parametrize("over", [{}, dict(Hqk=4), dict(segment_ids=4096, n_seqs=17), dict(T=64), dict(T=1)])
def test_workspace(over):
    p = problem(**over)
    lib = glc.load()
    need = lib.delta_bwd_workspace_size(ctypes.byref(p))
    BT = p.B * p.T
    chunks = min(BT, BT // 64 + p.n_seqs) if p.segment_ids else p.B * ((p.T + 63) // 64)
    least = 8 * p.H * (chunks * p.K * p.V + BT * p.V) + (8 * BT * p.H * p.K if p.Hqk != p.H else 0)
    assert least <= need <= 2 * least + (1 << 14)
    for kw in (dict(workspace=None), dict(workspace_bytes=need - 1), dict(workspace=4096 + 16)):
        assert bwd(problem(**over, **kw)) == glc.ERR_WORKSPACE
    if p.segment_ids:
        need = lib.delta_fwd_workspace_size(ctypes.byref(p))
        assert need >= 16 * (p.n_seqs + 1)
        assert fwd(problem(**over, workspace_bytes=need - 1)) == glc.ERR_WORKSPACE


def test_no_tokens_is_a_no_op():
    p = problem(T=0, n_seqs=0, q=None, k=None, v=None, g=None)
    assert fwd(p, NULL, NULL, NULL) == glc.OK
    assert bwd(p, *[NULL] * 9) == glc.OK
    assert step(p, NULL, NULL, 9, NULL, NULL) == glc.OK


@pytest.mark.parametrize("over,kw", [(o, {}) for o in BAD] + [
    (dict(chunk_size=64), {}), (dict(segment_ids=4096), {}), (dict(initial_state=4096), {}),
    ({}, dict(beta=NULL)), ({}, dict(beta=ODD)), ({}, dict(state=NULL)), ({}, dict(o=NULL)), ({}, dict(n_slots=-1)),
    ({}, dict(n_slots=2, idx=NULL)), ({}, dict(state=ODD)), ({}, dict(idx=ODD)),
])
def test_step_refusals(over, kw):
    assert step(problem(**over), **kw) == glc.ERR_INVALID_ARG


def qk(**over):
    p = glc.QkNorm(B=2, T=5, Hq=4, Hk=2, D=16, R=8, dtype=glc.BF16, l2=0, interleaved=0, eps=1e-6, q=256, k=512, wq=256,
                   wk=256, cos_table=256, sin_table=256, positions=256, n_positions=9, workspace=4096,
                   workspace_bytes=1 << 30)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over", [
    dict(B=0), dict(T=-1), dict(Hq=0), dict(Hk=0), dict(D=0), dict(D=257), dict(R=9), dict(R=-1), dict(dtype=2),
    dict(l2=2), dict(interleaved=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(reserved0=1), dict(q=None),
    dict(k=None), dict(q=257), dict(wq=258), dict(cos_table=None), dict(sin_table=None), dict(n_positions=0),
    dict(positions=257), dict(q_stride=63), dict(k_stride=-1)])
def test_qk_norm_refusals(over):
    lib = glc.load()
    assert lib.qk_norm_fwd(ctypes.byref(qk(**over)), A, A, NULL) == glc.ERR_INVALID_ARG
    assert lib.qk_norm_bwd(ctypes.byref(qk(**over)), A, A, A, A, A, A, NULL) == glc.ERR_INVALID_ARG


def test_qk_norm_pointers_and_workspace():
    lib = glc.load()
    p = ctypes.byref(qk())
    for bad in ((NULL, A), (A, NULL), (ODD, A)):
        assert lib.qk_norm_fwd(p, *bad, NULL) == glc.ERR_INVALID_ARG
    for i in range(6):
        for at in (NULL, ODD):
            args = [A] * 6
            args[i] = at
            assert lib.qk_norm_bwd(p, *args, NULL) == glc.ERR_INVALID_ARG
    need = lib.qk_norm_bwd_workspace_size(p)
    assert need > 0 and need % (2 * 16 * 4) == 0
    for over in (dict(workspace=None), dict(workspace_bytes=need - 1), dict(workspace=4100)):
        assert lib.qk_norm_bwd(ctypes.byref(qk(**over)), *[A] * 6, NULL) == glc.ERR_WORKSPACE
    assert lib.qk_norm_fwd(ctypes.byref(qk(T=0, q=None, k=None)), NULL, NULL, NULL) == glc.OK


def test_packed_qk_norm_matches_the_structure():
    """The binding's packed form of glacore_qk_norm, field by field."""
    fields = [2, 5, 4, 2, 16, 8, glc.BF16, 1, 1, 0.5, 0, 256, 512, 768, 1024, 1280, 1536, 1792, 9, 64, 72, 4096, 99]
    p = glc.QkNorm.from_buffer_copy(glc._QK_PACK.pack(*fields))
    assert [getattr(p, n) or 0 for n, _ in glc.QkNorm._fields_] == fields


def test_binding_refusals_on_the_host():
    z = lambda *s: torch.zeros(*s)
    q, v, g = z(2, 3, 2, 8), z(2, 3, 4, 8), z(2, 3, 4)
    with pytest.raises(ValueError):
        glc.delta_fwd(q, q, v, g, g)  # not on a GPU
    with pytest.raises(ValueError):
        glc.qk_norm_fwd(q, q[:, :2])
    with pytest.raises(ValueError):
        glc.qk_norm_fwd(q, q, norm="layer")
    with pytest.raises(ValueError):
        glc.qk_norm_fwd(q, q, cos=z(4, 4))
    with pytest.raises(TypeError):
        glc.qk_norm_fwd(q, q.double())
