"""GPU parity of gla_step / ssd_step (new tokens on a pool of states) against
the fp64 token-by-token oracle, and against the chunked calls they continue.

Metric max|a-b| / max|b|.  The state is fp32 and every step multiplies it by
exp(g) (about 2 ulp) and adds one rounded product: below 4 * 2^-24 of its size
per token, 1e-5 for up to 20 tokens.  o is a sum of up to 256 products (at most
16 in sequence, then a tree): 1e-5 in fp32; a bf16 o is within half an ulp, at
most 2^-8 of itself (8 significant bits), of that, element by element."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
import oracle

pytestmark = pytest.mark.gpu

TOL_STATE = TOL = 1e-5
ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def rel(a, b):
    a = a.detach().to("cpu", torch.float64).numpy()
    return float(np.abs(a - b).max() / max(np.abs(b).max(), 1e-30)) if b.size else 0.0


def close(a, b):
    tol = TOL * np.abs(b).max() + ULP[a.dtype] * np.abs(b)
    return bool((np.abs(a.detach().to("cpu", torch.float64).numpy() - b) <= tol).all())


def make(kind, B, T, H, Hqk, K, V, dtype, seed, slots=None, fused=False):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    q, v = r(B, T, Hqk, K).to(dtype), r(B, T, H, V).to(dtype)
    k = torch.nn.functional.normalize(r(B, T, Hqk, K), dim=-1).to(dtype)
    gate = -r(B, T, H, K).abs() / 4 if kind == "gla" else -r(B, T, H).abs() / 4
    slots = slots or B
    state = r(slots, H, K, V)
    idx = torch.randperm(slots, generator=g)[:B].to(torch.int32)
    if fused:  # one projection's output: token stride 2 Hqk K + H V, any alignment
        p = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], 2).cuda()
        cq, ck, cv = p.split([Hqk * K, Hqk * K, H * V], 2)
        dev = (cq.unflatten(2, (Hqk, K)), ck.unflatten(2, (Hqk, K)), cv.unflatten(2, (H, V)))
    else:
        dev = (q.cuda(), k.cuda(), v.cuda())
    return q, k, v, gate, state, idx, dev


def ref(q, k, v, gate, state, idx, scale):
    np_ = lambda t: t.to(torch.float64).numpy()
    h0 = state[idx.long()]
    return oracle.fwd(np_(q), np_(k), np_(v), np_(gate), scale, None, np_(h0))


CASES = [
    # kind, B, T, H, Hqk, K, V, dtype, slots, fused
    ("gla", 1, 1, 16, 16, 128, 128, torch.bfloat16, 1, False),
    ("gla", 5, 1, 4, 2, 128, 128, torch.bfloat16, 9, True),
    ("ssd", 6, 1, 8, 1, 128, 64, torch.bfloat16, 6, False),
    ("gla", 3, 5, 6, 2, 72, 41, torch.float32, 4, True),
    ("ssd", 2, 3, 4, 4, 256, 256, torch.float32, 2, False),
    ("gla", 2, 17, 2, 1, 100, 130, torch.bfloat16, 5, False),
    ("gla", 4, 8, 3, 3, 16, 8, torch.float32, 4, True),
    ("ssd", 3, 9, 2, 2, 1, 1, torch.float32, 3, False),
    ("gla", 2, 2, 2, 2, 200, 20, torch.bfloat16, 7, True),
    ("ssd", 1, 20, 5, 5, 65, 33, torch.float32, 1, False),
    ("gla", 7, 1, 2, 2, 64, 16, torch.bfloat16, 8, False),
    ("gla", 2, 4, 2, 2, 64, 32, torch.float32, 2, False),
    ("gla", 2, 4, 2, 2, 250, 30, torch.float32, 2, True),
]


@pytest.mark.parametrize("kind,B,T,H,Hqk,K,V,dtype,slots,fused", CASES)
def test_against_oracle(cuda_ok, kind, B, T, H, Hqk, K, V, dtype, slots, fused):
    q, k, v, gate, state, idx, dev = make(kind, B, T, H, Hqk, K, V, dtype, B + T + K + V, slots, fused)
    pool = state.cuda()
    step = glc.gla_step if kind == "gla" else glc.ssd_step
    o = step(*dev, gate.cuda(), pool, idx.cuda(), 0.37, poison=True)
    ro, rs = ref(q, k, v, gate, state, idx, 0.37)
    assert close(o, ro)
    assert rel(pool[idx.long().cuda()], rs) <= TOL_STATE
    others = [i for i in range(slots) if i not in idx.tolist()]
    assert torch.equal(pool[others].cpu(), state[others])  # nobody else's slot is touched


def test_default_slots_and_scale(cuda_ok):
    q, k, v, gate, state, _, dev = make("gla", 3, 1, 2, 2, 32, 32, torch.float32, 1, 4)
    pool = state.cuda()
    o = glc.gla_step(*dev, gate.cuda(), pool)
    ro, rs = ref(q, k, v, gate, state, torch.arange(3), 32 ** -0.5)
    assert close(o, ro) and rel(pool[:3], rs) <= TOL_STATE


@pytest.mark.parametrize("kind", ["gla", "ssd"])
def test_continues_a_prompt(cuda_ok, kind):
    """A prompt by the chunked call, then its tokens one at a time, equals the
    chunked call over all of them: bf16 tensor-core tolerance of the chunked
    path (5e-3 on o and the final state) on both sides."""
    K, V = 128, 128 if kind == "gla" else 64
    q, k, v, gate, _, _, dev = make(kind, 2, 77, 4, 4, K, V, torch.bfloat16, 3)
    gate = gate / 16
    fwd = glc.gla_fwd if kind == "gla" else glc.ssd_fwd
    step = glc.gla_step if kind == "gla" else glc.ssd_step
    cut = lambda a, b: [t[:, a:b].contiguous() for t in (*dev, gate.cuda())]
    _, pool = fwd(*cut(0, 70), 0.1, output_final_state=True)
    outs = [step(*cut(t, t + 1), pool, None, 0.1) for t in range(70, 77)]
    np_ = lambda t: t.to(torch.float64).numpy()
    ro, rs = oracle.fwd(np_(q), np_(k), np_(v), np_(gate), 0.1)
    assert rel(torch.cat(outs, 1), ro[:, 70:]) <= 5e-3 and rel(pool, rs) <= 5e-3
    glc.get_device_error()


def test_idle_rows_and_slots_out_of_range(cuda_ok):
    q, k, v, gate, state, _, dev = make("gla", 5, 2, 2, 2, 32, 32, torch.float32, 4, 4)
    idx = torch.tensor([2, -1, 0, -7, 4], dtype=torch.int32)
    pool = state.cuda()
    o = glc.gla_step(*dev, gate.cuda(), pool, idx.cuda(), 1.0, poison=True)
    with pytest.raises(glc.GlacoreError) as e:
        glc.get_device_error()
    assert e.value.status == glc.ERR_INDEX
    glc.get_device_error()  # read once, cleared
    ro, rs = ref(q, k, v, gate, state, idx.clamp(0, 3), 1.0)
    live = [0, 2]
    assert torch.all(o[[1, 3, 4]] == 0)
    assert close(o[live], ro[live]) and rel(pool[[2, 0]], rs[live]) <= TOL_STATE
    assert torch.equal(pool[[1, 3]].cpu(), state[[1, 3]])


def test_all_rows_idle_on_an_empty_pool(cuda_ok):
    _, _, _, gate, _, _, dev = make("gla", 2, 1, 2, 2, 8, 8, torch.float32, 4)
    pool = torch.empty(0, 2, 8, 8, device="cuda")
    o = glc.gla_step(*dev, gate.cuda(), pool, torch.full((2,), -1, dtype=torch.int32, device="cuda"), poison=True)
    assert torch.all(o == 0)


@pytest.mark.parametrize("kind", ["gla", "ssd"])
def test_full_decay_starts_over_whatever_the_slot_held(cuda_ok, kind):
    q, k, v, gate, state, idx, dev = make(kind, 2, 3, 2, 2, 40, 24, torch.float32, 5)
    gate[:, 0] = -float("inf")
    dirty = state.clone()
    dirty[0], dirty[1, 0, 0, 0] = float("nan"), float("inf")
    pool = dirty.cuda()
    step = glc.gla_step if kind == "gla" else glc.ssd_step
    o = step(*dev, gate.cuda(), pool, idx.cuda(), 1.0)
    ro, rs = ref(q, k, v, gate, torch.zeros_like(state), idx, 1.0)
    assert close(o, ro) and rel(pool[idx.long().cuda()], rs) <= TOL_STATE


def test_strong_decay_has_no_range(cuda_ok):
    q, k, v, gate, state, idx, dev = make("gla", 2, 6, 2, 2, 128, 128, torch.bfloat16, 6)
    gate = gate * 200
    pool = state.cuda()
    o = glc.gla_step(*dev, gate.cuda(), pool, idx.cuda(), 1.0)
    ro, rs = ref(q, k, v, gate, state, idx, 1.0)
    assert close(o, ro) and rel(pool[idx.long().cuda()], rs) <= TOL_STATE
    glc.get_device_error()


def test_a_pool_past_32_bit_offsets(cuda_ok):
    """The last slot of a pool of 2^31 + 2^14 floats, on an unaligned pool too."""
    H, K, V = 2, 64, 128
    slots = (1 << 31) // (H * K * V) + 1
    q, k, v, gate, state, _, dev = make("ssd", 1, 1, H, H, K, V, torch.float32, 7, 1)
    pool = torch.empty(slots, H, K, V, device="cuda")
    pool[-1] = state[0].cuda()
    o = glc.ssd_step(*dev, gate.cuda(), pool, torch.tensor([slots - 1], dtype=torch.int32, device="cuda"), 1.0)
    ro, rs = ref(q, k, v, gate, state, torch.zeros(1, dtype=torch.int32), 1.0)
    assert close(o, ro) and rel(pool[-1:], rs) <= TOL_STATE


def test_unaligned_pool_and_other_stream(cuda_ok):
    q, k, v, gate, state, idx, dev = make("gla", 2, 2, 2, 2, 32, 32, torch.float32, 8)
    buf = torch.empty(state.numel() + 1, device="cuda")
    pool = buf[1:].view(state.shape)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pool.copy_(state)
        o = glc.gla_step(*dev, gate.cuda(), pool, idx.cuda(), 1.0)
    side.synchronize()
    ro, rs = ref(q, k, v, gate, state, idx, 1.0)
    assert close(o, ro) and rel(pool[idx.long().cuda()], rs) <= TOL_STATE


def test_no_tokens(cuda_ok):
    pool = torch.ones(2, 2, 8, 8, device="cuda")
    z = lambda *s: torch.zeros(*s, device="cuda")
    o = glc.gla_step(z(2, 0, 2, 8), z(2, 0, 2, 8), z(2, 0, 2, 8), z(2, 0, 2, 8), pool)
    assert o.shape == (2, 0, 2, 8) and torch.all(pool == 1)


def test_refusals(cuda_ok):
    z = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)
    q, v, g, pool = z(2, 1, 2, 8), z(2, 1, 4, 8), z(2, 1, 4, 8), z(3, 4, 8, 8)
    assert glc.gla_step(q, q, v, g, pool).shape == (2, 1, 4, 8)
    for bad in (pool.double(), pool.cpu(), pool.transpose(2, 3), z(3, 4, 8, 9), z(3, 2, 8, 8)):
        with pytest.raises(ValueError):
            glc.gla_step(q, q, v, g, bad)
    with pytest.raises(ValueError):
        glc.gla_step(q, q, v, g[..., 0], pool)  # a gate per head is ssd_step's
    with pytest.raises(ValueError):
        glc.gla_step(q, q, v, g, pool, z(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        glc.gla_step(q, q, v, g, pool, z(2, dtype=torch.int64))
    with pytest.raises(glc.GlacoreError) as e:
        glc.gla_step(q, q, v, g, pool[:1])  # fewer slots than sequences, no indices
    assert e.value.status == glc.ERR_INVALID_ARG
    with pytest.raises(glc.GlacoreError):
        glc.gla_step(z(2, 1, 2, 300), z(2, 1, 2, 300), v, z(2, 1, 4, 300), z(3, 4, 300, 8))
    lib = glc.load()
    p, keep = glc._problem(q, q, v, g, 1.0, None, None, 0, 2, False)
    p.chunk_size = 16
    assert lib.gla_step(ctypes.byref(p), glc._ptr(pool), 3, None, glc._ptr(v), None) == glc.ERR_INVALID_ARG
    p.chunk_size = 0
    assert lib.gla_step(ctypes.byref(p), None, 3, None, glc._ptr(v), None) == glc.ERR_INVALID_ARG
    assert lib.gla_step(ctypes.byref(p), glc._ptr(pool), 3, None, None, None) == glc.ERR_INVALID_ARG
    del keep
