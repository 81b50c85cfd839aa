"""GPU parity of the gated delta rule (delta_fwd, delta_bwd, delta_step) with the
fp64 token-by-token definitions.

|a - b| <= tol * max|b| + half an ulp of a's type times |b|, element by element.
TOL = 2^-14: on the tensor cores a chunk's chain of products meets at most 8
matrices of 16 bits (two bf16 parts, off by 2^-17 of an element each), and what
a chunk is off by decays with its state; on the CUDA cores 4 roundings of
2^-24 for each of up to 256 tokens that a state remembers.  dg sums terms that cancel
(a query's, a key's and the states'), up to four times the size of what is
left: 4 TOL."""
import ctypes
import math

import numpy as np
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
from oracle import delta

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -14
ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def close(a, b, tol=TOL):
    if a.shape != b.shape:
        return False
    if not b.size:
        return True
    bound = tol * np.abs(b).max() + ULP[a.dtype] * np.abs(b) + 1e-30
    return bool((np.abs(a.detach().to("cpu", torch.float64).numpy() - b) <= bound).all())


def make(B, T, H, Hqk, K, V, dtype, seed, docs=1, states=False, fused=False, rate=0.3, same_key=False):
    gen = torch.Generator("cpu")
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    norm = torch.nn.functional.normalize
    q, v = norm(r(B, T, Hqk, K), dim=-1).to(dtype), r(B, T, H, V).to(dtype)
    k = norm(r(B, T, Hqk, K) + (0.5 if not same_key else 40.0), dim=-1).to(dtype)
    x = dict(q=q, k=k, v=v, g=-r(B, T, H).abs() * rate, beta=r(B, T, H).sigmoid(), do=r(B, T, H, V).to(dtype))
    seg = None
    if docs > 1:
        seg = torch.zeros(B, T, dtype=torch.int32)
        for b in range(B):
            seg[b, torch.randperm(T - 1, generator=gen)[:docs - 1] + 1] = 1
        seg = seg.cumsum(1).to(torch.int32)
    n = B * docs if T else 0
    h0, dht = (r(n, H, K, V), r(n, H, K, V)) if states else (None, None)
    dev = {n_: t.cuda() for n_, t in x.items()}
    if fused:  # one projection's output
        p = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], 2).cuda()
        cq, ck, cv = p.split([Hqk * K, Hqk * K, H * V], 2)
        dev.update(q=cq.unflatten(2, (Hqk, K)), k=ck.unflatten(2, (Hqk, K)), v=cv.unflatten(2, (H, V)))
    c = lambda t: None if t is None else t.cuda()
    return x, dev, dict(seg=seg, h0=h0, dht=dht, n=n), dict(segment_ids=c(seg), initial_state=c(h0), n_seqs=n), c(dht)


CASES = [
    # B, T, H, Hqk, K, V, dtype, extras
    (1, 1, 2, 2, 128, 128, BF, {}),
    (2, 1, 2, 1, 16, 8, F32, dict(states=True)),
    (1, 63, 2, 2, 128, 128, BF, dict(states=True)),
    (2, 64, 2, 2, 128, 128, BF, {}),
    (1, 65, 2, 1, 128, 128, BF, dict(fused=True)),
    (1, 300, 3, 3, 128, 128, BF, dict(states=True)),
    (2, 257, 4, 2, 128, 64, BF, dict(docs=5)),
    (1, 200, 2, 1, 64, 64, BF, dict(docs=3, states=True)),
    (2, 130, 2, 2, 64, 128, BF, dict(fused=True, states=True)),
    (1, 150, 4, 2, 72, 40, BF, dict(docs=9)),
    (2, 100, 2, 2, 8, 8, BF, dict(states=True)),
    (1, 90, 2, 1, 127, 65, BF, dict(states=True, fused=True)),
    (1, 70, 2, 2, 200, 136, BF, {}),
    (3, 133, 6, 2, 72, 41, F32, dict(states=True)),
    (2, 129, 4, 4, 128, 128, F32, dict(docs=4, fused=True)),
    (1, 77, 2, 1, 256, 256, F32, dict(states=True)),
    (2, 40, 2, 2, 1, 1, F32, dict(states=True)),
    (1, 50, 3, 1, 33, 17, F32, dict(docs=50, states=True)),
]


@pytest.mark.parametrize("B,T,H,Hqk,K,V,dtype,kw", CASES)
def test_forward(cuda_ok, B, T, H, Hqk, K, V, dtype, kw):
    x, dev, host, args, _ = make(B, T, H, Hqk, K, V, dtype, B + T + K + V, **kw)
    o, ht = glc.delta_fwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], 0.37, output_final_state=True, poison=True,
                          **args)
    ro, rt = delta.fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.37, host["seg"], host["h0"])
    assert close(o, ro) and close(ht, rt)
    o2, none = glc.delta_fwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], 0.37, **args)
    assert none is None and torch.equal(o, o2)
    glc.get_device_error()


@pytest.mark.parametrize("B,T,H,Hqk,K,V,dtype,kw", CASES)
def test_backward(cuda_ok, B, T, H, Hqk, K, V, dtype, kw):
    x, dev, host, args, dht = make(B, T, H, Hqk, K, V, dtype, B + T + K + V, **kw)
    got = glc.delta_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dev["do"], 0.37, dht=dht, poison=True, **args)
    want = delta.bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], 0.37, host["seg"], host["h0"], host["dht"])
    for name, a in zip(NAMES, got):
        if a is None:
            assert name == "dh0" and host["h0"] is None
        else:
            assert close(a, want[name], 4 * TOL if name == "dg" else TOL), name
    again = glc.delta_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dev["do"], 0.37, dht=dht, **args)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))  # nothing depends on an order
    glc.get_device_error()


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 128), (BF, 128, 64), (F32, 40, 24)])
@pytest.mark.parametrize("rate", [0.0, 3.0, 60.0, float("inf")])
def test_decays(cuda_ok, dtype, K, V, rate):
    """No decay at all, decays that leave nothing of a state within a few tokens, and a full one."""
    x, dev, host, args, dht = make(1, 150, 2, 2, K, V, dtype, 5, states=True, rate=rate if rate < 1e9 else 0.3)
    if rate > 1e9:
        for t in (0, 70, 149):
            x["g"][:, t] = -rate
        dev["g"] = x["g"].cuda()
    o, ht = glc.delta_fwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], 0.37, output_final_state=True, **args)
    ro, rt = delta.fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.37, None, host["h0"])
    assert close(o, ro) and close(ht, rt)
    got = glc.delta_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dev["do"], 0.37, dht=dht, **args)
    want = delta.bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], 0.37, None, host["h0"], host["dht"])
    for name, a in zip(NAMES, got):
        assert close(a, want[name], 4 * TOL if name == "dg" else TOL), name
    glc.get_device_error()


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 128), (F32, 40, 24)])
@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
def test_writing_strengths_and_keys_that_repeat(cuda_ok, dtype, K, V, beta):
    """beta of nothing, all and a reflection, with keys that nearly coincide."""
    x, dev, host, args, dht = make(1, 200, 2, 2, K, V, dtype, 6, states=True, rate=0.01, same_key=True)
    x["beta"].fill_(beta)
    dev["beta"].fill_(beta)
    o, ht = glc.delta_fwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], 1.0, output_final_state=True, **args)
    ro, rt = delta.fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 1.0, None, host["h0"])
    # keys of length 1 + d (d <= 2^-9 in bf16) under a reflection grow what came before by (1 + 4 d) a token, and
    # what it is off by with it: none of the sums is larger than the result
    assert close(o, ro, 4 * TOL) and close(ht, rt, 4 * TOL)
    got = glc.delta_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dev["do"], 1.0, dht=dht, **args)
    want = delta.bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], 1.0, None, host["h0"], host["dht"])
    for name, a in zip(NAMES, got):
        assert close(a, want[name], 16 * TOL if name == "dg" else 4 * TOL), name


def test_differences(cuda_ok):
    """The gradients against differences of the forward itself, fp32: the change of sum(o do) + sum(S dht)
    along a random direction of each operand, central, a step of 2^-6 of its size."""
    x, dev, host, args, dht = make(2, 90, 2, 2, 24, 16, F32, 7, states=True)
    ops = dict(q=dev["q"], k=dev["k"], v=dev["v"], g=dev["g"], beta=dev["beta"], h0=args["initial_state"])

    def loss(o_):
        o, ht = glc.delta_fwd(o_["q"], o_["k"], o_["v"], o_["g"], o_["beta"], 1.0, initial_state=o_["h0"],
                              output_final_state=True)
        return float((o.double() * dev["do"].double()).sum() + (ht.double() * dht.double()).sum())

    got = glc.delta_bwd(*(ops[n] for n in ("q", "k", "v", "g", "beta")), dev["do"], 1.0, initial_state=ops["h0"], dht=dht)
    for (name, t), grad in zip(ops.items(), got):
        d = torch.randn_like(t) * t.abs().mean()
        h = 2.0 ** -6
        slope = lambda s: (loss(dict(ops, **{name: t + s * d})) - loss(dict(ops, **{name: t - s * d}))) / (2 * s)  # noqa: B023
        # the cubic term cancels between two steps
        num = (4 * slope(h / 2) - slope(h)) / 3
        ana = float((grad.double() * d.double()).sum())
        size = float((grad.double() * d.double()).norm())  # what a sum of independent terms comes to
        assert abs(num - ana) <= 2e-3 * max(abs(ana), size), (name, num, ana)


def test_prompt_then_tokens(cuda_ok):
    """A prompt by delta_fwd and its tokens by delta_step, on a pool, give what one call over all gives."""
    for dtype, K, V in ((BF, 128, 128), (BF, 128, 64), (F32, 48, 20)):
        x, dev, host, _, _ = make(2, 140, 4, 2, K, V, dtype, 8)
        cut = lambda a, b: [dev[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")]
        _, last = glc.delta_fwd(*cut(0, 131), 0.5, output_final_state=True)
        pool = torch.full((5, 4, K, V), 3.0, device="cuda")
        idx = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
        pool[idx.long()] = last
        outs = [glc.delta_step(*cut(131, 134), pool, idx, 0.5, poison=True)]
        outs += [glc.delta_step(*cut(t, t + 1), pool, idx, 0.5) for t in range(134, 140)]
        ro, rt = delta.fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5)
        assert close(torch.cat(outs, 1), ro[:, 131:]) and close(pool[idx.long()], rt)
        assert torch.all(pool[[0, 2, 4]] == 3.0)


STEPS = [
    # B, T, H, Hqk, K, V, dtype, slots, fused
    (1, 1, 16, 16, 128, 128, BF, 1, False),
    (5, 1, 4, 2, 128, 128, BF, 9, True),
    (6, 1, 8, 1, 128, 64, BF, 6, False),
    (3, 5, 6, 2, 72, 41, F32, 4, True),
    (2, 3, 4, 4, 256, 256, F32, 2, False),
    (2, 17, 2, 1, 100, 130, BF, 5, False),
    (4, 8, 3, 3, 16, 8, F32, 4, True),
    (3, 9, 2, 2, 1, 1, F32, 3, False),
    (2, 2, 2, 2, 200, 20, BF, 7, True),
    (1, 20, 5, 5, 65, 33, F32, 1, False),
    (7, 1, 2, 2, 64, 16, BF, 8, False),
    (2, 4, 2, 2, 250, 30, F32, 2, True),
]


def pool_of(x, slots, seed=3):
    B, H, K, V = x["v"].shape[0], x["v"].shape[2], x["k"].shape[3], x["v"].shape[3]
    gen = torch.Generator("cpu")
    gen.manual_seed(seed)
    return torch.randn(slots, H, K, V, generator=gen), torch.randperm(slots, generator=gen)[:B].to(torch.int32)


@pytest.mark.parametrize("B,T,H,Hqk,K,V,dtype,slots,fused", STEPS)
def test_step(cuda_ok, B, T, H, Hqk, K, V, dtype, slots, fused):
    x, dev, _, _, _ = make(B, T, H, Hqk, K, V, dtype, B + T + K + V, fused=fused)
    state, idx = pool_of(x, slots)
    pool = state.cuda()
    o = glc.delta_step(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], pool, idx.cuda(), 0.37, poison=True)
    ro, rs = delta.step(x["q"], x["k"], x["v"], x["g"], x["beta"], state, idx, 0.37)
    assert close(o, ro, 1e-5) and close(pool[idx.long().cuda()], rs, 1e-5)  # fp32, up to 20 tokens of 8 roundings
    others = [i for i in range(slots) if i not in idx.tolist()]
    assert torch.equal(pool[others].cpu(), state[others])


def test_step_idle_rows_bad_slots_and_full_decay(cuda_ok):
    x, dev, _, _, _ = make(5, 2, 2, 2, 32, 32, F32, 4)
    state, _ = pool_of(x, 4)
    x["g"][0, 0] = -float("inf")
    dev["g"] = x["g"].cuda()
    idx = torch.tensor([2, -1, 0, -7, 4], dtype=torch.int32)
    dirty = state.clone()
    dirty[2] = float("nan")
    pool = dirty.cuda()
    o = glc.delta_step(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], pool, idx.cuda(), 1.0, poison=True)
    with pytest.raises(glc.GlacoreError) as e:
        glc.get_device_error()
    assert e.value.status == glc.ERR_INDEX
    glc.get_device_error()
    ro, rs = delta.step(x["q"], x["k"], x["v"], x["g"], x["beta"], state, idx.clamp(0, 3), 1.0)
    live = [0, 2]
    assert torch.all(o[[1, 3, 4]] == 0)
    assert close(o[live], ro[live], 1e-5) and close(pool[[2, 0]], rs[live], 1e-5)
    assert torch.equal(pool[[1, 3]].cpu(), state[[1, 3]])


def test_step_on_a_pool_past_32_bit_offsets_and_unaligned(cuda_ok):
    H, K, V = 2, 64, 128
    slots = (1 << 31) // (H * K * V) + 1
    x, dev, _, _, _ = make(1, 1, H, H, K, V, F32, 7)
    state, _ = pool_of(x, 1)
    args = (dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"])
    ro, rs = delta.step(x["q"], x["k"], x["v"], x["g"], x["beta"], state, [0], 1.0)
    pool = torch.empty(slots, H, K, V, device="cuda")
    pool[-1] = state[0].cuda()
    o = glc.delta_step(*args, pool, torch.tensor([slots - 1], dtype=torch.int32, device="cuda"), 1.0)
    assert close(o, ro, 1e-5) and close(pool[-1:], rs, 1e-5)
    pool = torch.empty(state.numel() + 1, device="cuda")[1:].view(state.shape)
    pool.copy_(state)
    o = glc.delta_step(*args, pool, None, 1.0)
    assert close(o, ro, 1e-5) and close(pool, rs, 1e-5)


def test_tokens_past_32_bit_offsets(cuda_ok):
    """Three tokens 2^30 elements apart: the last starts at element 2^31."""
    x, dev, _, _, _ = make(1, 3, 2, 2, 128, 64, BF, 9)
    want = glc.delta_fwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], 1.0)[0]
    grads = glc.delta_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dev["do"], 1.0)
    buf = torch.empty((1 << 31) + 1024, dtype=BF, device="cuda")
    far = {}
    for at, n in ((0, "q"), (256, "k"), (512, "v")):
        hd, d = dev[n].shape[2:]
        far[n] = buf[at:].as_strided((1, 3, hd, d), (3 << 30, 1 << 30, d, 1))
        far[n].copy_(dev[n])
    o = glc.delta_fwd(far["q"], far["k"], far["v"], dev["g"], dev["beta"], 1.0)[0]
    assert torch.equal(o, want)
    for a, b in zip(glc.delta_bwd(far["q"], far["k"], far["v"], dev["g"], dev["beta"], dev["do"], 1.0), grads):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype,K,V,docs", [(BF, 128, 128, 1), (BF, 128, 64, 4), (F32, 40, 24, 3)])
def test_captured_and_replayed(cuda_ok, dtype, K, V, docs):
    """A forward, its gradients and a decode step in one graph, replayed on other values: bit for bit what calls give."""
    def fresh(seed):
        x, dev, host, args, _ = make(2, 150, 4, 2, K, V, dtype, seed, docs=docs)
        d = dict(dev, state=torch.randn(7, 4, K, V, device="cuda"))
        d["seg"] = args["segment_ids"] if docs > 1 else torch.zeros(2, 150, dtype=torch.int32, device="cuda")
        return d

    def call(s):
        o, ht = glc.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], None, s["seg"], None, True, n_seqs=2 * docs)
        grads = glc.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], None, s["seg"], n_seqs=2 * docs)
        one = [s[n][:, :1] for n in ("q", "k", "v", "g", "beta")]
        return o, ht, *grads[:5], glc.delta_step(*one, s["state"]), s["state"]

    state = fresh(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(state)
    for seed in (2, 3):
        values = fresh(seed)
        for n, v in values.items():
            state[n].copy_(v)
        graph.replay()
        want = call({n: v.clone() for n, v in values.items()})
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    glc.get_device_error()


def test_two_streams_at_once(cuda_ok):
    """Calls on two streams with workspaces of their own, and outputs and a workspace that the caller gives."""
    sets = [make(2, 200, 2, 2, 128, 128, BF, s)[1] for s in (1, 2)]
    call = lambda d, **kw: glc.delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], **kw)
    want = [call(d) for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    spaces = [torch.empty(1 << 26, dtype=torch.uint8, device="cuda") for _ in sets]
    outs = [[torch.full_like(t, float("nan")) for t in w[:5]] + [None] for w in want]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, d, o, ws in zip(streams, sets, outs, spaces):
            with torch.cuda.stream(s):
                call(d, outs=o, workspace=ws)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(o, w))


def test_nothing_past_the_outputs_is_written(cuda_ok):
    """Outputs in the middle of a larger buffer keep their neighbours."""
    for K, V, T in ((128, 128, 70), (128, 64, 1), (64, 128, 129)):
        _, d, _, _, _ = make(1, T, 2, 1, K, V, BF, 11)
        want = glc.delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"])[:5] + \
            glc.delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"])[:1]
        bufs = [torch.full((w.numel() + 512,), 7.0, dtype=w.dtype, device="cuda") for w in want]
        mid = [b[256:256 + w.numel()].view(w.shape) for b, w in zip(bufs, want)]
        glc.delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], outs=(*mid[:5], None))
        glc.delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], out=mid[5])
        for b, m, w in zip(bufs, mid, want):
            assert torch.equal(m, w) and torch.all(b[:256] == 7) and torch.all(b[256 + w.numel():] == 7)


def test_addresses_and_strides_of_single_elements(cuda_ok):
    """bf16 operands at odd addresses give what aligned ones give, up to what either kernel may be off."""
    x, d, _, _, _ = make(1, 100, 2, 2, 128, 64, BF, 12)

    def shifted(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = b[1:].view(t.shape)
        v.copy_(t)
        return v

    s = {n: shifted(t) for n, t in d.items()}
    o, _ = glc.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], 1.0)
    ro, _ = delta.fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 1.0)
    assert close(o, ro)
    want = delta.bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], 1.0)
    for name, a in zip(NAMES, glc.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], 1.0)[:5]):
        assert close(a, want[name], 4 * TOL if name == "dg" else TOL), name


def test_wrong_number_of_documents(cuda_ok):
    x, d, host, args, _ = make(1, 130, 2, 2, 128, 64, BF, 13, docs=4)
    for n in (3, 5):
        glc.delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], segment_ids=args["segment_ids"], n_seqs=n)
        with pytest.raises(glc.GlacoreError) as e:
            glc.get_device_error()
        assert e.value.status == glc.ERR_DOCS


def test_no_tokens_and_refusals(cuda_ok):
    z = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)
    q, v, g = z(2, 0, 2, 8), z(2, 0, 4, 8), z(2, 0, 4)
    assert glc.delta_fwd(q, q, v, g, g)[0].shape == v.shape
    assert [t.shape for t in glc.delta_bwd(q, q, v, g, g, v)[:5]] == [t.shape for t in (q, q, v, g, g)]
    assert glc.delta_step(q, q, v, g, g, z(2, 4, 8, 8)).shape == v.shape
    q, v, g, pool = z(2, 1, 2, 8), z(2, 1, 4, 8), z(2, 1, 4), z(3, 4, 8, 8)
    assert glc.delta_step(q, q, v, g, g, pool).shape == v.shape
    for bad in (g[..., :1], z(2, 1, 4, 8), g.cpu()):
        with pytest.raises(ValueError):
            glc.delta_step(q, q, v, g, bad, pool)
        with pytest.raises(ValueError):
            glc.delta_fwd(q, q, v, g, bad)
        with pytest.raises(ValueError):
            glc.delta_bwd(q, q, v, g, bad, v)
    for bad in (pool.double(), pool.cpu(), pool.transpose(2, 3), z(3, 4, 8, 9)):
        with pytest.raises(ValueError):
            glc.delta_step(q, q, v, g, g, bad)
    with pytest.raises(TypeError):
        glc.delta_fwd(q, q, v, g, g.double())
    with pytest.raises(TypeError):
        glc.delta_bwd(q, q, v, g, g, v.double())
    with pytest.raises(ValueError):
        glc.delta_bwd(q, q, v, g, g, v[:, :0])
    with pytest.raises(ValueError):
        glc.delta_fwd(q, q, v, g, g, initial_state=z(2, 4, 8, 9))
    with pytest.raises(glc.GlacoreError) as e:
        glc.delta_fwd(z(1, 1, 1, 257), z(1, 1, 1, 257), z(1, 1, 1, 8), z(1, 1, 1), z(1, 1, 1))
    assert e.value.status == glc.ERR_INVALID_ARG
    p, keep = glc._problem(q, q, v, g, 1.0, None, None, 0, 2, True)
    p.chunk_size = 32
    assert glc.load().delta_fwd(ctypes.byref(p), glc._ptr(g), glc._ptr(v), None, None) == glc.ERR_UNSUPPORTED
    del keep


@pytest.mark.parametrize("B,T,H,Hqk,V,docs", [(4, 2048, 16, 16, 128, 1), (1, 8192, 16, 8, 128, 9), (2, 3001, 16, 4, 64, 5)])
def test_many_chunks_against_the_other_kernels(cuda_ok, B, T, H, Hqk, V, docs):
    """Dozens of chunks on every SM at once: the tensor-core kernels, ten times the same bits, against the token by
    token ones (which take outputs at odd addresses).  Both are within half an ulp and TOL of the same values."""
    gen = torch.Generator("cuda")
    gen.manual_seed(B + T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    norm = torch.nn.functional.normalize
    q, k = (norm(r(B, T, Hqk, 128), dim=-1).to(BF) for _ in range(2))
    v, do, g, b = r(B, T, H, V).to(BF), r(B, T, H, V).to(BF), -r(B, T, H).abs() / 8, r(B, T, H).sigmoid()
    seg = None
    if docs > 1:
        seg = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        for i in range(B):
            seg[i, torch.randperm(T - 1, generator=gen, device="cuda")[:docs - 1] + 1] = 1
        seg = seg.cumsum(1).to(torch.int32)

    def odd(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)

    def call(at_odd=False):
        outs = (*(odd(t) for t in (q, k, v, g, b)), None) if at_odd else None
        o, ht = glc.delta_fwd(q, k, v, g, b, segment_ids=seg, output_final_state=True, n_seqs=B * docs, poison=True,
                              out=odd(v) if at_odd else None)
        return (o, ht, *glc.delta_bwd(q, k, v, g, b, do, segment_ids=seg, n_seqs=B * docs, poison=True, outs=outs)[:5])

    want = call(at_odd=True)
    first = call()
    for _ in range(9):
        assert all(torch.equal(x, y) for x, y in zip(first, call()))
    for name, x, y in zip(("o", "ht", *NAMES), first, want):
        x, y = x.double(), y.double()
        bound = 2 * (4 if name == "dg" else 1) * TOL * y.abs().max() + (2 * ULP[BF] * y.abs() if first[0].dtype == BF else 0)
        assert bool(((x - y).abs() <= bound).all()), (name, float((x - y).abs().max()), float(y.abs().max()))
    glc.get_device_error()


@pytest.mark.parametrize("B,T,H,Hqk,K,V,kw", [
    (2, 640, 32, 32, 128, 128, {}), (4, 2048, 16, 4, 128, 128, {}), (1, 777, 76, 19, 64, 48, {"states": True}),
    (1, 64 * 41 + 1, 33, 11, 128, 64, {"states": True}), (4, 1000, 16, 16, 128, 128, {"same_key": True})])
def test_tiles_made_while_the_chains_walk(cuda_ok, B, T, H, Hqk, K, V, kw):
    """Sequences of one length on few SMs take one kernel; given as documents they take two: the same bits, every time,
    also from a graph beside another stream's calls."""
    x, dev, _, call, _ = make(B, T, H, Hqk, K, V, BF, 11, **kw)
    if kw.get("same_key"):
        dev["beta"].fill_(2.0)  # long rows of Z: their third part
    args = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    seg = torch.arange(B, device="cuda", dtype=torch.int32)[:, None].expand(B, T).contiguous()
    run = lambda **k: glc.delta_fwd(*args, initial_state=call["initial_state"], output_final_state=True, **k)
    with glc.LaunchTimer(8) as t:
        want = run(segment_ids=seg, n_seqs=B)
    assert t.labels[-2:] == ["delta_prep", "delta_chain"]
    with glc.LaunchTimer(8) as t:
        got = run(poison=True)
    if torch.cuda.get_device_properties(0).multi_processor_count // 2 >= B * H:
        assert t.labels == ["delta_overlap"]
    same = lambda a: all(torch.equal(x, y) for x, y in zip(a, want))
    assert same(got)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(20):
        side.wait_stream(torch.cuda.current_stream())
        for y in held:
            y.zero_()
        graph.replay()
        with torch.cuda.stream(side):
            other = run()
        torch.cuda.synchronize()
        assert same(held) and same(other)
    glc.get_device_error()


@pytest.mark.parametrize("B,T,H,Hqk,K,V,kw", [
    (1, 333, 6, 2, 72, 41, {"docs": 4}), (2, 150, 4, 4, 125, 77, {"states": True}), (1, 200, 3, 3, 9, 127, {"fused": True}),
    (2, 130, 4, 1, 128, 128, {"odd": True, "states": True}), (2, 700, 32, 32, 101, 128, {})])
def test_sizes_strides_and_addresses_that_take_padded_copies(cuda_ok, B, T, H, Hqk, K, V, kw):
    """Forwards and backwards on the tensor cores, whatever divides the operands: states, gradients and outputs of their own
    sizes, nothing past them written."""
    kw = dict(kw)
    at_odd = kw.pop("odd", False)
    x, dev, host, call, dht = make(B, T, H, Hqk, K, V, BF, 23, **kw)
    if at_odd:
        for n in "qkv":
            y = torch.empty(dev[n].numel() + 1, dtype=BF, device="cuda")[1:].view(dev[n].shape)
            dev[n] = y.copy_(dev[n])
    args = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    shapes = ((B, T, Hqk, K), (B, T, Hqk, K), (B, T, H, V), (B, T, H), (B, T, H), (host["n"], H, K, V))
    guard = 512
    bufs = [torch.full((math.prod(s) + guard,), 77.0, dtype=t, device="cuda")
            for s, t in zip(shapes, (BF, BF, BF, F32, F32, F32))]
    outs = [b_[:b_.numel() - guard].view(s) for b_, s in zip(bufs, shapes)]
    if not kw.get("states"):
        outs[5] = None
    o_buf = torch.full((B * T * H * V + guard,), 77.0, dtype=BF, device="cuda")
    with glc.LaunchTimer(12) as t:
        o, last = glc.delta_fwd(*args, output_final_state=True, out=o_buf[:-guard].view(B, T, H, V), **call)
    assert "delta_pad" in t.labels and t.labels[-1] == "delta_unpad"
    with glc.LaunchTimer(12) as t:
        got = glc.delta_bwd(*args, dev["do"], dht=dht, outs=outs, **call)
    assert "delta_pad" in t.labels
    h = [x[n] for n in ("q", "k", "v", "g", "beta")]
    want, state = delta.fwd(*h, K ** -0.5, host["seg"], host["h0"])
    assert close(o, want) and close(last, state)
    ref = delta.bwd(*h, x["do"], K ** -0.5, host["seg"], host["h0"], host["dht"])
    for name, a in zip(NAMES, got):
        assert a is None or close(a, ref[name], 4 * TOL if name == "dg" else TOL), name
    assert all(torch.all(b_[-guard:] == 77.0) for b_ in (*bufs, o_buf))
    glc.get_device_error()
