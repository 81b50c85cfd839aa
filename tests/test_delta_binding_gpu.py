"""What the binding of the gated delta rule and the head norm refuses before it hands an address to the library,
outputs and workspaces that the caller gives, and the measurement hook."""
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another GPU (there is one here)."""

    @property
    def device(self):
        return torch.device("cuda", 1)

    def get_device(self):
        return 1

    def is_contiguous(self, *a, **kw):
        return True


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, device="cuda", dtype=dtype)


def calls():
    """name: (call of keyword operands, outputs' keyword, outputs)."""
    q, v, g, pool = z(2, 3, 2, 8), z(2, 3, 4, 8), z(2, 3, 4), z(3, 4, 8, 8)
    idx = torch.arange(2, device="cuda", dtype=torch.int32)
    seg, w, cs = z(2, 3, dtype=torch.int32), z(8), z(9, 4)
    qkv = dict(q=q, k=q, v=v, g=g, beta=g)
    head = dict(q=q, k=v, wq=w, wk=w, cos=cs, sin=cs, positions=seg)
    grads = [z(2, 3, 2, 8), z(2, 3, 2, 8), z(2, 3, 4, 8), z(2, 3, 4), z(2, 3, 4)]
    return {
        "delta_fwd": (dict(qkv, segment_ids=seg, initial_state=pool[:2]), "out", [z(2, 3, 4, 8)]),
        "delta_bwd": (dict(qkv, do=v, segment_ids=seg, initial_state=pool[:2], dht=pool[:2]), "outs",
                      grads + [z(2, 4, 8, 8)]),
        "delta_step": (dict(qkv, state=pool, state_indices=idx), "out", [z(2, 3, 4, 8)]),
        "qk_norm_fwd": (head, "outs", [z(2, 3, 2, 8), z(2, 3, 4, 8)]),
        "qk_norm_bwd": (dict(head, dqo=q, dko=v), "outs", [z(2, 3, 2, 8), z(2, 3, 4, 8), z(8), z(8)]),
    }


NAMES = ["delta_fwd", "delta_bwd", "delta_step", "qk_norm_fwd", "qk_norm_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_operands_on_another_device(cuda_ok, name):
    args, _, _ = calls()[name]
    call = getattr(glc, name)
    call(**args)
    for key in args:
        with pytest.raises(ValueError):
            call(**dict(args, **{key: args[key].as_subclass(Elsewhere)}))
        with pytest.raises(ValueError):
            call(**dict(args, **{key: args[key].cpu()}))
    glc.get_device_error()


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_do_not_fit(cuda_ok, name):
    args, key, outs = calls()[name]
    call = getattr(glc, name)
    given = lambda o: {key: o[0] if key == "out" else tuple(o)}
    got = call(**args, **given(outs))
    got = got[:len(outs)] if isinstance(got, tuple) else (got,)
    assert all(a is b for a, b in zip(got, outs))
    call(**args, **given([o.flatten() for o in outs]))  # the axes are the caller's own
    for i, o in enumerate(outs):
        wide = torch.zeros(*o.shape[:-1], 2 * o.shape[-1], device="cuda")[..., ::2]
        for bad in (o[:1], o.flatten()[:-1], o.cpu(), o.as_subclass(Elsewhere), wide, o.double(), o.bfloat16()):
            with pytest.raises((ValueError, TypeError)):
                call(**args, **given(outs[:i] + [bad] + outs[i + 1:]))


@pytest.mark.parametrize("name", ["delta_fwd", "delta_bwd", "qk_norm_bwd"])
def test_workspaces(cuda_ok, name):
    args, _, _ = calls()[name]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    getattr(glc, name)(**args, workspace=ws)
    getattr(glc, name)(**args, workspace=ws[1:])  # one that does not serve is left alone
    assert ws.data_ptr() % 256 == 0
    for bad in (ws.cpu(), ws.as_subclass(Elsewhere)):
        with pytest.raises(ValueError):
            getattr(glc, name)(**args, workspace=bad)


def test_a_workspace_of_exactly_its_size(cuda_ok):
    """Nothing is written behind the bytes that the query names, whichever kernels run."""
    for dt, T, K, V, H in ((torch.bfloat16, 130, 128, 128, 2), (torch.bfloat16, 40, 64, 40, 4), (torch.float32, 70, 24, 40, 4)):
        r = lambda *s: torch.randn(*s, device="cuda")
        q, k = (torch.nn.functional.normalize(r(1, T, 2, K), dim=-1).to(dt) for _ in range(2))
        v, g, b = r(1, T, H, V).to(dt), -r(1, T, H).abs(), r(1, T, H).sigmoid()
        seg = (torch.arange(T, device="cuda") > 20).int()[None].contiguous()
        p, keep = glc._problem(q, k, v, g, 1.0, seg, None, 0, 2, True)
        for name, args in (("delta_fwd", (q, k, v, g, b)), ("delta_bwd", (q, k, v, g, b, v))):
            need = glc.workspace_size(p, name)
            buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
            at = -buf.data_ptr() % 256
            with_ws = getattr(glc, name)(*args, 1.0, seg, n_seqs=2, workspace=buf[at:at + need])
            alone = getattr(glc, name)(*args, 1.0, seg, n_seqs=2)
            assert torch.all(buf[at + need:] == 77) and torch.all(buf[:at] == 77)
            assert all(x is y is None or torch.equal(x, y) for x, y in zip(with_ws, alone))
        del keep


def test_launches_are_named(cuda_ok):
    r = lambda *s: torch.randn(*s, device="cuda")
    q, v, g = r(1, 200, 2, 128).bfloat16(), r(1, 200, 4, 64).bfloat16(), -r(1, 200, 4).abs()
    with glc.LaunchTimer(8) as t:
        glc.delta_fwd(q, q, v, g, g.sigmoid())
    assert t.labels == ["delta_prep", "delta_chain"]
    with glc.LaunchTimer(8) as t:
        glc.delta_bwd(q, q, v, g, g.sigmoid(), v)
    assert t.labels == ["delta_prep", "delta_walks", "delta_grads", "delta_reduce_heads", "delta_reduce_heads"]
    with glc.LaunchTimer(8) as t:
        glc.delta_bwd(q.float(), q.float(), v.float(), g, g.sigmoid(), v.float())
    assert t.labels == ["delta_scans", "delta_grads", "delta_reduce_heads", "delta_reduce_heads"]
    with glc.LaunchTimer(8) as t:
        glc.qk_norm_bwd(q, q, q, q)
    assert t.labels == ["qk_norm_bwd", "qk_norm_sum_dw"]
    torch.cuda.synchronize()


def test_infinities_behind_a_documents_end(cuda_ok):
    """NaN and infinities in one document, row or head reach no other."""
    r = lambda *s: torch.randn(*s, device="cuda")
    norm = torch.nn.functional.normalize
    for dt, K, V in ((torch.bfloat16, 128, 128), (torch.bfloat16, 64, 64), (torch.float32, 24, 40)):
        q, k = (norm(r(2, 150, 2, K), dim=-1).to(dt) for _ in range(2))
        v, do, g, b = r(2, 150, 2, V).to(dt), r(2, 150, 2, V).to(dt), -r(2, 150, 2).abs() / 4, r(2, 150, 2).sigmoid()
        seg = torch.zeros(2, 150, dtype=torch.int32, device="cuda")
        seg[:, 70:] = 1
        seg[:, 101:] = 2

        def run():
            o, ht = glc.delta_fwd(q, k, v, g, b, 1.0, seg, None, True, n_seqs=6)
            return (o, *glc.delta_bwd(q, k, v, g, b, do, 1.0, seg, n_seqs=6)[:5]), ht

        want, states = run()
        for x in (q, k, v, do):
            x[0, 70:101, 0] = float("inf")
            x[0, 85, 0] = float("nan")
        got, bad = run()
        for x, y in zip(got, want):
            assert torch.equal(x[1], y[1]) and torch.equal(x[0, :70], y[0, :70]) and torch.equal(x[0, 101:], y[0, 101:])
            assert torch.equal(x[0, :, 1], y[0, :, 1])
        assert torch.equal(bad[[0, 2, 3, 4, 5]], states[[0, 2, 3, 4, 5]]) and torch.equal(bad[1, 1], states[1, 1])
