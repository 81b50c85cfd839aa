"""What the binding refuses before it hands an address to the library: operands on another device
than the call's, and output tensors that the kernels would not fill as they are."""
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
    """name: (call of keyword operands, operands, outputs by their keyword)."""
    x, w, b, st = z(6, 16), z(16), z(16), z(6)
    q, v, g, pool = z(2, 1, 2, 8), z(2, 1, 4, 8), z(2, 1, 4, 8), z(3, 4, 8, 8)
    idx = torch.arange(2, device="cuda", dtype=torch.int32)
    h, head, t = z(5, 16), z(9, 16), torch.zeros(5, dtype=torch.int64, device="cuda")
    step = dict(q=q, k=q, v=v, state=pool, state_indices=idx)
    return {
        "layer_norm_fwd": (dict(x=x, w=w, b=b), "out", [z(6, 16)]),
        "layer_norm_bwd": (dict(x=x, w=w, mean=st, rstd=st, dy=x), "outs", [z(6, 16), z(16), z(16)]),
        "gla_step": (dict(step, g=g), "out", [z(2, 1, 4, 8)]),
        "ssd_step": (dict(step, g=g[..., 0].contiguous()), "out", [z(2, 1, 4, 8)]),
        "linear_ce_fwd": (dict(x=h, w=head, target=t), "outs", [z(5), z(5)]),
        "linear_ce_bwd": (dict(x=h, w=head, target=t, lse=z(5), dloss=z(5)), "outs", [z(5, 16), z(9, 16)]),
        "gla_fwd": (dict(q=q, k=q, v=v, g=g), "out", [z(2, 1, 4, 8)]),
        "gla_bwd": (dict(q=q, k=q, v=v, g=g, do=v), "outs", [z(2, 1, 2, 8), z(2, 1, 2, 8), z(2, 1, 4, 8), z(2, 1, 4, 8)]),
        "norm_gate_fwd": (dict(o=x, z=x, w=w), "out", [z(6, 16)]),
        "norm_gate_bwd": (dict(o=x, z=x, w=w, dy=x), "outs", [z(6, 16), z(6, 16), z(16)]),
        "short_conv_fwd": (dict(x=z(2, 3, 16), w=z(4, 16), b=b), "out", [z(2, 3, 16)]),
        "short_conv_bwd": (dict(x=z(2, 3, 16), w=z(4, 16), b=b, dy=z(2, 3, 16)), "outs",
                           [z(2, 3, 16), z(4, 16), z(16)]),
    }


NAMES = ["layer_norm_fwd", "layer_norm_bwd", "gla_step", "ssd_step", "linear_ce_fwd", "linear_ce_bwd", "gla_fwd",
         "gla_bwd", "norm_gate_fwd", "norm_gate_bwd", "short_conv_fwd", "short_conv_bwd"]


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


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_do_not_fit(cuda_ok, name):
    args, key, outs = calls()[name]
    call = getattr(glc, name)
    more = (None,) if name == "gla_bwd" else ()  # no dh0
    given = lambda o: {key: o[0] if key == "out" else tuple(o) + more}
    got = call(**args, **given(outs))
    got = got[:len(outs)] if isinstance(got, tuple) else (got,)
    assert all(a is b for a, b in zip(got, outs))
    call(**args, **given([o.flatten() for o in outs]))  # the axes are the caller's own
    for i, o in enumerate(outs):
        wide = torch.zeros(*o.shape[:-1], 2 * o.shape[-1], device="cuda")[..., ::2]
        for bad in (o[:1], o.flatten()[:-1], o.cpu(), o.as_subclass(Elsewhere), wide, o.double(), o.bfloat16()):
            with pytest.raises((ValueError, TypeError)):
                call(**args, **given(outs[:i] + [bad] + outs[i + 1:]))


@pytest.mark.parametrize("name", ["layer_norm_bwd", "linear_ce_fwd", "linear_ce_bwd", "gla_bwd", "norm_gate_bwd",
                                  "short_conv_bwd"])
def test_workspace_on_another_device(cuda_ok, name):
    args, _, _ = calls()[name]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    getattr(glc, name)(**args, workspace=ws)
    for bad in (ws.cpu(), ws.as_subclass(Elsewhere)):
        with pytest.raises(ValueError):
            getattr(glc, name)(**args, workspace=bad)
