"""The example model: its loss falls, its autograd wrappers agree with plain
torch in fp32, and serving token by token gives the chunked pass's logits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("linear_lm", os.path.join(ROOT, "examples", "linear_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trains_and_serves(cuda_ok, lm):
    r = lm.main(steps=150)
    assert r["losses"][-1] < 0.5 * r["losses"][0]  # log 96 = 4.6 at first
    # bf16 activations through two layers: a few roundings of 2^-8 each
    assert r["apart"] < 4e-2


def plain(lm, p, tokens, target):
    """The model in plain torch, fp32, the recurrence token by token."""
    x = torch.nn.functional.embedding(tokens, p["embed"])
    B, T, W = x.shape
    ln = lambda x, w, b: torch.nn.functional.layer_norm(x, (W,), w, b, 1e-5)
    for i in range(lm.LAYERS):
        h = ln(x, p[f"{i}.norm_w"], p[f"{i}.norm_b"])
        q, k, v, z = (h @ p[f"{i}.qkvz"]).view(B, T, 4, lm.HEADS, lm.DIM).unbind(2)
        k = torch.nn.functional.normalize(k, dim=-1)
        a = (torch.nn.functional.logsigmoid(h @ p[f"{i}.gate"]).view(B, T, lm.HEADS, lm.DIM) / 16).exp()
        S, o = 0, []
        for t in range(T):
            S = a[:, t, :, :, None] * S + k[:, t, :, :, None] * v[:, t, :, None]
            o.append(lm.DIM ** -0.5 * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
        o = torch.stack(o, 1)
        o = o * (o.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * p[f"{i}.out_norm"] * z * z.sigmoid()
        x = x + o.reshape(B, T, W) @ p[f"{i}.out"]
    z = ln(x, p["norm_w"], p["norm_b"]) @ p["head"]
    return torch.nn.functional.cross_entropy(z.reshape(B * T, -1), target.reshape(-1), ignore_index=-1)


def test_gradients_against_plain_torch(cuda_ok, lm):
    """Every weight's gradient points the way the fp32 model's does (bf16
    activations: cosine above 0.99) and has its length within 5%."""
    gen = torch.Generator("cpu")
    gen.manual_seed(3)
    p = lm.make(3, "cuda")
    tokens = lm.text(2, 33, gen, "cuda")
    target = tokens[:, 1:].clone()
    target[:, 0] = -1
    h = lm.trunk(p, tokens[:, :-1], lambda i, q, k, v, g: lm.Recurrence.apply(q, k, v, g))
    loss = lm.Loss.apply(h.reshape(-1, lm.WIDTH), p["head"].t().bfloat16().contiguous(), target.reshape(-1))
    loss.backward()
    got = {n: t.grad.clone() for n, t in p.items()}
    for t in p.values():
        t.grad = None
    ref = plain(lm, p, tokens[:, :-1], target)
    ref.backward()
    assert abs(float(loss.detach()) - float(ref.detach())) < 2e-2 * float(ref.detach())
    for n, t in p.items():
        a, b = got[n].double().flatten(), t.grad.double().flatten()
        assert float(a @ b / (a.norm() * b.norm())) > 0.99, n
        assert abs(float(a.norm() / b.norm()) - 1) < 0.05, n
