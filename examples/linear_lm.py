"""A small linear-attention language model, trained and then served with the
library's operators:

    training   embedding -> layers of [layer norm -> q, k, v, gate projections
               -> GLA recurrence -> RMSNorm x swish gate -> output projection]
               -> layer norm -> softmax cross entropy of the output projection
               (the logits are never kept), gradients by the library's backward
               calls
    serving    the prompt through the chunked recurrence, whose final states
               fill slots of a state pool; then one token at a time for all
               sequences on the pool

The text is synthetic: every sequence counts up modulo the vocabulary by a
step that its first two tokens give away, so that a model that has learned can
go on counting.

    python examples/linear_lm.py [--steps 150]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_linear_chunk_gb300 as glc  # noqa: E402

HEADS, DIM, VOCAB, LAYERS = 2, 128, 96, 2
WIDTH = HEADS * DIM


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b):
        y, mean, rstd = glc.layer_norm_fwd(x, w, b)
        ctx.save_for_backward(x, w, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        return glc.layer_norm_bwd(*ctx.saved_tensors, dy)


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g):
        ctx.save_for_backward(q, k, v, g)
        return glc.gla_fwd(q, k, v, g)[0]

    @staticmethod
    def backward(ctx, do):
        return glc.gla_bwd(*ctx.saved_tensors, do)[:4]


class NormGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, z, w):
        ctx.save_for_backward(o, z, w)
        return glc.norm_gate_fwd(o, z, w)

    @staticmethod
    def backward(ctx, dy):
        return glc.norm_gate_bwd(*ctx.saved_tensors, dy)


class Loss(torch.autograd.Function):
    """Mean loss over the scored tokens (target >= 0)."""

    @staticmethod
    def forward(ctx, x, w, target):
        loss, lse = glc.linear_ce_fwd(x, w, target)
        count = (target >= 0).sum()
        ctx.save_for_backward(x, w, target, lse, count)
        return loss.sum() / count

    @staticmethod
    def backward(ctx, dmean):
        x, w, target, lse, count = ctx.saved_tensors
        dloss = (dmean / count).float().expand(len(target)).contiguous()
        return *glc.linear_ce_bwd(x, w, target, lse, dloss), None


def make(seed, device):
    """fp32 weights; the products run in bf16."""
    gen = torch.Generator("cpu")
    gen.manual_seed(seed)

    def weight(rows, cols, scale=1.0):
        return (torch.randn(rows, cols, generator=gen) * scale * rows ** -0.5).to(device).requires_grad_()

    def flat(n, value):
        return torch.full((n,), value, device=device, requires_grad=True)

    p = {"embed": (torch.randn(VOCAB, WIDTH, generator=gen)).to(device).requires_grad_(),
         "norm_w": flat(WIDTH, 1.0), "norm_b": flat(WIDTH, 0.0), "head": weight(WIDTH, VOCAB)}
    for i in range(LAYERS):
        p[f"{i}.norm_w"], p[f"{i}.norm_b"] = flat(WIDTH, 1.0), flat(WIDTH, 0.0)
        p[f"{i}.qkvz"] = weight(WIDTH, 4 * WIDTH)
        p[f"{i}.gate"] = weight(WIDTH, WIDTH)
        p[f"{i}.out_norm"] = flat(DIM, 1.0)
        p[f"{i}.out"] = weight(WIDTH, WIDTH, 0.5)
    return p


def project(p, i, h):
    """q, k, v, z [B,T,H,D] bf16 (views of one projection) and the log decay."""
    B, T, _ = h.shape
    q, k, v, z = (h @ p[f"{i}.qkvz"].bfloat16()).view(B, T, 4, HEADS, DIM).unbind(2)
    k = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
    g = torch.nn.functional.logsigmoid((h @ p[f"{i}.gate"].bfloat16()).float()).view(B, T, HEADS, DIM) / 16
    return q, k, v.contiguous(), z.contiguous(), g


def trunk(p, tokens, recurrence):
    """Hidden states [B,T,WIDTH] before the output projection; recurrence(i, q,
    k, v, g) is layer i's token mixing."""
    x = torch.nn.functional.embedding(tokens, p["embed"]).bfloat16()
    B, T, _ = x.shape
    for i in range(LAYERS):
        q, k, v, z, g = project(p, i, Norm.apply(x, p[f"{i}.norm_w"], p[f"{i}.norm_b"]))
        o = NormGate.apply(recurrence(i, q, k, v, g), z, p[f"{i}.out_norm"])
        x = x + o.reshape(B, T, WIDTH) @ p[f"{i}.out"].bfloat16()
    return Norm.apply(x, p["norm_w"], p["norm_b"])


def text(batch, length, gen, device):
    start = torch.randint(0, VOCAB, (batch, 1), generator=gen)
    step = torch.randint(1, 8, (batch, 1), generator=gen)
    return ((start + step * torch.arange(length)) % VOCAB).to(device)


def train(p, steps, gen, device, batch=8, length=128, lr=3e-3):
    opt = torch.optim.Adam(list(p.values()), lr=lr)
    losses = []
    for n in range(steps):
        tokens = text(batch, length + 1, gen, device)
        target = tokens[:, 1:].clone()
        target[:, 0] = -1  # the second token cannot be foreseen
        h = trunk(p, tokens[:, :-1], lambda i, q, k, v, g: Recurrence.apply(q, k, v, g))
        loss = Loss.apply(h.reshape(-1, WIDTH), p["head"].t().bfloat16().contiguous(), target.reshape(-1))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def serve(p, prompt, new, slots=None):
    """Greedy continuation by `new` tokens: (tokens [B, new], logits of each)."""
    B = prompt.shape[0]
    slots = slots if slots is not None else torch.arange(B, dtype=torch.int32, device=prompt.device)
    pools = [torch.zeros(int(slots.max()) + 1, HEADS, DIM, DIM, device=prompt.device) for _ in range(LAYERS)]

    def first(i, q, k, v, g):
        o, final = glc.gla_fwd(q, k, v, g, output_final_state=True)
        pools[i][slots.long()] = final
        return o

    head = p["head"].bfloat16()
    logits = [(trunk(p, prompt, first)[:, -1] @ head).float()]
    tokens = [logits[-1].argmax(1)]
    while len(tokens) < new:
        h = trunk(p, tokens[-1][:, None], lambda i, q, k, v, g: glc.gla_step(q, k, v, g, pools[i], slots))
        logits.append((h[:, -1] @ head).float())
        tokens.append(logits[-1].argmax(1))
    return torch.stack(tokens, 1), torch.stack(logits, 1)


@torch.no_grad()
def whole(p, tokens):
    """Logits of every position by one chunked pass."""
    return (trunk(p, tokens, lambda i, q, k, v, g: glc.gla_fwd(q, k, v, g)[0]) @ p["head"].bfloat16()).float()


def main(steps=150, device="cuda", seed=0):
    gen = torch.Generator("cpu")
    gen.manual_seed(seed)
    p = make(seed, device)
    losses = train(p, steps, gen, device)
    tokens = text(6, 60, gen, device)
    prompt, rest = tokens[:, :40], tokens[:, 40:]
    slots = torch.tensor([7, 0, 3, 5, 2, 6], dtype=torch.int32, device=device)
    out, logits = serve(p, prompt, rest.shape[1], slots)
    again = whole(p, torch.cat([prompt, out], 1))[:, 39:-1]
    glc.get_device_error()
    return dict(losses=losses, right=float((out == rest).float().mean()),
                apart=float((logits - again).abs().max() / again.abs().max()))


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=150)
    r = main(ap.parse_args().steps)
    print("loss: first %.3f, last %.3f" % (r["losses"][0], r["losses"][-1]))
    print("continued tokens that are right: %.0f%%" % (100 * r["right"]))
    print("logits token by token against one chunked pass: %.1e of the largest" % r["apart"])
