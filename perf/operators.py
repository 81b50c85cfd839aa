"""Cases of the operators around the recurrence in a language model: the layer
norm in front of a layer (forward, backward with the weight gradients), the
recurrence one token at a time on a pool of states (per-key-channel and
per-head decay), and the softmax cross entropy of the output projection
(forward, backward) that keeps no logits.

listed() and draw() give cases, prepare() their inputs on the GPU, run() one
pass (the library's calls where `own` is true, plain torch operations in 32
bits where it is false), exact() the same outputs from the definitions in 64
bits, work() the bytes and operations that a pass cannot do without."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # decoding one sequence: the norm of one token of a 16 x 128 wide model
        dict(name="norm one token", op="norm_fwd", dtype="bf16", rows=1, D=2048),
        # a training batch of 4 x 2048 tokens of that model
        dict(name="norm batch", op="norm_fwd", dtype="bf16", rows=8192, D=2048),
        dict(name="norm grad batch", op="norm_bwd", dtype="bf16", rows=8192, D=2048),
        # fp32 training, a width and a token count that no vector length divides
        dict(name="norm grad odd f32", op="norm_bwd", dtype="f32", rows=4099, D=1111),
        # decoding one sequence: 16 heads of 128 x 128 states
        dict(name="gla step one", op="step", kind="gla", dtype="bf16", B=1, T=1, H=16, Hqk=16, K=128, V=128, spare=0,
             fused=False),
        # a serving batch of 256 sequences out of a pool of 300, q, k, v read from one projection
        dict(name="gla step batch", op="step", kind="gla", dtype="bf16", B=256, T=1, H=16, Hqk=16, K=128, V=128,
             spare=44, fused=True),
        # a serving batch with one decay per head: 32 heads of 128 x 64 states, one q / k head
        dict(name="ssd step batch", op="step", kind="ssd", dtype="bf16", B=128, T=1, H=32, Hqk=1, K=128, V=64,
             spare=16, fused=False),
        # a few new tokens at once (a draft to verify), odd head sizes, shared q / k heads, fp32
        dict(name="gla step odd f32", op="step", kind="gla", dtype="f32", B=33, T=5, H=6, Hqk=2, K=72, V=41, spare=3,
             fused=True),
        # scoring a few tokens: the vocabulary is read once and little else happens
        dict(name="loss few tokens", op="ce_fwd", dtype="bf16", N=16, D=2048, V=32000),
        # the loss of a training batch and its gradient
        dict(name="loss batch", op="ce_fwd", dtype="bf16", N=8192, D=2048, V=32000),
        dict(name="loss grad batch", op="ce_bwd", dtype="bf16", N=8192, D=2048, V=32000),
        # fp32 training of a small model, a vocabulary that is no multiple of anything
        dict(name="loss grad odd f32", op="ce_bwd", dtype="f32", N=1001, D=520, V=10007),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "step", "step", "ce_fwd", "ce_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 8, 8192)
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, max(1, min(16384, (1 << 24) // D))), D=D)
    if op == "step":
        kind = rng.choice(["gla", "ssd"])
        Hqk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hqk * rng.choice([1, 1, 2, 4])
        K = rng.choice([128, 64, _log(rng, 8, 256)])
        V = rng.choice([128, 64, _log(rng, 8, 256)])
        B = _log(rng, 1, max(1, min(512, (1 << 26) // (H * K * V))))
        T = rng.choice([1, 1, 1, rng.randint(2, 8)])
        return dict(op=op, kind=kind, dtype=dtype, B=B, T=T, H=H, Hqk=Hqk, K=K, V=V, spare=rng.randint(0, 9),
                    fused=rng.random() < 0.5)
    D = 8 * _log(rng, 4, 256)
    N, V = _log(rng, 1, 8192), _log(rng, 100, 32000)
    if dtype == "f32":  # fp32 products take several times as long
        N = min(N, 2048)
    return dict(op=op, dtype=dtype, N=N, D=D, V=V)


def work(case):
    es = SIZES[case["dtype"]]
    if case["op"] == "norm_fwd":
        n, D = case["rows"], case["D"]
        # x in; y, the two row statistics and the two weights
        return {"bytes": 2 * n * D * es + 8 * n + 8 * D, "flops": 8 * n * D}
    if case["op"] == "norm_bwd":
        n, D = case["rows"], case["D"]
        # x, dy, statistics, w in; dx, dw, db out
        return {"bytes": 3 * n * D * es + 8 * n + 12 * D, "flops": 14 * n * D}
    if case["op"] == "step":
        B, T, H, Hqk, K, V = (case[n] for n in ("B", "T", "H", "Hqk", "K", "V"))
        gate = K if case["kind"] == "gla" else 1
        state = 2 * B * H * K * V * 4  # read once, written once
        rows = B * T * ((2 * Hqk * K + 2 * H * V) * es + H * gate * 4) + 4 * B
        # decay, k v^T added, q . S
        return {"bytes": state + rows, "flops": 5 * B * T * H * K * V}
    N, D, V = case["N"], case["D"], case["V"]
    if case["op"] == "ce_fwd":
        return {"bytes": (N + V) * D * es + 16 * N, "flops": 2 * N * V * D}
    # x, w, targets, lse, dloss in; dx, dw out.  The logits are not kept, so
    # they are one product, the two gradients one each.
    return {"bytes": 2 * (N + V) * D * es + 16 * N, "flops": 6 * N * V * D}


# ----------------------------------------------------------------- inputs ----
def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] in ("norm_fwd", "norm_bwd"):
        n, D = case["rows"], case["D"]
        # a residual stream: channels of unlike size, some off centre
        x = (randn(n, D) * (1 + 2 * randn(D).abs()) + 0.3 * randn(D)).to(dt)
        s = dict(case=case, x=x, w=1 + 0.1 * randn(D), b=0.1 * randn(D))
        if case["op"] == "norm_bwd":
            xf = x.double()  # the statistics that the forward pass handed on
            mean = xf.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((xf - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            s["dy"] = randn(n, D).to(dt)
        return s

    if case["op"] == "step":
        B, T, H, Hqk, K, V = (case[n] for n in ("B", "T", "H", "Hqk", "K", "V"))
        q, v = randn(B, T, Hqk, K), randn(B, T, H, V)
        k = torch.nn.functional.normalize(randn(B, T, Hqk, K), dim=-1)
        if case["fused"]:  # one projection's output, q, k and v views of it
            p = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], dim=2).to(dt)
            q, k, v = p.split([Hqk * K, Hqk * K, H * V], dim=2)
            q, k, v = q.unflatten(2, (Hqk, K)), k.unflatten(2, (Hqk, K)), v.unflatten(2, (H, V))
        else:
            q, k, v = q.to(dt), k.to(dt), v.to(dt)
        if case["kind"] == "gla":
            g = torch.nn.functional.logsigmoid(randn(B, T, H, K)) / 16
            scale = K ** -0.5
        else:
            g = -torch.nn.functional.softplus(randn(B, T, H) - 4) * torch.linspace(0, math.log(16), H, device="cuda").exp()
            scale = 1.0
        slots = B + case["spare"]
        state = 0.5 * randn(slots, H, K, V)
        idx = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
        return dict(case=case, q=q, k=k, v=v, g=g, state=state, idx=idx, scale=scale)

    N, D, V = case["N"], case["D"], case["V"]
    w = (randn(V, D) * (2 * D ** -0.5)).to(dt)
    target = torch.randint(0, V, (N,), generator=gen, device="cuda")
    # a model part of the way through its training: some tokens are foreseen
    # well (the target's logit is up to 16 above its noise), some not at all
    x = (randn(N, D) + 4 * torch.rand(N, 1, generator=gen, device="cuda") * w[target].float()).to(dt)
    skipped = torch.rand(N, generator=gen, device="cuda") < 0.05
    skipped[0] = False
    target = torch.where(skipped, -100, target)
    s = dict(case=case, x=x, w=w, target=target)
    if case["op"] == "ce_bwd":
        s["lse"] = torch.logsumexp(x.float() @ w.float().T, dim=1)  # handed on by the forward pass
        s["dloss"] = torch.full((N,), 1.0, device="cuda") / (~skipped).sum()
    return s


# ------------------------------------------------------------ plain forms ----
def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["w"] + s["b"]
    return y.to(s["x"].dtype), mean, rstd


def _norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    a = dy * s["w"]
    dx = s["rstd"][:, None] * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * n).sum(0), dy.sum(0)


def _step(s):
    q, k, v, g = (s[n].float().transpose(1, 2) for n in ("q", "k", "v", "g"))  # [B, heads, T, ...]
    H, T = v.shape[1], v.shape[2]
    share = H // q.shape[1]
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    g = g[..., None] if g.dim() == 3 else g
    G = g.cumsum(2)
    idx = s["idx"].long()
    S = s["state"][idx]
    # what the tokens of this call add, decayed from token r to token t >= r
    seen = torch.ones(T, T, dtype=torch.bool, device=q.device).tril()[:, :, None]
    decay = (G[:, :, :, None] - G[:, :, None]).masked_fill(~seen, -math.inf).exp()
    A = (q[:, :, :, None] * k[:, :, None] * decay).sum(-1)
    o = s["scale"] * ((q * G.exp()) @ S + A @ v)
    end = G[:, :, -1:]
    S = S * end.exp().transpose(2, 3) + (k * (end - G).exp()).transpose(2, 3) @ v
    s["state"][idx] = S
    return o.transpose(1, 2).contiguous().to(s["q"].dtype), s["state"]


def _ce_fwd(s):
    z = s["x"].float() @ s["w"].float().T
    m = z.amax(1)
    lse = m + (z - m[:, None]).exp().sum(1).log()
    t = s["target"]
    loss = lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return torch.where(t < 0, 0.0, loss), lse


def _ce_bwd(s):
    x, w, t = s["x"].float(), s["w"].float(), s["target"]
    G = (x @ w.T - s["lse"][:, None]).exp()
    G.scatter_add_(1, t.clamp(min=0)[:, None], torch.full_like(G[:, :1], -1.0))
    G = G * torch.where(t < 0, 0.0, s["dloss"])[:, None]
    return (G @ w).to(s["x"].dtype), (G.T @ x).to(s["w"].dtype)


PLAIN = dict(norm_fwd=_norm_fwd, norm_bwd=_norm_bwd, step=_step, ce_fwd=_ce_fwd, ce_bwd=_ce_bwd)


def run(s):
    op = s["case"]["op"]
    if not own:
        return PLAIN[op](s)
    import chunked_gated_linear_chunk_gb300 as glc

    if op == "norm_fwd":
        return glc.layer_norm_fwd(s["x"], s["w"], s["b"], EPS)
    if op == "norm_bwd":
        return glc.layer_norm_bwd(s["x"], s["w"], s["mean"], s["rstd"], s["dy"])
    if op == "step":
        step = glc.gla_step if s["case"]["kind"] == "gla" else glc.ssd_step
        return step(s["q"], s["k"], s["v"], s["g"], s["state"], s["idx"], s["scale"]), s["state"]
    if op == "ce_fwd":
        return glc.linear_ce_fwd(s["x"], s["w"], s["target"])
    return glc.linear_ce_bwd(s["x"], s["w"], s["target"], s["lse"], s["dloss"])


# ---------------------------------------------------- definitions, 64 bits ----
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        x, w = s["x"].double(), s["w"].double()
        if case["op"] == "norm_fwd":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            std = (var + EPS).sqrt()
            return (x - mean[:, None]) / std[:, None] * w + s["b"].double(), mean, 1 / std
        dy, mean, r = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        D = x.shape[1]
        # dL/dn of the normalised row n, then through n's own row statistics
        n = (x - mean) * r
        dn = dy * w
        dx = r / D * (D * dn - dn.sum(1, keepdim=True) - n * torch.einsum("rd,rd->r", dn, n)[:, None])
        return dx, torch.einsum("rd,rd->d", dy, n), dy.sum(0)
    if case["op"] == "step":
        q, k, v, g = (s[n].double() for n in ("q", "k", "v", "g"))
        H, share = case["H"], case["H"] // case["Hqk"]
        head = torch.arange(H, device="cuda") // share
        idx = s["idx"].long()
        S, out = s["state"][idx].double(), []
        for t in range(case["T"]):
            a = g[:, t].exp()
            a = a[..., None, None] if case["kind"] == "ssd" else a[..., None]
            S = S * a + torch.einsum("bhk,bhv->bhkv", k[:, t][:, head], v[:, t])
            out.append(s["scale"] * torch.einsum("bhk,bhkv->bhv", q[:, t][:, head], S))
        state = s["state"].double()
        state[idx] = S
        return torch.stack(out, 1), state
    x, w, t = s["x"].double(), s["w"].double(), s["target"]
    z = torch.einsum("nd,vd->nv", x, w)
    here = torch.arange(case["V"], device="cuda")[None] == t[:, None]
    if case["op"] == "ce_fwd":
        lse = torch.logsumexp(z, 1)
        return (lse - (z * here).sum(1)) * (t >= 0), lse
    G = (z - s["lse"].double()[:, None]).exp().sub_(here.double()) * (s["dloss"].double() * (t >= 0))[:, None]
    return torch.einsum("nv,vd->nd", G, w), torch.einsum("nv,nd->vd", G, x)
