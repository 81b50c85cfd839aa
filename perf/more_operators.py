"""Cases of the gated delta rule (over whole sequences forward and backward,
and token by token on a pool of states) and of what stands in front of it: the
norm of every query and key head with the rotation by position in the same pass
(forward, backward with the weight gradients).

listed() and draw() give cases, prepare() their inputs on the GPU, run() one
pass (the library's calls where `own` is true, plain torch operations in 32
bits where it is false), exact() the same outputs from the definitions in 64
bits, token by token, work() the bytes and operations that a pass cannot do
without.

The gated delta rule, S of K x V for every sequence and head:
    u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t)
    S_t = exp(g_t) S_{t-1} + k_t u_t^T,   o_t = scale S_t^T q_t
The head norm of a row x of D channels, then the rotation of its first 2 R:
    n = x r w,  r = (mean(x^2) + eps)^(-1/2)   ("l2": the sum in the mean's place)
    (n_i, n_j) -> (n_i c - n_j s, n_j c + n_i s),  j = i + R, c, s of position and i"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
EPS = 1e-6
CHUNK = 64  # tokens that the plain form treats as one matrix
NORM_OPS = ("norm_fwd", "norm_bwd")


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # a short prompt of one sequence, its state kept for the tokens to come
        dict(name="delta prompt", op="fwd", dtype="bf16", B=1, T=96, H=16, Hqk=16, K=128, V=128, docs=1, states=True),
        # the layer of a training batch: 16 heads of 128 x 128
        dict(name="delta batch", op="fwd", dtype="bf16", B=4, T=2048, H=16, Hqk=16, K=128, V=128, docs=1, states=False),
        # 16 documents packed into one row of a training batch, q and k shared by pairs of heads
        dict(name="delta packed", op="fwd", dtype="bf16", B=1, T=16384, H=16, Hqk=8, K=128, V=128, docs=16,
             states=False),
        # the gradients of a training batch
        dict(name="delta grad batch", op="bwd", dtype="bf16", B=4, T=2048, H=16, Hqk=16, K=128, V=128, docs=1,
             states=False),
        # value heads of 64 over shared q and k heads, packed documents that end anywhere
        dict(name="delta grad packed", op="bwd", dtype="bf16", B=2, T=3001, H=16, Hqk=4, K=128, V=64, docs=5,
             states=False),
        # fp32 training of a small model, sizes that nothing divides, states handed in and out
        dict(name="delta grad odd f32", op="bwd", dtype="f32", B=3, T=333, H=6, Hqk=2, K=72, V=41, docs=1, states=True),
        # decoding one sequence
        dict(name="delta step one", op="step", dtype="bf16", B=1, T=1, H=16, Hqk=16, K=128, V=128, spare=0, fused=False),
        # a serving batch of 256 sequences out of a pool of 300, q, k, v read from one projection
        dict(name="delta step batch", op="step", dtype="bf16", B=256, T=1, H=16, Hqk=16, K=128, V=128, spare=44,
             fused=True),
        # one token's queries and keys
        dict(name="head norm one token", op="norm_fwd", dtype="bf16", B=1, T=1, Hq=16, Hk=16, D=128, R=64, norm="rms",
             fused=True),
        # those of a training batch, read from one projection
        dict(name="head norm batch", op="norm_fwd", dtype="bf16", B=4, T=2048, Hq=16, Hk=16, D=128, R=64, norm="rms",
             fused=True),
        dict(name="head norm grad batch", op="norm_bwd", dtype="bf16", B=4, T=2048, Hq=16, Hk=16, D=128, R=64,
             norm="rms", fused=True),
        # fp32, heads of 72 of which 48 turn, the norm to unit length that the delta rule takes
        dict(name="head norm grad odd f32", op="norm_bwd", dtype="f32", B=3, T=333, Hq=6, Hk=2, D=72, R=24, norm="l2",
             fused=False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in NORM_OPS:
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        D = rng.choice([128, 64, 256, _log(rng, 8, 256)])
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, (1 << 25) // (T * (Hq + Hk) * D))))
        return dict(op=op, dtype=dtype, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=rng.choice([0, D // 2, D // 4]),
                    norm=rng.choice(["rms", "l2"]), fused=rng.random() < 0.5)
    Hqk = rng.choice([1, 2, 3, 4, 8, 16])
    H = Hqk * rng.choice([1, 1, 2, 4])
    K = rng.choice([128, 128, 64, _log(rng, 8, 256)])
    V = rng.choice([128, 128, 64, _log(rng, 8, 256)])
    if op == "step":
        B = _log(rng, 1, max(1, min(512, (1 << 26) // (H * K * V))))
        return dict(op=op, dtype=dtype, B=B, T=rng.choice([1, 1, 1, rng.randint(2, 8)]), H=H, Hqk=Hqk, K=K, V=V,
                    spare=rng.randint(0, 9), fused=rng.random() < 0.5)
    most = (1 << 31) // (H * K * V)  # tokens that cost as much as the batch of the listed cases
    if dtype == "f32":
        most //= 4
    T = _log(rng, 1, min(16384, max(1, most)))
    B = _log(rng, 1, max(1, min(16, most // T)))
    docs = rng.choice([1, 1, max(1, min(T, _log(rng, 1, 40)))])
    return dict(op=op, dtype=dtype, B=B, T=T, H=H, Hqk=Hqk, K=K, V=V, docs=docs, states=docs == 1 and rng.random() < 0.5)


def work(case):
    es = SIZES[case["dtype"]]
    if case["op"] in NORM_OPS:
        B, T, Hq, Hk, D, R = (case[n] for n in ("B", "T", "Hq", "Hk", "D", "R"))
        n = B * T * (Hq + Hk)
        turn = T * R * 8 + B * T * 4 if R else 0  # the rows of the two tables that the positions name, the positions
        if case["op"] == "norm_fwd":  # x in, y out, two weights; squares, two scalings, the rotation
            return {"bytes": 2 * n * D * es + 8 * D + turn, "flops": n * (4 * D + 6 * R)}
        # x, dy in, dx out, the weights in and their gradients out
        return {"bytes": 3 * n * D * es + 16 * D + turn, "flops": n * (12 * D + 6 * R)}
    B, T, H, Hqk, K, V = (case[n] for n in ("B", "T", "H", "Hqk", "K", "V"))
    rows = B * T * (2 * Hqk * K * es + H * V * es + 8 * H)  # q, k, v, g, beta
    if case["op"] == "step":
        # the states read and written; S^T k, k u^T, S^T q of every token and the decay
        return {"bytes": 8 * B * H * K * V + rows + B * T * H * V * es + 4 * B, "flops": 7 * B * T * H * K * V}
    state = 4 * B * H * K * V if case["states"] else 0
    seg = 4 * B * T if case["docs"] > 1 else 0
    if case["op"] == "fwd":
        return {"bytes": rows + B * T * H * V * es + 2 * state + seg, "flops": 7 * B * T * H * K * V}
    # do in, every gradient out; the states again (5 K V), then S do, q do^T, dS^T k, k du^T, dS u, S du, the decay
    return {"bytes": 2 * rows + B * T * H * V * es + 3 * state + seg, "flops": 18 * B * T * H * K * V}


# ----------------------------------------------------------------- inputs ----
def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    F = torch.nn.functional

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    B, T = case["B"], case["T"]
    if case["op"] in NORM_OPS:
        Hq, Hk, D, R = (case[n] for n in ("Hq", "Hk", "D", "R"))
        q, k = 2 * randn(B, T, Hq, D), 2 * randn(B, T, Hk, D)
        if case["fused"]:  # q and k as views of one projection that holds as many value heads as key heads
            p = torch.cat([q.flatten(2), k.flatten(2), randn(B, T, Hk * D)], dim=2).to(dt)
            q, k, _ = p.split([Hq * D, Hk * D, Hk * D], dim=2)
            q, k = q.unflatten(2, (Hq, D)), k.unflatten(2, (Hk, D))
        else:
            q, k = q.to(dt), k.to(dt)
        s = dict(case=case, q=q, k=k, wq=1 + 0.2 * randn(D), wk=1 + 0.2 * randn(D), cos=None, sin=None, positions=None)
        if R:  # tables for 8192 positions, the sequences somewhere in them
            angle = torch.arange(8192, device="cuda").double()[:, None] * torch.pow(
                torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -torch.arange(R, device="cuda") / R)
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
            first = torch.randint(0, 8192 - T, (B, 1), generator=gen, device="cuda")
            s["positions"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
        if case["op"] == "norm_bwd":
            s["dq"], s["dk"] = randn(B, T, Hq, D).to(dt), randn(B, T, Hk, D).to(dt)
        return s

    H, Hqk, K, V = (case[n] for n in ("H", "Hqk", "K", "V"))
    # queries and keys of unit length after a SiLU, as a delta rule layer makes them
    q = F.normalize(F.silu(randn(B, T, Hqk, K) + 0.3), dim=-1)
    k = F.normalize(F.silu(randn(B, T, Hqk, K) + 0.3), dim=-1)
    v = randn(B, T, H, V)
    if case.get("fused"):  # one projection's output, q, k and v views of it
        p = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], dim=2).to(dt)
        q, k, v = p.split([Hqk * K, Hqk * K, H * V], dim=2)
        q, k, v = q.unflatten(2, (Hqk, K)), k.unflatten(2, (Hqk, K)), v.unflatten(2, (H, V))
    else:
        q, k, v = q.to(dt), k.to(dt), v.to(dt)
    # decays of heads that remember a few tokens up to those that remember thousands
    rate = torch.linspace(0, math.log(16), H, device="cuda").exp()
    g = -F.softplus(randn(B, T, H) - 4) * rate
    beta = randn(B, T, H).sigmoid()
    s = dict(case=case, q=q, k=k, v=v, g=g, beta=beta, scale=K ** -0.5)
    if case["op"] == "step":
        slots = B + case["spare"]
        s["state"] = 0.5 * randn(slots, H, K, V)
        s["idx"] = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
        return s
    s["h0"] = 0.1 * randn(B, H, K, V) if case["states"] else None
    s["seg"], s["n"] = None, B
    if case["docs"] > 1:  # every row starts its own documents, at other tokens than the other rows
        cut = torch.stack([torch.randperm(T - 1, generator=gen, device="cuda")[:case["docs"] - 1] for _ in range(B)]) + 1
        first = torch.zeros(B, T, dtype=torch.int32, device="cuda").scatter_(1, cut, 1)
        s["seg"], s["n"] = first.cumsum(1, dtype=torch.int32), B * case["docs"]
    if case["op"] == "bwd":
        s["do"] = randn(B, T, H, V).to(dt)
        s["dht"] = 0.1 * randn(B, H, K, V) if case["states"] else None
    return s


# ------------------------------------------------------------ plain forms ----
# One chunk of C tokens as matrices (G: the sum of g from the chunk's start,
# D_ts = exp(G_t - G_s) for s <= t within a document, N the part of D (k_t . k_s)
# below the diagonal): with Y = V - exp(G) K S the errors before the chunk's own
# tokens are counted,
#     E = (I + N diag(beta))^(-1) Y = Y + Z (beta Y),   U = beta E
#     O = scale (exp(G) Q S + (D (.) Q K^T) U),   S' = exp(G_C) S + K^T (exp(G_C - G) U)
def _chunks(x, share=1):
    """[B, T, heads, ...] as [B, heads, chunks, C, ...] in 32 bits; the tokens past T are zero."""
    x = x.float()
    B, T = x.shape[:2]
    n = -(-T // CHUNK)
    x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * CHUNK - T))
    return x.unflatten(1, (n, CHUNK)).movedim(3, 1).repeat_interleave(share, 1)


def _tokens(x, T, dtype):
    """The inverse of _chunks."""
    return x.movedim(1, 3).flatten(1, 2)[:, :T].contiguous().to(dtype)


def _per_head(s):
    """What a chunk takes from its own tokens."""
    share = s["case"]["H"] // s["case"]["Hqk"]
    c = dict(q=_chunks(s["q"], share), k=_chunks(s["k"], share), v=_chunks(s["v"]), g=_chunks(s["g"]),
             beta=_chunks(s["beta"]))
    seg = s["seg"] if s["seg"] is not None else torch.zeros_like(s["g"][..., 0], dtype=torch.int32)
    # which document of the chunk a token is in; documents start at a row's first token and where seg changes
    first = torch.cat([torch.ones_like(seg[:, :1]), (seg[:, 1:] != seg[:, :-1]).int()], 1)
    first[:, 0] = 0 if s["h0"] is not None else 1
    doc = _chunks(first[:, :, None])[:, :, :, :].cumsum(3)
    G = c["g"].cumsum(3)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    together = (doc[..., :, None] == doc[..., None, :]) & low
    c["D"] = (G[..., :, None] - G[..., None, :]).masked_fill(~together, -math.inf).exp()
    c["into"] = (G.exp() * (doc == 0))[..., None]  # of the state before the chunk
    last = doc[..., -1:]
    c["outof"] = ((G[..., -1:] - G).exp() * (doc == last))[..., None]
    c["over"] = (G[..., -1:].exp() * (last == 0))[..., None]
    c["A"] = c["k"] @ c["k"].mT
    N = (c["D"] * c["A"]).tril(-1)
    c["b"] = c["beta"][..., None]
    NB = N * c["b"].mT
    Z = -N
    for t in range(1, CHUNK):  # row t of (I + N diag(beta)) Z = -N, from those above
        Z[..., t:t + 1, :] -= NB[..., t:t + 1, :t] @ Z[..., :t, :]
    c["Z"] = Z
    c["P"] = s["scale"] * c["D"] * (c["q"] @ c["k"].mT)
    return c


def _states(s, c):
    """The state before each chunk, each chunk's E, the state after the last."""
    B, _, H, K, V = s["case"]["B"], s["case"]["T"], s["case"]["H"], s["case"]["K"], s["case"]["V"]
    S = s["h0"] if s["h0"] is not None else torch.zeros(B, H, K, V, device="cuda")
    before, errors = [], []
    for j in range(c["k"].shape[2]):
        before.append(S)
        k, b = c["k"][:, :, j], c["b"][:, :, j]
        Y = c["v"][:, :, j] - c["into"][:, :, j] * (k @ S)
        E = Y + c["Z"][:, :, j] @ (b * Y)
        errors.append(E)
        S = c["over"][:, :, j] * S + k.mT @ (c["outof"][:, :, j] * b * E)
    return torch.stack(before, 2), torch.stack(errors, 2), S


def _fwd(s):
    c = _per_head(s)
    before, E, S = _states(s, c)
    o = s["scale"] * c["into"] * (c["q"] @ before) + c["P"] @ (c["b"] * E)
    o = _tokens(o, s["case"]["T"], s["q"].dtype)
    return (o, S) if s["case"]["states"] else o


def _bwd(s):
    T, dt, scale = s["case"]["T"], s["q"].dtype, s["scale"]
    Hqk = s["case"]["Hqk"]
    c = _per_head(s)
    before, E, S = _states(s, c)
    do = _chunks(s["do"])
    dS = s["dht"] if s["dht"] is not None else torch.zeros_like(S)
    after, dR = [None] * do.shape[2], [None] * do.shape[2]
    PTdo, Qdo = c["P"].mT @ do, c["q"].mT @ (scale * c["into"] * do)
    for j in reversed(range(do.shape[2])):
        k, b = c["k"][:, :, j], c["b"][:, :, j]
        after[j] = dS
        dU = PTdo[:, :, j] + c["outof"][:, :, j] * (k @ dS)
        dR[j] = dU + c["Z"][:, :, j].mT @ (b * dU)
        dS = c["over"][:, :, j] * dS + Qdo[:, :, j] - k.mT @ (c["into"][:, :, j] * b * dR[j])
    after, dR = torch.stack(after, 2), torch.stack(dR, 2)
    U, dY = c["b"] * E, c["b"] * dR
    dbeta = (dR * E).sum(-1)
    dP = scale * c["D"] * (do @ U.mT)
    dA = -(c["D"] * (dY @ U.mT)).tril(-1)
    q_in = scale * c["into"] * (do @ before.mT)
    k_in = -c["into"] * (dY @ before.mT)
    k_out = c["outof"] * (U @ after.mT)
    dq = q_in + dP @ c["k"]
    dk = k_in + k_out + dP.mT @ c["q"] + (dA + dA.mT) @ c["k"]
    # g_t decays what the tokens before it handed to t and the tokens after: pairs r >= t > s, and the states
    W = (dP * (c["q"] @ c["k"].mT) + dA * c["A"]).tril(-1)
    pairs = (W.flip(3).cumsum(3).flip(3).cumsum(4) - W.flip(3).cumsum(3).flip(3)).diagonal(dim1=3, dim2=4)
    reads = ((c["q"] * q_in).sum(-1) + (c["k"] * k_in).sum(-1)).flip(3).cumsum(3).flip(3)
    adds = (c["k"] * k_out).sum(-1)
    dg = pairs + reads + adds.cumsum(3) - adds + (c["over"] * before * after).sum((-2, -1))[..., None]
    group = lambda x: x.unflatten(1, (Hqk, -1)).sum(2)  # noqa: E731  the heads that share one q and k
    out = (_tokens(group(dq), T, dt), _tokens(group(dk), T, dt), _tokens(dY, T, dt), _tokens(dg, T, torch.float32),
           _tokens(dbeta, T, torch.float32))
    return out + (dS,) if s["case"]["states"] else out


def _step(s):
    share = s["case"]["H"] // s["case"]["Hqk"]
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    q, k = q.repeat_interleave(share, 2), k.repeat_interleave(share, 2)
    idx = s["idx"].long()
    S, out = s["state"][idx], []
    for t in range(s["case"]["T"]):
        S = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None] @ S)[..., 0, :])
        S = S + k[:, t, :, :, None] * u[..., None, :]
        out.append(s["scale"] * (q[:, t, :, None] @ S)[..., 0, :])
    s["state"][idx] = S
    return torch.stack(out, 1).to(s["q"].dtype), s["state"]


def _turn(x, c, s, R):
    a, b = x[..., :R], x[..., R:2 * R]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * R:]], -1)


def _factors(s):
    """cos and sin of every token, [B, T, 1, R], or None."""
    if s["cos"] is None:
        return None, None
    p = s["positions"].long()
    return s["cos"][p][:, :, None], s["sin"][p][:, :, None]


def _rstd(x, norm):
    x2 = x.square()
    return ((x2.mean(-1, keepdim=True) if norm == "rms" else x2.sum(-1, keepdim=True)) + EPS).rsqrt()


def _norm_fwd(s):
    R, norm = s["case"]["R"], s["case"]["norm"]
    c, sn = _factors(s)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        y = y * _rstd(y, norm) * w
        y = _turn(y, c, sn, R) if R else y
        out.append(y.to(x.dtype))
    return tuple(out)


def _norm_bwd(s):
    R, norm = s["case"]["R"], s["case"]["norm"]
    c, sn = _factors(s)
    dx, dw = [], []
    for x, w, dy in ((s["q"], s["wq"], s["dq"]), (s["k"], s["wk"], s["dk"])):
        xf, d = x.float(), dy.float()
        d = _turn(d, c, -sn, R) if R else d  # the rotation back
        r = _rstd(xf, norm)
        n, a = xf * r, d * w
        an = a * n
        dx.append((r * (a - n * (an.mean(-1, keepdim=True) if norm == "rms" else an.sum(-1, keepdim=True)))).to(x.dtype))
        dw.append((d * n).sum((0, 1, 2)))
    return dx[0], dx[1], dw[0], dw[1]


PLAIN = dict(fwd=_fwd, bwd=_bwd, step=_step, norm_fwd=_norm_fwd, norm_bwd=_norm_bwd)


def run(s):
    op = s["case"]["op"]
    if not own:
        return PLAIN[op](s)
    import chunked_gated_linear_chunk_gb300 as glc

    if op == "norm_fwd":
        return glc.qk_norm_fwd(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], EPS,
                               s["case"]["norm"])
    if op == "norm_bwd":
        return glc.qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"],
                               EPS, s["case"]["norm"])
    if op == "step":
        return glc.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["idx"], s["scale"]), s["state"]
    if op == "fwd":
        o, ht = glc.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["seg"], s["h0"],
                              s["case"]["states"], n_seqs=s["n"])
        return (o, ht) if s["case"]["states"] else o
    out = glc.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], s["scale"], s["seg"], s["h0"], s["dht"],
                        n_seqs=s["n"])
    return out if s["case"]["states"] else out[:5]


# ---------------------------------------------------- definitions, 64 bits ----
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in NORM_OPS:
        out = []
        D, R = case["D"], case["R"]
        # the rotation of a token as a D x D matrix is the identity but for its R planes
        for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
            x, w = x.double(), w.double()
            m = x.pow(2).sum(-1, keepdim=True) / (D if case["norm"] == "rms" else 1) + EPS
            n = x / m.sqrt()
            z = torch.polar(torch.ones_like(m), torch.zeros_like(m))
            if R:
                z = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, :, None]
            y = (n * w if dy is None else dy.double()).clone()
            if R:
                t = torch.complex(y[..., :R].clone(), y[..., R:2 * R].clone()) * (z if dy is None else z.conj())
                y[..., :R], y[..., R:2 * R] = t.real, t.imag
            if dy is None:
                out.append(y)
                continue
            d = y * w  # dL/dn; n = x m^(-1/2), dm/dx = 2 x / D or 2 x
            dm = -(d * x).sum(-1, keepdim=True) / (2 * m.pow(1.5))
            out.append((d / m.sqrt() + dm * 2 * x / (D if case["norm"] == "rms" else 1),
                        torch.einsum("bthd,bthd->d", y, n)))
        return tuple(out) if case["op"] == "norm_fwd" else (out[0][0], out[1][0], out[0][1], out[1][1])

    B, T, H, Hqk, K, V = (case[n] for n in ("B", "T", "H", "Hqk", "K", "V"))
    if 3 * 8 * B * H * K * V * min(T, 64) > 60e9 or T > 20000:
        return None
    head = torch.arange(H, device="cuda") // (H // Hqk)
    q, k = s["q"].double()[:, :, head], s["k"].double()[:, :, head]
    v, a, beta = s["v"].double(), s["g"].double().exp()[..., None, None], s["beta"].double()[..., None]

    def token(S, t):
        S = a[:, t] * S
        e = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S)
        return S + torch.einsum("bhk,bhv->bhkv", k[:, t], beta[:, t] * e), e

    if case["op"] == "step":
        idx = s["idx"].long()
        S, out = s["state"][idx].double(), []
        for t in range(T):
            S, _ = token(S, t)
            out.append(s["scale"] * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
        state = s["state"].double()
        state[idx] = S
        return torch.stack(out, 1), state

    S = s["h0"].double() if s["h0"] is not None else torch.zeros(B, H, K, V, dtype=torch.float64, device="cuda")
    # 0 where a document starts within a row
    goes_on = torch.ones(B, T, dtype=torch.float64, device="cuda")
    if s["seg"] is not None:
        goes_on[:, 1:] = (s["seg"][:, 1:] == s["seg"][:, :-1]).double()
    goes_on = goes_on[:, :, None, None, None]
    if case["op"] == "fwd":
        out = []
        for t in range(T):
            S, _ = token(goes_on[:, t] * S, t)
            out.append(s["scale"] * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
        o = torch.stack(out, 1)
        return (o, S) if case["states"] else o

    # the tokens backwards, the states of a stretch of tokens computed again from its first
    step, kept = 64, []
    for t in range(T):
        if t % step == 0:
            kept.append(S)
        S, _ = token(goes_on[:, t] * S, t)
    do = s["do"].double()
    dS = s["dht"].double() if s["dht"] is not None else torch.zeros_like(S)
    grads = [None] * T
    for t0 in reversed(range(0, T, step)):
        S, states = kept.pop(), []
        for t in range(t0, min(T, t0 + step)):
            before = goes_on[:, t] * S
            S, e = token(before, t)
            states.append((before, S, e))
        for t in reversed(range(t0, min(T, t0 + step))):
            before, S, e = states[t - t0]
            dS = dS + s["scale"] * torch.einsum("bhk,bhv->bhkv", q[:, t], do[:, t])
            dq = s["scale"] * torch.einsum("bhkv,bhv->bhk", S, do[:, t])
            du = torch.einsum("bhk,bhkv->bhv", k[:, t], dS)
            db = (du * e).sum(-1)
            de = beta[:, t] * du
            decayed = a[:, t] * before
            dk = torch.einsum("bhkv,bhv->bhk", dS, beta[:, t] * e) - torch.einsum("bhkv,bhv->bhk", decayed, de)
            dS = dS - torch.einsum("bhk,bhv->bhkv", k[:, t], de)  # now of the decayed state
            grads[t] = (dq, dk, de, torch.einsum("bhkv,bhkv->bh", dS, decayed), db)
            dS = goes_on[:, t] * a[:, t] * dS
    dq, dk, dv, dg, db = (torch.stack(x, 1) for x in zip(*grads))
    group = lambda x: x.unflatten(2, (Hqk, H // Hqk)).sum(3)  # noqa: E731
    out = (group(dq), group(dk), dv, dg, db)
    return out + (dS,) if case["states"] else out
