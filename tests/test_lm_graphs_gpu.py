"""The operators around the recurrence in a captured CUDA graph, replayed on other
inputs: bit for bit what a call gives."""
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu


def r(*shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda").to(dtype)


def replayed(call, state, fresh, times=3):
    """call(state) captured once; then `fresh` values are copied into the state's
    tensors and the replay's outputs compared with a call's on the same values."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(state)  # attributes and addresses are looked up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(state)
    for _ in range(times):
        values = fresh()
        for k, v in values.items():
            state[k].copy_(v)
        graph.replay()
        want = call({k: v.clone() for k, v in values.items()})
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    glc.get_device_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 2048), (700, 1111), (900, 256)])
def test_layer_norm(cuda_ok, rows, D, dtype):
    fresh = lambda: dict(x=r(rows, D, dtype=dtype), w=r(D), b=r(D), dy=r(rows, D, dtype=dtype))

    def call(s):
        y, mean, rstd = glc.layer_norm_fwd(s["x"], s["w"], s["b"])
        return y, mean, rstd, *glc.layer_norm_bwd(s["x"], s["w"], mean, rstd, s["dy"])

    replayed(call, fresh(), fresh)


@pytest.mark.parametrize("kind", ["gla", "ssd"])
def test_a_decode_step(cuda_ok, kind):
    B, H, K, V, slots = 5, 4, 64, 40, 9

    def fresh():
        g = -r(B, 1, H, K).abs() if kind == "gla" else -r(B, 1, H).abs()
        return dict(q=r(B, 1, 2, K), k=r(B, 1, 2, K), v=r(B, 1, H, V), g=g, state=r(slots, H, K, V),
                    idx=torch.randperm(slots, device="cuda")[:B].int())

    def call(s):
        step = glc.gla_step if kind == "gla" else glc.ssd_step
        return step(s["q"], s["k"], s["v"], s["g"], s["state"], s["idx"]), s["state"]

    replayed(call, fresh(), fresh)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,D,V", [(7, 64, 900), (64, 33, 300), (65, 33, 300), (900, 128, 3000)])
def test_loss(cuda_ok, N, D, V, dtype):
    def fresh():
        t = torch.randint(0, V, (N,), device="cuda")
        t[N // 2] = -100
        return dict(x=r(N, D, dtype=dtype), w=r(V, D, dtype=dtype) / 8, t=t, dl=r(N))

    def call(s):
        loss, lse = glc.linear_ce_fwd(s["x"], s["w"], s["t"])
        return loss, lse, *glc.linear_ce_bwd(s["x"], s["w"], s["t"], lse, s["dl"])

    replayed(call, fresh(), fresh)
