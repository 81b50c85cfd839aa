"""Calls of different sizes from several host threads at once, each on a stream of
its own: what a launch may take of shared memory is a property of the kernel on
the device, which the threads share, so no call may leave it at less than
another's launch needs.  ctypes releases the interpreter's lock during a call."""
import ctypes
import threading

import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu


def run_together(calls, times):
    """Every call `times` times in a thread of its own; each result must be the
    first one's again."""
    want = [c() for c in calls]
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(len(calls))

    def work(call, ref):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for i in range(times):
                    got = call()
                    if i % 50 == 49:
                        stream.synchronize()
                        assert all(torch.equal(a, b) for a, b in zip(got, ref))
                stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    glc.get_device_error()


def loss_call(N, D, V, dtype, backward):
    g = torch.Generator("cuda")
    g.manual_seed(N)
    x = torch.randn(N, D, generator=g, device="cuda").to(dtype)
    w = (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).to(dtype)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    if not backward:
        return lambda: glc.linear_ce_fwd(x, w, t)
    lse = glc.linear_ce_fwd(x, w, t)[1]
    dl = torch.ones(N, device="cuda")
    return lambda: glc.linear_ce_bwd(x, w, t, lse, dl)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("backward", [False, True])
def test_losses_of_different_sizes(cuda_ok, dtype, backward):
    run_together([loss_call(N, 64, 900, dtype, backward) for N in (8, 70, 300, 1000)], 1500)


def test_layer_norms_of_different_sizes(cuda_ok):
    def call(rows, D, dtype):
        x = torch.randn(rows, D, device="cuda").to(dtype)
        w = torch.randn(D, device="cuda")
        _, mean, rstd = glc.layer_norm_fwd(x, w)
        return lambda: (*glc.layer_norm_fwd(x, w), *glc.layer_norm_bwd(x, w, mean, rstd, x))

    run_together([call(1500, D, torch.float32) for D in (511, 64, 2048, 8191)], 200)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_recurrences_of_different_sizes(cuda_ok, dtype):
    """The kernels of head sizes other than the tensor-core ones.  The C entry
    itself, in a tight loop: there is little between two launches."""
    lib, keep, statuses = glc.load(), [], []

    def problem(K, V):
        r = lambda *s: torch.randn(*s, device="cuda")
        q, k, v = r(1, 16, 1, K).to(dtype), r(1, 16, 1, K).to(dtype), r(1, 16, 1, V).to(dtype)
        p, args = glc._problem(q, k, v, -r(1, 16, 1, K).abs() / 16, 1.0, None, None, 16, None, False)
        ws = glc._workspace(p, "gla_fwd", q.device, None)
        o, stream = torch.empty_like(v), torch.cuda.Stream()
        keep.append((args, ws, o, stream))
        torch.cuda.synchronize()
        return ctypes.byref(p), glc._ptr(o), ctypes.c_void_p(stream.cuda_stream)

    problems = [problem(K, V) for K, V in ((16, 16), (112, 40), (48, 24), (120, 80))]
    start = threading.Barrier(len(problems))

    def work(p, o, stream):
        start.wait()
        statuses.append({lib.gla_fwd(p, o, None, stream) for _ in range(5000)})

    threads = [threading.Thread(target=work, args=a) for a in problems]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{glc.OK}] * len(problems)
    glc.get_device_error()
