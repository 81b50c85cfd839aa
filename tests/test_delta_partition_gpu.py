"""The gated delta rule on a stream that has a part of the device's SMs (a green context's)."""
import ctypes

import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu

SM, AT_SM = 1, 96  # CU_DEV_RESOURCE_TYPE_SM; where a CUdevResource holds its number of SMs


class Partition:
    """A stream of `sms` SMs of the current device."""

    def __init__(self, sms):
        torch.zeros(1, device="cuda")
        self.cu = cu = ctypes.CDLL("libcuda.so.1")
        self.ctx, self.stream = ctypes.c_void_p(), ctypes.c_void_p()
        res = lambda: ctypes.create_string_buffer(1024)
        dev, whole, part, rest = ctypes.c_int(), res(), res(), res()
        n, desc = ctypes.c_uint(1), ctypes.c_void_p()
        ref = ctypes.byref

        def do(name, *args):
            if getattr(cu, name)(*args):
                pytest.skip(f"{name}: this driver makes no partitions")

        do("cuDeviceGet", ref(dev), torch.cuda.current_device())
        do("cuDeviceGetDevResource", dev, whole, SM)
        do("cuDevSmResourceSplitByCount", part, ref(n), whole, rest, ctypes.c_uint(0), ctypes.c_uint(sms))
        self.sms = ctypes.c_uint.from_buffer(part, AT_SM).value
        do("cuDevResourceGenerateDesc", ref(desc), part, ctypes.c_uint(1))
        do("cuGreenCtxCreate", ref(self.ctx), desc, dev, ctypes.c_uint(1))
        do("cuGreenCtxStreamCreate", ref(self.stream), self.ctx, ctypes.c_uint(1), ctypes.c_int(0))

    def __enter__(self):
        return torch.cuda.ExternalStream(self.stream.value)

    def __exit__(self, *exc):
        self.cu.cuStreamSynchronize(self.stream)
        self.cu.cuStreamDestroy_v2(self.stream)
        self.cu.cuGreenCtxDestroy(self.ctx)


@pytest.mark.parametrize("sms", [64, 128])
def test_forward_and_backward_on_a_part_of_the_sms(cuda_ok, sms):
    """Where all SMs make tiles beside the walks, a part of them makes them first: the same bits."""
    gen = torch.Generator("cuda")
    gen.manual_seed(sms)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    B, T, H, K = 4, 650, 16, 128
    q, k = (torch.nn.functional.normalize(r(B, T, H, K), dim=-1).bfloat16() for _ in range(2))
    v, do, g, b = r(B, T, H, K).bfloat16(), r(B, T, H, K).bfloat16(), -r(B, T, H).abs() / 4, r(B, T, H).sigmoid()

    def run():
        with glc.LaunchTimer(8) as t:
            o, s = glc.delta_fwd(q, k, v, g, b, output_final_state=True, poison=True)
        return t.labels, (o, s, *glc.delta_bwd(q, k, v, g, b, do, poison=True)[:5])

    labels, want = run()
    if torch.cuda.get_device_properties(0).multi_processor_count >= 2 * B * H:
        assert labels == ["delta_overlap"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, held = run()
    assert captured == labels
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, want))
    with Partition(sms) as stream:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for _ in range(3):
                labels, got = run()
        stream.synchronize()
        assert labels == ["delta_prep", "delta_chain"]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        del got
    glc.get_device_error()
