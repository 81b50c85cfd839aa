"""The measurement hook: every entry call records from the first event on, so the
labels after several calls are the last one's alone."""
import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc

pytestmark = pytest.mark.gpu


def calls():
    z = lambda *s: torch.zeros(*s, device="cuda")
    x, w, st = z(6, 16), z(16), z(6)
    q, g, pool = z(2, 1, 2, 8), z(2, 1, 2, 8), z(2, 2, 8, 8)
    head, t = z(9, 16), torch.zeros(6, dtype=torch.int64, device="cuda")
    c, cw = z(2, 3, 16), z(4, 16)
    return {
        "layer_norm_fwd": lambda: glc.layer_norm_fwd(x, w, w),
        "layer_norm_bwd": lambda: glc.layer_norm_bwd(x, w, st, st, x),
        "linear_ce_fwd": lambda: glc.linear_ce_fwd(x, head, t),
        "linear_ce_bwd": lambda: glc.linear_ce_bwd(x, head, t, st, st),
        "gla_step": lambda: glc.gla_step(q, q, q, g, pool),
        "gla_fwd": lambda: glc.gla_fwd(q, q, q, g),
        "norm_gate_fwd": lambda: glc.norm_gate_fwd(x, x, w),
        "norm_gate_bwd": lambda: glc.norm_gate_bwd(x, x, w, x),
        "short_conv_fwd": lambda: glc.short_conv_fwd(c, cw),
        "short_conv_bwd": lambda: glc.short_conv_bwd(c, cw, None, c),
        "state_scan": lambda: glc.state_scan(z(2, 3, 8, 8), z(2, 3, 8), 1),
    }


@pytest.mark.parametrize("name", ["layer_norm_fwd", "layer_norm_bwd", "linear_ce_fwd", "linear_ce_bwd", "gla_step",
                                  "gla_fwd", "norm_gate_fwd", "norm_gate_bwd", "short_conv_fwd", "short_conv_bwd",
                                  "state_scan"])
def test_each_call_records_from_the_first_event(cuda_ok, name):
    call = calls()[name]
    with glc.LaunchTimer(16) as once:
        call()
    with glc.LaunchTimer(16) as t:
        for _ in range(20):
            call()
    torch.cuda.synchronize()
    assert once.labels and t.labels == once.labels
