"""Sizes of the gated delta rule's scratch for bf16 problems, as the header states them (no GPU needed)."""
import ctypes

import pytest

import chunked_gated_linear_chunk_gb300 as glc

FWD, BWD = 41 * 1024, 233 * 1024  # per chunk and head


def need(entry, B, T, H, Hqk, K, V, n=None, q=256):
    p = glc.Problem(B=B, T=T, H=H, Hqk=Hqk, K=K, V=V, dtype=glc.BF16, chunk_size=0, scale=1.0, reserved0=0, q=q, k=512,
                    v=768, g=1024, segment_ids=None if n is None else 4096, n_seqs=B if n is None else n,
                    initial_state=None)
    return getattr(glc.load(), entry)(ctypes.byref(p))


@pytest.mark.parametrize("B,T,H,Hqk,K,V,n,q", [
    (4, 2048, 16, 16, 128, 128, None, 256), (1, 65, 2, 1, 128, 64, None, 256), (2, 1, 4, 4, 8, 8, None, 256),
    (1, 16384, 16, 8, 128, 128, 16, 256), (1, 4096, 4, 4, 128, 128, 512, 256), (1, 50, 3, 3, 64, 64, 50, 256),
    (4, 2048, 16, 16, 125, 77, None, 256), (2, 300, 4, 2, 72, 41, 9, 256), (1, 300, 4, 4, 128, 128, None, 258)])
def test_bytes_of_a_bf16_problem(B, T, H, Hqk, K, V, n, q):
    BT = B * T
    chunks = B * -(-T // 64) if n is None else min(BT, BT // 64 + n)
    padded = K % 8 or V % 8 or q % 16
    up = lambda x: (x + 7) // 8 * 8
    rows = 2 * BT * (2 * Hqk * up(K) + 2 * H * up(V)) if padded else 0
    docs = 20 * (n or B)  # tables and launch order
    least = chunks * H * FWD + rows
    assert least <= need("delta_fwd_workspace_size", B, T, H, Hqk, K, V, n, q) <= least + 4 * chunks * H + docs + 4096
    copies = 2 * BT * (H * up(V) + 2 * H * up(K) * (2 if H != Hqk else 1)) if padded else 0
    least = chunks * H * BWD + rows + copies
    shared = 8 * BT * H * K if H != Hqk and not padded else 0
    assert least + shared <= need("delta_bwd_workspace_size", B, T, H, Hqk, K, V, n, q) <= least + shared + docs + 4096
