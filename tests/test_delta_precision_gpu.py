"""How far the fp32 results of the gated delta rule are off, in the root mean square over a tensor relative to its own.

On the tensor cores whatever is computed enters a product in two bf16 parts, which leave 2.5e-6 of it (root mean
square; 2^-17 at most), and a product of two such matrices is without that of their low parts (2.8e-6).  Roundings that
a result meets (a state that is carried on is kept in fp32):
  final state: S in S^T k; R, Z and their low parts' product; U                                              5
  dh0: dS in dS^T k; P; R, Z and their low parts' product; the scaled do; dX                                 7
  dbeta: those of E (S, R, Z, low parts) and of dR (dS, P, R, Z, low parts), and both as they are kept      11
  dg: dbeta's, S and dS as they are kept, U, dPd and dA, as a difference of sums twice as large             16
They are independent, so n of them make sqrt(n) times one; bounds are twice that, and twice as much for dg.  In fp32 a
value meets 4 roundings for each of up to 150 tokens that a state remembers and 8 exchanges: sqrt(608) 2^-25, bounds
four times that."""
import math

import pytest
import torch

import chunked_gated_linear_chunk_gb300 as glc
from oracle import delta

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ONE = 2.8e-6
TC = {n: 2 * math.sqrt(c) * ONE for n, c in (("ht", 5), ("dh0", 7), ("dbeta", 11))} | {"dg": 4 * 4 * ONE}
FULL = {n: 4 * math.sqrt(608) * 2.0 ** -25 * (2 if n == "dg" else 1) for n in TC}


@pytest.mark.parametrize("B,T,H,Hqk,K,V,dtype", [
    (2, 300, 4, 2, 128, 128, BF), (1, 1000, 2, 2, 128, 64, BF), (3, 200, 2, 1, 72, 41, BF),
    (2, 150, 4, 2, 72, 41, F32), (1, 130, 2, 2, 200, 136, F32)])
def test_states_and_gradients_in_fp32(cuda_ok, B, T, H, Hqk, K, V, dtype):
    gen = torch.Generator("cpu")
    gen.manual_seed(T + K)
    r = lambda *s: torch.randn(*s, generator=gen)
    norm = torch.nn.functional.normalize
    q, k = (norm(r(B, T, Hqk, K), dim=-1).to(dtype) for _ in range(2))
    v, do, g, b = r(B, T, H, V).to(dtype), r(B, T, H, V).to(dtype), -r(B, T, H).abs() / 8, r(B, T, H).sigmoid()
    h0, dht = r(B, H, K, V), r(B, H, K, V)
    x = [t.cuda() for t in (q, k, v, g, b)]
    got = {"ht": glc.delta_fwd(*x, 0.5, initial_state=h0.cuda(), output_final_state=True)[1]}
    grads = glc.delta_bwd(*x, do.cuda(), 0.5, initial_state=h0.cuda(), dht=dht.cuda())
    got.update(dg=grads[3], dbeta=grads[4], dh0=grads[5])
    want = delta.bwd(q, k, v, g, b, do, 0.5, None, h0, dht)
    want["ht"] = delta.fwd(q, k, v, g, b, 0.5, None, h0)[1]
    for name, bound in (TC if dtype == BF else FULL).items():
        w = torch.from_numpy(want[name])
        off = float((got[name].cpu().double() - w).norm() / w.norm())
        print(name, f"{off:.1e} of {bound:.1e}")
        assert off <= bound, name
