// delta.cuh -- the gated delta rule (delta*.cu): declarations shared by its
// host side and kernels.  Notation of the chunk form, for the C tokens of a
// chunk of one (document, value head), S0 the state before it, S1 after it:
//     G_t = sum of g from the chunk's start,  D_ts = exp(G_t - G_s) (s <= t)
//     N = strict lower part of D (.) K K^T,   Z = -(I + N diag(b))^-1 N
//     Y = V - e^G (.) K S0,  E = Y + Z (b Y),  U = b E
//     O = scale (e^G (.) Q S0 + P U),  P = lower part of D (.) Q K^T
//     S1 = e^{G_C} S0 + K^T (e^{G_C - G} (.) U)
// E_t = v_t - e^{g_t} S_{t-1}^T k_t is the error of token t's own prediction.
// Backward, with dS1 the gradient of S1:
//     dU = scale P^T dO + e^{G_C - G} (.) K dS1,  dE = b dU
//     dR = dU + Z^T (b dU),  dY = b dR = dV,  db = rowsum(E (.) dR)
//     dS0 = e^{G_C} dS1 + Q^T (scale e^G (.) dO) - K^T (e^G (.) dY)
//     dPd = scale D (.) lower(dO U^T),  dA = -D (.) strict lower(dY U^T)
//     dQ = scale e^G (.) dO S0^T + dPd K
//     dK = -e^G (.) dY S0^T + e^{G_C - G} (.) U dS1^T + dPd^T Q + (dA + dA^T) K
// and dg_t, the gradient of everything that g_t decays: the pairs r >= t > s
// of W = dPd (.) Q K^T + dA (.) K K^T, what the tokens r >= t read of S0, what
// the tokens s < t left in S1, and e^{G_C} <S0, dS1>.
#pragma once

#include <initializer_list>

#include "internal.cuh"

namespace glacore {
namespace delta {

constexpr int C = 64;  // tokens of a chunk

struct Call {
  Prob p;
  Docs docs;         // tables for chunks of C tokens
  int64_t slots;     // chunk slots (of all documents)
  int dtype;
  int64_t sK, sV;     // K and V of the states (p.K and p.V may be those of padded copies)
  const float *beta;  // [BT, H]
  cudaStream_t st;
};

// The chunk in a slot: its document d and tokens [tok, tok + len).  False: an
// unused slot (behind the last document's).  There are fewer than 2^31 slots.
__device__ __forceinline__ bool chunk_in_slot(const Docs &docs, int64_t slot, int64_t &tok, int &len) {
  int64_t d, j;
  if (docs.cbase) {
    if (slot >= docs.cbase[docs.n]) return false;
    int64_t lo = 0, hi = docs.n;  // cbase[lo] <= slot < cbase[hi]
    while (hi - lo > 1) {
      const int64_t m = (lo + hi) >> 1;
      if (docs.cbase[m] <= slot) lo = m; else hi = m;
    }
    d = lo;
    j = slot - docs.cbase[d];
  } else {
    const uint32_t per = (uint32_t)((docs.T + C - 1) / C), r = (uint32_t)slot / per;
    d = r;
    j = slot - (int64_t)r * per;
  }
  int64_t s0, s1;
  docs.range(d, s0, s1);
  tok = s0 + j * C;
  len = (int)min((int64_t)C, s1 - tok);
  return true;
}

// A token's log decay as a chunk's sums take it: below -10^4 e^g is 0 as well, and
// the sums stay finite.  (Not by fmaxf, which takes NaN for the bound.)
__device__ __forceinline__ float log_decay(float g) { return g < -1e4f ? -1e4f : g; }

// Scratch of the backward, all fp32: states before and state gradients after
// every chunk [slots, H, K, V], E and dR of every token [BT, H, V].
struct Saved {
  float *s0, *ds1, *e, *dr;
};

// ---- CUDA-core kernels (delta_simt.cu): any K, V up to 256, both types ----
// Token by token: o, ht (may be null).
cudaError_t simt_fwd(const Call &c, void *o, float *ht);
// The backward's passes forwards and backwards in time: what `saved` holds, dv, dh0 (may be null).
cudaError_t simt_scans(const Call &c, const void *dO, const float *dht, void *dv, float *dh0, const Saved &saved);
// dq, dk, dg, dbeta from what the two passes saved, every chunk by itself.
// dq and dk: [BT, H, K] fp32 per value head where heads share q and k (to be
// summed by reduce_heads), [BT, H, K] dtype otherwise.
cudaError_t simt_grads(const Call &c, const void *dO, const Saved &saved, void *dq, void *dk, bool per_head, float *dg,
                       float *dbeta);
// out [BT, Hqk, sK] dtype = sums of x [BT, H, p.K] fp32 over the heads of a group.
cudaError_t reduce_heads(const Call &c, const float *x, void *out);
// bf16 rows of D channels, `heads` to a token, `stride` values from token to
// token, copied to dense rows of Dp (a multiple of 8; the rest 0), and back.
struct Rows {
  const void *src;
  void *dst;
  int64_t stride;
  int heads, D, Dp;
};
cudaError_t pad_rows(const Call &c, std::initializer_list<Rows> tensors);
cudaError_t unpad_rows(const Call &c, std::initializer_list<Rows> tensors);

// ---- tensor-core kernels (delta_tc.cu): bf16, K and V multiples of 8 up to 128 ----
bool tc_supported(const glacore_problem *p);  // sizes, strides and addresses of q, k, v
bool tc_padded(const glacore_problem *p);     // not so, but dense copies of q, k, v with padded rows are
size_t tc_workspace(int64_t docs, int64_t slots, int64_t H, bool backward);
cudaError_t tc_fwd(const Call &c, void *o, float *ht, char *ws);
// dq and dk as in simt_grads
cudaError_t tc_bwd(const Call &c, const void *dO, const float *dht, void *dq, void *dk, bool per_head, void *dv, float *dg,
                   float *dbeta, float *dh0, char *ws);

// ---- token by token on a pool of states (delta_step.cu) -------------------
cudaError_t launch_step(const glacore_problem *p, const float *beta, float *state, int64_t n_slots,
                        const int32_t *slots, void *o, int *err, cudaStream_t st);

}  // namespace delta
}  // namespace glacore
