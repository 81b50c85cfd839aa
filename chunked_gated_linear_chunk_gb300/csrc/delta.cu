// delta.cu -- the gated delta rule: argument checks, workspace layout and
// launches (C ABI in include/glacore.h; formulas in delta.cuh).
#include <string.h>

#include <algorithm>

#include "delta.cuh"

namespace glacore {
namespace delta {

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// bf16 operands that the tensor-core kernels cannot read in place (heads of no
// multiple of 8, odd strides or addresses) go to them as padded copies, backwards always
// and forwards from this many tokens times rounds of blocks (run_fwd) on.  Token by
// token / copies, us forward and backward, heads of 72 x 41 and 6 of them: 8 tokens
// 6 / 31, 52 / 45; 100: 29 / 35, 93 / 52; 128: 35 / 35, 101 / 53; 333: 89 / 47, 160 / 70;
// 4 x 2048 tokens of 16 heads of 125 x 77: 756 / 207, 2127 / 522; 64 x 8 tokens of 16
// heads of 90 x 90: 47 / 88, 385 / 234.
constexpr int64_t PAD_TOKENS = 120;

struct Layout {
  size_t start, cbase;          // document tables (segment_ids only)
  size_t s0, ds1, e, dr;        // backward
  size_t dq, dk;                // backward, shared q / k heads: per value head, fp32
  size_t tc;                    // the tensor-core kernels' own
  size_t pq, pk, pv, po, pdv, pdq, pdk;  // padded copies (po: of o, of do in the backward)
  size_t total;
  int64_t slots, Kp, Vp;
  bool on_tc, pad;
};

Layout layout(const glacore_problem *p, bool backward) {
  Layout L;
  memset(&L, 0, sizeof(L));
  const int64_t BT = p->B * p->T, n = p->n_seqs;
  size_t off = 0;
  auto take = [&](size_t &at, size_t bytes) {
    at = off;
    off = align256(off + bytes);
  };
  if (p->segment_ids) {
    take(L.start, sizeof(int64_t) * (n + 1));
    take(L.cbase, sizeof(int64_t) * (n + 1));
  }
  // a document's last chunk may be short: at most one more than its tokens fill
  L.slots = p->segment_ids ? std::min(BT, BT / C + n) : p->B * ((p->T + C - 1) / C);
  const bool fits = L.slots * p->H < ((int64_t)1 << 30) && n * p->H < ((int64_t)1 << 30);  // units in 32 bits
  L.on_tc = fits && tc_supported(p);
  L.pad = fits && tc_padded(p);
  if (L.pad) {
    L.Kp = (p->K + 7) / 8 * 8;
    L.Vp = (p->V + 7) / 8 * 8;
    take(L.pq, 2 * (size_t)BT * p->Hqk * L.Kp);
    take(L.pk, 2 * (size_t)BT * p->Hqk * L.Kp);
    take(L.pv, 2 * (size_t)BT * p->H * L.Vp);
    take(L.po, 2 * (size_t)BT * p->H * L.Vp);
    take(L.tc, tc_workspace(n, L.slots, p->H, backward));
    if (backward) {
      const size_t each = p->Hqk != p->H ? sizeof(float) : 2;
      take(L.pdv, 2 * (size_t)BT * p->H * L.Vp);
      take(L.pdq, each * (size_t)BT * p->H * L.Kp);
      take(L.pdk, each * (size_t)BT * p->H * L.Kp);
    }
    L.total = off;
    return L;
  }
  // the scratch of one call serves either family: the addresses of the outputs decide (run_fwd, run_bwd)
  if (L.on_tc) take(L.tc, tc_workspace(n, L.slots, p->H, backward));
  if (backward) {
    if (L.on_tc) off = L.tc;
    const size_t states = sizeof(float) * (size_t)L.slots * p->H * p->K * p->V;
    const size_t rows = sizeof(float) * (size_t)BT * p->H * p->V;
    take(L.s0, states);
    take(L.ds1, states);
    take(L.e, rows);
    take(L.dr, rows);
    if (L.on_tc) off = std::max(off, L.tc + align256(tc_workspace(n, L.slots, p->H, true)));
    if (p->Hqk != p->H) {
      take(L.dq, sizeof(float) * (size_t)BT * p->H * p->K);
      take(L.dk, sizeof(float) * (size_t)BT * p->H * p->K);
    }
  }
  L.total = off;
  return L;
}

glacore_status check(const glacore_problem *p) {
  const glacore_status s = check_problem(p, true);
  if (s) return s;
  return p->chunk_size != 0 && p->chunk_size != C ? GLACORE_ERR_UNSUPPORTED : GLACORE_OK;
}

// Every pointer at a multiple of its elements' size.
bool aligned(const glacore_problem *p, std::initializer_list<const void *> data,
             std::initializer_list<const void *> floats) {
  const uintptr_t es = p->dtype == GLACORE_BF16 ? 1 : 3;
  uintptr_t d = (uintptr_t)p->q | (uintptr_t)p->k | (uintptr_t)p->v;
  uintptr_t f = (uintptr_t)p->g | (uintptr_t)p->initial_state | (uintptr_t)p->segment_ids;
  for (const void *x : data) d |= (uintptr_t)x;
  for (const void *x : floats) f |= (uintptr_t)x;
  return !(d & es) && !(f & 3);
}

glacore_status check_ws(const glacore_problem *p, const Layout &L) {
  if (L.total == 0) return GLACORE_OK;
  if (!p->workspace || p->workspace_bytes < L.total || ((uintptr_t)p->workspace & 255)) return GLACORE_ERR_WORKSPACE;
  return GLACORE_OK;
}

glacore_status begin(const glacore_problem *p, const float *beta, const Layout &L, cudaStream_t st, Call &c) {
  c.p = make_prob(p, true);
  if (!c.p.err) return GLACORE_ERR_CUDA;
  c.slots = L.slots;
  c.dtype = p->dtype;
  c.sK = p->K;
  c.sV = p->V;
  c.beta = beta;
  c.st = st;
  char *ws = (char *)p->workspace;
  c.docs.T = p->T;
  c.docs.n = p->n_seqs;
  c.docs.chunk = C;
  c.docs.start = p->segment_ids ? (const int64_t *)(ws + L.start) : nullptr;
  c.docs.cbase = p->segment_ids ? (const int64_t *)(ws + L.cbase) : nullptr;
  if (!p->segment_ids) return GLACORE_OK;
  return status_of(launch_prep(p->segment_ids, p->B, p->T, p->n_seqs, C, (int64_t *)(ws + L.start),
                               (int64_t *)(ws + L.cbase), c.p.err, st));
}

// The same call on padded copies of q, k, v (and do).
cudaError_t padded(const Call &c, const Layout &L, const void *dO, char *ws, Call &to) {
  to = c;
  Prob &p = to.p;
  p.q = ws + L.pq;
  p.k = ws + L.pk;
  p.v = ws + L.pv;
  p.K = L.Kp;
  p.V = L.Vp;
  p.qs = p.ks = p.Hqk * p.K;
  p.vs = p.H * p.V;
  const int H = (int)p.H, Hqk = (int)p.Hqk, K = (int)c.p.K, V = (int)c.p.V, Kp = (int)L.Kp, Vp = (int)L.Vp;
  const Rows q{c.p.q, ws + L.pq, c.p.qs, Hqk, K, Kp}, k{c.p.k, ws + L.pk, c.p.ks, Hqk, K, Kp},
      v{c.p.v, ws + L.pv, c.p.vs, H, V, Vp}, o{dO, ws + L.po, (int64_t)H * V, H, V, Vp};
  return dO ? pad_rows(c, {q, k, v, o}) : pad_rows(c, {q, k, v});
}

glacore_status run_fwd(const glacore_problem *p, const float *beta, void *o, float *ht, cudaStream_t st) {
  glacore_status s = check(p);
  if (s) return s;
  const int64_t BT = p->B * p->T;
  if (BT > 0 && (!beta || !o)) return GLACORE_ERR_INVALID_ARG;
  const Layout L = layout(p, false);
  if ((s = check_ws(p, L))) return s;
  if (!aligned(p, {o}, {beta, ht})) return GLACORE_ERR_INVALID_ARG;
  if (BT == 0) return GLACORE_OK;
  Call c;
  if ((s = begin(p, beta, L, st, c))) return s;
  // Short rows: token by token, all slices of all documents at once, 4 us and
  // 0.26 us per token and round of blocks, against 13 us and 4 us per chunk
  // (one row of 16 heads of 128 x 128: 48 tokens 16.6 us against 18.5, 56 tokens 18.7 against
  // 17.7, 64 tokens 20.7 against 17.0; 64 rows of 8 tokens 62 us against 80, of 16 tokens 98 against
  // 80).  Of packed documents the row bounds the longest, whose tokens are in sequence; their
  // number does not tell it: 64 of 8 tokens in a row would take 68 us against 92, but one of 1793 beside 255
  // of one token (2 heads of 32 x 32) 340 against 134.
  const int64_t blocks = c.docs.n * p->H * ((p->V + 31) / 32), rounds = (blocks + 607) / 608;
  if (L.on_tc && p->T * rounds > 56 && !((uintptr_t)o & 15))
    return status_of(tc_fwd(c, o, ht, (char *)p->workspace + L.tc));
  if (L.pad && p->T * rounds > PAD_TOKENS) {
    char *ws = (char *)p->workspace;
    Call t;
    cudaError_t e = padded(c, L, nullptr, ws, t);
    if (e == cudaSuccess) e = tc_fwd(t, ws + L.po, ht, ws + L.tc);
    if (e == cudaSuccess) e = unpad_rows(c, {{ws + L.po, o, 0, (int)p->H, (int)p->V, (int)L.Vp}});
    return status_of(e);
  }
  return status_of(simt_fwd(c, o, ht));
}

glacore_status run_bwd(const glacore_problem *p, const float *beta, const void *dO, const float *dht, void *dq,
                       void *dk, void *dv, float *dg, float *dbeta, float *dh0, cudaStream_t st) {
  glacore_status s = check(p);
  if (s) return s;
  const int64_t BT = p->B * p->T;
  if (BT > 0 && (!beta || !dO || !dq || !dk || !dv || !dg || !dbeta)) return GLACORE_ERR_INVALID_ARG;
  const Layout L = layout(p, true);
  if ((s = check_ws(p, L))) return s;
  if (!aligned(p, {dO, dq, dk, dv}, {beta, dht, dg, dbeta, dh0})) return GLACORE_ERR_INVALID_ARG;
  if (BT == 0) return GLACORE_OK;
  Call c;
  if ((s = begin(p, beta, L, st, c))) return s;
  char *ws = (char *)p->workspace;
  const Saved saved = {(float *)(ws + L.s0), (float *)(ws + L.ds1), (float *)(ws + L.e), (float *)(ws + L.dr)};
  const bool shared = p->Hqk != p->H;
  void *hq = shared ? (void *)(ws + L.dq) : dq, *hk = shared ? (void *)(ws + L.dk) : dk;
  cudaError_t e;
  if (L.pad) {
    Call t;
    e = padded(c, L, dO, ws, t);
    if (e == cudaSuccess)
      e = tc_bwd(t, ws + L.po, dht, ws + L.pdq, ws + L.pdk, shared, ws + L.pdv, dg, dbeta, dh0, ws + L.tc);
    const int H = (int)p->H, K = (int)p->K;
    const Rows v{ws + L.pdv, dv, 0, H, (int)p->V, (int)L.Vp}, q{ws + L.pdq, dq, 0, H, K, (int)L.Kp},
        k{ws + L.pdk, dk, 0, H, K, (int)L.Kp};
    if (e == cudaSuccess) e = shared ? unpad_rows(c, {v}) : unpad_rows(c, {v, q, k});
    if (e == cudaSuccess && shared) e = reduce_heads(t, (const float *)(ws + L.pdq), dq);
    if (e == cudaSuccess && shared) e = reduce_heads(t, (const float *)(ws + L.pdk), dk);
    return status_of(e);
  }
  if (L.on_tc && !(((uintptr_t)dO | (uintptr_t)dv | (uintptr_t)hq | (uintptr_t)hk) & 15)) {
    e = tc_bwd(c, dO, dht, hq, hk, shared, dv, dg, dbeta, dh0, ws + L.tc);
  } else {
    e = simt_scans(c, dO, dht, dv, dh0, saved);
    if (e == cudaSuccess) e = simt_grads(c, dO, saved, hq, hk, shared, dg, dbeta);
  }
  if (e == cudaSuccess && shared) e = reduce_heads(c, (const float *)hq, dq);
  if (e == cudaSuccess && shared) e = reduce_heads(c, (const float *)hk, dk);
  return status_of(e);
}

glacore_status run_step(const glacore_problem *p, const float *beta, float *state, int64_t n_slots,
                        const int32_t *slots, void *o, cudaStream_t st) {
  const glacore_status s = check_problem(p, true);
  if (s) return s;
  if (p->segment_ids || p->initial_state || p->chunk_size != 0) return GLACORE_ERR_INVALID_ARG;
  if (n_slots < 0 || (!slots && n_slots < p->B)) return GLACORE_ERR_INVALID_ARG;
  if (p->B * p->T == 0) return GLACORE_OK;
  if (!o || !beta || (n_slots > 0 && !state) || !aligned(p, {o}, {beta, state, slots})) return GLACORE_ERR_INVALID_ARG;
  int *err = device_error_ptr();
  if (!err) return GLACORE_ERR_CUDA;
  return status_of(launch_step(p, beta, state, n_slots, slots, o, err, st));
}

}  // namespace
}  // namespace delta
}  // namespace glacore

using namespace glacore;

extern "C" {

size_t delta_fwd_workspace_size(const glacore_problem *p) {
  return delta::check(p) == GLACORE_OK ? delta::layout(p, false).total : 0;
}
size_t delta_bwd_workspace_size(const glacore_problem *p) {
  return delta::check(p) == GLACORE_OK ? delta::layout(p, true).total : 0;
}
glacore_status delta_fwd(const glacore_problem *p, const float *beta, void *o, float *final_state,
                         glacore_stream_t stream) {
  begin_marks();
  return delta::run_fwd(p, beta, o, final_state, (cudaStream_t)stream);
}
glacore_status delta_bwd(const glacore_problem *p, const float *beta, const void *do_, const float *dht, void *dq,
                         void *dk, void *dv, float *dg, float *dbeta, float *dh0, glacore_stream_t stream) {
  begin_marks();
  return delta::run_bwd(p, beta, do_, dht, dq, dk, dv, dg, dbeta, dh0, (cudaStream_t)stream);
}
glacore_status delta_step(const glacore_problem *p, const float *beta, float *state, int64_t n_slots,
                          const int32_t *state_indices, void *o, glacore_stream_t stream) {
  begin_marks();
  return delta::run_step(p, beta, state, n_slots, state_indices, o, (cudaStream_t)stream);
}

}  // extern "C"
