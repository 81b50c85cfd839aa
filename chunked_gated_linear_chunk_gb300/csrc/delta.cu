// delta.cu -- the gated delta rule: argument checks, workspace layout and
// launches (C ABI in include/glacore.h; formulas in delta.cuh).
#include <string.h>

#include <algorithm>

#include "delta.cuh"

namespace glacore {
namespace delta {

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
  size_t start, cbase;          // document tables (segment_ids only)
  size_t s0, ds1, e, dr;        // backward
  size_t dq, dk;                // backward, shared q / k heads: per value head, fp32
  size_t tc;                    // the tensor-core kernels' own
  size_t total;
  int64_t slots;
  bool on_tc;
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
  L.on_tc = tc_supported(p) && L.slots * p->H < ((int64_t)1 << 30) && n * p->H < ((int64_t)1 << 30);  // units in 32 bits
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
  // 0.26 us per token and round of blocks, against 19 us and 4 us per further chunk
  // (one row of 16 heads of 128 x 128: 48 tokens 16.6 us against 18.6, 64 tokens
  // 20.8 against 18.6; 64 rows of 8 tokens 62 us against 84, of 16 tokens 98 against 82).
  const int64_t blocks = c.docs.n * p->H * ((p->V + 31) / 32), rounds = (blocks + 607) / 608;
  if (L.on_tc && p->T * rounds > 56 && !((uintptr_t)o & 15))
    return status_of(tc_fwd(c, o, ht, (char *)p->workspace + L.tc));
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
