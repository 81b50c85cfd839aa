// delta_step.cu -- the gated delta rule token by token on a pool of states,
// for decoding (C ABI in include/glacore.h):
//     u = beta_t (v_t - e^{g_t} S^T k_t),  S <- e^{g_t} S + k_t u^T,  o_t = scale S^T q_t
// for the T (usually one) new tokens of each of B sequences; sequence b's
// state is slot state_indices[b] of the pool and is updated in place.
//
// HBM-bound like the GLA step: a state is read once and written once per
// call, everything else is smaller by a factor of K or V.  A CTA owns
// 4 * COLT value columns of one (sequence, head); thread (row, col) holds four
// consecutive columns (V no multiple of 4: four columns COLT apart) of KR key
// rows in registers, all loads in flight before the first is used.  The rule
// needs S^T k before the state changes; S^T q is summed over the same state at
// the same time and the token's own share added to it,
//     o = scale (e^g S^T q + (q . k) u),
// so that a token costs one exchange over the CTA: partial sums of the warps
// in shared memory, added by every thread in a fixed order.  Arithmetic is
// fp32 throughout.  256 sequences of 16 heads of 128 x 128: 90 us in 8192 CTAs, 89%
// of the copy rate (one sequence: 6 us from a graph, its launch and two latencies).
#include <algorithm>

#include "delta.cuh"

namespace glacore {
namespace delta {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int TOKENS = 8;  // tokens whose q, k, v are staged at once

struct StepArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  float *state;
  const int32_t *slots;  // null: sequence b uses slot b
  void *o;
  int *err;
  int64_t n_slots, T, qs, ks, vs;
  int H, Hqk, K, V, slices, bf16;
  float scale;
};

__device__ __forceinline__ float load(const void *p, int bf16, int64_t i) {
  return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i])
              : reinterpret_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store(void *p, int bf16, int64_t i, float x) {
  if (bf16)
    reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
  else
    reinterpret_cast<float *>(p)[i] = x;
}

// COLT threads side by side cover 4 COLT value columns; VEC: V is a multiple
// of 4 and the pool 16-byte aligned.
template <int COLT, int KR, bool VEC>
__global__ void __launch_bounds__(THREADS, 4) delta_step_kernel(const StepArgs a) {
  constexpr int ROWT = THREADS / COLT, COLS = 4 * COLT, ROWS = ROWT * KR;
  static_assert(ROWS % 32 == 0, "");
  __shared__ float2 s_kq[TOKENS][ROWS];  // k, q of a key row
  __shared__ float s_v[TOKENS][COLS];
  __shared__ float s_gate[TOKENS], s_beta[TOKENS], s_qk[TOKENS][ROWS / 32];
  __shared__ float4 s_x[2][WARPS][COLT][2];  // partial sums of S^T k and S^T q, two tokens' worth
  const int slice = blockIdx.x % a.slices;
  const int64_t bh = blockIdx.x / a.slices;
  const int h = (int)(bh % a.H);
  const int64_t b = bh / a.H;
  const int hq = h / (a.H / a.Hqk), v0 = slice * COLS;
  const int col = threadIdx.x % COLT, row = threadIdx.x / COLT, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {  // an idle row (negative) or a slot that is not there: no state, o = 0
    if (slot >= a.n_slots && threadIdx.x == 0) set_device_error(a.err, GLACORE_ERR_INDEX);
    for (int64_t i = threadIdx.x; i < a.T * COLS; i += THREADS) {
      const int c = v0 + (int)(i % COLS);
      if (c < a.V) store(a.o, a.bf16, ((b * a.T + i / COLS) * a.H + h) * a.V + c, 0.f);
    }
    return;
  }
  float *S = a.state + (slot * a.H + h) * a.K * a.V;
  auto column = [&](int e) { return VEC ? 4 * col + e : col + e * COLT; };
  float st[KR][4];
#pragma unroll
  for (int j = 0; j < KR; ++j) {
    const int c = row + j * ROWT;
    if (VEC) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < a.K && v0 + 4 * col < a.V) f = *reinterpret_cast<const float4 *>(S + (int64_t)c * a.V + v0 + 4 * col);
      st[j][0] = f.x, st[j][1] = f.y, st[j][2] = f.z, st[j][3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int vc = v0 + column(e);
        st[j][e] = c < a.K && vc < a.V ? S[(int64_t)c * a.V + vc] : 0.f;
      }
    }
  }
  for (int64_t t0 = 0; t0 < a.T; t0 += TOKENS) {
    const int n = (int)(a.T - t0 < TOKENS ? a.T - t0 : TOKENS);
    if (t0) __syncthreads();  // the last tokens' rows have been used
    // q, k and, of every 32 channels (a warp's), q . k; whole warps take part or none
    for (int i = threadIdx.x; i < n * ROWS; i += THREADS) {
      const int t = i / ROWS, c = i % ROWS;
      const int64_t tok = b * a.T + t0 + t;
      float q = 0.f, k = 0.f;
      if (c < a.K) {
        q = load(a.q, a.bf16, tok * a.qs + (int64_t)hq * a.K + c);
        k = load(a.k, a.bf16, tok * a.ks + (int64_t)hq * a.K + c);
      }
      s_kq[t][c] = make_float2(k, q);
      float dot = q * k;
#pragma unroll
      for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
      if (lane == 0) s_qk[t][c / 32] = dot;
    }
    if (threadIdx.x < n) {
      const int64_t at = (b * a.T + t0 + threadIdx.x) * a.H + h;
      s_gate[threadIdx.x] = expf(a.g[at]);
      s_beta[threadIdx.x] = a.beta[at];
    }
    for (int i = threadIdx.x; i < n * COLS; i += THREADS) {
      const int t = i / COLS, c = i % COLS;
      s_v[t][c] = v0 + c < a.V ? load(a.v, a.bf16, (b * a.T + t0 + t) * a.vs + (int64_t)h * a.V + v0 + c) : 0.f;
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float d = s_gate[t];
      if (d == 0.f) {  // a decay of exactly 0 forgets whatever the slot held, NaN included
#pragma unroll
        for (int j = 0; j < KR; ++j) st[j][0] = st[j][1] = st[j][2] = st[j][3] = 0.f;
      }
      float xk[4] = {0.f, 0.f, 0.f, 0.f}, xq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KR; ++j) {
        const float2 r = s_kq[t][row + j * ROWT];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xk[e] = fmaf(r.x, st[j][e], xk[e]);
          xq[e] = fmaf(r.y, st[j][e], xq[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int m = COLT; m < 32; m <<= 1) {
          xk[e] += __shfl_xor_sync(0xffffffffu, xk[e], m);
          xq[e] += __shfl_xor_sync(0xffffffffu, xq[e], m);
        }
      }
      if (lane < COLT) {
        s_x[t & 1][warp][lane][0] = make_float4(xk[0], xk[1], xk[2], xk[3]);
        s_x[t & 1][warp][lane][1] = make_float4(xq[0], xq[1], xq[2], xq[3]);
      }
      __syncthreads();
      // s_x of token t is written again by token t + 2, after the barrier of t + 1
      float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 p = s_x[t & 1][w][col][0];
        sk.x += p.x, sk.y += p.y, sk.z += p.z, sk.w += p.w;
      }
      const float tk[4] = {sk.x, sk.y, sk.z, sk.w};
      float u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = s_beta[t] * (s_v[t][column(e)] - d * tk[e]);
      if (row == 0) {
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float4 p = s_x[t & 1][w][col][1];
          sq.x += p.x, sq.y += p.y, sq.z += p.z, sq.w += p.w;
        }
        const float tq[4] = {sq.x, sq.y, sq.z, sq.w};
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS / 32; ++i) qk += s_qk[t][i];
        const int64_t at = ((b * a.T + t0 + t) * a.H + h) * a.V + v0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (v0 + column(e) < a.V) store(a.o, a.bf16, at + column(e), a.scale * fmaf(qk, u[e], d * tq[e]));
      }
#pragma unroll
      for (int j = 0; j < KR; ++j) {
        const float k = s_kq[t][row + j * ROWT].x;
#pragma unroll
        for (int e = 0; e < 4; ++e) st[j][e] = fmaf(k, u[e], d * st[j][e]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < KR; ++j) {
    const int c = row + j * ROWT;
    if (VEC) {
      if (c < a.K && v0 + 4 * col < a.V)
        __stcs(reinterpret_cast<float4 *>(S + (int64_t)c * a.V + v0 + 4 * col),  // not read again in this call
               make_float4(st[j][0], st[j][1], st[j][2], st[j][3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int vc = v0 + column(e);
        if (c < a.K && vc < a.V) S[(int64_t)c * a.V + vc] = st[j][e];
      }
    }
  }
}

template <int COLT, int KR>
cudaError_t launch_as(StepArgs &a, int64_t B, bool vec, cudaStream_t st) {
  a.slices = (a.V + 4 * COLT - 1) / (4 * COLT);
  const int64_t ctas = B * a.H * a.slices;
  if (ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  if (vec)
    delta_step_kernel<COLT, KR, true><<<(unsigned)ctas, THREADS, 0, st>>>(a);
  else
    delta_step_kernel<COLT, KR, false><<<(unsigned)ctas, THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step(const glacore_problem *p, const float *beta, float *state, int64_t n_slots,
                        const int32_t *slots, void *o, int *err, cudaStream_t st) {
  StepArgs a;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.g = p->g;
  a.beta = beta;
  a.state = state;
  a.slots = slots;
  a.o = o;
  a.err = err;
  a.n_slots = n_slots;
  a.T = p->T;
  a.qs = p->q_stride ? p->q_stride : p->Hqk * p->K;
  a.ks = p->k_stride ? p->k_stride : p->Hqk * p->K;
  a.vs = p->v_stride ? p->v_stride : p->H * p->V;
  a.H = (int)p->H;
  a.Hqk = (int)p->Hqk;
  a.K = (int)p->K;
  a.V = (int)p->V;
  a.bf16 = p->dtype == GLACORE_BF16;
  a.scale = p->scale;
  const bool vec = p->V % 4 == 0 && ((uintptr_t)state & 15) == 0;
  // Columns of a CTA by V: 64 where they waste no more than 32 would; key rows
  // of a thread by K, no more than 8 (64 registers: four CTAs per SM).
  const int64_t over64 = (p->V + 63) / 64 * 64, over32 = (p->V + 31) / 32 * 32;
  cudaError_t e;
  if (p->V <= 16)
    e = p->K <= 64 ? launch_as<4, 1>(a, p->B, vec, st)
                   : p->K <= 128 ? launch_as<4, 2>(a, p->B, vec, st) : launch_as<4, 4>(a, p->B, vec, st);
  else if (p->K > 128)
    e = launch_as<8, 8>(a, p->B, vec, st);
  else if (over32 < over64)
    e = p->K <= 64 ? launch_as<8, 2>(a, p->B, vec, st) : launch_as<8, 4>(a, p->B, vec, st);
  else
    e = p->K <= 64 ? launch_as<16, 4>(a, p->B, vec, st) : launch_as<16, 8>(a, p->B, vec, st);
  mark_launch("delta_step", st);
  return e;
}

}  // namespace delta
}  // namespace glacore
