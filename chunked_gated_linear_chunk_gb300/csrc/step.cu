// step.cu -- the recurrence token by token on a pool of states, for decoding
// (C ABI in include/glacore.h):
//     S <- diag(exp(g_t)) S + k_t v_t^T,     o_t = scale * S^T q_t
// for the T (usually one) new tokens of each of B sequences; sequence b's
// state is slot state_indices[b] of the pool and is updated in place.
//
// HBM-bound: a state is K x V fp32 and is read once and written once per
// call, whatever T is; everything else (q, k, v, g, o) is smaller by a factor
// of K or V.  A CTA owns 4 * COLT value columns of one (sequence, head):
// thread (row, col) holds the four consecutive columns 4 col .. 4 col + 3
// (one 16-byte access; with V not a multiple of 4, columns col, col + COLT,
// ...) of KR key rows row, row + ROWT, ..., all in registers, so every load
// of the state is in flight before the first is used, and the tokens of a
// call walk over registers.  The sum over key rows is a shuffle within a
// warp and one pass over the warps' partial rows in shared memory, added in a
// fixed order.  State arithmetic is fp32 throughout.
// Measured: 256 sequences x 16 heads of 128 x 128 states, bf16, 85 us = 6.4 TB/s
// (94% of the copy rate); 128 x 32 heads of 128 x 64, 44.5 us = 6.1 TB/s.  With
// two CTAs per SM instead of four (registers): 121 us.
#include <algorithm>

#include "internal.cuh"
#include "step.cuh"

namespace glacore {
namespace step {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int TOKENS = 8;  // tokens whose q, k, v and decay are staged at once

struct Args {
  const void *q, *k, *v;
  const float *g;
  float *state;
  const int32_t *slots;  // null: sequence b uses slot b
  void *o;
  int *err;
  int64_t n_slots, T, qs, ks, vs;
  int H, Hqk, K, V, slices;
  int bf16, head_gate;
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

// Two fp32 operations per instruction: o = a b + c, and o = a b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 o;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
      : "=f"(o.x), "=f"(o.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return o;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 o;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(o.x), "=f"(o.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return o;
}

// COLT threads side by side cover 4 COLT value columns; VEC: V is a multiple
// of 4 and the pool 16-byte aligned.
template <int COLT, int KR, bool VEC>
__global__ void __launch_bounds__(THREADS, 4) step_kernel(const Args a) {
  constexpr int ROWT = THREADS / COLT, COLS = 4 * COLT;
  __shared__ float4 s_akq[TOKENS][ROWT * KR];  // decay, k, scale q of a key row
  __shared__ float s_v[TOKENS][COLS];
  __shared__ float s_o[TOKENS][WARPS][COLS];
  const int slice = blockIdx.x % a.slices;
  const int64_t bh = blockIdx.x / a.slices;
  const int h = (int)(bh % a.H);
  const int64_t b = bh / a.H;
  const int hq = h / (a.H / a.Hqk), v0 = slice * COLS;
  const int col = threadIdx.x % COLT, row = threadIdx.x / COLT;
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
  float2 st[KR][2];
#pragma unroll
  for (int j = 0; j < KR; ++j) {
    const int c = row + j * ROWT;
    if (VEC) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < a.K && v0 + 4 * col < a.V) f = *reinterpret_cast<const float4 *>(S + (int64_t)c * a.V + v0 + 4 * col);
      st[j][0] = make_float2(f.x, f.y);
      st[j][1] = make_float2(f.z, f.w);
    } else {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int vc = v0 + col + e * COLT;
        f[e] = c < a.K && vc < a.V ? S[(int64_t)c * a.V + vc] : 0.f;
      }
      st[j][0] = make_float2(f[0], f[1]);
      st[j][1] = make_float2(f[2], f[3]);
    }
  }
  for (int64_t t0 = 0; t0 < a.T; t0 += TOKENS) {
    const int n = (int)(a.T - t0 < TOKENS ? a.T - t0 : TOKENS);
    if (t0) __syncthreads();  // the last tokens' rows have been used
    bool forgets = false;
    for (int i = threadIdx.x; i < n * (ROWT * KR); i += THREADS) {
      const int t = i / (ROWT * KR), c = i % (ROWT * KR);
      const int64_t tok = b * a.T + t0 + t;
      float q = 0.f, k = 0.f, d = 0.f;
      if (c < a.K) {
        q = a.scale * load(a.q, a.bf16, tok * a.qs + (int64_t)hq * a.K + c);
        k = load(a.k, a.bf16, tok * a.ks + (int64_t)hq * a.K + c);
        d = expf(a.head_gate ? a.g[tok * a.H + h] : a.g[(tok * a.H + h) * a.K + c]);
      }
      forgets |= c < a.K && d == 0.f;
      s_akq[t][c] = make_float4(d, k, q, 0.f);
    }
    for (int i = threadIdx.x; i < n * COLS; i += THREADS) {
      const int t = i / COLS, c = i % COLS;
      s_v[t][c] = v0 + c < a.V ? load(a.v, a.bf16, (b * a.T + t0 + t) * a.vs + (int64_t)h * a.V + v0 + c) : 0.f;
    }
    forgets = __syncthreads_or(forgets);
    for (int t = 0; t < n; ++t) {
      if (forgets) {  // a decay of exactly 0 forgets whatever the slot held, NaN included
#pragma unroll
        for (int j = 0; j < KR; ++j)
          if (s_akq[t][row + j * ROWT].x == 0.f) st[j][0] = st[j][1] = make_float2(0.f, 0.f);
      }
      float2 v[2], acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        v[e] = make_float2(s_v[t][VEC ? 4 * col + 2 * e : col + 2 * e * COLT],
                           s_v[t][VEC ? 4 * col + 2 * e + 1 : col + (2 * e + 1) * COLT]);
#pragma unroll
      for (int j = 0; j < KR; ++j) {
        const float4 r = s_akq[t][row + j * ROWT];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          st[j][e] = fma2(make_float2(r.y, r.y), v[e], mul2(make_float2(r.x, r.x), st[j][e]));
          acc[e] = fma2(make_float2(r.z, r.z), st[j][e], acc[e]);
        }
      }
      float o[4] = {acc[0].x, acc[0].y, acc[1].x, acc[1].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int m = COLT; m < 32; m <<= 1) o[e] += __shfl_xor_sync(0xffffffffu, o[e], m);
      }
      if ((threadIdx.x & 31) < COLT)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_o[t][threadIdx.x >> 5][VEC ? 4 * col + e : col + e * COLT] = o[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * COLS; i += THREADS) {
      const int t = i / COLS, c = i % COLS;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) o += s_o[t][w][c];
      if (v0 + c < a.V) store(a.o, a.bf16, ((b * a.T + t0 + t) * a.H + h) * a.V + v0 + c, o);
    }
  }
#pragma unroll
  for (int j = 0; j < KR; ++j) {
    const int c = row + j * ROWT;
    if (VEC) {
      if (c < a.K && v0 + 4 * col < a.V)
        __stcs(reinterpret_cast<float4 *>(S + (int64_t)c * a.V + v0 + 4 * col),  // not read again in this call
               make_float4(st[j][0].x, st[j][0].y, st[j][1].x, st[j][1].y));
    } else {
      const float f[4] = {st[j][0].x, st[j][0].y, st[j][1].x, st[j][1].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int vc = v0 + col + e * COLT;
        if (c < a.K && vc < a.V) S[(int64_t)c * a.V + vc] = f[e];
      }
    }
  }
}

template <int COLT, int KR>
cudaError_t launch_as(Args &a, int64_t B, bool vec, cudaStream_t st) {
  a.slices = (a.V + 4 * COLT - 1) / (4 * COLT);
  const int64_t ctas = B * a.H * a.slices;
  if (ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  if (vec)
    step_kernel<COLT, KR, true><<<(unsigned)ctas, THREADS, 0, st>>>(a);
  else
    step_kernel<COLT, KR, false><<<(unsigned)ctas, THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch(const glacore_problem *p, bool head_gate, float *state, int64_t n_slots, const int32_t *slots,
                   void *o, int *err, cudaStream_t st) {
  Args a;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.g = p->g;
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
  a.head_gate = head_gate;
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
  mark_launch(head_gate ? "ssd_step" : "gla_step", st);
  return e;
}

}  // namespace step
}  // namespace glacore
