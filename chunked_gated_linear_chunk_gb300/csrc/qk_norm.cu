// qk_norm.cu -- the norm of every query and key head and the rotation by
// position in one pass, forward and backward (C ABI in include/glacore.h).
// Over a row x of D channels (one token, one head):
//     n = x r w,  r = (mean(x^2) + eps)^(-1/2)      (l2: the sum, not the mean)
//     (n_i, n_j) -> (n_i c - n_j s, n_j c + n_i s)  for the R pairs (i, j)
// with c, s the cosine and sine of the token's position.  Backward, with a the
// gradient rotated back:
//     dx = r (a w - x r m(a w x r)),  dw = sum over rows of a x r
// (m: the mean, or the sum for l2).
//
// HBM-bound: x in, y out (backward x, dy in, dx out); the statistics of a row
// are made again in the backward, which reads the row anyway.  A lane holds 8
// consecutive channels of a row (16 bytes of bf16), LPR lanes a row, so the
// row's sum is a few shuffles and a pair's other half one; a warp takes the
// heads of one token and keeps that token's cosines and sines and the weights
// in registers, with the loads of several rows in flight.  Rows that 16-byte accesses
// or 8-channel steps do not fit take a kernel with a warp per row and the
// row in shared memory.
// 8192 tokens of 32 heads of 128, bf16, rotated: 26.8 us forward (75% of the copy
// rate), 55 us backward (55%: three blocks' loads on an SM do not cover their
// latency; two or four of them are slower), 7 us of it the sum of the weight gradients.
// fp32: 48 and 81 us (84 and 75%).
// Heads of 101 channels, bf16: 122 and 162 us (single values, the table read for each; a row
// fetched ahead gains nothing and costs 20% at 250 channels).
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "internal.cuh"

namespace glacore {
namespace qkn {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int MAXD = 256;

struct Args {
  const void *x[2], *dy[2];  // q and k
  void *y[2];                // outputs (forward) or input gradients
  const float *w[2];         // null: 1
  const float *cs, *sn;      // [P, R]
  const int32_t *pos;        // null: the token's index in its row
  float *part;               // backward: weight gradients of every block, [blocks][2][D]
  int *err;
  int64_t tokens, T, P, xs[2];
  int H[2], D, R, mean, inter;
  int group[2], parts[2];  // heads of a warp, warps per token
  float eps;
};

// 8 channels of a row
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  // another lane's channels
  __device__ __forceinline__ Vec of(int lane) const {
    Vec o;
    o.a.x = __shfl_sync(0xffffffffu, a.x, lane);
    o.a.y = __shfl_sync(0xffffffffu, a.y, lane);
    o.a.z = __shfl_sync(0xffffffffu, a.z, lane);
    o.a.w = __shfl_sync(0xffffffffu, a.w, lane);
    return o;
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <> struct Vec<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ Vec of(int lane) const {
    Vec o;
    o.a.x = __shfl_sync(0xffffffffu, a.x, lane);
    o.a.y = __shfl_sync(0xffffffffu, a.y, lane);
    o.a.z = __shfl_sync(0xffffffffu, a.z, lane);
    o.a.w = __shfl_sync(0xffffffffu, a.w, lane);
    o.b.x = __shfl_sync(0xffffffffu, b.x, lane);
    o.b.y = __shfl_sync(0xffffffffu, b.y, lane);
    o.b.z = __shfl_sync(0xffffffffu, b.z, lane);
    o.b.w = __shfl_sync(0xffffffffu, b.w, lane);
    return o;
  }
  static __device__ __forceinline__ void store(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The row of the tables of a token (-1: no rotation, recorded as an error).
// x / y of values that nearly always fit in 32 bits
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}
__device__ __forceinline__ int64_t table_row(const Args &a, int64_t token) {
  const int64_t p = a.pos ? (int64_t)a.pos[token] : token - quotient(token, a.T) * a.T;
  if (p >= 0 && p < a.P) return p;
  set_device_error(a.err, GLACORE_ERR_INDEX);
  return -1;
}

// The rotation of a lane's 8 channels: c and s of each, s with the sign that
// it takes there, and where a pair's other half is.
struct Turn {
  float c[8], s[8];
  int other;  // lane of the other half (pairs (i, i + R)); the lane itself: no rotation
};
template <int LPR>
__device__ __forceinline__ void make_turn(const Args &a, int64_t token, int li, Turn &t) {
  const int c0 = 8 * li, lane = threadIdx.x & 31;
  t.other = lane;
#pragma unroll
  for (int e = 0; e < 8; ++e) t.c[e] = 1.f, t.s[e] = 0.f;
  if (a.R == 0) return;
  const int64_t p = table_row(a, token);
  if (p < 0 || c0 >= 2 * a.R) return;
  const float *cs = a.cs + p * a.R, *sn = a.sn + p * a.R;
  if (a.inter) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c = __ldg(cs + c0 / 2 + e), s = __ldg(sn + c0 / 2 + e);
      t.c[2 * e] = t.c[2 * e + 1] = c;
      t.s[2 * e] = -s;
      t.s[2 * e + 1] = s;
    }
  } else {
    const bool first = c0 < a.R;
    const int i0 = first ? c0 : c0 - a.R;
    t.other = first ? lane + a.R / 8 : lane - a.R / 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t.c[e] = __ldg(cs + i0 + e);
      const float s = __ldg(sn + i0 + e);
      t.s[e] = first ? -s : s;
    }
  }
}
// The 8 channels that a lane's are paired with, as they are in the row
// (interleaved: its own, neighbours swapped).  All lanes of the warp call it.
template <typename T>
__device__ __forceinline__ void paired(const Args &a, const Turn &t, const Vec<T> &x, const float (&f)[8], float (&o)[8]) {
  if (a.inter) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = f[e ^ 1];
  } else {
    x.of(t.other).get(o);
  }
}

__device__ __forceinline__ void weights(const float *w, int c0, bool in, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = w && in ? __ldg(w + c0 + e) : 1.f;
}

// With a row's rotation y_i = r (x_i w_i c + x_j w_j s) (s with its sign), c w
// and the pair's s w are made once for a token, and the pair's raw channels
// fetched while the row is summed.
template <typename T, int LPR, bool TURN>
__global__ void __launch_bounds__(THREADS, 4) fwd_kernel(const Args a) {
  constexpr int RPP = 32 / LPR, UNROLL = 2;  // rows of a pass, passes in flight
  const int lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
  const int64_t token = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const int z = (int)blockIdx.y >= a.parts[0], part = (int)blockIdx.y - (z ? a.parts[0] : 0);
  const int h0 = part * a.group[z], h1 = min(h0 + a.group[z], a.H[z]);
  const int c0 = 8 * li;
  const bool in = c0 < a.D;
  const T *x = (const T *)a.x[z] + token * a.xs[z] + c0;
  T *y = (T *)a.y[z] + token * a.H[z] * a.D + c0;
  const float inv = a.mean ? 1.f / (float)a.D : 1.f;
  Vec<T> v[UNROLL];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int hh = h + u * RPP + sub;
      if (in && hh < h1) v[u].load(x + (int64_t)hh * a.D); else v[u].clear();
    }
  };
  fetch(h0);
  float cw[8], sw[8];
  weights(a.w[z], c0, in, cw);
  Turn t;
  if (TURN) {
    make_turn<LPR>(a, token, li, t);
    // the weights of the paired channels
    float ow[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) ow[e] = a.inter ? cw[e ^ 1] : __shfl_sync(0xffffffffu, cw[e], t.other);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cw[e] *= t.c[e];
      sw[e] = ow[e] * t.s[e];
    }
  }
  for (int h = h0; h < h1; h += UNROLL * RPP) {
    Vec<T> w[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) w[u] = v[u];
    fetch(h + UNROLL * RPP);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      float f[8], o[8], ss = 0.f;
      w[u].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
      if (TURN) paired(a, t, w[u], f, o);
      const float r = rsqrtf(fmaf(row_sum<LPR>(ss), inv, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = r * (TURN ? fmaf(o[e], sw[e], f[e] * cw[e]) : f[e] * cw[e]);
      const int hh = h + u * RPP + sub;
      if (in && hh < h1) Vec<T>::store(y + (int64_t)hh * a.D, f);
    }
  }
}

// The blocks' sums of dw, in a fixed order: the block's rows of a channel are
// spread over its warps and the lane groups of a warp.
__device__ __forceinline__ void block_dw(const Args &a, const float *sums /* [rows][2][D] in shared memory */, int rows) {
  float *dst = a.part + (int64_t)blockIdx.x * 2 * a.D;
  for (int i = threadIdx.x; i < 2 * a.D; i += THREADS) {
    float x = 0.f;
    for (int r = 0; r < rows; ++r) x += sums[r * 2 * a.D + i];
    dst[i] = x;
  }
}

template <typename T, int LPR, bool TURN>
__global__ void __launch_bounds__(THREADS, 3) bwd_kernel(const Args a) {
  constexpr int RPP = 32 / LPR;
  extern __shared__ float sums[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
  const int c0 = 8 * li;
  const bool in = c0 < a.D;
  const float inv = a.mean ? 1.f / (float)a.D : 1.f;
  for (int z = 0; z < 2; ++z) {
    float w[8], dw[8];
    weights(a.w[z], c0, in, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = 0.f;
    // (query, key) x token x part of the heads, dealt to the warps of the grid in turn
    const int64_t all = (int64_t)gridDim.x * WARPS, mine = (int64_t)blockIdx.x * WARPS + warp;
    const int64_t skip = z ? a.tokens * a.parts[0] % all : 0;
    for (int64_t unit = (mine - skip + all) % all; unit < a.tokens * a.parts[z]; unit += all) {
      const int64_t token = a.parts[z] == 1 ? unit : unit >> 1;
      const int first = a.parts[z] == 1 ? 0 : (int)(unit & 1) * a.group[z], end = min(first + a.group[z], a.H[z]);
      Turn t;
      if (TURN) make_turn<LPR>(a, token, li, t);
      const T *x = (const T *)a.x[z] + token * a.xs[z] + c0;
      const T *dy = (const T *)a.dy[z] + token * a.H[z] * a.D + c0;
      T *dx = (T *)a.y[z] + token * a.H[z] * a.D + c0;
      Vec<T> nx, nd;  // the next row
      auto fetch = [&](int h) {
        if (in && h < end) {
          nx.load(x + (int64_t)h * a.D);
          nd.load(dy + (int64_t)h * a.D);
        } else {
          nx.clear();
          nd.clear();
        }
      };
      fetch(first + sub);
      for (int h = first + sub; h < end + sub; h += RPP) {  // all lanes as often
        const Vec<T> vx = nx, vd = nd;
        fetch(h + RPP);
        float f[8], d[8], g[8], ss = 0.f, sa = 0.f;
        vx.get(f);
        vd.get(d);
        if (TURN) {  // the gradient rotated back
          float o[8];
          paired(a, t, vd, d, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = fmaf(-t.s[e], o[e], t.c[e] * d[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          g[e] = d[e] * f[e];
          ss = fmaf(f[e], f[e], ss);
          sa = fmaf(g[e], w[e], sa);
        }
        ss = row_sum<LPR>(ss);
        sa = row_sum<LPR>(sa);
        const float r = rsqrtf(fmaf(ss, inv, a.eps));
        const float m = sa * r * r * r * inv;  // r m(a w n), for x itself
        const bool live = in && h < end;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[e] = fmaf(g[e], live ? r : 0.f, dw[e]);
          d[e] = fmaf(-f[e], m, r * (d[e] * w[e]));
        }
        if (live) Vec<T>::store(dx + (int64_t)h * a.D, d);
      }
    }
    if (in)
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[((warp * RPP + sub) * 2 + z) * a.D + c0 + e] = dw[e];
  }
  __syncthreads();
  block_dw(a, sums, WARPS * RPP);
  follow_allow();
}

// Rows of any D, R, stride and alignment: a warp per row, the row in shared memory.
template <typename T, bool BWD, int E>
__global__ void __launch_bounds__(THREADS) rows_kernel(const Args a) {
  __shared__ float buf[WARPS][32 * E];
  extern __shared__ float sums[];  // BWD: [WARPS][2][D]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv = a.mean ? 1.f / (float)a.D : 1.f;
  const int heads = a.H[0] + a.H[1];
  float *row = buf[warp];
  if (BWD) {
    for (int i = lane; i < 2 * a.D; i += 32) sums[warp * 2 * a.D + i] = 0.f;
    __syncwarp();
  }
  for (int64_t unit = (int64_t)blockIdx.x * WARPS + warp; unit < a.tokens * heads; unit += (int64_t)gridDim.x * WARPS) {
    const int64_t token = quotient(unit, heads);
    int h = (int)(unit - token * heads);
    const int z = h >= a.H[0];
    if (z) h -= a.H[0];
    const T *x = (const T *)a.x[z] + token * a.xs[z] + (int64_t)h * a.D;
    const int64_t at = (token * a.H[z] + h) * a.D;
    const float *w = a.w[z];
    int64_t p = -1;
    if (a.R) p = table_row(a, token);
    // channel c of a row in shared memory, rotated by dir
    const float *cs = a.cs + (p < 0 ? 0 : p) * a.R, *sn = a.sn + (p < 0 ? 0 : p) * a.R;
    auto turned = [&](int c, float dir) -> float {
      if (p < 0 || c >= 2 * a.R) return row[c];
      const bool first = a.inter ? (c & 1) == 0 : c < a.R;
      const int i = a.inter ? c / 2 : (first ? c : c - a.R), o = a.inter ? c ^ 1 : (first ? c + a.R : c - a.R);
      const float s = dir * __ldg(sn + i);
      return fmaf(first ? -s : s, row[o], __ldg(cs + i) * row[c]);
    };
    float f[E], d[E], ss = 0.f, sa = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane + 32 * e;
      f[e] = c < a.D ? to_f32(x[c]) : 0.f;
      ss = fmaf(f[e], f[e], ss);
      if (BWD && c < a.D) row[c] = to_f32(((const T *)a.dy[z])[at + c]);
    }
    __syncwarp();
    if (BWD) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = lane + 32 * e;
        d[e] = c < a.D ? turned(c, -1.f) : 0.f;
        sa = fmaf(c < a.D && w ? d[e] * __ldg(w + c) : d[e], f[e], sa);
      }
      sa = row_sum<32>(sa);
    }
    const float r = rsqrtf(fmaf(row_sum<32>(ss), inv, a.eps));
    if (BWD) {
      const float m = sa * r * inv;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = lane + 32 * e;
        if (c < a.D) {
          const float n = f[e] * r;
          ((T *)a.y[z])[at + c] = from_f32<T>(r * fmaf(-n, m, w ? d[e] * __ldg(w + c) : d[e]));
          float *dw = sums + (warp * 2 + z) * a.D + c;
          *dw = fmaf(d[e], n, *dw);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = lane + 32 * e;
        if (c < a.D) row[c] = f[e] * r * (w ? __ldg(w + c) : 1.f);
      }
      __syncwarp();
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = lane + 32 * e < a.D ? turned(lane + 32 * e, 1.f) : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (lane + 32 * e < a.D) ((T *)a.y[z])[at + lane + 32 * e] = from_f32<T>(y[e]);
    }
    __syncwarp();
  }
  if (BWD) {
    __syncthreads();
    block_dw(a, sums, WARPS);
    follow_allow();
  }
}

// dw = the blocks' sums, in block order: 32 columns of a block, its 16 warps
// take a 16th of the sums each.
__global__ void __launch_bounds__(512) sum_dw_kernel(const float *part, int blocks, int D, float *dwq, float *dwk) {
  __shared__ float s[16][33];
  follow_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  float x = 0.f;
  if (c < 2 * D)
#pragma unroll 8
    for (int b = warp; b < blocks; b += 16) x += part[(int64_t)b * 2 * D + c];
  s[warp][threadIdx.x & 31] = x;
  __syncthreads();
  if (warp == 0 && c < 2 * D) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) y += s[w][threadIdx.x & 31];
    (c < D ? dwq : dwk)[c < D ? c : c - D] = y;
  }
}

constexpr int64_t BWD_BLOCKS = 152 * 3;  // blocks of the backward at most (resident at once)

int64_t bwd_blocks(int64_t tokens) { return std::max<int64_t>(1, std::min<int64_t>((tokens + WARPS - 1) / WARPS, BWD_BLOCKS)); }

glacore_status check(const glacore_qk_norm *p) {
  if (!p || p->B < 1 || p->T < 0 || p->Hq < 1 || p->Hk < 1 || p->Hq > 65535 || p->Hk > 65535 || p->D < 1 ||
      p->D > MAXD || p->R < 0 || 2 * p->R > p->D || p->B > (int64_t)1 << 31 || p->T > (int64_t)1 << 31 ||
      p->B * p->T > (int64_t)1 << 33)
    return GLACORE_ERR_INVALID_ARG;
  if (p->dtype != GLACORE_F32 && p->dtype != GLACORE_BF16) return GLACORE_ERR_INVALID_ARG;
  if ((p->l2 != 0 && p->l2 != 1) || (p->interleaved != 0 && p->interleaved != 1) || !(p->eps >= 0.f) || p->reserved0)
    return GLACORE_ERR_INVALID_ARG;
  if ((p->q_stride && p->q_stride < p->Hq * p->D) || (p->k_stride && p->k_stride < p->Hk * p->D))
    return GLACORE_ERR_INVALID_ARG;
  if (p->R > 0 && (!p->cos_table || !p->sin_table || p->n_positions < 1)) return GLACORE_ERR_INVALID_ARG;
  const uintptr_t es = p->dtype == GLACORE_BF16 ? 1 : 3;
  if ((((uintptr_t)p->q | (uintptr_t)p->k) & es) ||
      (((uintptr_t)p->wq | (uintptr_t)p->wk | (uintptr_t)p->cos_table | (uintptr_t)p->sin_table |
        (uintptr_t)p->positions) & 3))
    return GLACORE_ERR_INVALID_ARG;
  if (p->B * p->T > 0 && (!p->q || !p->k)) return GLACORE_ERR_INVALID_ARG;
  return GLACORE_OK;
}

Args make_args(const glacore_qk_norm *p, void *yq, void *yk, int *err) {
  Args a;
  memset(&a, 0, sizeof(a));
  a.x[0] = p->q;
  a.x[1] = p->k;
  a.y[0] = yq;
  a.y[1] = yk;
  a.w[0] = p->wq;
  a.w[1] = p->wk;
  a.cs = p->cos_table;
  a.sn = p->sin_table;
  a.pos = p->positions;
  a.err = err;
  a.tokens = p->B * p->T;
  a.T = p->T;
  a.P = p->n_positions;
  a.xs[0] = p->q_stride ? p->q_stride : p->Hq * p->D;
  a.xs[1] = p->k_stride ? p->k_stride : p->Hk * p->D;
  a.H[0] = (int)p->Hq;
  a.H[1] = (int)p->Hk;
  a.D = (int)p->D;
  a.R = (int)p->R;
  a.mean = !p->l2;
  a.inter = p->interleaved;
  a.eps = p->eps;
  return a;
}

// Rows that the kernels with 8 channels per lane take: 16-byte steps everywhere.
bool vectors(const glacore_qk_norm *p, const Args &a) {
  const int64_t step = p->dtype == GLACORE_BF16 ? 8 : 4;
  const uintptr_t at = (uintptr_t)a.x[0] | (uintptr_t)a.x[1] | (uintptr_t)a.y[0] | (uintptr_t)a.y[1] |
                       (uintptr_t)a.dy[0] | (uintptr_t)a.dy[1];
  return p->D % 8 == 0 && (a.inter || p->R % 8 == 0) && (!a.inter || p->R % 4 == 0) && a.xs[0] % step == 0 &&
         a.xs[1] % step == 0 && !(at & 15);
}

// go(E), 32 E channels holding a row
template <typename F>
void by_channels(int64_t D, F go) {
  if (D <= 32) go(std::integral_constant<int, 1>());
  else if (D <= 64) go(std::integral_constant<int, 2>());
  else if (D <= 128) go(std::integral_constant<int, 4>());
  else go(std::integral_constant<int, 8>());
}

template <typename T>
cudaError_t run_fwd(const glacore_qk_norm *p, Args &a, cudaStream_t st) {
  if (!vectors(p, a)) {
    const int64_t rows = a.tokens * (a.H[0] + a.H[1]);
    const unsigned blocks = (unsigned)std::min<int64_t>((rows + WARPS - 1) / WARPS, 152 * 64);
    by_channels(p->D, [&](auto e) { rows_kernel<T, false, decltype(e)::value><<<blocks, THREADS, 0, st>>>(a); });
    return cudaGetLastError();
  }
  // A warp takes all heads of a token's queries (keys); few tokens: fewer heads,
  // down to one pass in flight, so that the card has work for its warps.
  const int lpr = p->D <= 64 ? 8 : p->D <= 128 ? 16 : 32, least = 32 / lpr;
  for (int z = 0; z < 2; ++z) {
    int g = a.H[z];
    while (g > least && a.tokens * 2 * ((a.H[z] + g - 1) / g) < 152 * 16) g = (g + 1) / 2;
    g = std::max(g, (a.H[z] + 16383) / 16384);  // the second axis of a grid has 65535 places
    a.group[z] = (g + least - 1) / least * least;
    a.parts[z] = (a.H[z] + a.group[z] - 1) / a.group[z];
  }
  const dim3 grid((unsigned)((a.tokens + WARPS - 1) / WARPS), a.parts[0] + a.parts[1]);
  auto go = [&](auto kernel) { kernel<<<grid, THREADS, 0, st>>>(a); };
  if (lpr == 8)
    a.R ? go(fwd_kernel<T, 8, true>) : go(fwd_kernel<T, 8, false>);
  else if (lpr == 16)
    a.R ? go(fwd_kernel<T, 16, true>) : go(fwd_kernel<T, 16, false>);
  else
    a.R ? go(fwd_kernel<T, 32, true>) : go(fwd_kernel<T, 32, false>);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_bwd(const glacore_qk_norm *p, Args &a, float *dwq, float *dwk, cudaStream_t st) {
  for (int z = 0; z < 2; ++z) {  // two warps to the heads of a token where there are enough: the last round is shorter
    a.parts[z] = a.H[z] >= 8 ? 2 : 1;
    a.group[z] = (a.H[z] + a.parts[z] - 1) / a.parts[z];
  }
  const int64_t blocks = bwd_blocks(a.tokens);
  const size_t row = 2 * sizeof(float) * a.D;
  if (!vectors(p, a)) {
    by_channels(p->D, [&](auto e) {
      rows_kernel<T, true, decltype(e)::value><<<(unsigned)blocks, THREADS, WARPS * row, st>>>(a);
    });
  } else {
    const int lpr = p->D <= 64 ? 8 : p->D <= 128 ? 16 : 32;
    auto go = [&](auto kernel) { kernel<<<(unsigned)blocks, THREADS, WARPS * (32 / lpr) * row, st>>>(a); };
    if (lpr == 8)
      a.R ? go(bwd_kernel<T, 8, true>) : go(bwd_kernel<T, 8, false>);
    else if (lpr == 16)
      a.R ? go(bwd_kernel<T, 16, true>) : go(bwd_kernel<T, 16, false>);
    else
      a.R ? go(bwd_kernel<T, 32, true>) : go(bwd_kernel<T, 32, false>);
  }
  cudaError_t e = cudaGetLastError();
  mark_launch("qk_norm_bwd", st);
  if (e != cudaSuccess) return e;
  e = launch_follow(sum_dw_kernel, dim3((unsigned)((2 * a.D + 31) / 32)), dim3(512), st, (const float *)a.part,
                    (int)blocks, a.D, dwq, dwk);
  mark_launch("qk_norm_sum_dw", st);
  return e;
}

}  // namespace
}  // namespace qkn
}  // namespace glacore

using namespace glacore;

extern "C" {

size_t qk_norm_bwd_workspace_size(const glacore_qk_norm *p) {
  if (qkn::check(p) != GLACORE_OK) return 0;
  return (size_t)qkn::bwd_blocks(p->B * p->T) * 2 * p->D * sizeof(float);
}

glacore_status qk_norm_fwd(const glacore_qk_norm *p, void *qo, void *ko, glacore_stream_t stream) {
  begin_marks();
  const glacore_status s = qkn::check(p);
  if (s) return s;
  if (p->B * p->T == 0) return GLACORE_OK;
  if (!qo || !ko || (((uintptr_t)qo | (uintptr_t)ko) & (p->dtype == GLACORE_BF16 ? 1 : 3)))
    return GLACORE_ERR_INVALID_ARG;
  int *err = device_error_ptr();
  if (!err) return GLACORE_ERR_CUDA;
  qkn::Args a = qkn::make_args(p, qo, ko, err);
  const cudaError_t e = p->dtype == GLACORE_BF16 ? qkn::run_fwd<__nv_bfloat16>(p, a, (cudaStream_t)stream)
                                                 : qkn::run_fwd<float>(p, a, (cudaStream_t)stream);
  mark_launch("qk_norm_fwd", (cudaStream_t)stream);
  return status_of(e);
}

glacore_status qk_norm_bwd(const glacore_qk_norm *p, const void *dqo, const void *dko, void *dq, void *dk, float *dwq,
                           float *dwk, glacore_stream_t stream) {
  begin_marks();
  const glacore_status s = qkn::check(p);
  if (s) return s;
  const uintptr_t es = p->dtype == GLACORE_BF16 ? 1 : 3;
  if (!dwq || !dwk || (((uintptr_t)dwq | (uintptr_t)dwk) & 3)) return GLACORE_ERR_INVALID_ARG;
  if (p->B * p->T > 0 && (!dqo || !dko || !dq || !dk ||
                          (((uintptr_t)dqo | (uintptr_t)dko | (uintptr_t)dq | (uintptr_t)dk) & es)))
    return GLACORE_ERR_INVALID_ARG;
  if (!p->workspace || p->workspace_bytes < qk_norm_bwd_workspace_size(p) || ((uintptr_t)p->workspace & 255))
    return GLACORE_ERR_WORKSPACE;
  int *err = device_error_ptr();
  if (!err) return GLACORE_ERR_CUDA;
  qkn::Args a = qkn::make_args(p, dq, dk, err);
  a.dy[0] = dqo;
  a.dy[1] = dko;
  a.part = (float *)p->workspace;
  return status_of(p->dtype == GLACORE_BF16 ? qkn::run_bwd<__nv_bfloat16>(p, a, dwq, dwk, (cudaStream_t)stream)
                                            : qkn::run_bwd<float>(p, a, dwq, dwk, (cudaStream_t)stream));
}

}  // extern "C"
