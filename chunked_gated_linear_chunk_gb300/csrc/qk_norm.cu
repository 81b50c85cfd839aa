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
#include <string.h>

#include <algorithm>

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
  int group[2], parts[2];  // forward: heads of a warp, warps per token
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
__device__ __forceinline__ int64_t table_row(const Args &a, int64_t token) {
  const int64_t p = a.pos ? (int64_t)a.pos[token] : token % a.T;
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
// v rotated (back: the other way).  All lanes of the warp call it.
__device__ __forceinline__ void turn(const Args &a, const Turn &t, float (&v)[8], float dir) {
  if (a.R == 0) return;
  float o[8];
  if (a.inter) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = v[e ^ 1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, v[e], t.other);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fmaf(dir * t.s[e], o[e], t.c[e] * v[e]);
}

__device__ __forceinline__ void weights(const float *w, int c0, bool in, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = w && in ? __ldg(w + c0 + e) : 1.f;
}

template <typename T, int LPR>
__global__ void __launch_bounds__(THREADS) fwd_kernel(const Args a) {
  constexpr int RPP = 32 / LPR, UNROLL = 4;  // rows of a pass, passes in flight
  const int lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
  const int64_t unit = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  const int per = a.parts[0] + a.parts[1];
  const int64_t token = unit / per;
  if (token >= a.tokens) return;
  int part = (int)(unit % per);
  const int z = part >= a.parts[0];
  if (z) part -= a.parts[0];
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
  Turn t;
  make_turn<LPR>(a, token, li, t);
  float w[8];
  weights(a.w[z], c0, in, w);
  for (int h = h0; h < h1; h += UNROLL * RPP) {
    float f[UNROLL][8], ss[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      v[u].get(f[u]);
      ss[u] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[u] = fmaf(f[u][e], f[u][e], ss[u]);
    }
    fetch(h + UNROLL * RPP);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const float r = rsqrtf(fmaf(row_sum<LPR>(ss[u]), inv, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) f[u][e] = f[u][e] * r * w[e];
      turn(a, t, f[u], 1.f);
      const int hh = h + u * RPP + sub;
      if (in && hh < h1) Vec<T>::store(y + (int64_t)hh * a.D, f[u]);
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

template <typename T, int LPR>
__global__ void __launch_bounds__(THREADS) bwd_kernel(const Args a) {
  constexpr int RPP = 32 / LPR, UNROLL = 2;
  extern __shared__ float sums[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
  const int c0 = 8 * li;
  const bool in = c0 < a.D;
  const float inv = a.mean ? 1.f / (float)a.D : 1.f;
  float w[2][8], dw[2][8];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    weights(a.w[z], c0, in, w[z]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[z][e] = 0.f;
  }
  for (int64_t token = (int64_t)blockIdx.x * WARPS + warp; token < a.tokens; token += (int64_t)gridDim.x * WARPS) {
    Turn t;
    make_turn<LPR>(a, token, li, t);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const T *x = (const T *)a.x[z] + token * a.xs[z] + c0;
      const T *dy = (const T *)a.dy[z] + token * a.H[z] * a.D + c0;
      T *dx = (T *)a.y[z] + token * a.H[z] * a.D + c0;
      for (int h = 0; h < a.H[z]; h += UNROLL * RPP) {
        Vec<T> vx[UNROLL], vd[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          const int hh = h + u * RPP + sub;
          if (in && hh < a.H[z]) {
            vx[u].load(x + (int64_t)hh * a.D);
            vd[u].load(dy + (int64_t)hh * a.D);
          } else {
            vx[u].clear();
            vd[u].clear();
          }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          float f[8], d[8], ss = 0.f, sa = 0.f;
          vx[u].get(f);
          vd[u].get(d);
          turn(a, t, d, -1.f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(f[e], f[e], ss);
            sa = fmaf(d[e] * w[z][e], f[e], sa);
          }
          ss = row_sum<LPR>(ss);
          sa = row_sum<LPR>(sa);
          const float r = rsqrtf(fmaf(ss, inv, a.eps));
          const int hh = h + u * RPP + sub;
          const bool live = in && hh < a.H[z];
          const float m = sa * r * inv;  // mean (sum) of a w n
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float n = f[e] * r;
            o[e] = r * fmaf(-n, m, d[e] * w[z][e]);
            if (live) dw[z][e] = fmaf(d[e], n, dw[z][e]);
          }
          if (live) Vec<T>::store(dx + (int64_t)hh * a.D, o);
        }
      }
    }
  }
#pragma unroll
  for (int z = 0; z < 2; ++z)
    if (in)
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[((warp * RPP + sub) * 2 + z) * a.D + c0 + e] = dw[z][e];
  __syncthreads();
  block_dw(a, sums, WARPS * RPP);
  follow_allow();
}

// Rows of any D, R, stride and alignment: a warp per row, the row in shared memory.
template <typename T, bool BWD>
__global__ void __launch_bounds__(THREADS) rows_kernel(const Args a) {
  __shared__ float buf[WARPS][MAXD];
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
    const int64_t token = unit / heads;
    int h = (int)(unit % heads);
    const int z = h >= a.H[0];
    if (z) h -= a.H[0];
    const T *x = (const T *)a.x[z] + token * a.xs[z] + (int64_t)h * a.D;
    const int64_t at = (token * a.H[z] + h) * a.D;
    const float *w = a.w[z];
    int64_t p = -1;
    if (a.R) p = table_row(a, token);
    // channel c of a row in shared memory, rotated by dir
    auto turned = [&](int c, float dir) -> float {
      if (p < 0 || c >= 2 * a.R) return row[c];
      const bool first = a.inter ? (c & 1) == 0 : c < a.R;
      const int i = a.inter ? c / 2 : (first ? c : c - a.R), o = a.inter ? c ^ 1 : (first ? c + a.R : c - a.R);
      const float s = dir * __ldg(a.sn + p * a.R + i);
      return fmaf(first ? -s : s, row[o], __ldg(a.cs + p * a.R + i) * row[c]);
    };
    float f[MAXD / 32], d[MAXD / 32], ss = 0.f, sa = 0.f;
#pragma unroll
    for (int e = 0; e < MAXD / 32; ++e) {
      const int c = lane + 32 * e;
      f[e] = c < a.D ? to_f32(x[c]) : 0.f;
      ss = fmaf(f[e], f[e], ss);
      if (BWD && c < a.D) row[c] = to_f32(((const T *)a.dy[z])[at + c]);
    }
    __syncwarp();
    if (BWD) {
#pragma unroll
      for (int e = 0; e < MAXD / 32; ++e) {
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
      for (int e = 0; e < MAXD / 32; ++e) {
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
      for (int e = 0; e < MAXD / 32; ++e) {
        const int c = lane + 32 * e;
        if (c < a.D) row[c] = f[e] * r * (w ? __ldg(w + c) : 1.f);
      }
      __syncwarp();
      for (int c = lane; c < a.D; c += 32) ((T *)a.y[z])[at + c] = from_f32<T>(turned(c, 1.f));
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

constexpr int64_t BWD_BLOCKS = 152 * 4;  // blocks of the backward at most (resident at once)

int64_t bwd_blocks(int64_t tokens) { return std::max<int64_t>(1, std::min<int64_t>((tokens + WARPS - 1) / WARPS, BWD_BLOCKS)); }

glacore_status check(const glacore_qk_norm *p) {
  if (!p || p->B < 1 || p->T < 0 || p->Hq < 1 || p->Hk < 1 || p->Hq > 65535 || p->Hk > 65535 || p->D < 1 ||
      p->D > MAXD || p->R < 0 || 2 * p->R > p->D || p->B > (int64_t)1 << 31 || p->T > (int64_t)1 << 31)
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

template <typename T>
cudaError_t run_fwd(const glacore_qk_norm *p, Args &a, cudaStream_t st) {
  if (!vectors(p, a)) {
    const int64_t rows = a.tokens * (a.H[0] + a.H[1]);
    rows_kernel<T, false><<<(unsigned)std::min<int64_t>((rows + WARPS - 1) / WARPS, 152 * 64), THREADS, 0, st>>>(a);
    return cudaGetLastError();
  }
  // A warp takes all heads of a token's queries (keys); few tokens: fewer heads,
  // down to one pass in flight, so that the card has work for its warps.
  const int lpr = p->D <= 64 ? 8 : p->D <= 128 ? 16 : 32, least = 32 / lpr;
  for (int z = 0; z < 2; ++z) {
    int g = a.H[z];
    while (g > least && a.tokens * 2 * ((a.H[z] + g - 1) / g) < 152 * 16) g = (g + 1) / 2;
    a.group[z] = (g + least - 1) / least * least;
    a.parts[z] = (a.H[z] + a.group[z] - 1) / a.group[z];
  }
  const int64_t units = a.tokens * (a.parts[0] + a.parts[1]), blocks = (units + WARPS - 1) / WARPS;
  if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  if (lpr == 8)
    fwd_kernel<T, 8><<<(unsigned)blocks, THREADS, 0, st>>>(a);
  else if (lpr == 16)
    fwd_kernel<T, 16><<<(unsigned)blocks, THREADS, 0, st>>>(a);
  else
    fwd_kernel<T, 32><<<(unsigned)blocks, THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_bwd(const glacore_qk_norm *p, const Args &a, float *dwq, float *dwk, cudaStream_t st) {
  const int64_t blocks = bwd_blocks(a.tokens);
  const size_t row = 2 * sizeof(float) * a.D;
  if (!vectors(p, a)) {
    rows_kernel<T, true><<<(unsigned)blocks, THREADS, WARPS * row, st>>>(a);
  } else if (p->D <= 64) {
    bwd_kernel<T, 8><<<(unsigned)blocks, THREADS, WARPS * 4 * row, st>>>(a);
  } else if (p->D <= 128) {
    bwd_kernel<T, 16><<<(unsigned)blocks, THREADS, WARPS * 2 * row, st>>>(a);
  } else {
    bwd_kernel<T, 32><<<(unsigned)blocks, THREADS, WARPS * row, st>>>(a);
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
