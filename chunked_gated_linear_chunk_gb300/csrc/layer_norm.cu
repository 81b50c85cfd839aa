// layer_norm.cu -- layer norm, forward and backward, with the gradients of
// its weights (C ABI in include/glacore.h).  Over each row of D values:
//     m = mean(x),  r = (mean((x - m)^2) + eps)^(-1/2),
//     n = (x - m) r,  y = n w + b
//   backward, a = dy w:
//     dx = r (a - mean(a) - n mean(a n)),  dw = sum_rows dy n,  db = sum_rows dy
//
// HBM-bound: the forward moves 2, the backward 3 rows of D values per token
// and nothing is read twice.  A row lives in the registers of L threads
// (column vectors t, t + L, ... of 16 bytes for thread t), so the mean and the
// squared deviations from it are two exact passes over registers.  A thread
// keeps its columns for the whole kernel: their weights and the column sums of
// the weight gradients stay in its registers (read for every row instead, w
// and b took the L1 more time than the rows took the memory: 8192 x 2048 bf16
// forward 22.5 us).  It takes up to two rows at a time and loads the next ones
// before it reduces these.  L <= 32 threads exchange sums by shuffles alone, L
// = 64 .. 256 through shared memory and a barrier of the row's own warps.
// Rows of more than MAX_COLS values are walked in a loop by a whole CTA
// instead.  All arithmetic is fp32; bf16 outputs are rounded once.  The weight
// gradients are deterministic: per-CTA partial sums in the workspace, then one
// kernel that adds the partial rows in a fixed order.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "internal.cuh"
#include "tc.cuh"

namespace glacore {
namespace ln {

constexpr int THREADS = 256;
constexpr int64_t MAX_COLS = 8192;  // a row in registers: at most 256 threads x 32 values
constexpr int LONG_THREADS = 512;   // a CTA per longer row
constexpr int RED_X = 32, RED_Y = 32;

// VEC consecutive values of T as they lie in memory (16 bytes, or one value
// where the row length or an address rules out 16-byte accesses).
template <typename T, int VEC> struct Vec;
template <> struct Vec<__nv_bfloat16, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec<float, 4> {
  float4 u;
  __device__ __forceinline__ void load(const float *p) { u = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
  static __device__ __forceinline__ void store(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <typename T> struct Vec<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T *p) { u = *p; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f32(u); }
  static __device__ __forceinline__ void store(T *p, const float (&v)[1]) { *p = from_f32<T>(v[0]); }
};

// VEC consecutive weights (null: all `otherwise`).
template <int VEC>
__device__ __forceinline__ void weights(const float *w, int64_t c, float otherwise, float (&v)[VEC]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = otherwise;
  } else if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4 *>(w + c + e));
      v[e] = f.x; v[e + 1] = f.y; v[e + 2] = f.z; v[e + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = __ldg(w + c + e);
  }
}

// N sums over the L threads of a row group, in every one of them.  Two
// buffers in turn: one barrier per call, since a thread writes a buffer again
// only after a barrier that everyone reaches after reading it.
template <int N> struct RowSum {
  float (*red)[THREADS / 32][N];
  int L, buf;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    for (int m = 1; m < L && m < 32; m <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    if (L > 32) {
      const int warp = threadIdx.x >> 5, wpr = L >> 5, first = warp & ~(wpr - 1);
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[buf][warp][i] = v[i];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / wpr), "r"(L) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.f;
      for (int k = 0; k < wpr; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += red[buf][first + k][i];
      buf ^= 1;
    }
  }
};

// Rows a thread takes at a time, and whether the next ones are loaded early:
// as far as registers allow.
constexpr int rows_of(int vec, int nv) { return vec * nv <= 8 ? 2 : 1; }
constexpr bool early(int vec, int nv) { return vec * nv * rows_of(vec, nv) <= 16; }

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(THREADS)
    layer_norm_fwd_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b,
                          T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd, int64_t rows, int D,
                          int64_t xs, int lg, float eps) {
  constexpr int R = rows_of(VEC, NV);
  __shared__ float red[2][THREADS / 32][R];
  const int L = 1 << lg, t = threadIdx.x & (L - 1), per = (THREADS >> lg) * R;
  RowSum<R> sum{red, L, 0};
  const float inv = 1.f / (float)D;
  float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((j * L + t) * VEC < D) {
      weights<VEC>(w, (j * L + t) * VEC, 1.f, wv[j]);
      weights<VEC>(b, (j * L + t) * VEC, 0.f, bv[j]);
    }
  Vec<T, VEC> xv[R][NV], next[R][NV];
  auto fetch = [&](int64_t r0, Vec<T, VEC>(&v)[R][NV]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = r0 + (threadIdx.x >> lg) * R + i;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (row < rows && (j * L + t) * VEC < D) v[i][j].load(x + row * xs + (j * L + t) * VEC);
    }
  };
  int64_t r0 = (int64_t)blockIdx.x * per;
  const int64_t step = (int64_t)gridDim.x * per;
  if (early(VEC, NV)) fetch(r0, xv);
  for (; r0 < rows; r0 += step) {
    if (early(VEC, NV))
      fetch(r0 + step, next);
    else
      fetch(r0, xv);
    const int64_t first = r0 + (threadIdx.x >> lg) * R;
    float m[R], r[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (first + i < rows && (j * L + t) * VEC < D) {
          float v[VEC];
          xv[i][j].get(v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) m[i] += v[e];
        }
    }
    sum(m);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] *= inv;
      r[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (first + i < rows && (j * L + t) * VEC < D) {
          float v[VEC];
          xv[i][j].get(v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) r[i] += (v[e] - m[i]) * (v[e] - m[i]);
        }
    }
    sum(r);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (first + i >= rows) continue;
      r[i] = rsqrtf(r[i] * inv + eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * L + t) * VEC;
        if (c < D) {
          float v[VEC];
          xv[i][j].get(v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] = (v[e] - m[i]) * r[i] * wv[j][e] + bv[j][e];
          Vec<T, VEC>::store(y + (first + i) * D + c, v);
        }
      }
      if (t == 0 && mean) {
        mean[first + i] = m[i];
        rstd[first + i] = r[i];
      }
    }
    if (early(VEC, NV))
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NV; ++j) xv[i][j] = next[i][j];
  }
}

// part: [gridDim.x][2][D] partial dw, db of the rows each CTA walked.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(THREADS)
    layer_norm_bwd_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ mean,
                          const float *__restrict__ rstd, const T *__restrict__ dy, T *__restrict__ dx,
                          float *__restrict__ part, int64_t rows, int D, int64_t xs, int64_t ys, int lg) {
  constexpr int R = rows_of(VEC, NV);
  __shared__ float red[2][THREADS / 32][2 * R];
  __shared__ float cols[MAX_COLS];
  const int L = 1 << lg, t = threadIdx.x & (L - 1), per = (THREADS >> lg) * R;
  RowSum<2 * R> sum{red, L, 0};
  const float inv = 1.f / (float)D;
  float wv[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if ((j * L + t) * VEC < D) weights<VEC>(w, (j * L + t) * VEC, 1.f, wv[j]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  struct Rows {
    Vec<T, VEC> x[R][NV], g[R][NV];
    float m[R], r[R];
  } cur, next;
  auto fetch = [&](int64_t r0, Rows &f) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = r0 + (threadIdx.x >> lg) * R + i;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (row < rows && (j * L + t) * VEC < D) {
          f.x[i][j].load(x + row * xs + (j * L + t) * VEC);
          f.g[i][j].load(dy + row * ys + (j * L + t) * VEC);
        }
      f.m[i] = row < rows ? mean[row] : 0.f;
      f.r[i] = row < rows ? rstd[row] : 0.f;
    }
  };
  int64_t r0 = (int64_t)blockIdx.x * per;
  const int64_t step = (int64_t)gridDim.x * per;
  if (early(VEC, NV)) fetch(r0, cur);
  for (; r0 < rows; r0 += step) {
    if (early(VEC, NV))
      fetch(r0 + step, next);
    else
      fetch(r0, cur);
    const int64_t first = r0 + (threadIdx.x >> lg) * R;
    float s[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[2 * i] = s[2 * i + 1] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (first + i < rows && (j * L + t) * VEC < D) {
          float v[VEC], g[VEC];
          cur.x[i][j].get(v);
          cur.g[i][j].get(g);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float n = (v[e] - cur.m[i]) * cur.r[i], a = g[e] * wv[j][e];
            dw[j][e] += g[e] * n;
            db[j][e] += g[e];
            s[2 * i] += a;
            s[2 * i + 1] += a * n;
          }
        }
    }
    sum(s);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float c1 = s[2 * i] * inv, c2 = s[2 * i + 1] * inv;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * L + t) * VEC;
        if (first + i < rows && c < D) {
          float v[VEC], g[VEC];
          cur.x[i][j].get(v);
          cur.g[i][j].get(g);
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            v[e] = cur.r[i] * (g[e] * wv[j][e] - c1 - (v[e] - cur.m[i]) * cur.r[i] * c2);
          Vec<T, VEC>::store(dx + (first + i) * D + c, v);
        }
      }
    }
    if (early(VEC, NV)) cur = next;
  }
  // Column sums of the CTA: rows that share a warp by shuffles, then the
  // warps one after another (in warp order) through shared memory.
  const int warp = threadIdx.x >> 5, turn = L > 32 ? threadIdx.x >> lg : warp,
            turns = L > 32 ? THREADS >> lg : THREADS / 32;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float(&acc)[NV][VEC] = which ? db : dw;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        for (int k = L; k < 32; k <<= 1) acc[j][e] += __shfl_xor_sync(0xffffffffu, acc[j][e], k);
    for (int i = 0; i < turns; ++i) {
      __syncthreads();
      if (turn == i && (L > 32 || (threadIdx.x & 31) < L))
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (j * L + t) * VEC;
          if (c < D)
#pragma unroll
            for (int e = 0; e < VEC; ++e) cols[c + e] = (i ? cols[c + e] : 0.f) + acc[j][e];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += THREADS) part[((int64_t)blockIdx.x * 2 + which) * D + c] = cols[c];
  }
}

// dw[c] / db[c] = sum over n partial rows, in order within each of RED_Y
// phases, then over the phases in order.
__global__ void __launch_bounds__(RED_X *RED_Y)
    layer_norm_dw_kernel(const float *__restrict__ part, int64_t n, int64_t D, float *__restrict__ dw,
                         float *__restrict__ db) {
  __shared__ float red[RED_Y][RED_X + 1];
  const int64_t c = (int64_t)blockIdx.x * RED_X + threadIdx.x;
  float acc = 0.f;
  if (c < 2 * D) {
    int64_t p = threadIdx.y;
    for (; p + 3 * RED_Y < n; p += 4 * RED_Y)
      acc += (part[p * 2 * D + c] + part[(p + RED_Y) * 2 * D + c]) +
             (part[(p + 2 * RED_Y) * 2 * D + c] + part[(p + 3 * RED_Y) * 2 * D + c]);
    for (; p < n; p += RED_Y) acc += part[p * 2 * D + c];
  }
  red[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.y == 0 && c < 2 * D) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < RED_Y; ++k) s += red[k][threadIdx.x];
    if (c < D)
      dw[c] = s;
    else
      db[c - D] = s;
  }
}

// ---- rows longer than MAX_COLS: a CTA walks the row -----------------------
__device__ __forceinline__ float2 cta_sum(float2 v, float2 *red) {
  for (int m = 1; m < 32; m <<= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, m);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, m);
  }
  __syncthreads();  // the last sum has been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = make_float2(0.f, 0.f);
  for (int i = 0; i < LONG_THREADS / 32; ++i) {
    v.x += red[i].x;
    v.y += red[i].y;
  }
  return v;
}

template <typename T>
__global__ void __launch_bounds__(LONG_THREADS)
    layer_norm_fwd_long_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b,
                               T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd, int64_t rows,
                               int64_t D, int64_t xs, float eps) {
  __shared__ float2 red[LONG_THREADS / 32];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * xs;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < D; c += LONG_THREADS) s += to_f32(xr[c]);
    const float m = cta_sum(make_float2(s, 0.f), red).x / (float)D;
    s = 0.f;
    for (int64_t c = threadIdx.x; c < D; c += LONG_THREADS) {
      const float d = to_f32(xr[c]) - m;
      s += d * d;
    }
    const float r = rsqrtf(cta_sum(make_float2(s, 0.f), red).x / (float)D + eps);
    for (int64_t c = threadIdx.x; c < D; c += LONG_THREADS)
      y[row * D + c] = from_f32<T>((to_f32(xr[c]) - m) * r * (w ? w[c] : 1.f) + (b ? b[c] : 0.f));
    if (threadIdx.x == 0 && mean) {
      mean[row] = m;
      rstd[row] = r;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(LONG_THREADS)
    layer_norm_bwd_long_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ mean,
                               const float *__restrict__ rstd, const T *__restrict__ dy, T *__restrict__ dx,
                               int64_t rows, int64_t D, int64_t xs, int64_t ys) {
  __shared__ float2 red[LONG_THREADS / 32];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * xs, *gr = dy + row * ys;
    const float m = mean[row], r = rstd[row];
    float2 s = make_float2(0.f, 0.f);
    for (int64_t c = threadIdx.x; c < D; c += LONG_THREADS) {
      const float a = to_f32(gr[c]) * (w ? w[c] : 1.f);
      s.x += a;
      s.y += a * (to_f32(xr[c]) - m) * r;
    }
    s = cta_sum(s, red);
    const float c1 = s.x / (float)D, c2 = s.y / (float)D;
    for (int64_t c = threadIdx.x; c < D; c += LONG_THREADS)
      dx[row * D + c] =
          from_f32<T>(r * (to_f32(gr[c]) * (w ? w[c] : 1.f) - c1 - (to_f32(xr[c]) - m) * r * c2));
  }
}

// Partial column sums of the long rows: a CTA takes 256 columns and every
// gridDim.y-th row.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    layer_norm_cols_long_kernel(const T *__restrict__ x, const float *__restrict__ mean,
                                const float *__restrict__ rstd, const T *__restrict__ dy, float *__restrict__ part,
                                int64_t rows, int64_t D, int64_t xs, int64_t ys) {
  const int64_t c = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  if (c >= D) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float g = to_f32(dy[row * ys + c]);
    dw += g * (to_f32(x[row * xs + c]) - mean[row]) * rstd[row];
    db += g;
  }
  part[(int64_t)blockIdx.y * 2 * D + c] = dw;
  part[((int64_t)blockIdx.y * 2 + 1) * D + c] = db;
}

// How a row is spread over threads: L threads (2^lg), nv vectors each.
struct Plan {
  int vec, nv, lg;
  int64_t ctas;  // that cover the rows once
};

inline int log2_up(int64_t v) {
  int lg = 0;
  while (((int64_t)1 << lg) < v) ++lg;
  return lg;
}

// vec values per vector (1 where 16-byte accesses are ruled out).  Up to 256
// threads share a row, one vector each, before a thread takes several.
inline Plan plan_of(int64_t rows, int64_t D, int vec) {
  const int64_t need = (D + vec - 1) / vec;
  Plan p;
  p.vec = vec;
  p.nv = vec == 1 ? 4 : 1;
  while (need > (int64_t)THREADS * p.nv) p.nv *= 2;
  p.lg = log2_up((need + p.nv - 1) / p.nv);
  const int64_t per = (int64_t)(THREADS >> p.lg) * rows_of(vec, p.nv);
  p.ctas = (rows + per - 1) / per;
  return p;
}

// CTAs of a persistent launch: what fits at once (looked up once per kernel).
template <typename K> int64_t resident(K kernel, std::atomic<int> &cache) {
  int n = cache.load(std::memory_order_relaxed);
  if (n <= 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, THREADS, 0) != cudaSuccess || n <= 0) n = 1;
    cache.store(n, std::memory_order_relaxed);
  }
  return n * tc::sm_count();
}

inline bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// CTAs of the backward, at most: few enough that the partial sums stay small.
inline int64_t bwd_ctas(int64_t ctas) { return std::max<int64_t>(1, std::min<int64_t>(ctas, 2 * tc::sm_count())); }
inline int64_t long_chunks(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(rows, 64)); }

// Calls f with the number of vectors as a constant: up to 8192 values per row
// over 256 threads.
template <int VEC, typename F> void pick(int nv, F f) {
  if constexpr (VEC == 1) {
    switch (nv) {
      case 4: f(std::integral_constant<int, 4>()); break;
      case 8: f(std::integral_constant<int, 8>()); break;
      case 16: f(std::integral_constant<int, 16>()); break;
      default: f(std::integral_constant<int, 32>()); break;
    }
  } else {
    switch (nv) {
      case 1: f(std::integral_constant<int, 1>()); break;
      case 2: f(std::integral_constant<int, 2>()); break;
      default:
        if constexpr (VEC == 4) {
          if (nv == 8) {
            f(std::integral_constant<int, 8>());
            break;
          }
        }
        f(std::integral_constant<int, 4>());
    }
  }
}

template <typename T, int VEC>
cudaError_t fwd(const Plan &p, const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                int64_t rows, int64_t D, int64_t xs, float eps, cudaStream_t st) {
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    static std::atomic<int> cache;
    auto *k = layer_norm_fwd_kernel<T, VEC, NV>;
    const unsigned grid = (unsigned)std::min<int64_t>(p.ctas, resident(k, cache));
    k<<<grid, THREADS, 0, st>>>((const T *)x, w, b, (T *)y, mean, rstd, rows, (int)D, xs, p.lg, eps);
  };
  pick<VEC>(p.nv, go);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t bwd(const Plan &p, int64_t &ctas, const void *x, const float *w, const float *mean, const float *rstd,
                const void *dy, void *dx, float *part, int64_t rows, int64_t D, int64_t xs, int64_t ys,
                cudaStream_t st) {
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    static std::atomic<int> cache;
    auto *k = layer_norm_bwd_kernel<T, VEC, NV>;
    ctas = std::min(bwd_ctas(p.ctas), resident(k, cache));
    k<<<(unsigned)ctas, THREADS, 0, st>>>((const T *)x, w, mean, rstd, (const T *)dy, (T *)dx, part, rows, (int)D, xs,
                                          ys, p.lg);
  };
  pick<VEC>(p.nv, go);
  return cudaGetLastError();
}

inline bool sizes_ok(int64_t rows, int64_t D, int64_t xs, int32_t dtype) {
  return rows >= 0 && D >= 1 && D < ((int64_t)1 << 31) && (xs == 0 || xs >= D) &&
         (dtype == GLACORE_BF16 || dtype == GLACORE_F32);
}

}  // namespace ln
}  // namespace glacore

using namespace glacore;
using namespace glacore::ln;

extern "C" {

glacore_status layer_norm_fwd(const void *x, const float *w, const float *b, int64_t rows, int64_t D,
                              int64_t x_stride, int32_t dtype, float eps, void *y, float *mean, float *rstd,
                              glacore_stream_t stream) {
  if (!sizes_ok(rows, D, x_stride, dtype) || !(eps >= 0.f)) return GLACORE_ERR_INVALID_ARG;
  if (rows == 0) return GLACORE_OK;
  if (!x || !y || !mean != !rstd) return GLACORE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t xs = x_stride ? x_stride : D;
  const bool bf = dtype == GLACORE_BF16;
  cudaError_t e;
  if (D > MAX_COLS) {
    const unsigned grid = (unsigned)std::min<int64_t>(rows, 4 * tc::sm_count());
    if (bf)
      layer_norm_fwd_long_kernel<__nv_bfloat16><<<grid, LONG_THREADS, 0, st>>>(
          (const __nv_bfloat16 *)x, w, b, (__nv_bfloat16 *)y, mean, rstd, rows, D, xs, eps);
    else
      layer_norm_fwd_long_kernel<float><<<grid, LONG_THREADS, 0, st>>>((const float *)x, w, b, (float *)y, mean, rstd,
                                                                       rows, D, xs, eps);
    e = cudaGetLastError();
  } else {
    const int full = bf ? 8 : 4;
    const bool wide = D % full == 0 && xs % full == 0 && al16(x) && al16(y) && al16(w) && al16(b);
    const Plan p = plan_of(rows, D, wide ? full : 1);
    if (bf)
      e = wide ? fwd<__nv_bfloat16, 8>(p, x, w, b, y, mean, rstd, rows, D, xs, eps, st)
               : fwd<__nv_bfloat16, 1>(p, x, w, b, y, mean, rstd, rows, D, xs, eps, st);
    else
      e = wide ? fwd<float, 4>(p, x, w, b, y, mean, rstd, rows, D, xs, eps, st)
               : fwd<float, 1>(p, x, w, b, y, mean, rstd, rows, D, xs, eps, st);
  }
  mark_launch("layer_norm_fwd", st);
  return status_of(e);
}

// Enough for every way a row can be spread (the spread also depends on the
// pointers, which the query does not see).
size_t layer_norm_bwd_workspace_size(int64_t rows, int64_t D) {
  if (rows < 0 || D < 1 || D >= ((int64_t)1 << 31)) return 0;
  const int64_t n = D > MAX_COLS ? long_chunks(rows) : bwd_ctas(rows);
  return (size_t)n * 2 * (size_t)D * sizeof(float);
}

glacore_status layer_norm_bwd(const void *x, const float *w, const float *mean, const float *rstd, const void *dy,
                              int64_t rows, int64_t D, int64_t x_stride, int64_t dy_stride, int32_t dtype, void *dx,
                              float *dw, float *db, void *workspace, size_t workspace_bytes,
                              glacore_stream_t stream) {
  if (!sizes_ok(rows, D, x_stride, dtype) || (dy_stride != 0 && dy_stride < D) || !dw || !db)
    return GLACORE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {
    const cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)D * sizeof(float), st);
    return status_of(e != cudaSuccess ? e : cudaMemsetAsync(db, 0, (size_t)D * sizeof(float), st));
  }
  if (!x || !mean || !rstd || !dy || !dx) return GLACORE_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < layer_norm_bwd_workspace_size(rows, D) || ((uintptr_t)workspace & 255))
    return GLACORE_ERR_WORKSPACE;
  const int64_t xs = x_stride ? x_stride : D, ys = dy_stride ? dy_stride : D;
  const bool bf = dtype == GLACORE_BF16;
  float *part = (float *)workspace;
  int64_t n;
  cudaError_t e;
  if (D > MAX_COLS) {
    n = long_chunks(rows);
    const unsigned grid = (unsigned)std::min<int64_t>(rows, 4 * tc::sm_count());
    const dim3 cgrid((unsigned)((D + THREADS - 1) / THREADS), (unsigned)n);
    if (bf) {
      typedef __nv_bfloat16 T;
      layer_norm_bwd_long_kernel<T><<<grid, LONG_THREADS, 0, st>>>((const T *)x, w, mean, rstd, (const T *)dy, (T *)dx,
                                                                   rows, D, xs, ys);
      layer_norm_cols_long_kernel<T><<<cgrid, THREADS, 0, st>>>((const T *)x, mean, rstd, (const T *)dy, part, rows, D,
                                                                xs, ys);
    } else {
      layer_norm_bwd_long_kernel<float><<<grid, LONG_THREADS, 0, st>>>((const float *)x, w, mean, rstd,
                                                                       (const float *)dy, (float *)dx, rows, D, xs, ys);
      layer_norm_cols_long_kernel<float><<<cgrid, THREADS, 0, st>>>((const float *)x, mean, rstd, (const float *)dy,
                                                                    part, rows, D, xs, ys);
    }
    e = cudaGetLastError();
  } else {
    const int full = bf ? 8 : 4;
    const bool wide = D % full == 0 && xs % full == 0 && ys % full == 0 && al16(x) && al16(dy) && al16(dx) && al16(w);
    const Plan p = plan_of(rows, D, wide ? full : 1);
    if (bf)
      e = wide ? bwd<__nv_bfloat16, 8>(p, n, x, w, mean, rstd, dy, dx, part, rows, D, xs, ys, st)
               : bwd<__nv_bfloat16, 1>(p, n, x, w, mean, rstd, dy, dx, part, rows, D, xs, ys, st);
    else
      e = wide ? bwd<float, 4>(p, n, x, w, mean, rstd, dy, dx, part, rows, D, xs, ys, st)
               : bwd<float, 1>(p, n, x, w, mean, rstd, dy, dx, part, rows, D, xs, ys, st);
  }
  mark_launch("layer_norm_bwd", st);
  if (e != cudaSuccess) return status_of(e);
  layer_norm_dw_kernel<<<(unsigned)((2 * D + RED_X - 1) / RED_X), dim3(RED_X, RED_Y), 0, st>>>(part, n, D, dw, db);
  mark_launch("layer_norm_dw", st);
  return status_of(cudaGetLastError());
}

}  // extern "C"
