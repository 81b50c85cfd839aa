// layer_norm.cu -- layer norm, forward and backward, with the gradients of
// its weights (C ABI in include/glacore.h).  Over each row of D values:
//     m = mean(x),  r = (mean((x - m)^2) + eps)^(-1/2),
//     n = (x - m) r,  y = n w + b
//   backward, a = dy w:
//     dx = r (a - mean(a) - n mean(a n)),  dw = sum_rows dy n,  db = sum_rows dy
//
// HBM-bound, with the instruction issue close behind: the forward moves 2, the
// backward 3 rows of D values per token and nothing is read twice.  A row
// lives in the registers of L threads (column vectors t, t + L, ... of 16
// bytes for thread t), so the mean and the squared deviations from it are two
// exact passes over registers; the next row is loaded before this one is
// reduced.  A sum over a row's threads costs some 30 instructions each, so a
// thread holds as many values of a row as registers allow: in the forward up
// to 64 (a warp holds a row of 2048 bf16 and needs no barrier; the weights
// wait in shared memory), in the backward 16 to 32 beside the column sums of
// the two weight gradients, with a barrier of the row's own warps.  (8 values
// per thread ran the forward at 77% of all issue slots and 28% of the DRAM
// rate.)  The arithmetic is fp32, two values per instruction; bf16 outputs are
// rounded once.  Rows of more than MAX_COLS values are walked in a loop by a
// whole CTA instead.  The weight gradients are deterministic: per-CTA partial
// sums in the workspace, then one kernel that adds the partial rows in a fixed
// order.
// Measured: 8192 x 2048 bf16 forward 14.5 us (4.6 TB/s), backward 25.5 us (3.9
// TB/s; 3.5 us of it the sum of the partial rows).  Forward / backward by what a
// row's length allows, 4554 rows of bf16: 1336 values (16-byte accesses) 9.0 /
// 16.3 us, 1334 (4 bytes) 11.1 / 18.7 us, 1335 (single values, the backward's
// copied as words) 17.4 / 24.7 us; 4099 rows of fp32: 1112 values 9.0 / 15.8 us,
// 1111 14.9 / 23.4 us.  Rows in registers and longer ones, 4096 of bf16: 8192
// values 32 / 66 us, 8200 (walked by a CTA, single values, three passes) 56 / 132
// us, 12288 77 / 187 us, where 8191, single values in registers, take 96 / 116 us.
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
constexpr size_t SMEM_DEFAULT = 46 << 10;  // dynamic shared memory that needs no leave (48 KB with the static part)

// VEC consecutive values of T as they lie in memory: 16 bytes, or 4 or one
// bf16 where the row length or an address rules that out.
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
template <> struct Vec<__nv_bfloat16, 2> {
  uint32_t u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint32_t *>(p); }
  __device__ __forceinline__ void get(float (&v)[2]) const {
    v[0] = __uint_as_float(u << 16);
    v[1] = __uint_as_float(u & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[2]) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
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

// Two fp32 operations per instruction.
__device__ __forceinline__ void fma2(float &x, float &y, float ax, float ay, float bx, float by, float cx, float cy) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
      : "=f"(x), "=f"(y)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by), "f"(cx), "f"(cy));
}
__device__ __forceinline__ void add2(float &x, float &y, float ax, float ay) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(x), "=f"(y)
      : "f"(ax), "f"(ay), "f"(x), "f"(y));
}
__device__ __forceinline__ void mul2(float &x, float &y, float ax, float ay, float bx, float by) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(x), "=f"(y)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
// The same over N values: o = a b + c, o += a, o = a b (b and c may be one
// number for all).
struct All {
  float v;
  __device__ __forceinline__ float operator[](int) const { return v; }
};
template <int N, typename B, typename C>
__device__ __forceinline__ void vfma(float (&o)[N], const float (&a)[N], const B &b, const C &c) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) fma2(o[i], o[i + 1], a[i], a[i + 1], b[i], b[i + 1], c[i], c[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(a[i], b[i], c[i]);
  }
}
template <int N> __device__ __forceinline__ void vadd(float (&o)[N], const float (&a)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) add2(o[i], o[i + 1], a[i], a[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] += a[i];
  }
}
template <int N, typename B>
__device__ __forceinline__ void vmul(float (&o)[N], const float (&a)[N], const B &b) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) mul2(o[i], o[i + 1], a[i], a[i + 1], b[i], b[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = a[i] * b[i];
  }
}
template <int N> __device__ __forceinline__ float total(const float (&a)[N]) {
  float s = a[0];
#pragma unroll
  for (int i = 1; i < N; ++i) s += a[i];
  return s;
}

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

// Shared-memory copy of D weights, 16-byte accesses of a warp free of bank
// conflicts: of 8 consecutive weights the first four lie in one half of the
// copy, the others in the other.
template <int VEC> __device__ __forceinline__ int staged_at(int c, int D) {
  return VEC == 8 ? ((c >> 2) & 1) * (D / 2) + (c >> 3) * 4 + (c & 3) : c;
}
template <int VEC> __device__ __forceinline__ void staged(const float *s, int c, int D, float (&v)[VEC]) {
  if constexpr (VEC < 4) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = s[c + e];
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(s + staged_at<VEC>(c + e, D));
      v[e] = f.x; v[e + 1] = f.y; v[e + 2] = f.z; v[e + 3] = f.w;
    }
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
      for (int i = 0; i < N; ++i) v[i] = red[buf][first][i];
      for (int k = 1; k < wpr; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += red[buf][first + k][i];
      buf ^= 1;
    }
  }
  __device__ __forceinline__ float operator()(float x) {
    float v[1] = {x};
    (*this)(v);
    return v[0];
  }
};

// Whether the forward loads a row's successor early: where registers allow.
constexpr bool early(int bytes) { return bytes <= 128; }

// STAGED: w and b go through shared memory (worth it where a CTA takes several
// rows).
template <typename T, int VEC, int NV, bool STAGED>
__global__ void __launch_bounds__(THREADS)
    layer_norm_fwd_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b,
                          T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd, int64_t rows, int D,
                          int64_t xs, int lg, float eps) {
  constexpr bool EARLY = STAGED && early(NV * VEC * (int)sizeof(T));
  extern __shared__ float4 smem[];
  __shared__ float red[2][THREADS / 32][1];
  const int L = 1 << lg, t = threadIdx.x & (L - 1), per = THREADS >> lg;
  RowSum<1> sum{red, L, 0};
  const float inv = 1.f / (float)D;
  float *sw = reinterpret_cast<float *>(smem), *sb = sw + (D + 3) / 4 * 4;
  Vec<T, VEC> xv[NV], next[NV];
  auto fetch = [&](int64_t row, Vec<T, VEC>(&v)[NV]) {
    if (row >= rows) return;
    const T *p = x + row * xs + t * VEC;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if ((j * L + t) * VEC < D) v[j].load(p + j * L * VEC);
  };
  int64_t row = (int64_t)blockIdx.x * per + (threadIdx.x >> lg);
  const int64_t step = (int64_t)gridDim.x * per;
  if (EARLY) fetch(row, xv);  // under way while the weights are staged
  if (STAGED) {
    for (int c = threadIdx.x; c < D; c += THREADS) {
      sw[staged_at<VEC>(c, D)] = w ? w[c] : 1.f;
      sb[staged_at<VEC>(c, D)] = b ? b[c] : 0.f;
    }
    __syncthreads();
  }
  // every thread of the CTA turns as often as its first row group (barriers)
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < rows; r0 += step, row += step) {
    if (EARLY)
      fetch(row + step, next);
    else
      fetch(row, xv);
    const bool live = row < rows;
    float acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (live && (j * L + t) * VEC < D) {
        float v[VEC];
        xv[j].get(v);
        vadd(acc, v);
      }
    const float m = sum(total(acc)) * inv;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (live && (j * L + t) * VEC < D) {
        float v[VEC], d[VEC];
        xv[j].get(v);
        vfma(d, v, All{1.f}, All{-m});
        vfma(acc, d, d, acc);
      }
    const float r = rsqrtf(sum(total(acc)) * inv + eps);
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * L + t) * VEC;
        if (c < D) {
          float v[VEC], wv[VEC], bv[VEC];
          xv[j].get(v);
          if (STAGED) {
            staged<VEC>(sw, c, D, wv);
            staged<VEC>(sb, c, D, bv);
          } else {
            weights<VEC>(w, c, 1.f, wv);
            weights<VEC>(b, c, 0.f, bv);
          }
          // the difference first: exact for x near m, however far off centre
          vfma(v, v, All{1.f}, All{-m});
          vmul(v, v, All{r});
          vfma(v, v, wv, bv);
          Vec<T, VEC>::store(y + row * D + c, v);
        }
      }
      if (t == 0 && mean) {
        mean[row] = m;
        rstd[row] = r;
      }
    }
    if (EARLY)
#pragma unroll
      for (int j = 0; j < NV; ++j) xv[j] = next[j];
  }
}

// Copy of BYTES (4 or 16) to shared memory, in flight until its group is
// waited for.
template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}

// The backward takes two rows at a time (one exchange of sums for both), and
// copies them to shared memory AHEAD turns before theirs, each thread its own
// columns (no barrier: a thread reads only what it copied).  In registers the
// rows in flight would have to share the space with the column sums: 8192 x
// 2048 bf16 ran with 32 KB in flight per SM and 35 us.  Rows that start between
// two vectors (odd lengths) are copied as the 16-byte words that hold them, by
// their whole row group, with a barrier of the group per turn (4554 x 1335 bf16:
// 66 us when they were read in place, 24.4 us so; 4099 x 1111 fp32: 26.6 us when
// they were copied value by value, 23.8 us so).
// Such a word may hold up to 15 bytes beside the row: they are in the same aligned
// 16 bytes as a value of it, so never on another page, and nothing uses them.
constexpr int AHEAD = 2, SLOTS = AHEAD + 1;
// by a thread's values of a row (shared memory)
constexpr int rows_at_once(int values) { return values <= 16 ? 2 : 1; }

// Shared memory of one row, or of the words that hold it (single values).
__host__ __device__ inline int slot_bytes(int row_bytes, int vec) {
  return (row_bytes + (vec == 1 ? 15 : 0) + 15) / 16 * 16;
}

// part: [gridDim.x][2][D] partial dw, db of the rows each CTA walked.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(THREADS, 2)
    layer_norm_bwd_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ mean,
                          const float *__restrict__ rstd, const T *__restrict__ dy, T *__restrict__ dx,
                          float *__restrict__ part, int64_t rows, int D, int64_t xs, int64_t ys, int lg) {
  follow_allow();
  constexpr int BYTES = VEC * (int)sizeof(T);
  constexpr bool WORDS = VEC == 1;
  constexpr int R = rows_at_once(NV * VEC);
  extern __shared__ float4 smem[];
  __shared__ float red[2][THREADS / 32][2 * R];
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
  // this thread's columns of its row group's slots: x, dy of each of R rows
  const int pitch = slot_bytes(D * (int)sizeof(T), VEC);
  char *slots = reinterpret_cast<char *>(smem) + (int64_t)(threadIdx.x >> lg) * SLOTS * R * 2 * pitch + t * BYTES;
  auto fetch = [&](int64_t row, int slot) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (row + i < rows) {
        const T *px = x + (row + i) * xs, *pg = dy + (row + i) * ys;
        char *to = slots + (slot * R + i) * 2 * pitch;
        if constexpr (WORDS) {
          to += t * (16 - BYTES);
          const char *wx = reinterpret_cast<const char *>((uintptr_t)px & ~(uintptr_t)15) + 16 * t;
          const char *wg = reinterpret_cast<const char *>((uintptr_t)pg & ~(uintptr_t)15) + 16 * t;
          const char *ex = reinterpret_cast<const char *>(px + D), *eg = reinterpret_cast<const char *>(pg + D);
          for (int k = 0; wx + k < ex; k += 16 * L) copy_async<16>(to + k, wx + k);
          for (int k = 0; wg + k < eg; k += 16 * L) copy_async<16>(to + pitch + k, wg + k);
        } else {
          px += t * VEC;
          pg += t * VEC;
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if ((j * L + t) * VEC < D) {
              copy_async<BYTES>(to + j * L * BYTES, px + j * L * VEC);
              copy_async<BYTES>(to + pitch + j * L * BYTES, pg + j * L * VEC);
            }
        }
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t row = (int64_t)blockIdx.x * per + (threadIdx.x >> lg) * R;
  const int64_t step = (int64_t)gridDim.x * per;
  float m_next[R], r_next[R];
  auto stats = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (row + i < rows) {
        m_next[i] = mean[row + i];
        r_next[i] = rstd[row + i];
      }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(row + i * step, i);
  stats(row);
  int slot = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < rows; r0 += step, row += step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
    if constexpr (WORDS) {  // the group's copies are in, and it is done with the slot copied to next
      if (L > 32)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (threadIdx.x >> lg)), "r"(L) : "memory");
      else
        __syncwarp();
    }
    fetch(row + AHEAD * step, slot == 0 ? SLOTS - 1 : slot - 1);
    float m[R], r[R], s[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = m_next[i];
      r[i] = r_next[i];
    }
    stats(row + step);
    auto get = [&](int i, int j, float(&v)[VEC], float(&g)[VEC]) {  // columns j of x and dy of row i
      Vec<T, VEC> vx, vg;
      const char *fx = slots + (slot * R + i) * 2 * pitch + j * L * BYTES, *fg = fx + pitch;
      if constexpr (WORDS) {  // where in its first word the row starts
        fx += (uintptr_t)(x + (row + i) * xs) & 15;
        fg += (uintptr_t)(dy + (row + i) * ys) & 15;
      }
      vx.load(reinterpret_cast<const T *>(fx));
      vg.load(reinterpret_cast<const T *>(fg));
      vx.get(v);
      vg.get(g);
    };
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float s0[VEC], s1[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) s0[e] = s1[e] = 0.f;
      if (row + i < rows)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (VEC == 1 && j * L >= D) {  // no thread of the row has this one: jump, do not predicate
            break;
          } else if ((j * L + t) * VEC < D) {
            float n[VEC], g[VEC], a[VEC];
            get(i, j, n, g);
            vfma(n, n, All{1.f}, All{-m[i]});  // as in the forward
            vmul(n, n, All{r[i]});
            vmul(a, g, wv[j]);
            vfma(dw[j], g, n, dw[j]);
            vadd(db[j], g);
            vadd(s0, a);
            vfma(s1, a, n, s1);
          }
      s[2 * i] = total(s0);
      s[2 * i + 1] = total(s1);
    }
    sum(s);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (row + i >= rows) continue;
      // dx = r a - r mean(a) - r mean(a n) n = r a + k0 + kx (x - m), the
      // difference first: as r a + kx x + k1 the row of a mean of 1000 deviations
      // lost 1.4e-5 of the largest dx in k1
      const float kx = -s[2 * i + 1] * inv * r[i] * r[i], k0 = -s[2 * i] * inv * r[i];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * L + t) * VEC;
        if (VEC == 1 && j * L >= D) break;
        if (c < D) {
          float v[VEC], g[VEC];
          get(i, j, v, g);
          vmul(g, g, wv[j]);
          vfma(v, v, All{1.f}, All{-m[i]});
          vfma(v, v, All{kx}, All{k0});
          vfma(v, g, All{r[i]}, v);
          Vec<T, VEC>::store(dx + (row + i) * D + c, v);
        }
      }
    }
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  }
  float *cols = reinterpret_cast<float *>(smem);  // the slots are done with
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
  follow_wait();
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

// Fewest vectors a thread is built for.
constexpr int least_nv(int vec) { return vec < 4 ? 4 / vec : 1; }

// vec values per vector.  A thread
// takes up to `most` values of a row before the row takes more threads than a
// warp, and more than that only where 256 threads do not hold the row.  Few
// rows are spread wider, so that more threads have loads in flight.
inline Plan plan_of(int64_t rows, int64_t D, int vec, int most) {
  const int64_t need = (D + vec - 1) / vec;
  const int least = least_nv(vec);
  Plan p;
  p.vec = vec;
  p.nv = least;
  while (p.nv * vec < most && need > 32 * p.nv) p.nv *= 2;
  while (p.nv > least && need <= (int64_t)THREADS * p.nv / 2 &&
         rows * ((need + 32 * p.nv - 1) / (32 * p.nv)) < 8 * tc::sm_count())
    p.nv /= 2;
  while (need > (int64_t)THREADS * p.nv) p.nv *= 2;
  p.lg = log2_up((need + p.nv - 1) / p.nv);
  p.ctas = (rows + (THREADS >> p.lg) - 1) / (THREADS >> p.lg);
  return p;
}

// CTAs of a persistent launch: what fits at once.  The part of it that hangs
// on registers is looked up once per kernel.
template <typename K> int64_t resident(K kernel, std::atomic<int> &cache, size_t smem = 0) {
  int n = cache.load(std::memory_order_relaxed);
  if (n <= 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, THREADS, 0) != cudaSuccess || n <= 0) n = 1;
    cache.store(n, std::memory_order_relaxed);
  }
  return std::min<int64_t>(n, (227 << 10) / (smem + 2048)) * tc::sm_count();
}

// Values per access: 16 bytes, else 4, else one, as rows, strides (elements)
// and addresses allow (weights: 16 bytes with the first only).
inline int vec_of(bool bf, int64_t D, int64_t s0, int64_t s1, uintptr_t data, uintptr_t w) {
  const int64_t all = D | s0 | s1;
  const int full = bf ? 8 : 4;
  if (all % full == 0 && ((data | w) & 15) == 0) return full;
  return bf && all % 2 == 0 && (data & 3) == 0 ? 2 : 1;
}

// Shared memory of the backward's rows, at most: 12 slots of each of 8 rows of
// 511 fp32 in the words that hold them are 198144 bytes, no other spread has more.
constexpr int RING_MAX = 12 * 8 * 2064;
// CTAs of the backward: two per SM at most (registers), one where the rows in
// flight take more than half the shared memory.
inline int64_t bwd_ctas(int64_t ctas, size_t smem) {
  return std::max<int64_t>(1, std::min<int64_t>(ctas, (smem <= (112u << 10) ? 2 : 1) * tc::sm_count()));
}
inline int64_t long_chunks(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(rows, 64)); }

// Calls f with the number of vectors as a constant: 1, 2, 4 or 8 times the
// least, up to MOST values.
template <int VEC, int MOST, typename F> void pick(int nv, F f) {
  constexpr int U = least_nv(VEC);
  switch (nv / U) {
    case 1: f(std::integral_constant<int, U>()); break;
    case 2: f(std::integral_constant<int, 2 * U>()); break;
    default:
      if constexpr (8 * U * VEC <= MOST) {
        if (nv == 8 * U) {
          f(std::integral_constant<int, 8 * U>());
          break;
        }
      }
      f(std::integral_constant<int, 4 * U>());
  }
}

template <typename T, int VEC>
cudaError_t fwd(const Plan &p, const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                int64_t rows, int64_t D, int64_t xs, float eps, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (p.ctas < 4 * tc::sm_count()) {  // a row or two per CTA: w and b straight from memory
      layer_norm_fwd_kernel<T, VEC, NV, false><<<(unsigned)p.ctas, THREADS, 0, st>>>(
          (const T *)x, w, b, (T *)y, mean, rstd, rows, (int)D, xs, p.lg, eps);
      return;
    }
    auto *k = layer_norm_fwd_kernel<T, VEC, NV, true>;
    static std::atomic<int> cache;
    const size_t smem = 2 * (size_t)((D + 3) / 4 * 4) * sizeof(float);
    if (smem > SMEM_DEFAULT) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * (int)MAX_COLS * (int)sizeof(float));
      if (e != cudaSuccess) return;
    }
    const unsigned grid = (unsigned)std::min<int64_t>(p.ctas, resident(k, cache, smem));
    k<<<grid, THREADS, smem, st>>>((const T *)x, w, b, (T *)y, mean, rstd, rows, (int)D, xs, p.lg, eps);
  };
  pick<VEC, 64>(p.nv, go);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t bwd(const Plan &p, int64_t &ctas, const void *x, const float *w, const float *mean, const float *rstd,
                const void *dy, void *dx, float *part, int64_t rows, int64_t D, int64_t xs, int64_t ys,
                cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    constexpr int R = rows_at_once(NV * VEC);
    auto *k = layer_norm_bwd_kernel<T, VEC, NV>;
    const size_t ring = (size_t)(THREADS >> p.lg) * SLOTS * R * 2 * slot_bytes((int)(D * sizeof(T)), VEC);
    const size_t smem = std::max(ring, (size_t)D * sizeof(float));
    if (smem > SMEM_DEFAULT) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_MAX);
      if (e != cudaSuccess) return;
    }
    ctas = bwd_ctas((p.ctas + R - 1) / R, smem);
    k<<<(unsigned)ctas, THREADS, smem, st>>>((const T *)x, w, mean, rstd, (const T *)dy, (T *)dx, part, rows, (int)D,
                                             xs, ys, p.lg);
  };
  pick<VEC, 32>(p.nv, go);  // 8192 values over 256 threads
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Every pointer at a multiple of its elements' size (null passes).
inline bool natural(int32_t dtype, uintptr_t data, uintptr_t fp32) {
  return (data & (dtype == GLACORE_BF16 ? 1 : 3)) == 0 && (fp32 & 3) == 0;
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
  begin_marks();
  if (!sizes_ok(rows, D, x_stride, dtype) || !(eps >= 0.f)) return GLACORE_ERR_INVALID_ARG;
  if (rows == 0) return GLACORE_OK;
  if (!x || !y || !mean != !rstd) return GLACORE_ERR_INVALID_ARG;
  if (!natural(dtype, (uintptr_t)x | (uintptr_t)y, (uintptr_t)w | (uintptr_t)b | (uintptr_t)mean | (uintptr_t)rstd))
    return GLACORE_ERR_INVALID_ARG;
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
    const int vec = vec_of(bf, D, xs, xs, (uintptr_t)x | (uintptr_t)y, (uintptr_t)w | (uintptr_t)b);
    const Plan p = plan_of(rows, D, vec, vec == 8 ? 64 : vec == 1 ? 16 : 32);
    auto go = bf ? vec == 8 ? fwd<__nv_bfloat16, 8> : vec == 2 ? fwd<__nv_bfloat16, 2> : fwd<__nv_bfloat16, 1>
              : vec == 4 ? fwd<float, 4> : fwd<float, 1>;
    e = go(p, x, w, b, y, mean, rstd, rows, D, xs, eps, st);
  }
  mark_launch("layer_norm_fwd", st);
  return status_of(e);
}

// Enough for every way a row can be spread (the spread also depends on the
// pointers, which the query does not see).
size_t layer_norm_bwd_workspace_size(int64_t rows, int64_t D) {
  if (rows < 0 || D < 1 || D >= ((int64_t)1 << 31)) return 0;
  const int64_t n = D > MAX_COLS ? long_chunks(rows) : bwd_ctas(rows, 0);
  return (size_t)n * 2 * (size_t)D * sizeof(float);
}

glacore_status layer_norm_bwd(const void *x, const float *w, const float *mean, const float *rstd, const void *dy,
                              int64_t rows, int64_t D, int64_t x_stride, int64_t dy_stride, int32_t dtype, void *dx,
                              float *dw, float *db, void *workspace, size_t workspace_bytes,
                              glacore_stream_t stream) {
  begin_marks();
  if (!sizes_ok(rows, D, x_stride, dtype) || (dy_stride != 0 && dy_stride < D) || !dw || !db ||
      !natural(dtype, (uintptr_t)x | (uintptr_t)dy | (uintptr_t)dx,
               (uintptr_t)w | (uintptr_t)mean | (uintptr_t)rstd | (uintptr_t)dw | (uintptr_t)db))
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
    const int vec = vec_of(bf, D, xs, ys, (uintptr_t)x | (uintptr_t)dy | (uintptr_t)dx, (uintptr_t)w);
    const Plan p = plan_of(rows, D, vec, 16);
    auto go = bf ? vec == 8 ? bwd<__nv_bfloat16, 8> : vec == 2 ? bwd<__nv_bfloat16, 2> : bwd<__nv_bfloat16, 1>
              : vec == 4 ? bwd<float, 4> : bwd<float, 1>;
    e = go(p, n, x, w, mean, rstd, dy, dx, part, rows, D, xs, ys, st);
  }
  mark_launch("layer_norm_bwd", st);
  if (e != cudaSuccess) return status_of(e);
  e = launch_follow(layer_norm_dw_kernel, dim3((unsigned)((2 * D + RED_X - 1) / RED_X)), dim3(RED_X, RED_Y), st,
                    (const float *)part, n, D, dw, db);
  mark_launch("layer_norm_dw", st);
  return status_of(e);
}

}  // extern "C"
