// delta_simt.cu -- the gated delta rule on the CUDA cores, in fp32, for any
// K and V up to 256 and both types (formulas in delta.cuh); sums over the heads
// of a group, and the copies with padded rows that odd bf16 sizes go to the tensor
// cores as.
//
// The forward and the two passes of the backward that carry a state run token
// by token: a state's value columns do not see each other, so a warp owns 8
// columns of one (document, head), each thread KR key rows of two of them in
// registers, and one exchange
// over the 8 lanes of a column pair gives S^T k and S^T q of a token at once:
//     o_t = scale (e^g S^T q + (q . k) u),  u = b (v - e^g S^T k)
// (both on the state before the token).  fp32 and backwards two tokens at a time
// read the same state, the second corrected by k_1 . k_2 and k_1 . q_2, so that they
// share that exchange.  The other half of the block's warps converts the next 16
// tokens' q, k, v into shared memory meanwhile.  Bound by the latency of that
// dependence: 0.21 us a token in fp32, 0.26 one by one; any decay is exact here.  The
// gradients of q, k, g and beta then take every chunk of 64 tokens by itself
// (simt_grads), as products of 64 x 64 tiles.  333 tokens of 3 x 6 heads of 72 x 41,
// fp32: passes 70 us (both in one launch; token by token 85), gradients 48 us.
#include <algorithm>

#include "delta.cuh"
#include "tc.cuh"

namespace glacore {
namespace delta {

namespace {

constexpr int LK = 8;          // lanes along the key rows
constexpr int TT = 16;         // tokens staged at once
constexpr int COLS = 32;       // value columns of a block
constexpr int STAGERS = 4;     // warps that stage, behind those that compute
constexpr int NC = 2;          // columns of a thread (1 or 4: 10 to 25% more time where tokens are in sequence)
constexpr int CW = COLS / (4 * NC), THREADS = 32 * (CW + STAGERS);  // warps that compute; threads

// A thread's columns, one operation each (packed pairs take two cycles
// and want the key's channel twice in a register pair).
struct Cols {
  float v[NC];
};
__device__ __forceinline__ Cols fma_cols(float a, const Cols &b, const Cols &c) {
  Cols r;
#pragma unroll
  for (int n = 0; n < NC; ++n) r.v[n] = fmaf(a, b.v[n], c.v[n]);
  return r;
}
__device__ __forceinline__ Cols mul_cols(float a, const Cols &b) {
  Cols r;
#pragma unroll
  for (int n = 0; n < NC; ++n) r.v[n] = a * b.v[n];
  return r;
}

enum Mode { FWD, STATES, BACK };

template <typename T>
struct ScanArgs {
  const T *q, *k, *v;  // v: do in BACK
  const float *g, *beta, *seed;  // seed: initial state / gradient of the final state, or null
  float *last;                   // final state / gradient of the initial state, or null
  T *out;                        // o / null / dv
  float *states;                 // states before / gradients after every chunk (STATES, BACK)
  float *rows;                   // E / dR
  Docs docs;
  int64_t qs, ks, vs;
  int H, share, K, V, slices;
  float scale;
};

template <int KR>
struct alignas(16) Tile {
  float q[TT][LK * KR], k[TT][LK * KR];
  float v[TT][COLS];
  float a[TT], b[TT], qk[TT];
  float kk[TT], kq[TT];  // of odd tokens: k of the token before with k and q
};

template <typename T, int KR, int MODE>
__device__ __forceinline__ void scan(const ScanArgs<T> &a, uint32_t block) {
  extern __shared__ __align__(16) uint8_t smem[];
  Tile<KR> *tiles = reinterpret_cast<Tile<KR> *>(smem);  // two
  constexpr int KP = LK * KR;
  constexpr bool NEEDQ = MODE != STATES;
  constexpr bool TWO = KR <= 16 && !(MODE == FWD && sizeof(T) == 2);  // two tokens at a time
  const int slice = (int)(block % a.slices);
  const uint32_t dh = block / a.slices;
  const int h = (int)(dh % a.H);
  const int64_t d = dh / a.H;
  const int hq = h / a.share, v0 = slice * COLS;
  int64_t s0, s1;
  a.docs.range(d, s0, s1);
  const int64_t n = s1 - s0;
  const int ntile = (int)((n + TT - 1) / TT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool stages = warp >= CW;
  const int64_t slot0 = a.docs.chunk_base(d);

  // tile i of the pass covers the tokens tile_of(i) * TT ... of the document
  auto tile_of = [&](int i) { return MODE == BACK ? ntile - 1 - i : i; };
  auto stage = [&](int i) {
    Tile<KR> &t = tiles[i & 1];
    const int64_t t0 = (int64_t)tile_of(i) * TT;
    const int len = (int)min((int64_t)TT, n - t0);
    // a warp's four tokens at once: their loads are all in flight before the first is used
    constexpr int N = TT / STAGERS;
    float kx[N][KP / 32], qx[N][KP / 32], vx[N], gx[N], bx[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = (warp - CW) * N + n;
      const int64_t tok = s0 + t0 + (r < len ? r : 0);
      const T *qr = a.q + tok * a.qs + (int64_t)hq * a.K, *kr = a.k + tok * a.ks + (int64_t)hq * a.K;
#pragma unroll
      for (int e = 0; e < KP / 32; ++e) {
        const int c = lane + 32 * e;
        kx[n][e] = c < a.K ? to_f32(kr[c]) : 0.f;
        qx[n][e] = NEEDQ && c < a.K ? to_f32(qr[c]) : 0.f;
      }
      vx[n] = v0 + lane < a.V ? to_f32(a.v[tok * a.vs + (int64_t)h * a.V + v0 + lane]) : 0.f;
      gx[n] = a.g[tok * a.H + h];
      bx[n] = a.beta[tok * a.H + h];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = (warp - CW) * N + n;
      const bool odd = n & 1;
      float dot = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
      for (int e = 0; e < KP / 32; ++e) {
        t.k[r][lane + 32 * e] = kx[n][e];
        if (NEEDQ) t.q[r][lane + 32 * e] = qx[n][e];
        dot = fmaf(kx[n][e], qx[n][e], dot);
        if (TWO && odd) kk = fmaf(kx[n - 1][e], kx[n][e], kk);
        if (TWO && odd) kq = fmaf(kx[n - 1][e], qx[n][e], kq);
      }
      t.v[r][lane] = vx[n];
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        if (NEEDQ) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (TWO && odd) kk += __shfl_xor_sync(0xffffffffu, kk, o);
        if (TWO && odd && NEEDQ) kq += __shfl_xor_sync(0xffffffffu, kq, o);
      }
      if (lane == 0) {
        t.a[r] = expf(gx[n]);
        t.b[r] = bx[n];
        t.qk[r] = dot;
        if (odd) t.kk[r] = kk;
        if (odd) t.kq[r] = kq;
      }
    }
  };

  // thread (lk, c): rows 4 lk + 32 i + 0..3 of columns v0 + 4 NC warp + NC c ...
  const int lk = lane & 7, cl = (warp % CW) * 4 * NC + NC * (lane >> 3), col = v0 + cl;
  bool in[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) in[n] = col + n < a.V;
  Cols S[KR];
  const int64_t mat = (d * a.H + h) * a.K * a.V;
  auto put_state = [&](float *dst) {
#pragma unroll
    for (int j = 0; j < KR; ++j) {
      const int row = 4 * lk + 32 * (j >> 2) + (j & 3);
      if (row < a.K)
#pragma unroll
        for (int n = 0; n < NC; ++n)
          if (in[n]) dst[(int64_t)row * a.V + col + n] = S[j].v[n];
    }
  };
  if (!stages) {
#pragma unroll
    for (int j = 0; j < KR; ++j) {
      const int row = 4 * lk + 32 * (j >> 2) + (j & 3);
#pragma unroll
      for (int n = 0; n < NC; ++n)
        S[j].v[n] = a.seed && row < a.K && in[n] ? a.seed[mat + (int64_t)row * a.V + col + n] : 0.f;
    }
  } else if (ntile > 0) {
    stage(0);
  }
  __syncthreads();
  for (int i = 0; i < ntile; ++i) {
    if (stages) {
      if (i + 1 < ntile) stage(i + 1);
    } else {
      const Tile<KR> &t = tiles[i & 1];
      const int64_t t0 = (int64_t)tile_of(i) * TT;
      const int len = (int)min((int64_t)TT, n - t0);
      // the states before a chunk; the gradients after one (its last tile, or the document's)
      if (MODE == STATES && t0 % C == 0) put_state(a.states + ((slot0 + t0 / C) * a.H + h) * a.K * a.V);
      if (MODE == BACK && ((t0 + TT) % C == 0 || i == 0))
        put_state(a.states + ((slot0 + t0 / C) * a.H + h) * a.K * a.V);
      const int64_t at0 = ((s0 + t0) * a.H + h) * a.V + col, step = (int64_t)a.H * a.V;
      auto token = [&](int r) {
        Cols xk = {}, xq = {}, xk2 = {};
        float4 kv[KR / 4], qv[KR / 4];
#pragma unroll
        for (int j = 0; j < KR / 4; ++j) {
          kv[j] = *reinterpret_cast<const float4 *>(&t.k[r][4 * lk + 32 * j]);
          if (NEEDQ) qv[j] = *reinterpret_cast<const float4 *>(&t.q[r][4 * lk + 32 * j]);
        }
        const float *kp = reinterpret_cast<const float *>(kv), *qp = reinterpret_cast<const float *>(qv);
#pragma unroll
        for (int j = 0; j < KR; j += 2) {
          xk = fma_cols(kp[j], S[j], xk);
          xk2 = fma_cols(kp[j + 1], S[j + 1], xk2);
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) xk.v[n] += xk2.v[n];
        if (MODE == FWD) {
#pragma unroll
          for (int j = 0; j < KR; ++j) xq = fma_cols(qp[j], S[j], xq);
        }
#pragma unroll
        for (int o = 1; o < LK; o <<= 1)
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            xk.v[n] += __shfl_xor_sync(0xffffffffu, xk.v[n], o);
            if (MODE == FWD) xq.v[n] += __shfl_xor_sync(0xffffffffu, xq.v[n], o);
          }
        Cols v;
#pragma unroll
        for (int n = 0; n < NC; ++n) v.v[n] = t.v[r][cl + n];
        const float dec = t.a[r], b = t.b[r];
        const int64_t at = at0 + r * step;
        if (MODE != BACK) {
          const Cols e = fma_cols(-dec, xk, v), u = mul_cols(b, e);
#pragma unroll
          for (int j = 0; j < KR; ++j) S[j] = fma_cols(kp[j], u, mul_cols(dec, S[j]));
          if (MODE == FWD) {
            if (a.out && lk == 0) {
              const Cols y = fma_cols(t.qk[r], u, mul_cols(dec, xq));
#pragma unroll
              for (int n = 0; n < NC; ++n)
                if (in[n]) a.out[at + n] = from_f32<T>(a.scale * y.v[n]);
            }
          } else if (lk == 0) {
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (in[n]) a.rows[at + n] = e.v[n];
          }
        } else {
          const Cols du = fma_cols(a.scale * t.qk[r], v, xk), dy = mul_cols(b, du), w = mul_cols(a.scale, v);
#pragma unroll
          for (int j = 0; j < KR; ++j) S[j] = mul_cols(dec, fma_cols(-kp[j], dy, fma_cols(qp[j], w, S[j])));
          if (lk == 0) {
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (in[n]) a.rows[at + n] = du.v[n], a.out[at + n] = from_f32<T>(dy.v[n]);
          }
        }
      };
      // tokens r and r + 1 (1 and 2): both read the state before, or the gradient behind, the two of them
      auto two_tokens = [&](int r) {
        float4 kv[2][KR / 4], qv[2][KR / 4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < KR / 4; ++j) {
            kv[m][j] = *reinterpret_cast<const float4 *>(&t.k[r + m][4 * lk + 32 * j]);
            if (NEEDQ) qv[m][j] = *reinterpret_cast<const float4 *>(&t.q[r + m][4 * lk + 32 * j]);
          }
        const float *k1 = reinterpret_cast<const float *>(kv[0]), *k2 = reinterpret_cast<const float *>(kv[1]);
        const float *q1 = reinterpret_cast<const float *>(qv[0]), *q2 = reinterpret_cast<const float *>(qv[1]);
        Cols x1 = {}, x2 = {}, y1 = {}, y2 = {}, v1, v2;
#pragma unroll
        for (int n = 0; n < NC; ++n) v1.v[n] = t.v[r][cl + n], v2.v[n] = t.v[r + 1][cl + n];
        const float d1 = t.a[r], d2 = t.a[r + 1], b1 = t.b[r], b2 = t.b[r + 1], kk = t.kk[r + 1], kq = t.kq[r + 1];
        const float over = d1 * d2;
#pragma unroll
        for (int j = 0; j < KR; ++j) {
          x1 = fma_cols(k1[j], S[j], x1);
          x2 = fma_cols(k2[j], S[j], x2);
          if (MODE == FWD) {
            y1 = fma_cols(q1[j], S[j], y1);
            y2 = fma_cols(q2[j], S[j], y2);
          }
        }
#pragma unroll
        for (int o = 1; o < LK; o <<= 1)
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            x1.v[n] += __shfl_xor_sync(0xffffffffu, x1.v[n], o);
            x2.v[n] += __shfl_xor_sync(0xffffffffu, x2.v[n], o);
            if (MODE == FWD) {
              y1.v[n] += __shfl_xor_sync(0xffffffffu, y1.v[n], o);
              y2.v[n] += __shfl_xor_sync(0xffffffffu, y2.v[n], o);
            }
          }
        const int64_t at = at0 + r * step;
        if (MODE != BACK) {
          const Cols e1 = fma_cols(-d1, x1, v1), u1 = mul_cols(b1, e1);
          const Cols e2 = fma_cols(-d2, fma_cols(kk, u1, mul_cols(d1, x2)), v2), u2 = mul_cols(b2, e2);
          const Cols w1 = mul_cols(d2, u1);
#pragma unroll
          for (int j = 0; j < KR; ++j) S[j] = fma_cols(k2[j], u2, fma_cols(k1[j], w1, mul_cols(over, S[j])));
          if (MODE == FWD) {
            if (a.out && lk == 0) {
              const Cols o1 = fma_cols(t.qk[r], u1, mul_cols(d1, y1));
              const Cols o2 = fma_cols(t.qk[r + 1], u2, mul_cols(d2, fma_cols(kq, u1, mul_cols(d1, y2))));
#pragma unroll
              for (int n = 0; n < NC; ++n)
                if (in[n]) {
                  a.out[at + n] = from_f32<T>(a.scale * o1.v[n]);
                  a.out[at + step + n] = from_f32<T>(a.scale * o2.v[n]);
                }
            }
          } else if (lk == 0) {
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (in[n]) a.rows[at + n] = e1.v[n], a.rows[at + step + n] = e2.v[n];
          }
        } else {
          const Cols w1 = mul_cols(a.scale, v1), w2 = mul_cols(a.scale, v2);
          const Cols du2 = fma_cols(t.qk[r + 1], w2, x2), dy2 = mul_cols(b2, du2);
          const Cols du1 = fma_cols(t.qk[r], w1, mul_cols(d2, fma_cols(-kk, dy2, fma_cols(kq, w2, x1))));
          const Cols dy1 = mul_cols(b1, du1);
          const Cols aq1 = mul_cols(d1, w1), ak1 = mul_cols(-d1, dy1), aq2 = mul_cols(over, w2), ak2 = mul_cols(-over, dy2);
#pragma unroll
          for (int j = 0; j < KR; ++j)
            S[j] = fma_cols(k1[j], ak1, fma_cols(q1[j], aq1, fma_cols(k2[j], ak2, fma_cols(q2[j], aq2, mul_cols(over, S[j])))));
          if (lk == 0) {
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (in[n]) {
                a.rows[at + n] = du1.v[n], a.out[at + n] = from_f32<T>(dy1.v[n]);
                a.rows[at + step + n] = du2.v[n], a.out[at + step + n] = from_f32<T>(dy2.v[n]);
              }
          }
        }
      };
      // The last token of an odd number by itself; past 128 key rows registers do not hold two tokens, and
      // forwards the build for bf16 is slower with two (2048 tokens of 16 heads of 128 x 128: 659 instead of 523 us;
      // fp32: 436 instead of 512).
      const int even = TWO ? len & ~1 : 0;
      if (MODE == BACK) {
        for (int r = len - 1; r >= even; --r) token(r);
        for (int r = even - 2; r >= 0; r -= 2) two_tokens(r);
      } else {
        for (int r = 0; r < even; r += 2) two_tokens(r);
        for (int r = even; r < len; ++r) token(r);
      }
    }
    __syncthreads();
  }
  if (!stages && a.last) put_state(a.last + mat);
}

template <typename T, int KR>
__global__ void __launch_bounds__(THREADS) scan_kernel(const ScanArgs<T> a) {
  scan<T, KR, FWD>(a, blockIdx.x);
}
// The backward's two passes do not need one another: the first half of the
// blocks goes backwards in time, the second forwards.  Two blocks to an SM (EACH) cost 16 rows
// some spills: with 128 key channels 128 blocks of 2048 tokens take 504 us (one) or 610,
// 512 of 1024 tokens 838 or 715.
template <typename T, int KR, int EACH>
__global__ void __launch_bounds__(THREADS, EACH) scans_kernel(const ScanArgs<T> back, const ScanArgs<T> states, uint32_t half) {
  if (blockIdx.x < half)
    scan<T, KR, BACK>(back, blockIdx.x);
  else
    scan<T, KR, STATES>(states, blockIdx.x - half);
}

template <typename T>
ScanArgs<T> scan_args(const Call &c, const void *v, int64_t vs, const float *seed, float *last, void *out, float *states,
                      float *rows) {
  ScanArgs<T> a;
  a.q = (const T *)c.p.q;
  a.k = (const T *)c.p.k;
  a.v = (const T *)v;
  a.g = c.p.g;
  a.beta = c.beta;
  a.seed = seed;
  a.last = last;
  a.out = (T *)out;
  a.states = states;
  a.rows = rows;
  a.docs = c.docs;
  a.qs = c.p.qs;
  a.ks = c.p.ks;
  a.vs = vs;
  a.H = (int)c.p.H;
  a.share = (int)(c.p.H / c.p.Hqk);
  a.K = (int)c.p.K;
  a.V = (int)c.p.V;
  a.slices = (a.V + COLS - 1) / COLS;
  a.scale = c.p.scale;
  return a;
}

// go(kernel, bytes of shared memory) with the kernel for K's rows; few: no more blocks than SMs
template <template <int> class Kernel, typename F>
cudaError_t by_rows(int64_t K, bool few, F go) {
  if (K <= 32) return go(Kernel<4>::get(few), 2 * sizeof(Tile<4>));
  if (K <= 64) return go(Kernel<8>::get(few), 2 * sizeof(Tile<8>));
  if constexpr (Kernel<12>::ROWS == 12)
    if (K <= 96) return go(Kernel<12>::get(few), 2 * sizeof(Tile<12>));
  if (K <= 128) return go(Kernel<16>::get(few), 2 * sizeof(Tile<16>));
  return go(Kernel<32>::get(few), 2 * sizeof(Tile<32>));
}
// 65 to 96 channels: 12 rows of a thread but for fp32 forwards, which take 16 (12 rows / 16, us, forward: 3 x 333 tokens of
// 6 heads of 72 x 41 bf16 82 / 88, fp32 99 / 74; 2048 of 16 of 96 x 128 477 / 522, 579 / 436; 16 x 256 of 16 of 72 x 128
// 275 / 340, 371 / 308; 64 x 128 of 8 of 96 x 64 142 / 174, 191 / 158; 48 of 16 of 96 x 128 17 / 17, 19 / 15.  Backward, whole
// call, fp32: 123 / 135, 633 / 701, 887 / 1018, 538 / 602, 82 / 84; bf16 9 to 15% the same way).
template <typename T> struct Scan {
  template <int KR> struct One {
    enum { ROWS = KR == 12 && sizeof(T) == 4 ? 0 : KR };
    static auto get(bool) { return scan_kernel<T, KR>; }
  };
  template <int KR> struct Two {
    enum { ROWS = KR };
    static auto get(bool few) {
      if constexpr (KR == 16) return few ? scans_kernel<T, KR, 1> : scans_kernel<T, KR, 2>;
      else return scans_kernel<T, KR, KR < 16 ? 2 : 1>;
    }
  };
};

template <typename T>
cudaError_t scan_fwd(const Call &c, void *o, float *ht) {
  const ScanArgs<T> a = scan_args<T>(c, c.p.v, c.p.vs, c.p.h0, ht, o, nullptr, nullptr);
  const int64_t ctas = c.docs.n * c.p.H * a.slices;
  if (ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  const cudaError_t e = by_rows<Scan<T>::template One>(c.p.K, ctas <= tc::sm_count(), [&](auto kernel, size_t smem) -> cudaError_t {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)ctas, THREADS, smem, c.st>>>(a);
    return cudaGetLastError();
  });
  mark_launch("delta_scan", c.st);
  return e;
}
template <typename T>
cudaError_t scans_bwd(const Call &c, const void *dO, const float *dht, void *dv, float *dh0, const Saved &saved) {
  const ScanArgs<T> st = scan_args<T>(c, c.p.v, c.p.vs, c.p.h0, nullptr, nullptr, saved.s0, saved.e);
  const ScanArgs<T> bk = scan_args<T>(c, dO, c.p.H * c.p.V, dht, dh0, dv, saved.ds1, saved.dr);
  const int64_t ctas = c.docs.n * c.p.H * st.slices;
  if (2 * ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  const cudaError_t e = by_rows<Scan<T>::template Two>(c.p.K, 2 * ctas <= tc::sm_count(), [&](auto kernel, size_t smem) -> cudaError_t {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(2 * ctas), THREADS, smem, c.st>>>(bk, st, (uint32_t)ctas);
    return cudaGetLastError();
  });
  mark_launch("delta_scans", c.st);
  return e;
}

// ---- gradients of q, k, g, beta ---------------------------------------------
//
// One block per (chunk, head), 256 threads; thread (tx, ty) owns the 4 x 4
// entries (ty + 16 i, tx + 16 j) of a 64 x 64 result (rows and columns 16
// apart, so that its shared-memory reads, four along the contraction at once, are free of
// bank conflicts at a row pitch of PITCH).  Bound by those reads, and where
// the chunks are few by the staging: all of a slice's loads are in flight at once.
// 128 registers for two blocks on an SM: 1024 chunk heads of 128 x 128 fp32 551 -> 454 us,
// 108 of 72 x 41 (a block on an SM) 54 -> 55 us.
constexpr int W = 32;      // columns of a staged slice of the contraction
constexpr int PITCH = 36;  // its row pitch
constexpr int CP = C + 4;  // pitch of the C x C matrices
constexpr int PER = C * W / 256;  // values of a slice that a thread stages

template <typename T>
struct GradArgs {
  const T *q, *k, *dO;
  const float *g, *beta;
  Saved s;
  Docs docs;
  int64_t qs, ks;
  int H, share, K, V;
  float scale;
  void *dq, *dk;
  int per_head;  // dq, dk fp32 (to be summed), else T
  float *dg, *dbeta;
};

struct alignas(16) GradSmem {
  union {
    float x[5][C][PITCH];  // staged slices
    float kq[2][C][C + 1];  // 64 channels of k and q
    float w[C][CP];         // W_rs
  };
  float dP[C][CP], dPT[C][CP], dA[C][CP];  // dPd and its transpose, dA + dA^T
  double G[C], half_total;
  float into[C], outof[C], beta[C];
  float gq[C], gk[C], gadd[C], db[C], pair[C];
  float red[32];
};

// acc[i][j] += sum over the slice of a[ty + 16 i][.] b[tx + 16 j][.]
__device__ __forceinline__ void slice_product(float (&acc)[4][4], const float (*a)[PITCH], const float (*b)[PITCH],
                                              int tx, int ty) {
#pragma unroll 4
  for (int w = 0; w < W; w += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = *reinterpret_cast<const float4 *>(&a[ty + 16 * i][w]);
      y[i] = *reinterpret_cast<const float4 *>(&b[tx + 16 * i][w]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, acc[i][j]))));
  }
}
__device__ __forceinline__ void zero(float (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
}

template <typename T>
__global__ void __launch_bounds__(256, 2) grads_kernel(const GradArgs<T> a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  GradSmem &s = *reinterpret_cast<GradSmem *>(smem_raw);
  const int h = (int)(blockIdx.x % a.H);
  const int64_t slot = blockIdx.x / a.H;
  int64_t tok0;
  int L;
  if (!chunk_in_slot(a.docs, slot, tok0, L)) return;
  const int hq = h / a.share;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const T *q = a.q + (int64_t)hq * a.K, *k = a.k + (int64_t)hq * a.K;

  double G = 0.0;
  if (tid < C) {
    if (tid < L) G = (double)log_decay(a.g[(tok0 + tid) * a.H + h]);
    s.beta[tid] = tid < L ? a.beta[(tok0 + tid) * a.H + h] : 0.f;
    s.gq[tid] = s.gk[tid] = s.gadd[tid] = 0.f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, G, o);
      if ((tid & 31) >= o) G += y;
    }
    if (tid == 31) s.half_total = G;
  }
  __syncthreads();
  if (tid < C) s.G[tid] = tid < 32 ? G : G + s.half_total;
  __syncthreads();
  if (tid < C) {
    s.into[tid] = expf((float)s.G[tid]);
    s.outof[tid] = expf((float)(s.G[L - 1] - s.G[tid]));
  }
  const float over = expf((float)s.G[L - 1]);

  // token rows [tok0, tok0 + L) x columns [c0, c0 + W) of a per-head fp32 or T tensor
  auto load_rows = [&](float (&v)[PER], auto *src, int64_t stride, int c0, int width) {
#pragma unroll
    for (int n = 0; n < PER; ++n) {
      const int r = (tid + 256 * n) / W, c = tid % W;
      v[n] = r < L && c0 + c < width ? to_f32(src[(tok0 + r) * stride + c0 + c]) : 0.f;
    }
  };
  auto put_rows = [&](float (*dst)[PITCH], const float (&v)[PER]) {
#pragma unroll
    for (int n = 0; n < PER; ++n) dst[(tid + 256 * n) / W][tid % W] = v[n];
  };
  const int64_t hv = (int64_t)a.H * a.V;
  const float *e = a.s.e + (int64_t)h * a.V, *dr = a.s.dr + (int64_t)h * a.V;
  const T *dO = a.dO + (int64_t)h * a.V;

  // C x C products over the value columns, then over the key channels
  float b1[4][4], b2[4][4], db = 0.f;
  zero(b1);
  zero(b2);
  for (int c0 = 0; c0 < a.V; c0 += W) {
    float v0[PER], v1[PER], v2[PER];
    load_rows(v0, dO, hv, c0, a.V);
    load_rows(v1, dr, hv, c0, a.V);
    load_rows(v2, e, hv, c0, a.V);
    __syncthreads();
    put_rows(s.x[0], v0);
    put_rows(s.x[1], v1);
    put_rows(s.x[2], v2);
    __syncthreads();
    slice_product(b1, s.x[0], s.x[2], tx, ty);
    slice_product(b2, s.x[1], s.x[2], tx, ty);
#pragma unroll
    for (int n = 0; n < W / 4; ++n)  // four threads to a row
      db = fmaf(s.x[1][tid >> 2][(tid & 3) + 4 * n], s.x[2][tid >> 2][(tid & 3) + 4 * n], db);
  }
  db += __shfl_xor_sync(0xffffffffu, db, 1);
  db += __shfl_xor_sync(0xffffffffu, db, 2);
  if ((tid & 3) == 0) s.db[tid >> 2] = db;
  float qk[4][4], kk[4][4];
  zero(qk);
  zero(kk);
  for (int c0 = 0; c0 < a.K; c0 += W) {
    float v0[PER], v1[PER];
    load_rows(v0, q, a.qs, c0, a.K);
    load_rows(v1, k, a.ks, c0, a.K);
    __syncthreads();
    put_rows(s.x[0], v0);
    put_rows(s.x[1], v1);
    __syncthreads();
    slice_product(qk, s.x[0], s.x[1], tx, ty);
    slice_product(kk, s.x[1], s.x[1], tx, ty);
  }
  // dPd and dA; W_rs of the pairs r > s, kept in the staging area
  float (*Wm)[CP] = s.w;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int t = ty + 16 * i, r = tx + 16 * jj;
      float dp = 0.f, da = 0.f;
      if (r <= t && t < L) {
        const float D = expf((float)(s.G[t] - s.G[r])) * s.beta[r];  // U = beta E
        dp = a.scale * D * b1[i][jj];
        if (r < t) da = -D * s.beta[t] * b2[i][jj];
      }
      s.dP[t][r] = s.dPT[r][t] = dp;
      if (r <= t) s.dA[t][r] = s.dA[r][t] = da;
      Wm[t][r] = r < t ? fmaf(dp, qk[i][jj], da * kk[i][jj]) : 0.f;
    }
  __syncthreads();
  // pair[t] = sum over r >= t > s of W_rs: first every column's sums from below, then along each row
  if (tid < C) {
    float x = 0.f;
    for (int r = C - 8; r >= 0; r -= 8) {
      float y[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) y[n] = Wm[r + n][tid];
#pragma unroll
      for (int n = 7; n >= 0; --n) {
        x += y[n];
        Wm[r + n][tid] = x;
      }
    }
  }
  __syncthreads();
  {  // four threads to a row
    float x = 0.f;
#pragma unroll
    for (int n = 0; n < C / 4; ++n) {
      const int c = (tid & 3) + 4 * n;
      x += c < tid >> 2 ? Wm[tid >> 2][c] : 0.f;
    }
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if ((tid & 3) == 0) s.pair[tid >> 2] = x;
  }

  // dq, dk for 64 channels at a time; <S0, dS1> on the way
  const float *S0 = a.s.s0 + (slot * a.H + h) * (int64_t)a.K * a.V, *S1 = a.s.ds1 + (slot * a.H + h) * (int64_t)a.K * a.V;
  float sd = 0.f;
  for (int k0 = 0; k0 < a.K; k0 += 64) {
    float m1[4][4], m2[4][4], m3[4][4];
    zero(m1);
    zero(m2);
    zero(m3);
    for (int c0 = 0; c0 < a.V; c0 += W) {
      float v0[PER], v1[PER], v2[PER], v3[PER], v4[PER];
      load_rows(v0, dO, hv, c0, a.V);
      load_rows(v1, dr, hv, c0, a.V);
      load_rows(v2, e, hv, c0, a.V);
#pragma unroll
      for (int n = 0; n < PER; ++n) {
        const int r = (tid + 256 * n) / W, c = tid % W;
        const bool in = k0 + r < a.K && c0 + c < a.V;
        const int64_t at = (int64_t)(k0 + r) * a.V + c0 + c;
        v3[n] = in ? S0[at] : 0.f;
        v4[n] = in ? S1[at] : 0.f;
      }
      __syncthreads();
      put_rows(s.x[0], v0);
      put_rows(s.x[1], v1);
      put_rows(s.x[2], v2);
      put_rows(s.x[3], v3);
      put_rows(s.x[4], v4);
#pragma unroll
      for (int n = 0; n < PER; ++n) sd = fmaf(v3[n], v4[n], sd);
      __syncthreads();
      slice_product(m1, s.x[0], s.x[3], tx, ty);
      slice_product(m2, s.x[1], s.x[3], tx, ty);
      slice_product(m3, s.x[2], s.x[4], tx, ty);
    }
    {
      float kv[C / 4], qv[C / 4];
#pragma unroll
      for (int n = 0; n < C / 4; ++n) {
        const int r = tid / 64 + 4 * n, c = tid % 64;
        const bool in = r < L && k0 + c < a.K;
        kv[n] = in ? to_f32(k[(tok0 + r) * a.ks + k0 + c]) : 0.f;
        qv[n] = in ? to_f32(q[(tok0 + r) * a.qs + k0 + c]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < C / 4; ++n) {
        s.kq[0][tid / 64 + 4 * n][tid % 64] = kv[n];
        s.kq[1][tid / 64 + 4 * n][tid % 64] = qv[n];
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = ty + 16 * i;
      float rq = 0.f, rk = 0.f, ra = 0.f;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int c = tx + 16 * jj;
        m1[i][jj] *= a.scale * s.into[t];
        m2[i][jj] *= -s.into[t] * s.beta[t];
        m3[i][jj] *= s.outof[t] * s.beta[t];
        rq = fmaf(s.kq[1][t][c], m1[i][jj], rq);
        rk = fmaf(s.kq[0][t][c], m2[i][jj], rk);
        ra = fmaf(s.kq[0][t][c], m3[i][jj], ra);
        m2[i][jj] += m3[i][jj];
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) {
        rq += __shfl_xor_sync(0xffffffffu, rq, o);
        rk += __shfl_xor_sync(0xffffffffu, rk, o);
        ra += __shfl_xor_sync(0xffffffffu, ra, o);
      }
      if (tx == 0) {
        s.gq[t] += rq;
        s.gk[t] += rk;
        s.gadd[t] += ra;
      }
    }
    for (int r = 0; r < L; r += 4) {  // what is past L is 0
      float4 pr[4], pc[4], ar[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[i] = *reinterpret_cast<const float4 *>(&s.dP[ty + 16 * i][r]);
        pc[i] = *reinterpret_cast<const float4 *>(&s.dPT[ty + 16 * i][r]);
        ar[i] = *reinterpret_cast<const float4 *>(&s.dA[ty + 16 * i][r]);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float kx = s.kq[0][r + n][tx + 16 * jj], qx = s.kq[1][r + n][tx + 16 * jj];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = (&pr[i].x)[n], pt = (&pc[i].x)[n], at = (&ar[i].x)[n];
            m1[i][jj] = fmaf(p, kx, m1[i][jj]);
            m2[i][jj] = fmaf(pt, qx, fmaf(at, kx, m2[i][jj]));
          }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int t = ty + 16 * i, c = k0 + tx + 16 * jj;
        if (t < L && c < a.K) {
          const int64_t at = ((tok0 + t) * a.H + h) * a.K + c;
          if (a.per_head) {
            ((float *)a.dq)[at] = m1[i][jj];
            ((float *)a.dk)[at] = m2[i][jj];
          } else {
            ((T *)a.dq)[at] = from_f32<T>(m1[i][jj]);
            ((T *)a.dk)[at] = from_f32<T>(m2[i][jj]);
          }
        }
      }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
  if ((tid & 31) == 0) s.red[tid >> 5] = sd;
  __syncthreads();
  if (tid < L) {
    float x = s.pair[tid], sum = 0.f;
    for (int r = tid; r < L; ++r) x += s.gq[r] + s.gk[r];
    for (int r = 0; r < tid; ++r) x += s.gadd[r];
    for (int w = 0; w < 8; ++w) sum += s.red[w];
    a.dg[(tok0 + tid) * a.H + h] = fmaf(over, sum, x);
    a.dbeta[(tok0 + tid) * a.H + h] = s.db[tid];
  }
}

template <typename T>
cudaError_t grads_as(const Call &c, const void *dO, const Saved &saved, void *dq, void *dk, bool per_head, float *dg,
                     float *dbeta) {
  GradArgs<T> a;
  a.q = (const T *)c.p.q;
  a.k = (const T *)c.p.k;
  a.dO = (const T *)dO;
  a.g = c.p.g;
  a.beta = c.beta;
  a.s = saved;
  a.docs = c.docs;
  a.qs = c.p.qs;
  a.ks = c.p.ks;
  a.H = (int)c.p.H;
  a.share = (int)(c.p.H / c.p.Hqk);
  a.K = (int)c.p.K;
  a.V = (int)c.p.V;
  a.scale = c.p.scale;
  a.dq = dq;
  a.dk = dk;
  a.per_head = per_head;
  a.dg = dg;
  a.dbeta = dbeta;
  const int64_t ctas = c.slots * c.p.H;
  if (ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(grads_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(GradSmem));
  if (e != cudaSuccess) return e;
  grads_kernel<T><<<(unsigned)ctas, 256, sizeof(GradSmem), c.st>>>(a);
  mark_launch("delta_grads", c.st);
  return cudaGetLastError();
}

template <typename T>
__global__ void __launch_bounds__(256) reduce_heads_kernel(const float *x, T *out, int64_t n, int64_t K, int64_t pitch,
                                                           int share) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const float *src = x + (i / K) * share * pitch + i % K;
    float s = 0.f;
    for (int e = 0; e < share; ++e) s += src[e * pitch];
    out[i] = from_f32<T>(s);
  }
}

struct RowsArgs {
  Rows t[4];
  int64_t BT;
};
// Eight channels of a row to a thread; a tensor to blockIdx.y.
template <bool BACK>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ RowsArgs a) {
  const Rows r = a.t[blockIdx.y];
  const int per = r.Dp / 8;
  const int64_t n = a.BT * r.heads * per;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, t = row / r.heads;
    const int c = (int)(i % per) * 8;
    uint16_t x[8];
    if (BACK) {
      *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>((const uint16_t *)r.src + row * r.Dp + c);
      uint16_t *dst = (uint16_t *)r.dst + row * r.D + c;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < r.D) dst[e] = x[e];
    } else {
      const uint16_t *src = (const uint16_t *)r.src + t * r.stride + (row - t * r.heads) * r.D + c;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = c + e < r.D ? src[e] : (uint16_t)0;
      *reinterpret_cast<uint4 *>((uint16_t *)r.dst + row * r.Dp + c) = *reinterpret_cast<const uint4 *>(x);
    }
  }
}
template <bool BACK>
cudaError_t copy_rows(const Call &c, std::initializer_list<Rows> tensors, const char *label) {
  RowsArgs a;
  int64_t most = 0;
  int n = 0;
  a.BT = c.p.BT;
  for (const Rows &r : tensors) {
    a.t[n++] = r;
    most = std::max(most, a.BT * r.heads * (r.Dp / 8));
  }
  const dim3 grid((unsigned)std::min<int64_t>((most + 255) / 256, 152 * 8), n);
  rows_kernel<BACK><<<grid, 256, 0, c.st>>>(a);
  mark_launch(label, c.st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t simt_fwd(const Call &c, void *o, float *ht) {
  return c.dtype == GLACORE_BF16 ? scan_fwd<__nv_bfloat16>(c, o, ht) : scan_fwd<float>(c, o, ht);
}

cudaError_t simt_scans(const Call &c, const void *dO, const float *dht, void *dv, float *dh0, const Saved &saved) {
  return c.dtype == GLACORE_BF16 ? scans_bwd<__nv_bfloat16>(c, dO, dht, dv, dh0, saved)
                                 : scans_bwd<float>(c, dO, dht, dv, dh0, saved);
}

cudaError_t simt_grads(const Call &c, const void *dO, const Saved &saved, void *dq, void *dk, bool per_head, float *dg,
                       float *dbeta) {
  return c.dtype == GLACORE_BF16 ? grads_as<__nv_bfloat16>(c, dO, saved, dq, dk, per_head, dg, dbeta)
                                 : grads_as<float>(c, dO, saved, dq, dk, per_head, dg, dbeta);
}

cudaError_t pad_rows(const Call &c, std::initializer_list<Rows> tensors) {
  return copy_rows<false>(c, tensors, "delta_pad");
}
cudaError_t unpad_rows(const Call &c, std::initializer_list<Rows> tensors) {
  return copy_rows<true>(c, tensors, "delta_unpad");
}
cudaError_t reduce_heads(const Call &c, const float *x, void *out) {
  const int64_t n = c.p.BT * c.p.Hqk * c.sK;
  const int blocks = (int)std::min<int64_t>((n + 255) / 256, 152 * 16);
  const int share = (int)(c.p.H / c.p.Hqk);
  if (c.dtype == GLACORE_BF16)
    reduce_heads_kernel<<<blocks, 256, 0, c.st>>>(x, (__nv_bfloat16 *)out, n, c.sK, c.p.K, share);
  else
    reduce_heads_kernel<<<blocks, 256, 0, c.st>>>(x, (float *)out, n, c.sK, c.p.K, share);
  mark_launch("delta_reduce_heads", c.st);
  return cudaGetLastError();
}

}  // namespace delta
}  // namespace glacore
