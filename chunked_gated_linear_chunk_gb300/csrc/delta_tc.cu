// delta_tc.cu -- the gated delta rule on the tensor cores (formulas in
// delta.cuh): bf16, K and V multiples of 8 up to 128 (read as 128, the missing
// channels zero-filled by TMA), chunks of C = 64 tokens.
//
// Precision.  q, k, v and do are bf16 and enter products as they are.  Every
// matrix that is computed (the state, Z, P, R = b Y, U) enters a product in
// two bf16 parts, x = hi + lo to 2^-17 of x, and a product of two such matrices
// as hi hi + hi lo + lo hi; sums and the state itself are fp32.  With one part
// the outputs are off by 3e-3, twice what rounding them to bf16 costs,
// with two by 5e-6.  Where Z's rows are long (sum of |Z_ts| b_s above WIDE in a
// quarter of a row: keys that nearly coincide, written with b near 2), Y + Z (b Y)
// cancels and what Z and b Y are off by counts that much more: in such a chunk
// that product takes both in three parts (exact to 2^-25).  Chunks of unit keys that
// differ and b up to 1 stay below 3.
//
// delta_prep_kernel makes of every chunk by itself what the recurrence over
// chunks needs: Z and P (two 64 x 64 tiles each, laid out as the matrix
// operands that they become) and the chunk's decays.  delta_chain_kernel walks
// the chunks of one (document, head) with the state on chip; delta_overlap_kernel
// does both at once where few sequences leave SMs over.
#include <string.h>

#include <algorithm>
#include <atomic>

#include "delta.cuh"
#include "tc_common.cuh"

namespace glacore {
namespace delta {

namespace {

using namespace tc;  // ptx helpers, tensor maps (tc::C is 64 as well)

constexpr int CH = delta::C;
constexpr int D128 = 128;
constexpr uint32_t TILE = CH * CH * 2;          // a 64 x 64 bf16 tile
constexpr uint32_t TILES = 5 * TILE;            // Z hi, Z lo, P hi, P lo; of a wide chunk Z's third part
constexpr int GATES = 256;                      // floats of a chunk's gate slot:
constexpr int G_INTO = 0, G_OUT = 64, G_BETA = 128, G_OVER = 192;  // e^G, e^{G_C - G}, b, e^{G_C}
constexpr int G_WIDE = 193;                     // 1: Z (b Y) is to be taken in three parts
constexpr float WIDE = 4.f;
constexpr int NP = 68;                          // row pitch of the fp32 64 x 64 matrices

// hi and lo parts of two neighbours, packed.  What hi leaves is a product with
// -1 of the packed half itself, added to the fp32 value.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  float ra, rb;
  hi = pack_bf16(a, b);
  asm("{\n .reg .b16 x, y, m;\n mov.b32 {x, y}, %2;\n mov.b16 m, 0xBF80;\n fma.rn.f32.bf16 %0, x, m, %3;\n"
      " fma.rn.f32.bf16 %1, y, m, %4;\n}\n"
      : "=f"(ra), "=f"(rb)
      : "r"(hi), "f"(a), "f"(b));
  lo = pack_bf16(ra, rb);
}
// c + a b for both halves of two packed pairs
__device__ __forceinline__ float fma_pairs(uint32_t a, uint32_t b, float c) {
  asm("{\n .reg .b16 x, y, u, v;\n mov.b32 {x, y}, %1;\n mov.b32 {u, v}, %2;\n fma.rn.f32.bf16 %0, x, u, %0;\n"
      " fma.rn.f32.bf16 %0, y, v, %0;\n}\n"
      : "+f"(c)
      : "r"(a), "r"(b));
  return c;
}
// 2^x to 2 ulp; results below 2^-126 become 0
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// what hi and lo leave of them
__device__ __forceinline__ uint32_t split3(float a, float b, uint32_t hi, uint32_t lo) {
  return pack_bf16((a - __uint_as_float(hi << 16)) - __uint_as_float(lo << 16),
                   (b - __uint_as_float(hi & 0xffff0000u)) - __uint_as_float(lo & 0xffff0000u));
}

// ---------------------------------------------------------------------------
// One block per (chunk, q / k head): Q K^T and K K^T as one product of the
// stacked tiles [q; k] (128 rows) with k, then for each value head of the group
// P and N with the decays, and Z = -(I + N diag(b))^-1 N.  Z is made by
// blocks: those of 16 on the diagonal by forward substitution, a thread per
// column in registers, then twice the block below a pair of them, with
// (I + N b)^-1 = I + Z b,
//     Z21 = W + Z22 (b W),   W = -(N21 + N21 (b Z11)).
// (Substitution over the whole chunk is a sequence four times as long, and most
// of this kernel's time.)  Decays are e^{G_t - G_s} of the difference itself, G (in units
// of log 2) kept in two fp32 parts, so that neither a strong decay nor a long
// chunk costs digits.  Bound by barriers and shared-memory wavefronts: 2048 chunk
// heads 48 us on 152 SMs (four blocks on each), 24% of the memory's rate.
// ---------------------------------------------------------------------------
struct PrepArgs {
  const float *g, *beta;
  Docs docs;
  int H, Hqk, share;
  float scale;
  char *tiles;   // [slot, H] x TILES
  float *gates;  // [slot, H] x GATES
  int *err;
};
struct PrepMaps {
  CUtensorMap q, k;
};
struct PrepSmem {
  float N[CH][NP];  // N, block by block replaced by Z
  float2 G[CH];     // two parts of the decay exponent
  float beta[CH];
};
constexpr int WPITCH = 36;  // of W, in the place of Z's tiles until those are made
constexpr uint32_t PREP_BYTES = 32768 + sizeof(PrepSmem) + 1024;
constexpr int PREP_THREADS = 256;

__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
}
__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

// A flag per chunk and head, for blocks of the same kernel.
constexpr uint32_t READY = 1, READY_WIDE = 3;
__device__ __forceinline__ void st_release(uint32_t *p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_relaxed(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// ROWS rows of COLS columns of the block below a pair of diagonal ones (rows
// and columns r .. r + M - 1 and r + M .. r + 2 M - 1): W, a barrier, then Z21.
// Bound by shared-memory reads: a row's four entries serve all columns, a
// column pair's entry all rows.
template <int M, int ROWS, int COLS, typename B>
__device__ __forceinline__ void below(PrepSmem &s, float *W, int r, int j, int i0, B barrier) {
  auto pair = [](const float *p, float (&v)[COLS]) {
    if (COLS == 2) {
      const float2 x = *reinterpret_cast<const float2 *>(p);
      v[0] = x.x;
      v[COLS - 1] = x.y;
    } else {
      v[0] = *p;
    }
  };
  float w[ROWS][COLS];
  auto product = [&](const float *left, const float *right, int pitch, const float *beta, float sign) {
#pragma unroll
    for (int c = 0; c < M; c += 4) {
      const float4 b4 = *reinterpret_cast<const float4 *>(beta + c);
      const float b[4] = {b4.x, b4.y, b4.z, b4.w};
      float z[4][COLS];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        pair(right + (c + x) * pitch, z[x]);
#pragma unroll
        for (int y = 0; y < COLS; ++y) z[x][y] *= sign * b[x];
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float4 n = *reinterpret_cast<const float4 *>(left + i * NP + c);
#pragma unroll
        for (int y = 0; y < COLS; ++y)
          w[i][y] = fmaf(n.x, z[0][y], fmaf(n.y, z[1][y], fmaf(n.z, z[2][y], fmaf(n.w, z[3][y], w[i][y]))));
      }
    }
  };
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    pair(&s.N[r + M + i0 + i][r + j], w[i]);
#pragma unroll
    for (int y = 0; y < COLS; ++y) w[i][y] = -w[i][y];
  }
  product(&s.N[r + M + i0][r], &s.N[r][r + j], NP, &s.beta[r], -1.f);
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int y = 0; y < COLS; ++y) W[(i0 + i) * WPITCH + j + y] = w[i][y];
  barrier();
  product(&s.N[r + M + i0][r + M], W + j, WPITCH, &s.beta[r + M], 1.f);
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int y = 0; y < COLS; ++y) s.N[r + M + i0 + i][r + j + y] = w[i][y];
}

// What a team of PREP_THREADS threads works with: its shared memory, barriers
// `bar` .. `bar` + 3 of the block, 64 columns of tensor memory.
struct PrepTeam {
  uint8_t *sm;  // [q; k] tiles, then Z and P; behind them PrepSmem
  uint64_t *full, *done;
  uint32_t *tmem;
  double *warp0_total;
  int tid, bar;
};
__device__ __forceinline__ void prep_load(const PrepMaps &maps, const PrepTeam &w, int hq, int64_t tok) {
  mbar_expect_tx(w.full, 32768);
#pragma unroll
  for (int cb = 0; cb < 2; ++cb) {  // 64 channels: 64 rows of q, then 64 of k
    tma_load_3d(w.sm + cb * 16384, &maps.q, cb * 64, hq, (int)tok, w.full);
    tma_load_3d(w.sm + cb * 16384 + 8192, &maps.k, cb * 64, hq, (int)tok, w.full);
  }
}
// The chunk in `slot`, whose tiles prep_load has asked for; `phase` of the
// barriers.  `flags`: told of each head when its results are in memory.
template <bool FLAGS>
__device__ __forceinline__ bool prep_chunk(const PrepArgs &a, const PrepTeam &w, int64_t slot, int h0, int heads, int64_t tok,
                                           int L, uint32_t phase, uint32_t *flags) {
  uint8_t *sm = w.sm;
  PrepSmem &s = *reinterpret_cast<PrepSmem *>(sm + 32768);
  float *W = reinterpret_cast<float *>(sm);
  const int tid = w.tid, warp = tid >> 5, lane = tid & 31;
  auto team = [&] { named_bar(w.bar, PREP_THREADS); };
  // gates of head e of the group, loaded a head ahead; then their prefix sums
  float g_next = 0.f, b_next = 0.f;
  auto fetch = [&](int e) {
    g_next = b_next = 0.f;
    if (tid < L && tid < CH && e < heads) {
      const int64_t at = (tok + tid) * a.H + h0 + e;
      g_next = a.g[at];
      b_next = a.beta[at];
    }
  };
  auto scan = [&]() {  // begins and ends with a barrier of the team
    double G = (double)log_decay(g_next) * 1.4426950408889634;
    const float b = b_next;
    if (tid < CH) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, G, o);
        if (lane >= o) G += y;
      }
      if (tid == 31) *w.warp0_total = G;
    }
    team();
    if (tid < CH) {
      if (warp == 1) G += *w.warp0_total;
      const float gh = (float)G;
      s.G[tid] = make_float2(gh, (float)(G - (double)gh));
      s.beta[tid] = b;
    }
    team();
  };
  fetch(0);
  tc_fence_before();
  scan();
  tc_fence_after();
  const uint32_t tb = *w.tmem;
  fetch(1);
  bool ok = true;
  if (tid == 0) {
    ok = mbar_wait(w.full, phase, WAIT_CYCLES);
    const uint32_t base = smem_u32(sm);
    if (ok) {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_bf16(tb, kdesc(base, ks, 128), kdesc(base + 8192, ks, 128), idesc_bf16(128, 64, false, false), ks);
    }
    mma_commit(w.done);
  }
  __syncwarp();
  ok = mbar_wait(w.done, phase, WAIT_CYCLES) && ok;
  ok = !named_bar_any(w.bar, PREP_THREADS, !ok);
  uint32_t kind = 0;  // thread 0: of the last head
  auto publish = [&](int64_t sh) {
    bulk_wait_all();
    fence_async_all();
    st_release(flags + sh, kind);
  };
  if (ok) {
    tc_fence_after();
    // thread (row of the stack, half of the columns): rows < 64 of Q K^T, the others of K K^T
    const int row = (warp & 3) * 32 + lane, t = row & 63, half = warp >> 2;
    const bool isP = (warp & 3) < 2;
    const uint32_t at = tb + ((uint32_t)((warp & 3) * 32) << 16);
    for (int e = 0; e < heads; ++e) {
      const int64_t sh = slot * a.H + h0 + e;
      if (e) {
        if (tid == 0) {  // the tiles of the last head have left shared memory
          if (FLAGS)
            publish(sh - 1);
          else
            bulk_wait_read_all();
        }
        scan();
        fetch(e + 1);
      }
      const float2 gt = s.G[t];
      if (isP && half == 0) {
        const float2 last = s.G[63];
        float *gs = a.gates + sh * GATES;
        gs[G_INTO + t] = pow2(gt.x + gt.y);
        gs[G_OUT + t] = pow2((last.x - gt.x) + (last.y - gt.y));  // tokens past the end add no decay
        gs[G_BETA + t] = s.beta[t];
        if (t == 0) gs[G_OVER] = pow2(last.x + last.y);
      }
      // row t, columns s <= t (P) or s < t (N): scale D (.) QK^T, D (.) KK^T
      const int last = t < L ? (isP ? t : t - 1) : -1;
      const float f = isP ? a.scale : 1.f;
#pragma unroll
      for (int n = 0; n < 32; n += 8) {
        const int c0 = 32 * half + n;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (c0 <= (t | 31)) {  // for the warp: one of its rows reaches these columns
          uint32_t m[8];
          tmem_ld8(at + c0, m);
          tmem_ld_wait8(m);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 gc = *reinterpret_cast<const float4 *>(&s.G[c0 + i]);
            x[i] = c0 + i <= last ? f * pow2((gt.x - gc.x) + (gt.y - gc.y)) * __uint_as_float(m[i]) : 0.f;
            x[i + 1] = c0 + i + 1 <= last ? f * pow2((gt.x - gc.z) + (gt.y - gc.w)) * __uint_as_float(m[i + 1]) : 0.f;
          }
        }
        if (isP) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) split2(x[2 * i], x[2 * i + 1], hi[i], lo[i]);
          const uint32_t o = smem_u32(sm) + 2 * TILE + sw128_off(t, c0, 64);
          st_shared_v4(o, hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(o + TILE, lo[0], lo[1], lo[2], lo[3]);
        } else {
          *reinterpret_cast<float4 *>(&s.N[t][c0]) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4 *>(&s.N[t][c0 + 4]) = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
      if (!isP) {
        named_bar(w.bar + 1, 128);
        if (half == 0) {  // Z of the four diagonal blocks, two by a warp, a column by a thread, in N's place
          const int r = (warp - 2) * 32 + (lane & 16), j = lane & 15;
          float zb[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float z0 = -s.N[r + i][r + j], z1 = 0.f;
#pragma unroll
            for (int c = 0; c < i; c += 4) {
              const float4 n = *reinterpret_cast<const float4 *>(&s.N[r + i][r + c]);
              z0 = fmaf(-n.x, zb[c], z0);
              if (c + 1 < i) z1 = fmaf(-n.y, zb[c + 1], z1);
              if (c + 2 < i) z0 = fmaf(-n.z, zb[c + 2], z0);
              if (c + 3 < i) z1 = fmaf(-n.w, zb[c + 3], z1);
            }
            const float z = z0 + z1;
            zb[i] = z * s.beta[r + i];
            __syncwarp();
            s.N[r + i][r + j] = z;
          }
        }
      }
      team();
      // the block below each pair of them, then the one below both
      if ((warp & 3) < 2)
        below<16, 2, 2>(s, W + half * 16 * WPITCH, half * 32, 2 * (lane & 7), 8 * (warp & 1) + 2 * (lane >> 3),
                        [&] { named_bar(w.bar + 2 + half, 64); });
      team();
      if (warp < 4) below<32, 4, 2>(s, W, 0, 2 * (lane & 15), 8 * warp + 4 * (lane >> 4), [&] { named_bar(w.bar + 1, 128); });
      team();
      const int zr = tid & 63, z0 = (tid >> 6) * 16;
      float sum = 0.f;
      uint32_t third[8];
#pragma unroll
      for (int n = 0; n < 16; n += 8) {
        uint32_t hi[4], lo[4];
        alignas(16) float z[8];
        *reinterpret_cast<float4 *>(z) = *reinterpret_cast<const float4 *>(&s.N[zr][z0 + n]);
        *reinterpret_cast<float4 *>(z + 4) = *reinterpret_cast<const float4 *>(&s.N[zr][z0 + n + 4]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(fabsf(z[i]), fabsf(s.beta[z0 + n + i]), sum);  // a quarter of the row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          split2(z[2 * i], z[2 * i + 1], hi[i], lo[i]);
          third[n / 2 + i] = split3(z[2 * i], z[2 * i + 1], hi[i], lo[i]);
        }
        const uint32_t o = smem_u32(sm) + sw128_off(zr, z0 + n, 64);
        st_shared_v4(o, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(o + TILE, lo[0], lo[1], lo[2], lo[3]);
      }
      const bool wide = named_bar_any(w.bar, PREP_THREADS, !(sum <= WIDE));
      if (wide) {  // the third part takes Z's place
#pragma unroll
        for (int i = 0; i < 2; ++i)
          st_shared_v4(smem_u32(&s.N[0][0]) + sw128_off(zr, z0 + 8 * i, 64), third[4 * i], third[4 * i + 1],
                       third[4 * i + 2], third[4 * i + 3]);
      }
      fence_async_smem();
      team();
      if (tid == 0) {
        a.gates[sh * GATES + G_WIDE] = wide ? 1.f : 0.f;
        kind = wide ? READY_WIDE : READY;
        bulk_store(a.tiles + sh * TILES, sm, 4 * TILE);
        if (wide) bulk_store(a.tiles + sh * TILES + 4 * TILE, &s.N[0][0], TILE);
        bulk_commit();
      }
    }
    if (!FLAGS) follow_allow();
    if (tid == 0) {
      if (FLAGS)
        publish(slot * a.H + h0 + heads - 1);
      else
        bulk_wait_all();
    }
  } else if (tid == 0) {
    mbar_wait(w.full, phase, WAIT_CYCLES);
    set_device_error(a.err, GLACORE_ERR_TIMEOUT);
  }
  tc_fence_before();
  return ok;
}

__global__ void __launch_bounds__(PREP_THREADS, 4) delta_prep_kernel(const __grid_constant__ PrepMaps maps,
                                                                     const PrepArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full, done;
  __shared__ uint32_t tmem_base;
  __shared__ double warp0_total;
  const PrepTeam w{(uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023), &full, &done, &tmem_base, &warp0_total,
                   (int)threadIdx.x, 1};
  const int hq = (int)(blockIdx.x % a.Hqk);
  const int64_t slot = blockIdx.x / a.Hqk;
  int64_t tok;
  int L;
  if (!chunk_in_slot(a.docs, slot, tok, L)) return;
  if (w.tid == 0) {
    mbar_init(&full, 1);
    mbar_init(&done, 1);
    fence_mbar_init();
    prep_load(maps, w, hq, tok);
  }
  if (w.tid >> 5 == 1) {
    tmem_alloc(&tmem_base, 64);
    tmem_relinquish();
  }
  prep_chunk<false>(a, w, slot, hq * a.share, a.share, tok, L, 0, nullptr);
  __syncthreads();
  if (w.tid >> 5 == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 64);
  }
}

// ---------------------------------------------------------------------------
// The recurrence over the chunks of one (document, head).  The state is kept
// transposed, value column v in lane v of tensor memory, so that every
// elementwise step belongs to one thread and no operand that the chain makes
// goes through shared memory:
//     X^T  = S^T k^T                 A: S^T (hi, lo), B: k    -> Y = v - e^G X, R = b Y
//     E^T  = Y^T + R^T Z^T           A: R^T (hi, lo), B: Z    -> U = b E, U' = e^{G_C - G} U
//     S'^T = e^{G_C} S^T + U'^T k    A: U'^T (hi, lo), B: k (as rows of the contraction)
//     O^T  = scale e^G (S^T q^T) + U^T P^T
// Three products and three elementwise steps per chunk are in sequence, and
// the kernel is bound by that sequence: one block per (document, head), about
// half of a chunk's time in the products (a product of N <= 128 columns takes
// the tensor core the time of 128).  So S^T q^T shares X's instructions (B: [k; q], 128
// rows), U^T P^T runs where the sequence leaves the tensor core idle, and the
// output has warps of its own.  3.6 us a chunk, tensor pipe active 31%; 64 x 32
// chunks 119 us.
//   warps 0..15  the chain: lanes of quarter w % 4, group w / 4 holds 32 of the
//                state's key rows and 16 of the chunk's tokens (of its column v)
//   warps 16..19 the output (none in STATES)
//   warps 20, 21 products, copies (a thread each)
// TMEM columns: [0, 128) S^T, per group of 32 rows 16 columns of hi and 16 of
// lo; the same columns take U'^T k once X and S^T q^T have read S.  [128, 384)
// [X | S^T q^T] of even and odd chunks; E^T and then U^T P^T take X's place.  [384, 448)
// R, then U'; [448, 512) U.
// STATES (the backward's first pass) has no q, P and o; it saves the state before
// every chunk and E as the images that delta_grads_kernel multiplies with.
// ---------------------------------------------------------------------------
constexpr uint32_t T_S = 0, T_XQ = 128, T_R = 384, T_U = 448;
constexpr uint32_t T_R3 = T_S;  // R's third part, between X and the new state

// Images: units of 16 bytes, 8 channels (tokens) of a value column, the 128
// columns of a unit one after another: lanes write and read whole lines, and it
// is an operand with the value columns along the contraction.  (Rows of 128 swizzled
// bytes, a row to a lane, took 5000 cycles a chunk to write.)
constexpr uint32_t UNITS = 128 * 16;         // the columns of a unit
constexpr uint32_t S_IMAGE = 2 * 16 * UNITS;  // [hi, lo][16 units of 8 channels][128 columns]
constexpr uint32_t E_IMAGE = 2 * 8 * UNITS;   // [hi, lo][8 units of 8 tokens][128 columns]
// K-step ks (16 value columns) of an image
__device__ __forceinline__ SDesc image_desc(uint32_t base, int ks) {
  return sdesc_mn16(base, 128, UNITS) + (uint32_t)ks * 256u;
}

struct ChainMaps {
  CUtensorMap q, k, v;
};
struct ChainArgs {
  Docs docs;
  const int32_t *order;  // documents, longest first, or null
  int H, share, V, sK, sV;  // V of o and dv; K and V of the states
  float scale;
  const float *h0;
  float *ht;
  __nv_bfloat16 *o;
  const char *tiles;
  const float *gates;
  const uint32_t *flags;  // of each chunk and head, when tiles and gates are made meanwhile; else null
  char *s_images, *e_images;  // STATES
  int *err;
};

// Shared memory: two stages of k, (q), v, Z, gates; three of P; the output
// tile.
template <bool STATES>
struct ChainSmem {
  static constexpr uint32_t KQ = 0, V = STATES ? 16384 : 32768, Z = V + 16384, GT = Z + 3 * TILE, STAGE = GT + 1024;
  static constexpr uint32_t P = 2 * STAGE, OUT = P + (STATES ? 0 : 3 * 2 * TILE);
  static constexpr uint32_t BYTES = OUT + (STATES ? 0 : 16384) + 1024;
  static_assert(STAGE % 1024 == 0 && OUT % 1024 == 0 && BYTES <= 226 * 1024, "");
};
// 24 warps of 80 registers at launch (the last two or three of them idle), dealt out again by
// warpgroup: 512 x 88 + 256 x 64 = 768 x 80.  (88, 80 and 48: more spills, the walks 169 instead of 164 us;
// 96, 64 and 32: 10% slower.  22 warps without dealing out: 280 bytes spilt, 182 us.)
constexpr int CHAIN_WARPS = 16, CHAIN_THREADS = 768;
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// A warp's arrival, after what its lanes did (with their fences) is done: one
// arrival instead of 32 that would queue for the barrier.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// columns of K-step ks of S^T's hi part; lo: 16 further
__device__ __forceinline__ uint32_t s_col(uint32_t tb, int ks) {
  return tb + T_S + (uint32_t)(ks >> 1) * 32u + (uint32_t)(ks & 1) * 8u;
}
// 32 values of a column as hi and lo parts, into tensor memory; with IMG into
// an image as well, behind `arrive`.
template <bool IMG, typename F>
__device__ __forceinline__ void put_state(uint32_t at, const float (&S)[32], char *img, F arrive) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) split2(S[2 * i], S[2 * i + 1], hi[i], lo[i]);
  tmem_st16(at, hi);
  tmem_st16(at + 16, lo);
  tmem_st_wait();
  tc_fence_before();
  arrive();
  if (IMG) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      st_global_v4(img + i * UNITS, hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
      st_global_v4(img + S_IMAGE / 2 + i * UNITS, lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
    }
  }
}

template <bool STATES, bool FLAGS = false>
__device__ __forceinline__ void chain_walk(const ChainMaps &maps, const ChainArgs &a, int64_t unit) {
  using L_ = ChainSmem<STATES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[2], s_ready, x_full, r_ready, e_full, u_ready, s_full, pu_full[2], o_free[2], stage_free[2], drain;
  __shared__ alignas(16) float o_into[2][CH];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (int)((uint32_t)unit % (uint32_t)a.H);
  const uint32_t rank = (uint32_t)unit / (uint32_t)a.H;
  const int64_t d = a.order ? a.order[rank] : (int64_t)rank;
  int64_t s0, s1;
  a.docs.range(d, s0, s1);
  const int nch = (int)((s1 - s0 + CH - 1) / CH);
  const int64_t slot0 = a.docs.chunk_base(d);
  auto chunk_tok = [&](int j) -> int64_t { return s0 + (int64_t)j * CH; };
  auto chunk_len = [&](int j) -> int { return (int)min((int64_t)CH, s1 - chunk_tok(j)); };

  if (warp == 20) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&pu_full[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&stage_free[i], 1);
    }
    for (uint64_t *b : {&x_full, &e_full, &s_full, &drain}) mbar_init(b, 1);
    for (uint64_t *b : {&s_ready, &r_ready, &u_ready}) mbar_init(b, CHAIN_WARPS);
    fence_mbar_init();
  }
  follow_wait();
  fence_async_all();  // what the kernel before wrote with plain stores is read by copies here
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base;
  const uint32_t sb = smem_u32(sm);
  auto stage = [&](int j) -> uint32_t { return (uint32_t)(j & 1) * L_::STAGE; };
  auto wait_full = [&](int j) -> bool { return mbar_wait(&full[j & 1], (uint32_t)(j >> 1) & 1u, WAIT_CYCLES); };

  if (warp >= 20) {
    fewer_registers<64>();
    if (warp == 20 && lane == 0) {
      constexpr uint32_t id64 = idesc_bf16(128, 64, false, false), id128 = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idS = idesc_bf16(128, 128, false, true);
      constexpr uint32_t KROWS = STATES ? 64 : 128;  // rows of a 64-channel block of [k; q]
      // U^T P^T of chunk j: hi hi, then the rest
      auto pu = [&](int j, bool rest) {
        const uint32_t D = tb + T_XQ + (uint32_t)(j & 1) * 128u, p = sb + L_::P + (uint32_t)(j % 3) * 2 * TILE;
        if (!rest) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_U + 8u * ks, kdesc(p, ks, 64), id64, ks);
        } else {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_U + 32u + 8u * ks, kdesc(p, ks, 64), id64, 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_U + 8u * ks, kdesc(p + TILE, ks, 64), id64, 1);
          mma_commit(&pu_full[j & 1]);
        }
      };
      bool ok = true;
      for (int j = 0; j < nch; ++j) {
        const uint32_t ph = (uint32_t)j & 1u, D = tb + T_XQ + ph * 128u;
        const uint32_t k = sb + stage(j) + L_::KQ, z = sb + stage(j) + L_::Z;
        ok = wait_full(j) && mbar_wait(&s_ready, ph, WAIT_CYCLES);
        // the output has read this buffer's last values
        if (ok && !STATES && j >= 2) ok = mbar_wait(&o_free[ph], (uint32_t)((j - 2) >> 1) & 1u, WAIT_CYCLES);
        if (!ok) break;
        // chunk j - 1 is through with its stage (its last product with k came before s_ready), j - 2 with its P
        if (j) mbar_arrive(&stage_free[ph ^ 1u]);
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(D, s_col(tb, ks), kdesc(k, ks, KROWS), STATES ? id64 : id128, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(D, s_col(tb, ks) + 16u, kdesc(k, ks, KROWS), STATES ? id64 : id128, 1);
        mma_commit(&x_full);
        if (!STATES && j >= 1) pu(j - 1, true);
        ok = mbar_wait(&r_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_R + 8u * ks, kdesc(z, ks, 64), id64, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_R + 32u + 8u * ks, kdesc(z, ks, 64), id64, 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_R + 8u * ks, kdesc(z + TILE, ks, 64), id64, 1);
        if (lds_f1(sb + stage(j) + L_::GT + 4u * G_WIDE) != 0.f) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_R + 32u + 8u * ks, kdesc(z + TILE, ks, 64), id64, 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_R3 + 8u * ks, kdesc(z, ks, 64), id64, 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(D, tb + T_R + 8u * ks, kdesc(z + 2 * TILE, ks, 64), id64, 1);
        }
        mma_commit(&e_full);
        ok = mbar_wait(&u_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16_ta(tb + T_S, tb + T_R + 8u * ks, mdesc(k, ks, KROWS * 128u), idS, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16_ta(tb + T_S, tb + T_R + 32u + 8u * ks, mdesc(k, ks, KROWS * 128u), idS, 1);
        mma_commit(&s_full);
        if (!STATES) pu(j, false);
      }
      if (!STATES && ok && nch > 0) pu(nch - 1, true);
      // no product of this block is in flight when it leaves
      mma_commit(&drain);
      if (!mbar_wait(&drain, 0, WAIT_CYCLES)) ok = false;
      if (!ok) atomicExch(&abort_flag, 1);
    } else if (warp == 21 && lane == 0) {
      const int hq = h / a.share;
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
      bool ok = true;
      int loaded = 0;
      // whether chunk j is a wide one, read a chunk ahead of its copies; with FLAGS told with its being ready, of
      // up to AHEAD chunks at once: those before `ready`, in the bits of `wides`
      constexpr int AHEAD = 8;
      int ready = 0;
      uint32_t wides = 0;
      auto wide_of = [&](int j) -> bool {
        if (j >= nch) return false;
        const int64_t sh = (slot0 + j) * a.H + h;
        if (!FLAGS) return ldg_early(a.gates + sh * GATES + G_WIDE) != 0.f;
        if (j == ready) {
          const long long t0 = clock64();
          uint32_t f[AHEAD];
          do {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) f[i] = j + i < nch ? ld_relaxed(a.flags + sh + (int64_t)i * a.H) : 0u;
            if (clock64() - t0 > WAIT_CYCLES) ok = false;
          } while (!f[0] && ok);
          __threadfence();
          fence_async_all();  // what was written before the flags is read by copies here
          wides = 0;
#pragma unroll
          for (int i = 0; i < AHEAD; ++i)
            if (ready == j + i && f[i]) {
              ++ready;
              wides |= f[i] == READY_WIDE ? 1u << ((j + i) % AHEAD) : 0u;
            }
        }
        return wides >> (j % AHEAD) & 1u;
      };
      bool wide = wide_of(0);
      for (int j = 0; j < nch; ++j) {
        ok = ok && (j < 2 || mbar_wait(&stage_free[j & 1], (uint32_t)((j - 2) >> 1) & 1u, WAIT_CYCLES));
        if (!ok) break;
        uint8_t *p = sm + stage(j);
        uint64_t *bar = &full[j & 1];
        const int tok = (int)chunk_tok(j);
        mbar_expect_tx(bar, (STATES ? 2 : 3) * 16384 + (STATES ? 2 : 4) * TILE + (wide ? TILE : 0) + GATES * 4);
        if (STATES) {
          tma_load_3d(p + L_::KQ, &maps.k, 0, hq, tok, bar);
          tma_load_3d(p + L_::KQ + 8192, &maps.k, 64, hq, tok, bar);
        } else {
          tma_load_3d(p + L_::KQ, &maps.k, 0, hq, tok, bar);
          tma_load_3d(p + L_::KQ + 8192, &maps.q, 0, hq, tok, bar);
          tma_load_3d(p + L_::KQ + 16384, &maps.k, 64, hq, tok, bar);
          tma_load_3d(p + L_::KQ + 24576, &maps.q, 64, hq, tok, bar);
        }
        tma_load_3d(p + L_::V, &maps.v, 0, h, tok, bar);
        tma_load_3d(p + L_::V + 8192, &maps.v, 64, h, tok, bar);
        const int64_t sh = (slot0 + j) * a.H + h;
        bulk_load(p + L_::Z, a.tiles + sh * TILES, 2 * TILE, bar);
        if (wide) bulk_load(p + L_::Z + 2 * TILE, a.tiles + sh * TILES + 4 * TILE, TILE, bar);
        if (!STATES) bulk_load(sm + L_::P + (uint32_t)(j % 3) * 2 * TILE, a.tiles + sh * TILES + 2 * TILE, 2 * TILE, bar);
        bulk_load(p + L_::GT, a.gates + sh * GATES, GATES * 4, bar);
        loaded = j + 1;
        wide = wide_of(j + 1);
      }
      // no copy of this block is in flight when it leaves
      for (int j = max(0, loaded - 2); j < loaded; ++j)
        if (!wait_full(j)) ok = false;
      if (!ok) atomicExch(&abort_flag, 1);
    }
    __syncwarp();
  } else if (warp < CHAIN_WARPS) {
    more_registers<88>();
    const int grp = warp >> 2, qw = warp & 3, v = qw * 32 + lane;
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;  // this warp's lanes of tensor memory
    const bool in = v < a.sV;
    float S[32];
    {
      const int64_t at = ((d * a.H + h) * a.sK + 32 * grp) * (int64_t)a.sV + v;
#pragma unroll
      for (int i = 0; i < 32; ++i) S[i] = a.h0 && in && 32 * grp + i < a.sK ? a.h0[at + (int64_t)i * a.sV] : 0.f;
    }
    // Rows past the document's end hold other tokens: as zeros, nothing in them reaches a sum.  Those of the
    // products' operands, which wait for every warp (s_ready); v is masked where it is read, right behind this
    // warp's own share.
    auto clear_rows = [&](int j) -> bool {
      const int L = chunk_len(j);
      if (L == CH) return true;
      if (!wait_full(j)) return false;
      constexpr int BLOCKS = STATES ? 2 : 4;  // tiles of 64 rows: k, (q)
      for (int i = threadIdx.x; i < (CH - L) * BLOCKS * 8; i += 32 * CHAIN_WARPS) {
        const int c = i % 8, b = i / 8 % BLOCKS, r = L + i / (8 * BLOCKS);
        st_shared_v4(sb + stage(j) + b * 8192u + r * 128u + c * 16u, 0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      return true;
    };
    bool ok = true;
    // the state before chunk j, handed to the products
    auto hand_state = [&](int j) {
      put_state<STATES>(tb + lanes + T_S + 32u * grp, S,
                        a.s_images + ((slot0 + j) * a.H + h) * S_IMAGE + 4 * grp * UNITS + v * 16, [&] {
                          ok = ok && clear_rows(j);
                          warp_arrive(&s_ready);
                        });
    };
    if (nch > 0) hand_state(0);
    for (int j = 0; j < nch; ++j) {
      const uint32_t ph = (uint32_t)j & 1u, D = tb + lanes + T_XQ + ph * 128u + 16u * grp;
      const float *gates = reinterpret_cast<const float *>(sm + stage(j) + L_::GT);
      const float4 *into = reinterpret_cast<const float4 *>(gates + G_INTO + 16 * grp);
      const float4 *out = reinterpret_cast<const float4 *>(gates + G_OUT + 16 * grp);
      const float4 *beta = reinterpret_cast<const float4 *>(gates + G_BETA + 16 * grp);
      float Y[16];
      ok = ok && wait_full(j);
      {
        const ColBf16 col(sb + stage(j) + L_::V, 16 * grp, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) Y[i] = bf16_bits_to_f32(lds_u16(col.at(i)));
        // rows past the end hold other tokens: an infinity there times their b = 0 would be NaN in R
        const int left = chunk_len(j) - 16 * grp;
        if (left < 16)
#pragma unroll
          for (int i = 0; i < 16; ++i) Y[i] = i < left ? Y[i] : 0.f;
      }
      const bool wide = gates[G_WIDE] != 0.f;
      ok = ok && mbar_wait(&x_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[16];
        tmem_ld16(D, x);
        tmem_ld_wait(x);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 e = into[i / 4], b = beta[i / 4];
          Y[i] = fmaf(-e.x, __uint_as_float(x[i]), Y[i]);
          Y[i + 1] = fmaf(-e.y, __uint_as_float(x[i + 1]), Y[i + 1]);
          Y[i + 2] = fmaf(-e.z, __uint_as_float(x[i + 2]), Y[i + 2]);
          Y[i + 3] = fmaf(-e.w, __uint_as_float(x[i + 3]), Y[i + 3]);
          split2(b.x * Y[i], b.y * Y[i + 1], hi[i / 2], lo[i / 2]);
          split2(b.z * Y[i + 2], b.w * Y[i + 3], hi[i / 2 + 1], lo[i / 2 + 1]);
        }
        tmem_st8(tb + lanes + T_R + 8u * grp, hi);
        tmem_st8(tb + lanes + T_R + 32u + 8u * grp, lo);
        if (wide) {
          uint32_t l3[8];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 b = beta[i / 4];
            l3[i / 2] = split3(b.x * Y[i], b.y * Y[i + 1], hi[i / 2], lo[i / 2]);
            l3[i / 2 + 1] = split3(b.z * Y[i + 2], b.w * Y[i + 3], hi[i / 2 + 1], lo[i / 2 + 1]);
          }
          tmem_st8(tb + lanes + T_R3 + 8u * grp, l3);
        }
        // scale e^G for the output, which outlives the stage; X of this chunk began behind o_free of the one
        // before the last, whose factors were here
        if (!STATES && qw == 0 && lane < 16) o_into[ph][16 * grp + lane] = a.scale * gates[G_INTO + 16 * grp + lane];
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&r_ready);
      }
      ok = ok && mbar_wait(&e_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[16];
        tmem_ld16(D, x);
        tmem_ld_wait(x);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 b = beta[i / 4], r = out[i / 4];
#pragma unroll
          for (int n = 0; n < 4; ++n) Y[i + n] += __uint_as_float(x[i + n]);
          split2(r.x * (b.x * Y[i]), r.y * (b.y * Y[i + 1]), hi[i / 2], lo[i / 2]);
          split2(r.z * (b.z * Y[i + 2]), r.w * (b.w * Y[i + 3]), hi[i / 2 + 1], lo[i / 2 + 1]);
        }
        tmem_st8(tb + lanes + T_R + 8u * grp, hi);
        tmem_st8(tb + lanes + T_R + 32u + 8u * grp, lo);
        if (!STATES) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 b = beta[i / 4];
            split2(b.x * Y[i], b.y * Y[i + 1], hi[i / 2], lo[i / 2]);
            split2(b.z * Y[i + 2], b.w * Y[i + 3], hi[i / 2 + 1], lo[i / 2 + 1]);
          }
          tmem_st8(tb + lanes + T_U + 8u * grp, hi);
          tmem_st8(tb + lanes + T_U + 32u + 8u * grp, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&u_ready);
        if (STATES) {  // E
          char *img = a.e_images + ((slot0 + j) * a.H + h) * E_IMAGE + 2 * grp * UNITS + v * 16;
#pragma unroll
          for (int i = 0; i < 16; i += 2) split2(Y[i], Y[i + 1], hi[i / 2], lo[i / 2]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            st_global_v4(img + i * UNITS, hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
            st_global_v4(img + E_IMAGE / 2 + i * UNITS, lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
          }
        }
      }
      const float over = gates[G_OVER];
      ok = ok && mbar_wait(&s_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[32];
        tmem_ld32(tb + lanes + T_S + 32u * grp, x);
        tmem_ld_wait32(x);
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = fmaf(over, S[i], __uint_as_float(x[i]));
      }
      if (j + 1 < nch) hand_state(j + 1);
    }
    if (!ok) atomicExch(&abort_flag, 1);
    if (a.ht && in && ok) {
      float *dst = a.ht + ((d * a.H + h) * a.sK + 32 * grp) * (int64_t)a.sV + v;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (32 * grp + i < a.sK) dst[(int64_t)i * a.sV] = S[i];
    }
  } else {
    fewer_registers<64>();
    const int qw = warp & 3, v = qw * 32 + lane, tid = threadIdx.x - 32 * CHAIN_WARPS;
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    bool ok = true;
    for (int j = 0; !STATES && j < nch; ++j) {
      const uint32_t ph = (uint32_t)j & 1u, D = tb + lanes + T_XQ + ph * 128u;
      ok = ok && mbar_wait(&pu_full[ph], (uint32_t)(j >> 1) & 1u, WAIT_CYCLES);
      tc_fence_after();
      // the last tile has been read; everyone hears of a wait that ran out
      if (named_bar_any(1, 128, !ok)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        uint32_t x[16], p[16];
        tmem_ld16(D + 64u + c, x);
        tmem_ld16(D + c, p);
        tmem_ld_wait(x);
        tmem_ld_wait(p);
        const ColBf16 col(smem_u32(sm + L_::OUT), c, v);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 e = lds_f4(smem_u32(&o_into[ph][c + i]));
          const float f[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int n = 0; n < 4; ++n)
            sts_u16(col.at(i + n), f32_to_bf16_bits(fmaf(f[n], __uint_as_float(x[i + n]), __uint_as_float(p[i + n]))));
        }
      }
      tc_fence_before();
      warp_arrive(&o_free[ph]);
      named_bar(2, 128);
      const int L = chunk_len(j);
      __nv_bfloat16 *dst = a.o + (chunk_tok(j) * a.H + h) * (int64_t)a.V;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int i = tid + 128 * n, r = i >> 4, c = (i & 15) * 8;
        if (r < L && c < a.V) {
          const uint4 x = lds_u4(smem_u32(sm + L_::OUT) + sw128_off(r, c, 64));
          st_global_v4(dst + (int64_t)r * a.H * a.V + c, x.x, x.y, x.z, x.w);
        }
      }
    }
    if (!ok) atomicExch(&abort_flag, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile int *)&abort_flag) set_device_error(a.err, GLACORE_ERR_TIMEOUT);
  if (warp == 20) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// ---------------------------------------------------------------------------
// The same walk backwards, with the gradient of the state: value column v in
// lane v, per chunk
//     dU^T  = dO^T (P) + e^{G_C - G} (dS1^T k^T)       A: dO (rows of the contraction), dS1^T; B: P, k
//     dR^T  = dU^T + (b dU)^T Z                        -> dY = b dR (= dV), dX = -e^G dY
//     dS0^T = e^{G_C} dS1^T + (scale e^G dO)^T q + dX^T k
// dO^T P and the product with q do not wait for the chain.  Saved for
// delta_grads_kernel: dS1 of every chunk (an image as S0's) and dR (as rows of a
// token, [hi, lo][two blocks of 64 columns][64 rows]).
//   warps 0..15  the chain, as in the forward
//   warps 16..19 scale e^G dO as an operand, dv and dR on their way out
//   warp 20      copies and products, one thread (copies by another one, as in the forward, gain nothing here)
// TMEM columns: [0, 128) dS1^T (hi, lo); [128, 192) dS1^T k^T, then (b dU)^T Z;
// [192, 256) dO^T P; [256, 320) b dU, then dX; [320, 384) scale e^G dO;
// [384, 512) the new part of dS0^T.
// ---------------------------------------------------------------------------
constexpr uint32_t B_D1 = 128, B_PDO = 192, B_R = 256, B_DO = 320, B_DS = 384;
constexpr uint32_t R_IMAGE = 2 * 16384;

struct BackMaps {
  CUtensorMap q, k, dO;
};
struct BackArgs {
  Docs docs;
  const int32_t *order;
  int H, share, V, sK, sV;  // V of o and dv; K and V of the states
  float scale;
  const float *dht;
  float *dh0;
  __nv_bfloat16 *dv;
  const char *tiles;
  const float *gates;
  char *ds_images, *r_images;
  int *err;
};
struct BackSmem {
  static constexpr uint32_t K = 0, Q = 16384, DO = 32768, Z = 49152, P = Z + 2 * TILE, Z3 = P + 2 * TILE, GT = Z3 + TILE,
                            STAGE = GT + 1024;
  static constexpr uint32_t R = 2 * STAGE, BYTES = R + R_IMAGE + 1024;
};
static_assert(BackSmem::STAGE % 1024 == 0 && BackSmem::BYTES <= 226 * 1024, "");

__device__ __forceinline__ void back_walk(const BackMaps &maps, const BackArgs &a, int64_t unit) {
  using L_ = BackSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[2], s_ready, x_full, r_ready, e_full, u_ready, s_full, q_full, do_ready, dr_ready, dr_free, drain;
  __shared__ float w_beta[3][CH];  // of three steps: read behind the next step's barrier
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (int)((uint32_t)unit % (uint32_t)a.H);
  const uint32_t rank = (uint32_t)unit / (uint32_t)a.H;
  const int64_t d = a.order ? a.order[rank] : (int64_t)rank;
  int64_t s0, s1;
  a.docs.range(d, s0, s1);
  const int nch = (int)((s1 - s0 + CH - 1) / CH);
  const int64_t slot0 = a.docs.chunk_base(d);
  // step i of the walk takes chunk nch - 1 - i
  auto chunk_tok = [&](int i) -> int64_t { return s0 + (int64_t)(nch - 1 - i) * CH; };
  auto chunk_len = [&](int i) -> int { return (int)min((int64_t)CH, s1 - chunk_tok(i)); };
  auto chunk_sh = [&](int i) -> int64_t { return (slot0 + nch - 1 - i) * a.H + h; };

  if (warp == 20) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (uint64_t *b : {&full[0], &full[1], &x_full, &e_full, &s_full, &q_full, &drain}) mbar_init(b, 1);
    for (uint64_t *b : {&s_ready, &r_ready, &u_ready, &dr_ready}) mbar_init(b, CHAIN_WARPS);
    for (uint64_t *b : {&do_ready, &dr_free}) mbar_init(b, 4);
    fence_mbar_init();
  }
  follow_wait();
  fence_async_all();  // what the kernel before wrote with plain stores is read by copies here
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base;
  const uint32_t sb = smem_u32(sm);
  auto stage = [&](int i) -> uint32_t { return (uint32_t)(i & 1) * L_::STAGE; };
  auto wait_full = [&](int i) -> bool { return mbar_wait(&full[i & 1], (uint32_t)(i >> 1) & 1u, WAIT_CYCLES); };

  if (warp >= 20) {
    fewer_registers<64>();
    if (warp == 20 && lane == 0) {
      const int hq = h / a.share;
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.dO);
      int loaded = 0;
      auto wide_of = [&](int i) -> float { return i < nch ? ldg_early(a.gates + chunk_sh(i) * GATES + G_WIDE) : 0.f; };
      float wide_next = wide_of(0);
      auto load = [&](int i) {
        uint8_t *p = sm + stage(i);
        uint64_t *bar = &full[i & 1];
        const int tok = (int)chunk_tok(i);
        const bool wide = wide_next != 0.f;
        wide_next = wide_of(i + 1);
        mbar_expect_tx(bar, 3 * 16384 + 4 * TILE + (wide ? TILE : 0) + GATES * 4);
        tma_load_3d(p + L_::K, &maps.k, 0, hq, tok, bar);
        tma_load_3d(p + L_::K + 8192, &maps.k, 64, hq, tok, bar);
        tma_load_3d(p + L_::DO, &maps.dO, 0, h, tok, bar);
        tma_load_3d(p + L_::DO + 8192, &maps.dO, 64, h, tok, bar);
        tma_load_3d(p + L_::Q, &maps.q, 0, hq, tok, bar);
        tma_load_3d(p + L_::Q + 8192, &maps.q, 64, hq, tok, bar);
        const char *tiles = a.tiles + chunk_sh(i) * TILES;
        bulk_load(p + L_::Z, tiles, (wide ? 5 : 4) * TILE, bar);  // Z, P, Z's third part
        bulk_load(p + L_::GT, a.gates + chunk_sh(i) * GATES, GATES * 4, bar);
        loaded = i + 1;
      };
      constexpr uint32_t id64 = idesc_bf16(128, 64, false, false), id64n = idesc_bf16(128, 64, false, true);
      constexpr uint32_t idP = idesc_bf16(128, 64, true, true), idS = idesc_bf16(128, 128, false, true);
      auto pdo = [&](int i) {  // dO^T P
        const uint32_t dO = sb + stage(i) + L_::DO, p = sb + stage(i) + L_::P;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16(tb + B_PDO, mdesc(dO, ks, 8192), mdesc(p, ks, 8192), idP, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16(tb + B_PDO, mdesc(dO, ks, 8192), mdesc(p + TILE, ks, 8192), idP, 1);
      };
      bool ok = true;
      if (nch > 0) load(0);
      for (int i = 0; i < nch; ++i) {
        const uint32_t ph = (uint32_t)i & 1u;
        const uint32_t st = sb + stage(i), k = st + L_::K, q = st + L_::Q, z = st + L_::Z;
        // every row of the chunk is what it should be (rows past the end cleared) with the state of the step
        ok = wait_full(i) && mbar_wait(&s_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(tb + B_D1, s_col(tb, ks), kdesc(k, ks, 64), id64, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(tb + B_D1, s_col(tb, ks) + 16u, kdesc(k, ks, 64), id64, 1);
        if (i == 0) pdo(0);
        mma_commit(&x_full);
        // step i - 1 is through with its stage (its last product before s_ready, dO's copy in TMEM, gates copied)
        if (i + 1 < nch) load(i + 1);
        ok = mbar_wait(&r_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_D1, tb + B_R + 8u * ks, mdesc(z, ks, 8192), id64n, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_D1, tb + B_R + 32u + 8u * ks, mdesc(z, ks, 8192), id64n, 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_D1, tb + B_R + 8u * ks, mdesc(z + TILE, ks, 8192), id64n, 1);
        if (lds_f1(st + L_::GT + 4u * G_WIDE) != 0.f) {
          const uint32_t z3 = st + L_::Z3;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_D1, tb + B_R + 32u + 8u * ks, mdesc(z + TILE, ks, 8192), id64n, 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_D1, tb + T_R3 + 8u * ks, mdesc(z, ks, 8192), id64n, 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_D1, tb + B_R + 8u * ks, mdesc(z3, ks, 8192), id64n, 1);
        }
        mma_commit(&e_full);
        ok = mbar_wait(&do_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_DS, tb + B_DO + 8u * ks, mdesc(q, ks, 8192), idS, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_DS, tb + B_DO + 32u + 8u * ks, mdesc(q, ks, 8192), idS, 1);
        mma_commit(&q_full);
        ok = mbar_wait(&u_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_DS, tb + B_R + 8u * ks, mdesc(k, ks, 8192), idS, 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + B_DS, tb + B_R + 32u + 8u * ks, mdesc(k, ks, 8192), idS, 1);
        mma_commit(&s_full);
        if (i + 1 < nch) {  // a whole chunk, no rows to be cleared
          if (!(ok = wait_full(i + 1))) break;
          pdo(i + 1);
        }
      }
      // no copy or product of this block is in flight when it leaves
      for (int i = max(0, loaded - 2); i < loaded; ++i)
        if (!wait_full(i)) ok = false;
      mma_commit(&drain);
      if (!mbar_wait(&drain, 0, WAIT_CYCLES)) ok = false;
      if (!ok) atomicExch(&abort_flag, 1);
    }
    __syncwarp();
  } else if (warp < CHAIN_WARPS) {
    more_registers<88>();
    const int grp = warp >> 2, qw = warp & 3, v = qw * 32 + lane;
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    const bool in = v < a.sV;
    float S[32];
    {
      const int64_t at = ((d * a.H + h) * a.sK + 32 * grp) * (int64_t)a.sV + v;
#pragma unroll
      for (int i = 0; i < 32; ++i) S[i] = a.dht && in && 32 * grp + i < a.sK ? a.dht[at + (int64_t)i * a.sV] : 0.f;
    }
    auto clear_rows = [&](int i) -> bool {
      const int L = chunk_len(i);
      if (L == CH) return true;
      if (!wait_full(i)) return false;
      for (int n = threadIdx.x; n < (CH - L) * 6 * 8; n += 32 * CHAIN_WARPS) {  // k, q, dO: six tiles of 64 rows
        const int c = n % 8, b = n / 8 % 6, r = L + n / 48;
        st_shared_v4(sb + stage(i) + b * 8192u + r * 128u + c * 16u, 0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      return true;
    };
    const uint32_t img0 = 4 * grp * UNITS + v * 16;  // this thread's units in an image of the state
    bool ok = true;
    // the gradient behind the chunk of step i, handed to the products and to the grads kernel
    auto hand_state = [&](int i) {
      put_state<true>(tb + lanes + T_S + 32u * grp, S, a.ds_images + chunk_sh(i) * S_IMAGE + img0, [&] {
        ok = ok && clear_rows(i);
        warp_arrive(&s_ready);
      });
    };
    if (nch > 0) hand_state(0);
    for (int i = 0; i < nch; ++i) {
      const uint32_t ph = (uint32_t)i & 1u, D = tb + lanes + 16u * grp;
      const float *gates = reinterpret_cast<const float *>(sm + stage(i) + L_::GT);
      const float4 *into = reinterpret_cast<const float4 *>(gates + G_INTO + 16 * grp);
      const float4 *out = reinterpret_cast<const float4 *>(gates + G_OUT + 16 * grp);
      const float4 *beta = reinterpret_cast<const float4 *>(gates + G_BETA + 16 * grp);
      float Y[16];
      ok = ok && wait_full(i);
      const bool wide = gates[G_WIDE] != 0.f;
      ok = ok && mbar_wait(&x_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[16], p[16], hi[8], lo[8];
        tmem_ld16(D + B_D1, x);
        tmem_ld16(D + B_PDO, p);
        tmem_ld_wait(x);
        tmem_tie(p);
#pragma unroll
        for (int n = 0; n < 16; n += 4) {
          const float4 r = out[n / 4], b = beta[n / 4];
          Y[n] = fmaf(r.x, __uint_as_float(x[n]), __uint_as_float(p[n]));
          Y[n + 1] = fmaf(r.y, __uint_as_float(x[n + 1]), __uint_as_float(p[n + 1]));
          Y[n + 2] = fmaf(r.z, __uint_as_float(x[n + 2]), __uint_as_float(p[n + 2]));
          Y[n + 3] = fmaf(r.w, __uint_as_float(x[n + 3]), __uint_as_float(p[n + 3]));
          split2(b.x * Y[n], b.y * Y[n + 1], hi[n / 2], lo[n / 2]);
          split2(b.z * Y[n + 2], b.w * Y[n + 3], hi[n / 2 + 1], lo[n / 2 + 1]);
        }
        tmem_st8(tb + lanes + B_R + 8u * grp, hi);
        tmem_st8(tb + lanes + B_R + 32u + 8u * grp, lo);
        if (wide) {
          uint32_t l3[8];
#pragma unroll
          for (int n = 0; n < 16; n += 4) {
            const float4 b = beta[n / 4];
            l3[n / 2] = split3(b.x * Y[n], b.y * Y[n + 1], hi[n / 2], lo[n / 2]);
            l3[n / 2 + 1] = split3(b.z * Y[n + 2], b.w * Y[n + 3], hi[n / 2 + 1], lo[n / 2 + 1]);
          }
          tmem_st8(tb + lanes + T_R3 + 8u * grp, l3);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&r_ready);
      }
      ok = ok && mbar_wait(&e_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[16], hi[8], lo[8];
        tmem_ld16(D + B_D1, x);
        tmem_ld_wait(x);
#pragma unroll
        for (int n = 0; n < 16; n += 4) {
          const float4 b = beta[n / 4], e = into[n / 4];
#pragma unroll
          for (int m = 0; m < 4; ++m) Y[n + m] += __uint_as_float(x[n + m]);
          split2(-e.x * (b.x * Y[n]), -e.y * (b.y * Y[n + 1]), hi[n / 2], lo[n / 2]);
          split2(-e.z * (b.z * Y[n + 2]), -e.w * (b.w * Y[n + 3]), hi[n / 2 + 1], lo[n / 2 + 1]);
        }
        tmem_st8(tb + lanes + B_R + 8u * grp, hi);
        tmem_st8(tb + lanes + B_R + 32u + 8u * grp, lo);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&u_ready);
      }
      // dR, a column of the tile
      if (i >= 1) ok = ok && mbar_wait(&dr_free, (uint32_t)(i - 1) & 1u, WAIT_CYCLES);
      {
        const ColBf16 col(sb + L_::R, 16 * grp, v);
#pragma unroll
        for (int n = 0; n < 16; n += 2) {
          uint32_t hi, lo;
          split2(Y[n], Y[n + 1], hi, lo);
          sts_u16(col.at(n), (uint16_t)hi);
          sts_u16(col.at(n + 1), (uint16_t)(hi >> 16));
          sts_u16(col.at(n) + 16384u, (uint16_t)lo);
          sts_u16(col.at(n + 1) + 16384u, (uint16_t)(lo >> 16));
        }
        fence_async_smem();
        warp_arrive(&dr_ready);
      }
      const float over = gates[G_OVER];
      ok = ok && mbar_wait(&s_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[32];
        tmem_ld32(tb + lanes + B_DS + 32u * grp, x);
        tmem_ld_wait32(x);
#pragma unroll
        for (int n = 0; n < 32; ++n) S[n] = fmaf(over, S[n], __uint_as_float(x[n]));
      }
      if (i + 1 < nch) hand_state(i + 1);
    }
    if (!ok) atomicExch(&abort_flag, 1);
    if (a.dh0 && in && ok) {
      float *dst = a.dh0 + ((d * a.H + h) * a.sK + 32 * grp) * (int64_t)a.sV + v;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (32 * grp + i < a.sK) dst[(int64_t)i * a.sV] = S[i];
    }
  } else {
    fewer_registers<64>();
    const int qw = warp & 3, v = qw * 32 + lane, tid = threadIdx.x - 32 * CHAIN_WARPS;
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    bool ok = true;
    // scale e^G dO of step i into tensor memory (the product that read the last one is done)
    auto put_do = [&](int i) {
      ok = ok && wait_full(i);
      const float *gates = reinterpret_cast<const float *>(sm + stage(i) + L_::GT);
      const int L = chunk_len(i);
      if (tid < CH) w_beta[i % 3][tid] = gates[G_BETA + tid];
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        const ColBf16 col(sb + stage(i) + L_::DO, c, v);
        uint32_t hi[8], lo[8];
        uint16_t x[16];
#pragma unroll
        for (int n = 0; n < 16; ++n) x[n] = ld_u16(sm + (col.at(n) - sb));
#pragma unroll
        for (int n = 0; n < 16; n += 4) {
          const float4 e = *reinterpret_cast<const float4 *>(gates + G_INTO + c + n);
          const float f[4] = {e.x, e.y, e.z, e.w};
          float y[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) y[m] = bf16_bits_to_f32(x[n + m]) * (a.scale * f[m]);
          if (L < CH)  // rows past the end may be cleared or not yet
#pragma unroll
            for (int m = 0; m < 4; ++m) y[m] = c + n + m < L ? y[m] : 0.f;
          split2(y[0], y[1], hi[n / 2], lo[n / 2]);
          split2(y[2], y[3], hi[n / 2 + 1], lo[n / 2 + 1]);
        }
        tmem_st8(tb + lanes + B_DO + c / 2, hi);
        tmem_st8(tb + lanes + B_DO + 32u + c / 2, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&do_ready);
    };
    if (nch > 0) put_do(0);
    for (int i = 0; i < nch; ++i) {
      const uint32_t ph = (uint32_t)i & 1u;
      ok = ok && mbar_wait(&q_full, ph, WAIT_CYCLES);
      tc_fence_after();
      if (i + 1 < nch) put_do(i + 1);
      ok = ok && mbar_wait(&dr_ready, ph, WAIT_CYCLES);
      // w_beta is there; everyone hears of a wait that ran out
      if (named_bar_any(1, 128, !ok)) {
        ok = false;
        break;
      }
      if (tid == 0) {
        bulk_store(a.r_images + chunk_sh(i) * R_IMAGE, sm + L_::R, R_IMAGE);
        bulk_commit();
      }
      const int L = chunk_len(i);
      __nv_bfloat16 *dst = a.dv + (chunk_tok(i) * a.H + h) * (int64_t)a.V;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int e = tid + 128 * n, r = e >> 4, c = (e & 15) * 8;
        if (r < L && c < a.V) {
          const uint32_t o = L_::R + sw128_off(r, c, 64);
          const uint4 x = *reinterpret_cast<const uint4 *>(sm + o), y = *reinterpret_cast<const uint4 *>(sm + o + 16384u);
          const float b = w_beta[i % 3][r];
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
          uint32_t w[4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
            w[m] = pack_bf16(b * (__uint_as_float(xs[m] << 16) + __uint_as_float(ys[m] << 16)),
                             b * (__uint_as_float(xs[m] & 0xffff0000u) + __uint_as_float(ys[m] & 0xffff0000u)));
          st_global_v4(dst + (int64_t)r * a.H * a.V + c, w[0], w[1], w[2], w[3]);
        }
      }
      if (tid == 0) bulk_wait_read_all();
      warp_arrive(&dr_free);
    }
    if (tid == 0) bulk_wait_all();
    if (!ok) atomicExch(&abort_flag, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile int *)&abort_flag) set_device_error(a.err, GLACORE_ERR_TIMEOUT);
  if (warp == 20) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

__global__ void __launch_bounds__(CHAIN_THREADS, 1) delta_chain_kernel(const __grid_constant__ ChainMaps maps,
                                                                       const ChainArgs a) {
  chain_walk<false>(maps, a, blockIdx.x);
}
// Few sequences leave most SMs without a walk: those make the tiles meanwhile,
// chunk after chunk of all sequences, three teams of delta_prep_kernel's kind to a block.  Walks wait
// for blocks of their launch, so it is a cooperative one: all of them run at once.
struct OverlapArgs {
  ChainArgs chain;
  PrepArgs prep;
  uint32_t *flags;  // 0 before the launch
  uint32_t units, makers;  // blocks that walk, blocks that make tiles
};
constexpr int TEAMS = CHAIN_THREADS / PREP_THREADS;
constexpr uint32_t TEAM_BYTES = 50 * 1024;
static_assert(32768 + sizeof(PrepSmem) <= TEAM_BYTES && TEAMS * TEAM_BYTES + 1024 <= ChainSmem<false>::BYTES, "");

__device__ __forceinline__ void make_tiles(const PrepMaps &maps, const OverlapArgs &a, uint32_t maker) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[TEAMS], done[TEAMS];
  __shared__ uint32_t tmem_base[TEAMS];
  __shared__ double warp0_total[TEAMS];
  const int t = threadIdx.x / PREP_THREADS;
  const PrepTeam w{(uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023) + t * TEAM_BYTES, &full[t], &done[t],
                   &tmem_base[t], &warp0_total[t], (int)threadIdx.x % PREP_THREADS, 1 + 4 * t};
  const PrepArgs &p = a.prep;
  if (w.tid == 0) {
    mbar_init(w.full, 1);
    mbar_init(w.done, 1);
    fence_mbar_init();
  }
  if (w.tid >> 5 == 1) tmem_alloc(w.tmem, 64);
  __syncthreads();
  const uint32_t wide = (uint32_t)p.docs.n * (uint32_t)p.H;  // (sequence, head) pairs
  const uint32_t per = (uint32_t)((p.docs.T + CH - 1) / CH), n = wide * per;
  uint32_t phase = 0;
  for (uint32_t i = maker * TEAMS + t; i < n; i += a.makers * TEAMS, phase ^= 1u) {
    const uint32_t j = i / wide, r = i % wide;
    const int h = (int)(r % (uint32_t)p.H);
    const int64_t slot = (int64_t)(r / (uint32_t)p.H) * per + j;
    int64_t tok;
    int L;
    chunk_in_slot(p.docs, slot, tok, L);
    if (w.tid == 0) prep_load(maps, w, h / p.share, tok);
    if (!prep_chunk<true>(p, w, slot, h, 1, tok, L, phase, a.flags)) break;
  }
  __syncthreads();
  if (w.tid >> 5 == 1) {
    tc_fence_after();
    tmem_dealloc(*w.tmem, 64);
  }
}
struct OverlapMaps {
  ChainMaps chain;
  PrepMaps prep;
};
__global__ void __launch_bounds__(CHAIN_THREADS, 1) delta_overlap_kernel(const __grid_constant__ OverlapMaps maps,
                                                                         const __grid_constant__ OverlapArgs a) {
  if (blockIdx.x < a.units)
    chain_walk<false, true>(maps.chain, a.chain, blockIdx.x);
  else
    make_tiles(maps.prep, a, blockIdx.x - a.units);
}

// The backward's two walks do not need one another: the first half of the
// blocks goes backwards (the longer way), the second forwards.  4 x 16 heads: 128
// of 152 SMs at work instead of 64 twice, 32 chunks in 156 us.
struct WalkMaps {
  ChainMaps states;
  BackMaps back;
};
struct WalkArgs {
  ChainArgs states;
  BackArgs back;
  int64_t units;
};
__global__ void __launch_bounds__(CHAIN_THREADS, 1) delta_walks_kernel(const __grid_constant__ WalkMaps maps,
                                                                       const __grid_constant__ WalkArgs a) {
  if (blockIdx.x < a.units)
    back_walk(maps.back, a.back, blockIdx.x);
  else
    chain_walk<true>(maps.states, a.states, blockIdx.x - a.units);
}

// ---------------------------------------------------------------------------
// Gradients of q, k, g and beta, every chunk of a head by itself.  Key channel
// in lane (128 of them), tokens in columns:
//     B1 = dO E^T, B2 = dR E^T (token in lane: the stacked [dO; dR], twice over for
//     the two parts of dR, so that rows of dO come out doubled)
//     dPd = scale D (.) B1 diag(b), dA = -D (.) diag(b) B2 diag(b), db = diag(B2)
//     dQ^T = scale e^G (S0 dO^T) + K^T dPd^T
//     dK^T = -e^G b (S0 dR^T) + e^{G_C - G} b (dS1 E^T) + Q^T dPd + K^T (dA + dA^T)
// One block per SM walks over (chunk, head) pairs: 16 warps of elementwise
// work, one that copies and multiplies.  dS1's image takes the place of the
// stacks once those have been multiplied, beside S0's, in whose place the masked
// tiles come when <S0, dS1> has been summed and dq and dk when all is multiplied.  The
// next pair's operands are on their way while this one's gradients leave (S0's low
// part behind them, and the products with it last).  Products with two parts of a matrix put both into one operand of
// 128 columns where tensor memory has room for the two results (a product of 64
// columns is bound by its other operand's way through shared memory).
// 2048 pairs take 138 us on 152 SMs: 561 MB from and to memory (61% of the copy
// rate), issue slots and the barriers between steps.
// TMEM columns: [0, 64) [q; k] k^T, [64, 192) B1, B2 of E's two parts, later [0, 128)
// the pairs' part of dK^T (two halves); [192, 320) S0 dO^T, S0 dR^T; [320, 384)
// K^T dPd^T; [384, 512) dS1 E^T (two halves).
// ---------------------------------------------------------------------------
constexpr uint32_t Q_QK = 0, Q_B = 64, Q_1 = 192, Q_2 = 256, Q_4 = 320, Q_3 = 384, Q_5 = 0;

struct GradMaps {
  CUtensorMap q, k, dO;
};
struct GradArgs {
  Docs docs;
  int64_t units;  // slots x H
  int H, share, K;
  float scale;
  const float *g, *beta;
  const char *s_images, *ds_images, *e_images, *r_images;
  void *dq, *dk;  // bf16, or per value head in fp32
  float *dg, *dbeta;
  int *err;
};
struct GradSmem {
  // S: S0's image, then T: dPd hi, lo, dA hi, lo, and OUT: dq, dk; X1, X2: per 64 columns 64 rows of dO, 64 of dR
  // (hi, lo), then DS: dS1's image; QK: per 64 channels 64 rows of q, 64 of k
  static constexpr uint32_t S = 0, X1 = S + S_IMAGE, X2 = X1 + 32768, E = X2 + 32768, QK = E + E_IMAGE,
                            BYTES = QK + 32768 + 1024;
  static constexpr uint32_t T = S, OUT = S + S_IMAGE / 2, DS = X1;
  static_assert(4 * TILE == S_IMAGE / 2 && S_IMAGE == 2 * 32768, "");
};
// 20 warps of 96 registers at launch (the last three of them idle), dealt out again by warpgroup:
// 512 x 104 + 128 x 64 = 640 x 96.  (Nothing may spill: shared memory leaves the first-level cache a few KB.)
constexpr int GRAD_WARPS = 16, GRAD_THREADS = 640;

template <bool PER_HEAD>
__global__ void __launch_bounds__(GRAD_THREADS, 1) delta_grads_kernel(const __grid_constant__ GradMaps maps,
                                                                      const GradArgs a) {
  using L_ = GradSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full_a, full_b, full_ds, cleared, qk_read, g1, g2, tiles, g3, left, drain;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ alignas(16) float4 s_g[CH];  // two parts of G (in units of log 2), b
  __shared__ alignas(16) float s_into[CH], s_ki[CH], s_ko[CH];  // scale e^G, -e^G b, e^{G_C - G} b
  __shared__ alignas(16) float s_tot[2 * CH][4];
  // s_over, s_dot: of two units, the last one's are read while the next is begun
  __shared__ float s_db[CH], s_pair[4][CH], s_red[2][4][CH], s_over[2], s_dot[2][GRAD_WARPS];
  __shared__ double warp0_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == GRAD_WARPS) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    abort_flag = 0;
    for (uint64_t *b : {&full_a, &full_b, &full_ds, &g1, &g2, &g3, &drain}) mbar_init(b, 1);
    for (uint64_t *b : {&cleared, &qk_read, &tiles, &left}) mbar_init(b, GRAD_WARPS);
    fence_mbar_init();
  }
  follow_wait();
  fence_async_all();  // what the kernel before wrote with plain stores is read by copies here
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base, sb = smem_u32(sm);
  const uint32_t q = sb + L_::QK, k = q + 8192, x1 = sb + L_::X1, x2 = sb + L_::X2, e = sb + L_::E, si = sb + L_::S, ds = sb + L_::DS;
  // the first used unit from u on (units of unused slots are passed over)
  const uint32_t H = (uint32_t)a.H, units = (uint32_t)a.units;
  auto find = [&](uint32_t u, int64_t &tok, int &L) -> uint32_t {
    while (u < units && !chunk_in_slot(a.docs, u / H, tok, L)) u += gridDim.x;
    return u;
  };
  bool ok = true;
  int64_t tok = 0;
  int L = 0;
  if (warp >= GRAD_WARPS) {
    fewer_registers<64>();
    if (warp == GRAD_WARPS && lane == 0) {
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.dO);
      int loads_a = 0, loads_b = 0, loads_ds = 0;
      auto load_a = [&](uint32_t unit) {  // all but the low part of S0
        const int64_t u = unit;
        const int h = (int)(unit % H), hq = h / a.share;
        mbar_expect_tx(&full_a, E_IMAGE + S_IMAGE / 2 + 3 * 32768);
        bulk_load(sm + L_::E, a.e_images + u * E_IMAGE, E_IMAGE, &full_a);
#pragma unroll
        for (int cb = 0; cb < 2; ++cb) {
          tma_load_3d(sm + L_::QK + cb * 16384, &maps.q, cb * 64, hq, (int)tok, &full_a);
          tma_load_3d(sm + L_::QK + cb * 16384 + 8192, &maps.k, cb * 64, hq, (int)tok, &full_a);
          tma_load_3d(sm + L_::X1 + cb * 16384, &maps.dO, cb * 64, h, (int)tok, &full_a);
          tma_load_3d(sm + L_::X2 + cb * 16384, &maps.dO, cb * 64, h, (int)tok, &full_a);
          bulk_load(sm + L_::X1 + cb * 16384 + 8192, a.r_images + u * R_IMAGE + cb * 8192, 8192, &full_a);
          bulk_load(sm + L_::X2 + cb * 16384 + 8192, a.r_images + u * R_IMAGE + 16384 + cb * 8192, 8192, &full_a);
        }
        bulk_load(sm + L_::S, a.s_images + u * S_IMAGE, S_IMAGE / 2, &full_a);
        bulk_prefetch_l2(a.s_images + u * S_IMAGE + S_IMAGE / 2, S_IMAGE / 2);
        bulk_prefetch_l2(a.ds_images + u * S_IMAGE, S_IMAGE);
        ++loads_a;
      };
      auto load_b = [&](uint32_t unit) {
        mbar_expect_tx(&full_b, S_IMAGE / 2);
        bulk_load(sm + L_::S + S_IMAGE / 2, a.s_images + (int64_t)unit * S_IMAGE + S_IMAGE / 2, S_IMAGE / 2, &full_b);
        ++loads_b;
      };
      constexpr uint32_t idQK = idesc_bf16(128, 64, false, false), idB = idesc_bf16(128, 128, false, true);
      constexpr uint32_t idKN = idesc_bf16(128, 64, true, false), idMN = idesc_bf16(128, 64, true, true);
      constexpr uint32_t idKN2 = idesc_bf16(128, 128, true, false), idMN2 = idesc_bf16(128, 128, true, true);
      const uint32_t dp = sb + L_::T, da = dp + 2 * TILE;
      uint32_t u = find(blockIdx.x, tok, L);
      if (u < units) load_a(u);
      for (int it = 0; u < units; ++it) {
        const uint32_t ph = (uint32_t)it & 1u;
        // the last unit's gradients have left (S0's low part and tensor memory are free)
        if (it >= 1 && !(ok = mbar_wait(&left, ph ^ 1u, WAIT_CYCLES))) break;
        load_b(u);
        ok = mbar_wait(&full_a, ph, WAIT_CYCLES) && mbar_wait(&cleared, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_QK, kdesc(q, ks, 128), kdesc(k, ks, 128), idQK, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_B, kdesc(x1, ks, 128), image_desc(e, ks), idB, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_B, kdesc(x2, ks, 128), image_desc(e, ks), idB, 1);
        mma_commit(&g1);
        // S0 hi [dO | dR hi], S0 hi dR lo, S0 lo [dO | dR hi]
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_1, image_desc(si, ks), kdesc(x1, ks, 128), idKN2, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_2, image_desc(si, ks), kdesc(x2 + 8192, ks, 128), idKN, 1);
        if (!(ok = mbar_wait(&full_b, ph, WAIT_CYCLES))) break;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_1, image_desc(si + S_IMAGE / 2, ks), kdesc(x1, ks, 128), idKN2, 1);
        mma_commit(&g2);
        if (!(ok = mbar_wait(&g2, ph, WAIT_CYCLES))) break;
        mbar_expect_tx(&full_ds, S_IMAGE);
        bulk_load(sm + L_::DS, a.ds_images + (int64_t)u * S_IMAGE, S_IMAGE, &full_ds);
        ++loads_ds;
        if (!(ok = mbar_wait(&full_ds, ph, WAIT_CYCLES) && mbar_wait(&tiles, ph, WAIT_CYCLES))) break;
        tc_fence_after();
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16(tb + Q_4, mdesc(k, ks, 16384), kdesc(dp + p * TILE, ks, 64), idKN, p | ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16(tb + Q_5, mdesc(q, ks, 16384), mdesc(dp, ks, TILE), idMN2, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16(tb + Q_5, mdesc(k, ks, 16384), mdesc(da, ks, TILE), idMN2, 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16(tb + Q_5, mdesc(k, ks, 16384), kdesc(da, ks, 128), idKN2, 1);
        // dS1 (there when the tiles are) hi [E hi | E lo], dS1 lo E hi
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_3, image_desc(ds, ks), image_desc(e, ks), idMN2, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16(tb + Q_3, image_desc(ds + S_IMAGE / 2, ks), image_desc(e, ks), idMN, 1);
        mma_commit(&g3);
        u = find(u + gridDim.x, tok, L);
        if (!(ok = mbar_wait(&g3, ph, WAIT_CYCLES) && mbar_wait(&qk_read, ph, WAIT_CYCLES))) break;
        if (u < units) load_a(u);
      }
      if (!ok) {  // nothing of this block's is in flight when it leaves
        if (loads_a) mbar_wait(&full_a, (uint32_t)(loads_a - 1) & 1u, WAIT_CYCLES);
        if (loads_b) mbar_wait(&full_b, (uint32_t)(loads_b - 1) & 1u, WAIT_CYCLES);
        if (loads_ds) mbar_wait(&full_ds, (uint32_t)(loads_ds - 1) & 1u, WAIT_CYCLES);
        mma_commit(&drain);
        mbar_wait(&drain, 0, WAIT_CYCLES);
        atomicExch(&abort_flag, 1);
      }
    }
    __syncwarp();
  } else {
    more_registers<104>();
    // thread (row of the stack, later key channel: lane of tensor memory; 16 of the columns, tokens)
    const int grp = warp >> 2, qw = warp & 3, row = qw * 32 + lane, t = row & 63, c0 = 16 * grp;
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    const bool isA = qw >= 2;
    // the next unit, its tokens and gates, looked up while this one is worked on
    uint32_t next = 0;
    int64_t tok_next = 0;
    int L_next = 0;
    float g_next = 0.f, b_next = 0.f;
    auto look = [&](uint32_t from) {
      next = find(from, tok_next, L_next);
      g_next = b_next = 0.f;
      if (next < units && tid < CH && tid < L_next) {
        const int64_t at = (tok_next + tid) * a.H + next % H;
        g_next = a.g[at];
        b_next = a.beta[at];
      }
    };
    look(blockIdx.x);
    for (int it = 0; next < units; ++it) {
      const uint32_t ph = (uint32_t)it & 1u, u = next;
      const int h = (int)(u % H);
      tok = tok_next;
      L = L_next;
      // decays, while the copies run
      double G = (double)log_decay(g_next) * 1.4426950408889634;
      const float b = b_next;
      if (tid < CH) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, G, o);
          if (lane >= o) G += y;
        }
        if (tid == 31) warp0_total = G;
      }
      if (tid < CH) {
        named_bar(3, CH);
        if (warp == 1) G += warp0_total;
        const float gh = (float)G;
        s_g[tid] = make_float4(gh, (float)(G - (double)gh), b, 0.f);
        named_bar(3, CH);
        const float4 x = s_g[tid], z = s_g[63];
        const float into = pow2(x.x + x.y), out = pow2((z.x - x.x) + (z.y - x.y));
        s_into[tid] = a.scale * into;
        s_ki[tid] = -into * b;
        s_ko[tid] = out * b;
        if (tid == 63) s_over[ph] = into;
      }
      if (L < CH) {  // rows past the end hold other tokens: as zeros, nothing in them reaches a sum
        ok = ok && mbar_wait(&full_a, ph, WAIT_CYCLES);
        for (int n = tid; n < (CH - L) * 8 * 8; n += 32 * GRAD_WARPS) {  // q, k (four tiles), dO (twice two)
          const int c = n % 8, x = n / 8 % 8, r = L + n / 64;
          st_shared_v4(sb + (x < 4 ? L_::QK + x * 8192u : L_::X1 + (x - 4) * 16384u) + r * 128u + c * 16u, 0u, 0u, 0u, 0u);
        }
        fence_async_smem();
      }
      warp_arrive(&cleared);
      named_bar(1, 32 * GRAD_WARPS);  // the decays are there, the last unit's sums have been read
      ok = ok && mbar_wait(&g1, ph, WAIT_CYCLES);
      tc_fence_after();
      float w[16];
      uint32_t hi[8], lo[8];
      {
        uint32_t x[16], y[16];
        tmem_ld16(tb + lanes + Q_B + c0, x);
        tmem_ld16(tb + lanes + Q_B + 64u + c0, y);
        tmem_ld_wait(x);
        tmem_tie(y);
        const float4 gt = s_g[t];
        const float f = isA ? -gt.z : 0.5f * a.scale;
        const int last = t < L ? (isA ? t - 1 : t) : -1;
        if (c0 <= (t | 31)) {  // for the warp: one of its rows reaches these columns
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const int c = c0 + n;
            const float B = __uint_as_float(x[n]) + __uint_as_float(y[n]);
            if (isA && c == t) s_db[t] = B;
            const float4 gc = s_g[c];
            w[n] = c <= last ? f * gc.z * pow2((gt.x - gc.x) + (gt.y - gc.y)) * B : 0.f;
          }
        } else {
#pragma unroll
          for (int n = 0; n < 16; ++n) w[n] = 0.f;
        }
        tmem_ld16(tb + lanes + Q_QK + c0, x);
        tmem_ld_wait(x);
        tc_fence_before();
#pragma unroll
        for (int n = 0; n < 8; ++n) split2(w[2 * n], w[2 * n + 1], hi[n], lo[n]);
#pragma unroll
        for (int n = 0; n < 16; ++n) w[n] = c0 + n < t ? w[n] * __uint_as_float(x[n]) : 0.f;
      }
      look(u + gridDim.x);
      // sums of the pairs r >= t > s, dPd's part and dA's each by itself: along the row, then down the columns
#pragma unroll
      for (int n = 1; n < 16; ++n) w[n] += w[n - 1];
      s_tot[row][grp] = w[15];
      named_bar(1, 32 * GRAD_WARPS);
      {
        const float4 tot = *reinterpret_cast<const float4 *>(s_tot[row]);
        const float before = (grp > 0 ? tot.x : 0.f) + (grp > 1 ? tot.y : 0.f) + (grp > 2 ? tot.z : 0.f);
        // token c + 1 takes the sums up to column c of the rows from it on
#pragma unroll
        for (int n = 0; n < 16; ++n) w[n] = t > c0 + n ? w[n] + before : 0.f;
#pragma unroll
        for (int n = 0; n < 16; ++n) w[n] += __shfl_xor_sync(0xffffffffu, w[n], 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) {
          const bool up = (lane & o) != 0;
#pragma unroll
          for (int n = 0; n < o; ++n) {
            const float y = __shfl_xor_sync(0xffffffffu, up ? w[n] : w[n + o], o);
            w[n] = (up ? w[n + o] : w[n]) + y;
          }
        }
        if (lane < 16 && c0 + lane + 1 < CH) s_pair[qw][c0 + lane + 1] = w[0];
        if (lane == 0 && grp == 0) s_pair[qw][0] = 0.f;
      }
      {  // <S0, dS1>; then the tiles in S0's place
        ok = ok && mbar_wait(&full_a, ph, WAIT_CYCLES) && mbar_wait(&full_b, ph, WAIT_CYCLES) &&
             mbar_wait(&full_ds, ph, WAIT_CYCLES);
        float dot = 0.f, low = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t at = tid * 16 + n * 8192;
          const uint4 sh = lds_u4(si + at), sl = lds_u4(si + S_IMAGE / 2 + at);
          const uint4 dh = lds_u4(ds + at), dl = lds_u4(ds + S_IMAGE / 2 + at);
          const uint32_t x[4] = {sh.x, sh.y, sh.z, sh.w}, y[4] = {sl.x, sl.y, sl.z, sl.w};
          const uint32_t v[4] = {dh.x, dh.y, dh.z, dh.w}, z[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            dot = fma_pairs(x[m], v[m], dot);
            low = fma_pairs(x[m], z[m], fma_pairs(y[m], v[m], low));
          }
        }
        named_bar(1, 32 * GRAD_WARPS);  // everyone has read S0
        const uint32_t tile = sb + L_::T + (isA ? 2 * TILE : 0);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t o = tile + sw128_off(t, c0 + 8 * n, 64);
          st_shared_v4(o, hi[4 * n], hi[4 * n + 1], hi[4 * n + 2], hi[4 * n + 3]);
          st_shared_v4(o + TILE, lo[4 * n], lo[4 * n + 1], lo[4 * n + 2], lo[4 * n + 3]);
        }
        fence_async_smem();
        warp_arrive(&tiles);
        dot += low;
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) s_dot[ph][warp] = dot;
      }
      // q and k of the thread's channel and tokens, before the next unit's take their place
      uint32_t qv[8], kv[8];
      {
        const ColBf16 cq(q, c0, row, 16384u), ck(k, c0, row, 16384u);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          qv[n] = (uint32_t)lds_u16(cq.at(2 * n)) | (uint32_t)lds_u16(cq.at(2 * n + 1)) << 16;
          kv[n] = (uint32_t)lds_u16(ck.at(2 * n)) | (uint32_t)lds_u16(ck.at(2 * n + 1)) << 16;
        }
        warp_arrive(&qk_read);
      }
      auto half_of = [](uint32_t x, int n) { return __uint_as_float(n & 1 ? x & 0xffff0000u : x << 16); };
      ok = ok && mbar_wait(&g3, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        // lane: key channel; tokens c0 .. c0 + 15
        const int ch = row;
        float rd[16], ad[16];  // what token t's query and key read of S0, what its key left in S1, of this channel
        const ColBf16 oq(sb + L_::OUT, c0, ch), ok_(sb + L_::OUT + 16384, c0, ch);
        float *fq = (float *)a.dq + ((tok + c0) * a.H + h) * (int64_t)a.K + ch;
        float *fk = (float *)a.dk + ((tok + c0) * a.H + h) * (int64_t)a.K + ch;
        const int64_t step = (int64_t)a.H * a.K;
        const int rows = PER_HEAD && ch < a.K ? L - c0 : 0;
        {
          uint32_t x[16], y[16];
          tmem_ld16(tb + lanes + Q_1 + c0, x);
          tmem_ld16(tb + lanes + Q_4 + c0, y);
          tmem_ld_wait(x);
          tmem_tie(y);
#pragma unroll
          for (int n = 0; n < 16; n += 4) {
            const float4 f4 = *reinterpret_cast<const float4 *>(s_into + c0 + n);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float qi = f[m] * __uint_as_float(x[n + m]);
              rd[n + m] = qi * half_of(qv[(n + m) / 2], m);
              const float dq = qi + __uint_as_float(y[n + m]);
              if (PER_HEAD) {
                if (n + m < rows) fq[(n + m) * step] = dq;
              } else {
                sts_u16(oq.at(n + m), f32_to_bf16_bits(dq));
              }
            }
          }
        }
#pragma unroll
        for (int n0 = 0; n0 < 16; n0 += 8) {
          uint32_t x[8], y[8], z[8];
          float ko[8];
          tmem_ld8(tb + lanes + Q_3 + c0 + n0, x);
          tmem_ld8(tb + lanes + Q_3 + 64u + c0 + n0, y);
          tmem_ld_wait8(x);
          tmem_ld_wait8(y);
#pragma unroll
          for (int n = 0; n < 8; n += 4) {
            const float4 f4 = *reinterpret_cast<const float4 *>(s_ko + c0 + n0 + n);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) ko[n + m] = f[m] * (__uint_as_float(x[n + m]) + __uint_as_float(y[n + m]));
          }
          tmem_ld8(tb + lanes + Q_2 + c0 + n0, x);
          tmem_ld8(tb + lanes + Q_5 + c0 + n0, y);
          tmem_ld8(tb + lanes + Q_5 + 64u + c0 + n0, z);
          tmem_ld_wait8(x);
          tmem_ld_wait8(y);
          tmem_ld_wait8(z);
#pragma unroll
          for (int n = 0; n < 8; n += 4) {
            const float4 f4 = *reinterpret_cast<const float4 *>(s_ki + c0 + n0 + n);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const int r = n0 + n + m;
              const float ki = f[m] * __uint_as_float(x[n + m]), kx = half_of(kv[r / 2], m);
              rd[r] = fmaf(kx, ki, rd[r]);
              ad[r] = kx * ko[n + m];
              const float dk = (ki + ko[n + m]) + (__uint_as_float(y[n + m]) + __uint_as_float(z[n + m]));
              if (PER_HEAD) {
                if (r < rows) fk[r * step] = dk;
              } else {
                sts_u16(ok_.at(r), f32_to_bf16_bits(dk));
              }
            }
          }
        }
        // summed over the warp's channels: lanes n and n + 16 get token c0 + n
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          rd[n] += __shfl_xor_sync(0xffffffffu, rd[n], 16);
          ad[n] += __shfl_xor_sync(0xffffffffu, ad[n], 16);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) {
          const bool up = (lane & o) != 0;
#pragma unroll
          for (int n = 0; n < o; ++n) {
            const float r1 = __shfl_xor_sync(0xffffffffu, up ? rd[n] : rd[n + o], o);
            const float r2 = __shfl_xor_sync(0xffffffffu, up ? ad[n] : ad[n + o], o);
            rd[n] = (up ? rd[n + o] : rd[n]) + r1;
            ad[n] = (up ? ad[n + o] : ad[n]) + r2;
          }
        }
        if (lane < 16) {
          s_red[0][qw][c0 + lane] = rd[0];
          s_red[1][qw][c0 + lane] = ad[0];
        }
      }
      tc_fence_before();
      // the gradients are in shared memory; everyone hears of a wait that ran out
      if (named_bar_any(1, 32 * GRAD_WARPS, !ok)) {
        ok = false;
        break;
      }
      if (!PER_HEAD) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int i = tid + 512 * (n & 1), r = i >> 4, c = (i & 15) * 8;
          if (r < L && c < a.K) {
            const uint4 x = lds_u4(sb + L_::OUT + (n >> 1) * 16384 + sw128_off(r, c, 64));
            __nv_bfloat16 *dst = (__nv_bfloat16 *)(n >> 1 ? a.dk : a.dq) + ((tok + r) * a.H + h) * (int64_t)a.K + c;
            st_global_v4(dst, x.x, x.y, x.z, x.w);
          }
        }
      }
      fence_async_smem();
      warp_arrive(&left);
      if (warp == GRAD_WARPS - 1) {  // not one of those that begin the next unit
        // tokens lane and lane + 32: sums over the tokens from them on of what is read, over those before of what is left
        float r0 = 0.f, r1 = 0.f, d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          r0 += s_red[0][n][lane];
          r1 += s_red[0][n][lane + 32];
          d0 += s_red[1][n][lane];
          d1 += s_red[1][n][lane + 32];
        }
        const float p0 = (s_pair[0][lane] + s_pair[1][lane]) + (s_pair[2][lane] + s_pair[3][lane]);
        const float p1 = (s_pair[0][lane + 32] + s_pair[1][lane + 32]) + (s_pair[2][lane + 32] + s_pair[3][lane + 32]);
        const float own0 = d0, own1 = d1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float a0 = __shfl_down_sync(0xffffffffu, r0, o), a1 = __shfl_down_sync(0xffffffffu, r1, o);
          const float b0 = __shfl_up_sync(0xffffffffu, d0, o), b1 = __shfl_up_sync(0xffffffffu, d1, o);
          if (lane + o < 32) r0 += a0, r1 += a1;
          if (lane >= o) d0 += b0, d1 += b1;
        }
        r0 += __shfl_sync(0xffffffffu, r1, 0);
        d1 += __shfl_sync(0xffffffffu, d0, 31);
        float over = 0.f;
#pragma unroll
        for (int n = 0; n < GRAD_WARPS; ++n) over += s_dot[ph][n];
        over *= s_over[ph];
        if (lane < L) {
          a.dg[(tok + lane) * a.H + h] = (p0 + over) + (r0 + (d0 - own0));
          a.dbeta[(tok + lane) * a.H + h] = s_db[lane];
        }
        if (lane + 32 < L) {
          a.dg[(tok + lane + 32) * a.H + h] = (p1 + over) + (r1 + (d1 - own1));
          a.dbeta[(tok + lane + 32) * a.H + h] = s_db[lane + 32];
        }
      }
    }
    if (!ok) atomicExch(&abort_flag, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *(volatile int *)&abort_flag) set_device_error(a.err, GLACORE_ERR_TIMEOUT);
  if (warp == GRAD_WARPS) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

inline size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

bool tc_supported(const glacore_problem *p) {
  return p->dtype == GLACORE_BF16 && p->K % 8 == 0 && p->V % 8 == 0 && p->K <= D128 && p->V <= D128 &&
         p->q_stride % 8 == 0 && p->k_stride % 8 == 0 && p->v_stride % 8 == 0 && p->B * p->T < ((int64_t)1 << 31) - CH &&
         !(((uintptr_t)p->q | (uintptr_t)p->k | (uintptr_t)p->v) & 15);
}
bool tc_padded(const glacore_problem *p) {
  return p->dtype == GLACORE_BF16 && p->K <= D128 && p->V <= D128 && p->B * p->T < ((int64_t)1 << 31) - CH &&
         !tc_supported(p);
}

// Scratch (byte offsets): tiles and gates of every chunk and head, the backward's images.
namespace {
struct TcLayout {
  size_t order, flags, tiles, gates, s, ds, e, r, total;
};
TcLayout tc_layout(int64_t docs, int64_t slots, int64_t H, bool backward) {
  TcLayout l;
  memset(&l, 0, sizeof(l));
  size_t off = al256((size_t)docs * sizeof(int32_t));
  auto take = [&](size_t &at, size_t each) {
    at = off;
    off = al256(off + (size_t)slots * H * each);
  };
  take(l.tiles, TILES);
  take(l.gates, GATES * sizeof(float));
  if (!backward) {  // a flag per chunk and head
    l.flags = off;
    off = al256(off + (size_t)slots * H * sizeof(uint32_t));
  }
  if (backward) {
    take(l.s, S_IMAGE);
    take(l.ds, S_IMAGE);
    take(l.e, E_IMAGE);
    take(l.r, R_IMAGE);
  }
  l.total = off;
  return l;
}

struct Maps {
  CUtensorMap q, k, v, dO;
};
cudaError_t make_maps(const Call &c, const void *dO, Maps &m) {
  if (const cudaError_t e = bind_context()) return e;
  memset(&m, 0, sizeof(m));
  const bool ok = make_map(&m.q, c.p.q, true, c.p.K, c.p.Hqk, c.p.BT, 64, c.p.qs) &&
                  make_map(&m.k, c.p.k, true, c.p.K, c.p.Hqk, c.p.BT, 64, c.p.ks) &&
                  make_map(&m.v, c.p.v, true, c.p.V, c.p.H, c.p.BT, 64, c.p.vs) &&
                  (!dO || make_map(&m.dO, dO, true, c.p.V, c.p.H, c.p.BT, 64));
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}
// follow: the kernel begins while the last one ends, and waits for it (follow_wait); together: all blocks at once.
enum class Start { behind, follow, together };
template <auto kernel, typename M, typename A>
cudaError_t launch(int64_t blocks, int threads, uint32_t smem, const Call &c, const M &maps, const A &a,
                   const char *label, Start start) {
  if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  // shared memory is asked for once per kernel and device (the answer is the same for every call)
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.st;
  cudaLaunchAttribute attr[1];
  if (start == Start::together) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = start == Start::behind ? 0 : 1;
  const cudaError_t r = cudaLaunchKernelEx(&cfg, kernel, maps, a);
  if (r == cudaSuccess) mark_launch(label, c.st);
  return r;
}
// Whether a stream's kernels may run on all SMs of the device: not one that a
// partition of it (a green context) made.
bool on_all_sms(cudaStream_t st) {
  typedef CUresult(CUDAAPI * Fn)(CUstream, CUgreenCtx *);
  static const Fn partition_of = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuStreamGetGreenCtx", &p, 12040, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? (Fn)p : nullptr;
  }();
  CUgreenCtx partition = nullptr;
  return !partition_of || (partition_of((CUstream)st, &partition) == CUDA_SUCCESS && !partition);
}
PrepArgs prep_args(const Call &c, char *ws, const TcLayout &l) {
  PrepArgs a;
  a.g = c.p.g;
  a.beta = c.beta;
  a.docs = c.docs;
  a.H = (int)c.p.H;
  a.Hqk = (int)c.p.Hqk;
  a.share = a.H / a.Hqk;
  a.scale = c.p.scale;
  a.tiles = ws + l.tiles;
  a.gates = (float *)(ws + l.gates);
  a.err = c.p.err;
  return a;
}
cudaError_t prep(const Call &c, const Maps &m, char *ws, const TcLayout &l) {
  return launch<delta_prep_kernel>(c.slots * c.p.Hqk, PREP_THREADS, PREP_BYTES, c, PrepMaps{m.q, m.k}, prep_args(c, ws, l),
                                   "delta_prep", Start::behind);
}
// Packed documents that do not all run at once: the longest first, so that none
// of them is begun when the others are done.
cudaError_t launch_order(const Call &c, int64_t blocks, char *ws, const int32_t *&order) {
  if (!c.docs.start || blocks <= tc::sm_count()) return cudaSuccess;
  Units u;
  memset(&u, 0, sizeof(u));
  u.docs = c.docs;
  order = (const int32_t *)ws;
  return tc::launch_order_units(u, c.docs.n, (int32_t *)ws, c.st);
}
// Whether the tiles of the forward are made while the chains walk: sequences
// of one length on at most half of the SMs (of packed documents the longest
// would wait for the others' tiles), where what the tiles take alone, 0.019 us
// a chunk and head, is more than what the walk loses, 0.4 us a chunk (its
// copies wait for flags), and 2 to 6 us to begin with.  Heads x sequences, tokens,
// us one after the other / at once: 64 x 2048: 165 / 137; 64 x 8192: 612 / 475; 76 x
// 2048: 173 / 142; 64 x 640: 60 / 58; but 64 x 512: 49 / 50, 16 x 2048: 132 / 133,
// 16 x 512: 41 / 49, 16 x 96: 21 / 27.
bool overlaps(const Call &c, int64_t units) {
  return !c.docs.start && units <= tc::sm_count() / 2 && (units - 24) * ((c.docs.T + CH - 1) / CH) > 320 &&
         c.slots * c.p.H < ((int64_t)1 << 31);
}
ChainArgs chain_args(const Call &c, char *ws, const TcLayout &l) {
  ChainArgs a;
  memset(&a, 0, sizeof(a));
  a.docs = c.docs;
  a.H = (int)c.p.H;
  a.share = (int)(c.p.H / c.p.Hqk);
  a.V = (int)c.p.V;
  a.sK = (int)c.sK;
  a.sV = (int)c.sV;
  a.scale = c.p.scale;
  a.h0 = c.p.h0;
  a.tiles = ws + l.tiles;
  a.gates = (const float *)(ws + l.gates);
  a.err = c.p.err;
  return a;
}
}  // namespace

size_t tc_workspace(int64_t docs, int64_t slots, int64_t H, bool backward) {
  return tc_layout(docs, slots, H, backward).total;
}

cudaError_t tc_fwd(const Call &c, void *o, float *ht, char *ws) {
  const TcLayout l = tc_layout(c.docs.n, c.slots, c.p.H, false);
  Maps m;
  const int32_t *order = nullptr;
  cudaError_t e = make_maps(c, nullptr, m);
  const int64_t units = c.docs.n * c.p.H;
  ChainArgs a = chain_args(c, ws, l);
  a.o = (__nv_bfloat16 *)o;
  a.ht = ht;
  if (e == cudaSuccess && overlaps(c, units) && on_all_sms(c.st)) {
    OverlapArgs x;
    x.chain = a;
    x.prep = prep_args(c, ws, l);
    x.flags = (uint32_t *)(ws + l.flags);
    x.units = (uint32_t)units;
    x.chain.flags = x.flags;
    x.makers = (uint32_t)std::min(tc::sm_count() - units, (c.slots * c.p.H + TEAMS - 1) / TEAMS);
    e = cudaMemsetAsync(x.flags, 0, (size_t)(c.slots * c.p.H) * sizeof(uint32_t), c.st);
    if (e == cudaSuccess)
      e = launch<delta_overlap_kernel>(x.makers + units, CHAIN_THREADS, ChainSmem<false>::BYTES, c,
                                       OverlapMaps{{m.q, m.k, m.v}, {m.q, m.k}}, x, "delta_overlap", Start::together);
    // fewer SMs than the device has are to be had (a share of them): one kernel after the other
    if (e != cudaErrorCooperativeLaunchTooLarge) return e;
    cudaGetLastError();
    e = cudaSuccess;
  }
  if (e == cudaSuccess) e = launch_order(c, units, ws + l.order, order);
  if (e == cudaSuccess) e = prep(c, m, ws, l);
  if (e != cudaSuccess) return e;
  a.order = order;
  return launch<delta_chain_kernel>(units, CHAIN_THREADS, ChainSmem<false>::BYTES, c,
                ChainMaps{m.q, m.k, m.v}, a, "delta_chain", Start::follow);
}

cudaError_t tc_bwd(const Call &c, const void *dO, const float *dht, void *dq, void *dk, bool per_head, void *dv, float *dg,
                   float *dbeta, float *dh0, char *ws) {
  const TcLayout l = tc_layout(c.docs.n, c.slots, c.p.H, true);
  Maps m;
  const int32_t *order = nullptr;
  cudaError_t e = make_maps(c, dO, m);
  if (e == cudaSuccess) e = launch_order(c, 2 * c.docs.n * c.p.H, ws + l.order, order);
  if (e == cudaSuccess) e = prep(c, m, ws, l);
  if (e != cudaSuccess) return e;
  ChainArgs a = chain_args(c, ws, l);
  a.order = order;
  a.s_images = ws + l.s;
  a.e_images = ws + l.e;
  BackArgs b;
  b.docs = a.docs;
  b.order = order;
  b.H = a.H;
  b.share = a.share;
  b.V = a.V;
  b.sK = a.sK;
  b.sV = a.sV;
  b.scale = a.scale;
  b.dht = dht;
  b.dh0 = dh0;
  b.dv = (__nv_bfloat16 *)dv;
  b.tiles = a.tiles;
  b.gates = a.gates;
  b.ds_images = ws + l.ds;
  b.r_images = ws + l.r;
  b.err = a.err;
  const int64_t units = c.docs.n * c.p.H;
  e = launch<delta_walks_kernel>(2 * units, CHAIN_THREADS, std::max(ChainSmem<true>::BYTES, BackSmem::BYTES), c,
             WalkMaps{{m.q, m.k, m.v}, {m.q, m.k, m.dO}}, WalkArgs{a, b, units}, "delta_walks", Start::follow);
  if (e != cudaSuccess) return e;
  GradArgs g;
  g.docs = a.docs;
  g.H = a.H;
  g.share = a.share;
  g.K = (int)c.p.K;
  g.scale = a.scale;
  g.g = c.p.g;
  g.beta = c.beta;
  g.s_images = a.s_images;
  g.ds_images = b.ds_images;
  g.e_images = a.e_images;
  g.r_images = b.r_images;
  g.dq = dq;
  g.dk = dk;
  g.dg = dg;
  g.dbeta = dbeta;
  g.err = a.err;
  g.units = c.slots * c.p.H;
  const int64_t blocks = std::min(g.units, tc::sm_count());
  return per_head ? launch<delta_grads_kernel<true>>(blocks, GRAD_THREADS, GradSmem::BYTES, c, GradMaps{m.q, m.k, m.dO}, g,
                           "delta_grads", Start::follow)
                  : launch<delta_grads_kernel<false>>(blocks, GRAD_THREADS, GradSmem::BYTES, c, GradMaps{m.q, m.k, m.dO}, g,
                           "delta_grads", Start::follow);
}

}  // namespace delta
}  // namespace glacore
