// delta_tc.cu -- the gated delta rule on the tensor cores (formulas in
// delta.cuh): bf16, K and V multiples of 8 up to 128 (read as 128, the missing
// channels zero-filled by TMA), chunks of C = 64 tokens.
//
// Precision.  q, k, v and do are bf16 and enter products as they are.  Every
// matrix that is computed (the state, Z, P, R = b Y, U) enters a product in
// two bf16 parts, x = hi + lo to 2^-17 of x, and a product of two such matrices
// as hi hi + hi lo + lo hi; sums and the state itself are fp32.  With one part
// the outputs are off by 3e-3, twice what rounding them to bf16 costs,
// with two by 5e-6.  Where Z's rows are long (sum of |Z_ts| b_s above WIDE: keys
// that nearly coincide, written with b near 2), Y + Z (b Y) cancels and what Z
// and b Y are off by counts that much more: in such a chunk that product takes
// both in three parts (exact to 2^-25).  Chunks of unit keys that differ and b up to 1
// stay below 10.
//
// delta_prep_kernel makes of every chunk by itself what the recurrence over
// chunks needs: Z and P (two 64 x 64 tiles each, laid out as the matrix
// operands that they become) and the chunk's decays.  delta_chain_kernel walks
// the chunks of one (document, head) with the state on chip.
#include <string.h>

#include <algorithm>

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
constexpr float WIDE = 16.f;
constexpr int NP = 68;                          // row pitch of the fp32 64 x 64 matrices

// hi and lo parts of two neighbours, packed
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(a, b);
  lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
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
// blocks of 32: the diagonal ones by forward substitution, a thread per column in
// registers, and with (I + N b)^-1 = I + Z b
//     Z21 = W + Z22 (b W),   W = -(N21 + N21 (b Z11)).
// Decays are e^{G_t - G_s} of the difference itself, G kept in two fp32 parts, so that
// neither a strong decay nor a long chunk costs digits.
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
  float N[CH][NP], Z[CH][NP], W[32][36];
  float Gh[CH], Gl[CH], beta[CH];
};
constexpr uint32_t PREP_BYTES = 32768 + sizeof(PrepSmem) + 1024;

__global__ void __launch_bounds__(128) delta_prep_kernel(const __grid_constant__ PrepMaps maps, const PrepArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);  // [q; k] tiles, then Z and P
  PrepSmem &s = *reinterpret_cast<PrepSmem *>(sm + 32768);
  __shared__ uint64_t full, done;
  __shared__ uint32_t tmem_base;
  __shared__ double warp0_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hq = (int)(blockIdx.x % a.Hqk);
  const int64_t slot = blockIdx.x / a.Hqk;
  int64_t tok;
  int L;
  if (!chunk_in_slot(a.docs, slot, tok, L)) return;
  if (warp == 0) {
    tmem_alloc(&tmem_base, 64);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&full, 1);
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base;
  bool ok = true;
  if (tid == 0) {
    mbar_expect_tx(&full, 32768);
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {  // 64 channels: 64 rows of q, then 64 of k
      tma_load_3d(sm + cb * 16384, &maps.q, cb * 64, hq, (int)tok, &full);
      tma_load_3d(sm + cb * 16384 + 8192, &maps.k, cb * 64, hq, (int)tok, &full);
    }
    ok = mbar_wait(&full, 0, WAIT_CYCLES);
    const uint32_t base = smem_u32(sm);
    if (ok) {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_bf16(tb, kdesc(base, ks, 128), kdesc(base + 8192, ks, 128), idesc_bf16(128, 64, false, false), ks);
    }
    mma_commit(&done);
  }
  ok = mbar_wait(&done, 0, WAIT_CYCLES) && ok;
  ok = !__syncthreads_or(!ok);
  if (ok) {
    tc_fence_after();
    // thread tid < 64: row tid of Q K^T; else row tid - 64 of K K^T
    uint32_t r0[32], r1[32];
    const uint32_t at = tb + ((uint32_t)(warp * 32) << 16);
    tmem_ld32(at, r0);
    tmem_ld32(at + 32, r1);
    tmem_ld_wait32(r0);
    tmem_ld_wait32(r1);
    const int t = tid & 63;
    for (int e = 0; e < a.share; ++e) {
      const int h = hq * a.share + e;
      const int64_t sh = slot * a.H + h;
      if (e) {  // the tiles of the last head have left shared memory
        if (tid == 0) bulk_wait_read_all();
        __syncthreads();
      }
      double G = 0.0;
      float b = 0.f;
      if (tid < 64) {
        if (t < L) {
          G = (double)fmaxf(a.g[(tok + t) * a.H + h], -1e4f);  // e^g of less is 0 as well
          b = a.beta[(tok + t) * a.H + h];
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, G, o);
          if (lane >= o) G += y;
        }
        if (tid == 31) warp0_total = G;
      }
      __syncthreads();
      if (tid < 64) {
        if (warp == 1) G += warp0_total;
        s.Gh[t] = (float)G;
        s.Gl[t] = (float)(G - (double)(float)G);
        s.beta[t] = b;
      }
      __syncthreads();
      const float gh = s.Gh[t], gl = s.Gl[t];
      if (tid < 64) {
        float *gs = a.gates + sh * GATES;
        gs[G_INTO + t] = expf(gh + gl);
        gs[G_OUT + t] = expf((s.Gh[63] - gh) + (s.Gl[63] - gl));  // tokens past the end add no decay
        gs[G_BETA + t] = b;
        if (t == 0) gs[G_OVER] = expf(s.Gh[63] + s.Gl[63]);
      }
      // row t, columns s <= t (P) or s < t (N): scale D (.) QK^T, D (.) KK^T
      const int last = t < L ? (tid < 64 ? t : t - 1) : -1;
      const float f = tid < 64 ? a.scale : 1.f;
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 8) {
        float x[8];
        const bool some = c0 <= (t | 31);  // for the warp: one of its rows reaches these columns
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = c0 + i;
          x[i] = 0.f;
          if (some && c <= last)
            x[i] = f * expf((gh - s.Gh[c]) + (gl - s.Gl[c])) * __uint_as_float(c < 32 ? r0[c & 31] : r1[c & 31]);
        }
        if (tid < 64) {
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
      if (warp >= 2) {  // Z of the diagonal blocks: warp 2 the first, warp 3 the second
        named_bar(1, 64);
        const int r = (warp - 2) * 32;
        float zb[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float z0 = -s.N[r + i][r + lane], z1 = 0.f;
#pragma unroll
          for (int c = 0; c < i; c += 4) {
            const float4 n = *reinterpret_cast<const float4 *>(&s.N[r + i][r + c]);
            z0 = fmaf(-n.x, zb[c], z0);
            if (c + 1 < i) z1 = fmaf(-n.y, zb[c + 1], z1);
            if (c + 2 < i) z0 = fmaf(-n.z, zb[c + 2], z0);
            if (c + 3 < i) z1 = fmaf(-n.w, zb[c + 3], z1);
          }
          const float z = z0 + z1;
          s.Z[r + i][r + lane] = z;
          zb[i] = z * s.beta[r + i];
        }
      }
      __syncthreads();
      const int j = lane, i0 = warp * 8;
      {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = -s.N[32 + i0 + i][j];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          float z[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) z[x] = s.beta[c + x] * s.Z[c + x][j];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 n = *reinterpret_cast<const float4 *>(&s.N[32 + i0 + i][c]);
            w[i] = fmaf(-n.x, z[0], fmaf(-n.y, z[1], fmaf(-n.z, z[2], fmaf(-n.w, z[3], w[i]))));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s.W[i0 + i][j] = w[i];
      }
      __syncthreads();
      {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = s.W[i0 + i][j];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          float z[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) z[x] = s.beta[32 + c + x] * s.W[c + x][j];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 n = *reinterpret_cast<const float4 *>(&s.Z[32 + i0 + i][32 + c]);
            w[i] = fmaf(n.x, z[0], fmaf(n.y, z[1], fmaf(n.z, z[2], fmaf(n.w, z[3], w[i]))));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s.Z[32 + i0 + i][j] = w[i];
          s.Z[i0 + i][32 + j] = 0.f;
        }
      }
      __syncthreads();
      float sum = 0.f;
      uint32_t third[16];
      const int row = tid >> 1, c1 = (tid & 1) * 32;
#pragma unroll
      for (int c0 = 0; c0 < 32; c0 += 8) {
        uint32_t hi[4], lo[4];
        float z[8];
        *reinterpret_cast<float4 *>(z) = *reinterpret_cast<const float4 *>(&s.Z[row][c1 + c0]);
        *reinterpret_cast<float4 *>(z + 4) = *reinterpret_cast<const float4 *>(&s.Z[row][c1 + c0 + 4]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(fabsf(z[i]), fabsf(s.beta[c1 + c0 + i]), sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          split2(z[2 * i], z[2 * i + 1], hi[i], lo[i]);
          third[c0 / 2 + i] = split3(z[2 * i], z[2 * i + 1], hi[i], lo[i]);
        }
        const uint32_t o = smem_u32(sm) + sw128_off(row, c1 + c0, 64);
        st_shared_v4(o, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(o + TILE, lo[0], lo[1], lo[2], lo[3]);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      const bool wide = __syncthreads_or(!(sum <= WIDE));
      if (wide) {  // the third part takes N's place
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(smem_u32(&s.N[0][0]) + sw128_off(row, c1 + 8 * i, 64), third[4 * i], third[4 * i + 1],
                       third[4 * i + 2], third[4 * i + 3]);
      }
      fence_async_smem();
      __syncthreads();
      if (tid == 0) {
        a.gates[sh * GATES + G_WIDE] = wide ? 1.f : 0.f;
        bulk_store(a.tiles + sh * TILES, sm, 4 * TILE);
        if (wide) bulk_store(a.tiles + sh * TILES + 4 * TILE, &s.N[0][0], TILE);
        bulk_commit();
      }
    }
    if (tid == 0) bulk_wait_all();
  } else if (tid == 0) {
    set_device_error(a.err, GLACORE_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tb, 64);
  }
}

// ---------------------------------------------------------------------------
// The recurrence over the chunks of one (document, head).  The state is kept
// transposed, value column v in lane v of tensor memory, so that every
// elementwise step belongs to one thread and no operand that the chain makes
// goes through shared memory:
//     X^T  = S^T k^T             A: S^T (hi, lo), B: k    -> Y = v - e^G X, R = b Y
//     E^T  = Y^T + R^T Z^T       A: R^T (hi, lo), B: Z    -> U = b E, U' = e^{G_C - G} U
//     S'^T = e^{G_C} S^T + U'^T k    A: U'^T (hi, lo), B: k (as rows of the contraction)
//     O^T  = scale e^G (S^T q^T) + U^T P^T
// 256 threads of 8 warps compute: thread (lane v, half w) holds 64 of the
// state's key rows of its column and 32 of the chunk's tokens; one thread of a ninth warp issues
// copies and products.  Three exchanges per chunk are in sequence (X, E, S');
// S^T q^T runs while R is made, U^T P^T while the state is updated, and o is
// stored while the next X runs.
// TMEM columns: [0, 128) S^T as hi / lo of rows 0..63, hi / lo of rows 64..127;
// the same columns take U'^T k, once X and S^T q^T have read S.
// ---------------------------------------------------------------------------
constexpr uint32_t T_S = 0, T_X = 128, T_QS = 192, T_R = 256, T_U2 = 320, T_U = 384, T_PU = 448;
constexpr uint32_t T_R3 = T_U2;  // R's third part, until U' is made

struct ChainMaps {
  CUtensorMap q, k, v;
};
struct ChainArgs {
  Docs docs;
  int H, share, K, V;
  float scale;
  const float *h0;
  float *ht;
  __nv_bfloat16 *o;
  const char *tiles;
  const float *gates;
  int *err;
};
namespace cs {  // shared memory: two stages, the output tile
constexpr uint32_t KQ = 0, V = 32768, ZP = 49152, GT = 90112, STAGE = 91136;  // GT: 1 KB
constexpr uint32_t STAGES = 2;
constexpr uint32_t O = STAGES * STAGE;  // 16 KB
constexpr uint32_t BYTES = O + 16384 + 1024;
}  // namespace cs
static_assert(cs::STAGE % 1024 == 0 && cs::O % 1024 == 0, "tiles are 1024-byte aligned");
constexpr int CHAIN_THREADS = 288;

__global__ void __launch_bounds__(CHAIN_THREADS, 1) delta_chain_kernel(const __grid_constant__ ChainMaps maps,
                                                                       const ChainArgs a) {
  using namespace cs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[STAGES], s_ready, x_full, r_ready, e_full, u_ready, s_full, pu_full, o_free, drain;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (int)(blockIdx.x % a.H);
  const int64_t d = blockIdx.x / a.H;
  int64_t s0, s1;
  a.docs.range(d, s0, s1);
  const int nch = (int)((s1 - s0 + CH - 1) / CH);
  const int64_t slot0 = a.docs.chunk_base(d);
  auto chunk_tok = [&](int j) -> int64_t { return s0 + (int64_t)j * CH; };
  auto chunk_len = [&](int j) -> int { return (int)min((int64_t)CH, s1 - chunk_tok(j)); };

  if (warp == 8) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (uint32_t i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
    mbar_init(&x_full, 1);
    mbar_init(&e_full, 1);
    mbar_init(&s_full, 1);
    mbar_init(&pu_full, 1);
    mbar_init(&drain, 1);
    mbar_init(&s_ready, 256);
    mbar_init(&r_ready, 256);
    mbar_init(&u_ready, 256);
    mbar_init(&o_free, 256);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base;
  const uint32_t sb = smem_u32(sm);

  if (warp == 8) {
    if (lane == 0) {
      const int hq = h / a.share;
      tma_prefetch_desc(&maps.q);
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
      int loaded = 0;
      // whether chunk j is a wide one, read a chunk ahead of its copies
      auto wide_of = [&](int j) -> float { return j < nch ? ldg_early(a.gates + ((slot0 + j) * a.H + h) * GATES + G_WIDE) : 0.f; };
      float wide_next = wide_of(0);
      auto load = [&](int j) {
        const uint32_t st = (uint32_t)j % STAGES;
        uint8_t *p = sm + st * STAGE;
        const int tok = (int)chunk_tok(j);
        const bool wide = wide_next != 0.f;
        wide_next = wide_of(j + 1);
        mbar_expect_tx(&full[st], wide ? STAGE : STAGE - TILE);
        tma_load_3d(p + KQ, &maps.k, 0, hq, tok, &full[st]);
        tma_load_3d(p + KQ + 8192, &maps.q, 0, hq, tok, &full[st]);
        tma_load_3d(p + KQ + 16384, &maps.k, 64, hq, tok, &full[st]);
        tma_load_3d(p + KQ + 24576, &maps.q, 64, hq, tok, &full[st]);
        tma_load_3d(p + V, &maps.v, 0, h, tok, &full[st]);
        tma_load_3d(p + V + 8192, &maps.v, 64, h, tok, &full[st]);
        const int64_t sh = (slot0 + j) * a.H + h;
        bulk_load(p + ZP, a.tiles + sh * TILES, wide ? TILES : 4 * TILE, &full[st]);
        bulk_load(p + GT, a.gates + sh * GATES, GATES * 4, &full[st]);
        loaded = j + 1;
      };
      constexpr uint32_t id64 = idesc_bf16(128, 64, false, false), idS = idesc_bf16(128, 128, false, true);
      // columns of K-step ks of S^T (hi), of a 64-token operand
      auto sA = [&](int ks) { return tb + T_S + (uint32_t)(ks >> 2) * 64u + (uint32_t)(ks & 3) * 8u; };
      bool ok = true;
      for (int j = 0; j < nch && j < (int)STAGES - 1; ++j) load(j);
      for (int j = 0; ok && j < nch; ++j) {
        const uint32_t st = (uint32_t)j % STAGES, ph = (uint32_t)j & 1u;
        const uint32_t k = sb + st * STAGE + KQ, q = k + 8192, z = sb + st * STAGE + ZP, p = z + 2 * TILE;
        ok = ok && mbar_wait(&full[st], (uint32_t)(j / (int)STAGES) & 1u, WAIT_CYCLES) &&
             mbar_wait(&s_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(tb + T_X, sA(ks), kdesc(k, ks, 128), id64, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(tb + T_X, sA(ks) + 32u, kdesc(k, ks, 128), id64, 1);
        mma_commit(&x_full);
        // chunk j - 1 is done with its stage and with S^T q^T and U^T P^T
        if (j >= 1) ok = mbar_wait(&o_free, (uint32_t)(j - 1) & 1u, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
        if (j + 1 < nch) load(j + 1);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(tb + T_QS, sA(ks), kdesc(q, ks, 128), id64, ks);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(tb + T_QS, sA(ks) + 32u, kdesc(q, ks, 128), id64, 1);
        ok = mbar_wait(&r_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_X, tb + T_R + 8u * ks, kdesc(z, ks, 64), id64, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_X, tb + T_R + 32u + 8u * ks, kdesc(z, ks, 64), id64, 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_X, tb + T_R + 8u * ks, kdesc(z + TILE, ks, 64), id64, 1);
        if (lds_f1(sb + st * STAGE + GT + 4u * G_WIDE) != 0.f) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_bf16_ta(tb + T_X, tb + T_R + 32u + 8u * ks, kdesc(z + TILE, ks, 64), id64, 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_X, tb + T_R3 + 8u * ks, kdesc(z, ks, 64), id64, 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_X, tb + T_R + 8u * ks, kdesc(z + 4 * TILE, ks, 64), id64, 1);
        }
        mma_commit(&e_full);
        ok = mbar_wait(&u_ready, ph, WAIT_CYCLES);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_S, tb + T_U2 + 8u * ks, mdesc(k, ks, 16384), idS, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_S, tb + T_U2 + 32u + 8u * ks, mdesc(k, ks, 16384), idS, 1);
        mma_commit(&s_full);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_PU, tb + T_U + 8u * ks, kdesc(p, ks, 64), id64, ks);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_PU, tb + T_U + 32u + 8u * ks, kdesc(p, ks, 64), id64, 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_bf16_ta(tb + T_PU, tb + T_U + 8u * ks, kdesc(p + TILE, ks, 64), id64, 1);
        mma_commit(&pu_full);
      }
      // no copy or product of this block is in flight when it leaves
      for (int j = max(0, loaded - (int)STAGES); j < loaded; ++j)
        if (!mbar_wait(&full[j % (int)STAGES], (uint32_t)(j / (int)STAGES) & 1u, WAIT_CYCLES)) ok = false;
      mma_commit(&drain);
      if (!mbar_wait(&drain, 0, WAIT_CYCLES)) ok = false;
      if (!ok) atomicExch(&abort_flag, 1);
    }
    __syncwarp();
  } else {
    const int w = warp >> 2, qw = warp & 3, v = qw * 32 + lane;
    const uint32_t lo = (uint32_t)(qw * 32) << 16;  // this warp's lanes of tensor memory
    const bool in = v < a.V;
    float S[64];
    {
      const float *src = a.h0 && in ? a.h0 + ((d * a.H + h) * a.K + 64 * w) * (int64_t)a.V + v : nullptr;
#pragma unroll
      for (int i = 0; i < 64; ++i) S[i] = src && 64 * w + i < a.K ? src[(int64_t)i * a.V] : 0.f;
    }
    // S^T's hi and lo parts into tensor memory
    auto put_state = [&]() {
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t hi[16], l[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) split2(S[c + 2 * i], S[c + 2 * i + 1], hi[i], l[i]);
        tmem_st16(tb + lo + T_S + 64u * w + c / 2, hi);
        tmem_st16(tb + lo + T_S + 64u * w + 32u + c / 2, l);
      }
      tmem_st_wait();
      tc_fence_before();
    };
    // Rows past the document's end hold other tokens: as zeros, nothing in them reaches a sum.
    auto clear_rows = [&](int j) -> bool {
      const int L = chunk_len(j);
      if (L == CH) return true;
      const uint32_t st = (uint32_t)j % STAGES;
      if (!mbar_wait(&full[st], (uint32_t)(j / (int)STAGES) & 1u, WAIT_CYCLES)) return false;
      const int tid = threadIdx.x;
      for (int i = tid; i < (CH - L) * 48; i += 256) {  // rows of k, q (two blocks each) and v (two)
        const int r = L + i / 48, c = i % 48, b = c / 8;
        const uint32_t base = sb + st * STAGE + (b < 4 ? KQ + b * 8192u : V + (b - 4) * 8192u);
        st_shared_v4(base + r * 128u + (c % 8) * 16u, 0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      return true;
    };
    put_state();
    bool ok = nch == 0 || clear_rows(0);
    mbar_arrive(&s_ready);
    for (int j = 0; j < nch; ++j) {
      const uint32_t st = (uint32_t)j % STAGES, ph = (uint32_t)j & 1u;
      const uint8_t *sp = sm + st * STAGE;
      const float *gs = reinterpret_cast<const float *>(sp + GT);
      float Y[32];
      ok = ok && mbar_wait(&full[st], (uint32_t)(j / (int)STAGES) & 1u, WAIT_CYCLES);
      {
        const ColBf16 col(smem_u32(sp + V), 32 * w, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) Y[i] = bf16_bits_to_f32(lds_u16(col.at(i)));
      }
      ok = ok && mbar_wait(&x_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[32];
        tmem_ld32(tb + lo + T_X + 32u * w, x);
        tmem_ld_wait32(x);
        uint32_t hi[16], l[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 e = lds_f4(smem_u32(gs + G_INTO + 32 * w + i)), b = lds_f4(smem_u32(gs + G_BETA + 32 * w + i));
          Y[i] = fmaf(-e.x, __uint_as_float(x[i]), Y[i]);
          Y[i + 1] = fmaf(-e.y, __uint_as_float(x[i + 1]), Y[i + 1]);
          Y[i + 2] = fmaf(-e.z, __uint_as_float(x[i + 2]), Y[i + 2]);
          Y[i + 3] = fmaf(-e.w, __uint_as_float(x[i + 3]), Y[i + 3]);
          split2(b.x * Y[i], b.y * Y[i + 1], hi[i / 2], l[i / 2]);
          split2(b.z * Y[i + 2], b.w * Y[i + 3], hi[i / 2 + 1], l[i / 2 + 1]);
        }
        tmem_st16(tb + lo + T_R + 16u * w, hi);
        tmem_st16(tb + lo + T_R + 32u + 16u * w, l);
        if (lds_f1(smem_u32(gs + G_WIDE)) != 0.f) {
          uint32_t l3[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float b0 = lds_f1(smem_u32(gs + G_BETA + 32 * w + i)), b1 = lds_f1(smem_u32(gs + G_BETA + 32 * w + i + 1));
            l3[i / 2] = split3(b0 * Y[i], b1 * Y[i + 1], hi[i / 2], l[i / 2]);
          }
          tmem_st16(tb + lo + T_R3 + 16u * w, l3);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&r_ready);
      }
      ok = ok && mbar_wait(&e_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[32];
        tmem_ld32(tb + lo + T_X + 32u * w, x);
        tmem_ld_wait32(x);
        uint32_t hi[16], l[16], hi2[16], l2[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 b = lds_f4(smem_u32(gs + G_BETA + 32 * w + i)), r = lds_f4(smem_u32(gs + G_OUT + 32 * w + i));
          const float u0 = b.x * (Y[i] + __uint_as_float(x[i])), u1 = b.y * (Y[i + 1] + __uint_as_float(x[i + 1]));
          const float u2 = b.z * (Y[i + 2] + __uint_as_float(x[i + 2])), u3 = b.w * (Y[i + 3] + __uint_as_float(x[i + 3]));
          split2(u0, u1, hi[i / 2], l[i / 2]);
          split2(u2, u3, hi[i / 2 + 1], l[i / 2 + 1]);
          split2(r.x * u0, r.y * u1, hi2[i / 2], l2[i / 2]);
          split2(r.z * u2, r.w * u3, hi2[i / 2 + 1], l2[i / 2 + 1]);
        }
        tmem_st16(tb + lo + T_U2 + 16u * w, hi2);
        tmem_st16(tb + lo + T_U2 + 32u + 16u * w, l2);
        tmem_st16(tb + lo + T_U + 16u * w, hi);
        tmem_st16(tb + lo + T_U + 32u + 16u * w, l);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&u_ready);
      }
      ok = ok && mbar_wait(&s_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        const float over = lds_f1(smem_u32(gs + G_OVER));
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t x[32];
          tmem_ld32(tb + lo + T_S + 64u * w + c, x);
          tmem_ld_wait32(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) S[c + i] = fmaf(over, S[c + i], __uint_as_float(x[i]));
        }
        if (j + 1 < nch) {
          put_state();
          ok = ok && clear_rows(j + 1);
          mbar_arrive(&s_ready);
        }
      }
      // o of the chunk, while the next X runs
      ok = ok && mbar_wait(&pu_full, ph, WAIT_CYCLES);
      tc_fence_after();
      {
        uint32_t x[32], p[32];
        tmem_ld32(tb + lo + T_QS + 32u * w, x);
        tmem_ld32(tb + lo + T_PU + 32u * w, p);
        tmem_ld_wait32(x);
        tmem_ld_wait32(p);
        const ColBf16 col(smem_u32(sm + O), 32 * w, v);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 e = lds_f4(smem_u32(gs + G_INTO + 32 * w + i));
          const float f[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int n = 0; n < 4; ++n)
            sts_u16(col.at(i + n),
                    f32_to_bf16_bits(fmaf(a.scale * f[n], __uint_as_float(x[i + n]), __uint_as_float(p[i + n]))));
        }
        tc_fence_before();
        mbar_arrive(&o_free);
      }
      // the 256 threads leave together: the barrier tells everyone of a wait that ran out
      if (named_bar_any(1, 256, !ok)) {
        ok = false;
        break;
      }
      const int L = chunk_len(j);
      __nv_bfloat16 *dst = a.o + (chunk_tok(j) * a.H + h) * (int64_t)a.V;
      for (int i = threadIdx.x; i < CH * 16; i += 256) {
        const int r = i >> 4, c = (i & 15) * 8;
        if (r < L && c < a.V) {
          const uint4 x = lds_u4(smem_u32(sm + O) + sw128_off(r, c, 64));
          st_global_v4(dst + (int64_t)r * a.H * a.V + c, x.x, x.y, x.z, x.w);
        }
      }
    }
    if (!ok) atomicExch(&abort_flag, 1);
    if (a.ht && in && ok) {
      float *dst = a.ht + ((d * a.H + h) * a.K + 64 * w) * (int64_t)a.V + v;
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (64 * w + i < a.K) dst[(int64_t)i * a.V] = S[i];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile int *)&abort_flag) set_device_error(a.err, GLACORE_ERR_TIMEOUT);
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

inline size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

cudaError_t prep(const Call &c, const PrepMaps &maps, char *tiles, float *gates) {
  PrepArgs a;
  a.g = c.p.g;
  a.beta = c.beta;
  a.docs = c.docs;
  a.H = (int)c.p.H;
  a.Hqk = (int)c.p.Hqk;
  a.share = a.H / a.Hqk;
  a.scale = c.p.scale;
  a.tiles = tiles;
  a.gates = gates;
  a.err = c.p.err;
  cudaError_t e = cudaFuncSetAttribute(delta_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PREP_BYTES);
  if (e != cudaSuccess) return e;
  delta_prep_kernel<<<(unsigned)(c.slots * c.p.Hqk), 128, PREP_BYTES, c.st>>>(maps, a);
  mark_launch("delta_prep", c.st);
  return cudaGetLastError();
}

}  // namespace

bool tc_supported(const glacore_problem *p) {
  return p->dtype == GLACORE_BF16 && p->K % 8 == 0 && p->V % 8 == 0 && p->K <= D128 && p->V <= D128 &&
         p->q_stride % 8 == 0 && p->k_stride % 8 == 0 && p->v_stride % 8 == 0 && p->B * p->T < ((int64_t)1 << 31) - CH &&
         !(((uintptr_t)p->q | (uintptr_t)p->k | (uintptr_t)p->v) & 15);
}

size_t tc_workspace(int64_t slots, int64_t H, bool backward) {
  (void)backward;
  return al256((size_t)slots * H * TILES) + al256((size_t)slots * H * GATES * sizeof(float));
}

cudaError_t tc_fwd(const Call &c, void *o, float *ht, char *ws) {
  if (const cudaError_t be = bind_context()) return be;
  const int64_t units = c.docs.n * c.p.H;
  if (units >= ((int64_t)1 << 31) || c.slots * c.p.Hqk >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  ChainMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!make_map(&maps.q, c.p.q, true, c.p.K, c.p.Hqk, c.p.BT, 64, c.p.qs) ||
      !make_map(&maps.k, c.p.k, true, c.p.K, c.p.Hqk, c.p.BT, 64, c.p.ks) ||
      !make_map(&maps.v, c.p.v, true, c.p.V, c.p.H, c.p.BT, 64, c.p.vs))
    return cudaErrorInvalidValue;
  PrepMaps pm;
  pm.q = maps.q;
  pm.k = maps.k;
  char *tiles = ws;
  float *gates = (float *)(ws + al256((size_t)c.slots * c.p.H * TILES));
  cudaError_t e = prep(c, pm, tiles, gates);
  if (e != cudaSuccess) return e;
  ChainArgs a;
  a.docs = c.docs;
  a.H = (int)c.p.H;
  a.share = (int)(c.p.H / c.p.Hqk);
  a.K = (int)c.p.K;
  a.V = (int)c.p.V;
  a.scale = c.p.scale;
  a.h0 = c.p.h0;
  a.ht = ht;
  a.o = (__nv_bfloat16 *)o;
  a.tiles = tiles;
  a.gates = gates;
  a.err = c.p.err;
  e = cudaFuncSetAttribute(delta_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, cs::BYTES);
  if (e != cudaSuccess) return e;
  delta_chain_kernel<<<(unsigned)units, CHAIN_THREADS, cs::BYTES, c.st>>>(maps, a);
  mark_launch("delta_chain", c.st);
  return cudaGetLastError();
}

}  // namespace delta
}  // namespace glacore
