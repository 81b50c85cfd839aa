// linear_ce.cu -- softmax cross entropy of an output projection, forward and
// backward, without keeping the logits (C ABI in include/glacore.h):
//     z = x w^T  (x [N, D], w [V, D]),  lse_n = log sum_v exp(z_nv),
//     loss_n = lse_n - z_n,target(n)
//   backward, from lse and dloss:
//     G_nv = (exp(z_nv - lse_n) - [v = target(n)]) dloss_n,
//     dx = G w,  dw = G^T x
//
// Bound by the tensor cores: 2 N V D operations forward, 6 N V D backward
// (the logits once more and two products).  One kernel body does all of it, a
// persistent tcgen05 product of a pair of CTAs (M = 256, cta_group::2: each
// CTA loads half of either operand, so every byte brought to an SM feeds
// twice the products a single CTA's tile would) with three epilogues:
//   STATS    a tile of logits becomes, per row, its maximum and its sum of
//            exponentials, the target left out (one pass, the running sum
//            rescaled every 64 columns), and the target's logit; the tiles' pairs are merged by
//            ce_merge_kernel.  The logits leave TMEM and are gone.
//   GRAD     a tile of logits becomes a tile of G in bf16 (its products with w
//            and x are bf16 tensor-core products), for one piece of the
//            vocabulary at a time, so G takes a bounded workspace.  Of few
//            tokens in two bf16 parts (FEW_TOKENS).
//   PRODUCT  dx^T += w_piece^T G_piece^T and dw_piece = G_piece^T x as one
//            list of units: dw's fill the last wave that dx's would leave
//            open.  dx is summed over pieces and splits of the vocabulary in
//            fp32 and rounded once.
// Operand layouts: a B operand with its N axis contiguous (MN-major) ran the
// same product a quarter slower than a K-major one (8192 x 2048 x 15872: 425
// against 334 us), an A operand did not (334 against 326 us).  So dx is
// computed transposed (A = w^T as it lies, B = G as it lies), and x is
// transposed once per call for dw's B.
// Warps of a CTA (352 threads): 0..7 epilogue (a TMEM lane per thread, two
// warps per lane quarter, each half of the tile's columns), 8 TMA, 9 and 10 MMA
// (of the pair's leader).  Two accumulators in TMEM (four with fp32 operands),
// so the epilogue of one runs under the products of the next.  The two MMA
// warps fill accumulators in turn: the queue of issued products covers some 500
// cycles, less than one warp takes from its last product of an accumulator to
// its first of the next (two commits and two waits; fp32 1000 x 1000 x 8000
// forward: 18 us more with one warp).
// Measured (8192 x 2048 x 32000 bf16, cool card): forward 549 us, 1960 TFLOP/s;
// backward 1680 us, 1920 TFLOP/s (kept busy, the card's power limit takes 5 to
// 15% off both).
//
// fp32 operands: each value is cut exactly into three bf16 parts (the nearest
// bf16 to the value, to what that leaves, and the rest) and a product of two
// values is six of the nine products of their parts (the rest is below 2^-25 of
// it).  Parts cut off instead of rounded leave a rest of the product's own sign,
// which adds up: gradients of 1001 x 520 x 10007 were 1.1e-6 off, now 7.4e-7.
// Wherever a result is fp32 (the loss; everything of fp32 operands) the
// accumulators are added up in fp32 registers every few k-blocks (chunk_of):
// the tensor core's running sum is not rounded to nearest, and over hundreds
// of steps that shows (loss of 8192 x 2048 x 32000: 1.2e-6 off with one sum
// over K = 2048).  With fp32 operands that is every k-block, the small products
// of its parts first, so that only the large one's four steps lose anything
// (the gradients above with the small products summed apart and all four
// k-blocks at a time: 2.7e-6 off, in 12% less time; with a hand-over every two
// steps of a k-block no better, in 30% more).
#include <string.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "tc_pair.cuh"

namespace glacore {
namespace ce {

using namespace ptx;
using tc::pack_bf16;
using tc::tmem_ld32;
using tc::tmem_ld_wait32;
using tc::WAIT_CYCLES;

constexpr int THREADS = 352, EPI_WARPS = 8, TMA_WARP = 8, MMA_WARP = 9;  // and MMA_WARP + 1
enum Kind { STATS = 0, GRAD = 1, PRODUCT = 2 };
constexpr int BM = 256, BK = 64;      // rows of a pair's tile, columns of a k-block
constexpr uint32_t A_BYTES = 128 * BK * 2;
constexpr int MAX_STAGES = 12;
constexpr int SMEM = 231040;          // shared memory of ring and output staging, at most
constexpr int SMEM_LEAVE = SMEM + 1024;  // with a KB for alignment; 227 KB less the barriers' own
// Output staging of a warp: 32 rows of 128 bytes, stored by TMA; with fp32
// operands 8 rows at a time, stored by the warp, which leaves room for a third
// stage of the ring (gradients of 1001 x 520 x 10007: 33 us more with two stages).
constexpr int out_bytes_of(int parts) { return parts == 3 ? 1024 : 4096; }
constexpr int GROUP_M = 8;            // row tiles that share a walk over the columns (L2 reuse)
constexpr float LOG2E = 1.4426950408889634f;

// One product C[m, n] = A B^T over k-blocks, tiles of BM x bn.
struct Gemm {
  CUtensorMap a, b, o;      // o: the output, where bf16 operands' leaves by TMA
  int64_t m, n;
  int32_t a_mn;             // A stored with its M axis contiguous (B: always its K axis)
  int32_t mt, nt, kb;       // tiles, k-blocks
  int32_t a_box, b_box;     // rows of a K-major operand's load (fewer than a CTA's share where there are no more)
  int32_t splits, kb_split; // K cut into `splits` runs of kb_split blocks
  // PRODUCT: where C (C^T if `trans`) goes.  out_f32: fp32, split s at
  // out + s * m * n, added to what is there if `add`; otherwise the tensors'
  // dtype.  wide_out: its rows start at 16-byte steps, and leave through shared
  // memory.  GRAD of fp32 operands: G, out_pitch elements between rows.
  void *out;
  int64_t out_pitch;
  int32_t out_f32, add, trans, wide_out;
};

struct Args {
  Gemm g[2];
  int64_t units0, units;  // units of g[0], of both
  int32_t skip;           // rounds of g[1]'s units that the pairs with one unit of g[0] more sit out
  int32_t bn, stages, a_bytes;  // a_bytes: a CTA's rows of A in a k-block, as far as they are there
  int64_t N, V, v0;  // tokens, vocabulary, first column of the piece
  const int64_t *target;
  float2 *part;      // STATS: [2 * nt][N] (maximum, sum of e^(z - maximum)), the target left out
  float *zt;         // STATS: [N] the target's logit
  const float *lse, *dloss;  // GRAD
  const float *unit;         // G is in units of *unit (null: 1)
  const float *at_target;    // GRAD of few tokens: [N] p - 1 at the target
  int *err;
};

struct Tile {
  int64_t m0, n0;
  int which, split, kb0, kb1, nt;
};

// The units of pair p of P: g[0]'s dealt out in turn, then g[1]'s, whose first
// `skip` rounds pass over the first units0 % P pairs (they got a unit of g[0]
// more, worth about so many of g[1]'s).
struct Walk {
  int64_t p, P, units0, units1, u0, i;
  int32_t skip;
  __device__ __forceinline__ Walk(const Args &a, int64_t pair, int64_t pairs)
      : p(pair), P(pairs), units0(a.units0), units1(a.units - a.units0), u0(pair), i(0), skip(a.skip) {}
  // the next unit (g[1]'s counted on from units0), or -1
  __device__ __forceinline__ int64_t next() {
    if (u0 < units0) {
      const int64_t u = u0;
      u0 += P;
      return u;
    }
    const int64_t r = units0 % P, rest = P - r;
    int64_t u;
    if (p < r)
      u = skip * rest + i * P + p;
    else
      u = i < skip ? i * rest + p - r : skip * rest + (i - skip) * P + p;
    ++i;
    return u < units1 ? units0 + u : -1;
  }
};

__device__ __forceinline__ Tile tile_of(const Args &a, int64_t u) {
  Tile t;
  t.which = u >= a.units0;
  const Gemm &g = a.g[t.which];
  int64_t r = t.which ? u - a.units0 : u;
  const int64_t tiles = (int64_t)g.mt * g.nt;
  t.split = (int)(r / tiles);
  r -= t.split * tiles;
  const int64_t band = (int64_t)GROUP_M * g.nt, first = r / band * GROUP_M;
  const int64_t rows = g.mt - first < GROUP_M ? g.mt - first : GROUP_M;
  r -= first * g.nt;
  t.m0 = (first + r % rows) * BM;
  t.nt = (int)(r / rows);
  t.n0 = (int64_t)t.nt * a.bn;
  t.kb0 = t.split * g.kb_split;
  t.kb1 = min(t.kb0 + g.kb_split, g.kb);
  return t;
}

// Accumulators in TMEM (fp32 operands: tiles of 128 columns, handed over every
// k-block).
constexpr int bufs_of(int parts) { return parts == 3 ? 4 : 2; }
constexpr int block_bytes_of(int parts, int a_bytes, int bn) { return parts * (a_bytes + bn * BK); }
// G and dw leave through shared memory and TMA: a warp's direct stores of 32
// rows touch 32 lines each, and a product over few k-blocks is bound by them
// (backward of 16 x 2048 x 32000: 116 us with direct stores, 110 us so).
constexpr bool staged_out(int kind) { return kind != STATS; }
// k-blocks of a stage.  Two for the logits: half the waits and commits (8192 x
// 2048 x 32000 forward 571 -> 546 us on a cool card).  The gradients' products,
// with an operand in 64-row boxes, ran 3% slower so.
constexpr int join_of(int kind, int parts) { return parts == 1 && kind != PRODUCT ? 2 : 1; }
// Shared memory of the output staging, and of the last stage's A rows that are
// not there: a product reads 128 rows of A, whatever is in them.
constexpr int extra_of(int kind, int parts, int a_bytes) {
  return (staged_out(kind) ? EPI_WARPS * out_bytes_of(parts) : 0) + (int)A_BYTES - a_bytes;
}
constexpr int stages_of(int kind, int parts, int a_bytes, int bn) {
  const int n = (SMEM - extra_of(kind, parts, a_bytes)) / (join_of(kind, parts) * block_bytes_of(parts, a_bytes, bn));
  return n < MAX_STAGES ? n : MAX_STAGES;
}
// k-blocks whose products one accumulator sums.  The logits of bf16 operands (8192
// x 2048 x 32000, loss): 16 k-blocks 5.4e-7 off in 544 us, 8 2.5e-7 in 549, 4
// 1.3e-7 in 596.  Of few tokens, where w's way from memory bounds the call (16
// tokens): 8 in 32.6 us, 4 in 34.9; with 8 a single token's loss was up to 2e-6
// off, where sums in fp32 rounded to nearest give 5e-7.
constexpr int chunk_of(int kind, int parts, bool few) {
  return parts == 3 ? 1 : kind != STATS ? 1 << 30 : few ? 4 : 8;
}

// The six products of parts (a, b), small ones first; the last is the large
// one (bf16 operands: the only one).
__device__ constexpr int PA[6] = {2, 0, 1, 1, 0, 0}, PB[6] = {0, 2, 1, 0, 1, 0};

// (x - r) f and (y - r) f, two operations at once.
__device__ __forceinline__ float2 scaled_difference(float x, float y, float r, float f) {
  float2 o;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 b, {%5, %5};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(o.x), "=f"(o.y)
      : "f"(x), "f"(y), "f"(-r), "f"(f));
  return o;
}

// Bytes of one k-block (and part) that CTA `rank` loads for a tile.  What lies
// wholly past the end of M or N is not loaded: whatever is in its place only
// reaches accumulator rows and columns that nobody reads.
// `beside`: B is two parts of the same rows side by side, one for each CTA.
__device__ __forceinline__ uint32_t load_bytes(const Gemm &g, const Tile &t, int bn, int rank, bool beside) {
  const int64_t am = t.m0 + rank * 128, bn0 = t.n0 + (beside ? 0 : rank * (bn / 2));
  uint32_t n = bn0 < g.n ? (uint32_t)g.b_box * (BK * 2) : 0;
  if (g.a_mn)
    n += (am < g.m ? 8192 : 0) + (am + 64 < g.m ? 8192 : 0);
  else
    n += am < g.m ? (uint32_t)g.a_box * (BK * 2) : 0;
  return n;
}

// Parts of G (FEW: few tokens).  Two bf16 parts: GRAD writes them; of PRODUCT's
// sums dx has them side by side along its N axis (the tokens fill less than half
// a tile, so they cost it nothing) and leaves each as a split of its own, dw one
// after the other along K.
constexpr int g_parts_of(int parts, bool few) { return parts == 3 ? 3 : few ? 2 : 1; }

template <int KIND, int PARTS, bool FEW>
__global__ void __launch_bounds__(THREADS, 1) ce_product_kernel(const __grid_constant__ Args a) {
  constexpr int G_PARTS = g_parts_of(PARTS, FEW);
  constexpr bool TWO = KIND == PRODUCT && PARTS == 1 && G_PARTS == 2;
  constexpr int CHUNK = chunk_of(KIND, PARTS, FEW);
  constexpr bool CHUNKED = KIND == STATS || PARTS == 3;
  static_assert(CHUNK % join_of(KIND, PARTS) == 0);  // an accumulator's k-blocks fill whole stages
  constexpr int BUFS = bufs_of(PARTS), BUF_COLS = 512 / BUFS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[BUFS], acc_empty[BUFS], turn[2], drained;
  __shared__ uint32_t tmem_ptr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t b_bytes = (uint32_t)a.bn * BK;  // bn / 2 rows of BK bf16
  const uint32_t a_bytes = a.a_bytes;
  const uint32_t block_bytes = PARTS * (a_bytes + b_bytes), stage_bytes = join_of(KIND, PARTS) * block_bytes;
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * EPI_WARPS);
    }
    mbar_init(&turn[0], 1);
    mbar_init(&turn[1], 1);
    mbar_init(&drained, 2);
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc_pair(&tmem_ptr, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_ptr;
  follow_wait();  // what came before is needed from here on
  follow_allow();

  // Everything the two issuing threads use per k-block is in registers: a
  // parameter read again behind each of their asm statements costs them more
  // than the products take.
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
  const int stages = a.stages;
  if (warp == TMA_WARP) {
    if (lane == 0) {
      // ---- tile loads of this CTA; bytes complete on the leader's barrier
      bool ok = true, wrapped = false;
      int s = 0;
      uint32_t phase = 0;  // of the ring's current turn
      const uint32_t bar0 = mapa_shared(full0, 0);
      Walk walk(a, pair, pairs);
      for (int64_t u; ok && (u = walk.next()) >= 0;) {
        const Tile t = tile_of(a, u);
        const Gemm &g = a.g[t.which];
        const CUtensorMap *ma = &g.a, *mb = &g.b;
        const int am = (int)(t.m0 + rank * 128), bn0 = TWO && !t.which ? 0 : (int)(t.n0 + rank * (a.bn / 2));
        const bool a_mn = g.a_mn, a0 = am < g.m, a1 = am + 64 < g.m, b0 = bn0 < g.n;
        const bool beside = TWO && !t.which;
        const uint32_t bytes = PARTS * (load_bytes(g, t, a.bn, 0, beside) + load_bytes(g, t, a.bn, 1, beside));
        const bool behind = TWO && t.which;
        int k = behind ? t.kb0 / 2 * BK : t.kb0 * BK, za = behind ? t.kb0 % 2 : 0;
        const int zb = beside ? (int)rank : 0;
        for (int n = t.kb1 - t.kb0; n > 0; n -= join_of(KIND, PARTS)) {
          if (!mbar_wait_at(empty0 + 8 * s, phase ^ 1, WAIT_CYCLES)) {
            set_device_error(a.err, GLACORE_ERR_TIMEOUT);
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx_at(full0 + 8 * s, bytes * (uint32_t)min(n, join_of(KIND, PARTS)));
          const uint32_t bar = bar0 + 8 * s;
#pragma unroll
          for (int q = 0; q < join_of(KIND, PARTS); ++q) {
            if (q >= n) break;
            const uint32_t sa = smem + s * stage_bytes + q * block_bytes, sb = sa + PARTS * a_bytes;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
              if (a_mn) {
                if (a0) tma_load_3d_pair(sa + p * a_bytes, ma, am, k, p + za, bar);
                if (a1) tma_load_3d_pair(sa + p * a_bytes + 8192, ma, am + 64, k, p + za, bar);
              } else if (a0) {
                tma_load_3d_pair(sa + p * a_bytes, ma, k, am, p, bar);
              }
              if (b0) tma_load_3d_pair(sb + p * b_bytes, mb, k, bn0, p + zb, bar);
            }
            if (behind && za == 0) {
              za = 1;
            } else {
              za = 0;
              k += BK;
            }
          }
          if (++s == stages) {
            s = 0;
            phase ^= 1;
            wrapped = true;
          }
        }
      }
      // every load has landed, and every release has arrived, before the CTA ends
      for (int i = 0; i < stages; ++i) {
        if (i >= s && !wrapped) break;  // never used
        const uint32_t used = i < s ? phase : phase ^ 1;
        if (rank == 0) mbar_wait_at(full0 + 8 * i, used, WAIT_CYCLES);
        if (ok) ok = mbar_wait_at(empty0 + 8 * i, used, WAIT_CYCLES);
      }
    }
    __syncwarp();
  } else if (warp >= MMA_WARP) {
    if (lane == 0 && rank == 0) {
      // ---- products of the pair: every second accumulator's
      bool ok = true;
      const uint32_t side = warp - MMA_WARP;
      uint32_t hand = 0, ring = 0;  // accumulators handed over, stages used (modulo two turns), by both
      const uint32_t acc_full0 = smem_u32(acc_full);
      Walk walk(a, pair, pairs);
      for (int64_t u; ok && (u = walk.next()) >= 0;) {
        const Tile t = tile_of(a, u);
        const bool a_mn = a.g[t.which].a_mn;
        const uint32_t idesc = idesc_bf16(BM, a.bn, a_mn, false);
        const uint32_t astep = a_mn ? 2048 : 32;  // bytes between 16-element steps of K
        const SDesc ad0 = sdesc_sw128(smem, a_mn ? 8192 : 16, 1024);
        const SDesc bd0 = sdesc_sw128(smem + PARTS * a_bytes, 16, 1024);
        for (int left = t.kb1 - t.kb0; left > 0 && ok; ++hand) {
          const int run = min(left, CHUNK);
          left -= run;
          int s = ring;
          uint32_t phase = 0;
          ring = (ring + (run + join_of(KIND, PARTS) - 1) / join_of(KIND, PARTS)) % (2 * stages);
          if ((hand & 1) != side) continue;
          if (s >= stages) {
            s -= stages;
            phase = 1;
          }
          const uint32_t buf = hand % BUFS;
          // The accumulator has been read; and the other warp has seen all its
          // stages arrive (a stage's barrier tells two turns of the ring apart,
          // no more, so nobody waits for one further ahead).
          if (!mbar_wait_at(smem_u32(&acc_empty[buf]), (hand / BUFS + 1) & 1, WAIT_CYCLES) ||
              (hand > 0 && !mbar_wait_at(smem_u32(&turn[side]), ((hand - 1) >> 1) & 1, WAIT_CYCLES))) {
            set_device_error(a.err, GLACORE_ERR_TIMEOUT);
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t more = 0;  // the run's first products overwrite the accumulator
          for (int n = run; n > 0; n -= join_of(KIND, PARTS)) {
            if (!mbar_wait_at(full0 + 8 * s, phase, WAIT_CYCLES)) {
              set_device_error(a.err, GLACORE_ERR_TIMEOUT);
              ok = false;
              break;
            }
            if (n <= join_of(KIND, PARTS)) mbar_arrive(&turn[side ^ 1]);
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < join_of(KIND, PARTS); ++q) {
              if (q >= n) break;
              const uint32_t at = s * stage_bytes + q * block_bytes;
#pragma unroll
              for (int i = PARTS == 1 ? 5 : 0; i < 6; ++i) {
                const uint32_t d = tmem + buf * BUF_COLS;
                const SDesc ad = ad0 + (at + (PARTS == 1 ? 0 : PA[i] * a_bytes));
                const SDesc bd = bd0 + (at + (PARTS == 1 ? 0 : PB[i] * b_bytes));
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                  mma_bf16_pair(d, ad + k * astep, bd + k * 32, idesc,
                                more | (uint32_t)(k > 0 || i > (PARTS == 1 ? 5 : 0)));
              }
              more = 1;
            }
            mma_commit_pair(empty0 + 8 * s);
            if (++s == stages) {
              s = 0;
              phase ^= 1;
            }
          }
          if (ok) mma_commit_pair(acc_full0 + 8 * buf);
        }
      }
      mma_commit_pair(smem_u32(&drained));
    }
    // the products in flight end before TMEM and the operands of either CTA go
    if (lane == 0) mbar_wait_at(smem_u32(&drained), 0, WAIT_CYCLES);
    __syncwarp();
  } else {
    // ---- epilogue: thread = row, half = which half of the tile's columns
    const int quarter = warp & 3, half = warp >> 2, cols = a.bn / 2;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + half * cols;
    // The warp's staging: rows of 128 bytes, 16-byte chunks swizzled by row.
    const uint32_t stage = smem + stages * stage_bytes + warp * out_bytes_of(PARTS);
    auto put = [&](int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
      tc::st_shared_v4(stage + lane * 128 + ((chunk ^ (lane & 7)) << 4), x, y, z, w);
    };
    auto begin_out = [&]() {  // the last store has read the staging
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
    };
    auto send_out = [&](const CUtensorMap *map, int x, int y, int z) {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d_at(map, stage, x, y, z);
        bulk_commit();
      }
    };
    // `w`: 128 bytes of this lane's row; rows `pitch` bytes apart from `to` on,
    // of which the first `rows` are there, and the first `bytes` of each.
    auto store_rows = [&](const uint4 (&w)[8], char *to, int64_t pitch, int64_t rows, int bytes) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if ((lane >> 3) == r)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            tc::st_shared_v4(stage + (lane & 7) * 128 + ((i ^ (lane & 7)) << 4), w[i].x, w[i].y, w[i].z, w[i].w);
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          const int y = (lane >> 3) + h, c = lane & 7;
          const uint4 f = ld_shared_v4(stage + y * 128 + ((c ^ y) << 4));
          if (8 * r + y < rows && 16 * c < bytes) *reinterpret_cast<uint4 *>(to + (8 * r + y) * pitch + 16 * c) = f;
        }
        __syncwarp();
      }
    };
    auto release = [&](int buf) {  // this warp has read the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(mapa_shared(smem_u32(&acc_empty[buf]), 0));
    };
    const float unit = KIND != STATS && a.unit ? *a.unit : 1.f;
    uint32_t hand = 0;
    bool ok = true;
    Walk walk(a, pair, pairs);
    for (int64_t u; ok && (u = walk.next()) >= 0;) {
      const Tile t = tile_of(a, u);
      const Gemm &g = a.g[t.which];
      const int64_t row = t.m0 + rank * 128 + quarter * 32 + lane;
      const bool live = row < g.m;
      const bool beside = TWO && !t.which;
      const int64_t c0 = beside ? 0 : t.n0 + half * cols;  // first column of this warp (in the piece)
      // per-row state of the epilogue
      float mx = -INFINITY, sum = 0.f, lse = 0.f, dl = 0.f;
      int64_t tgt = -1;
      if (KIND != PRODUCT) {
        if (live) tgt = a.target[row];
        if (KIND == GRAD && live) {
          lse = a.lse[row];
          if (tgt >= a.V) {
            set_device_error(a.err, GLACORE_ERR_INDEX);
            tgt = -1;
          }
          dl = a.dloss[row] / unit;
        }
      }
      // 64 columns c0 + c .. of the row
      auto use = [&](int c, float (&v)[64]) {
        const int64_t col = c0 + c;
        if constexpr (KIND == STATS) {
          const int64_t room = min(a.V - col, (int64_t)(cols - c));  // columns of the vocabulary, of this warp here
          if (room <= 0) return;
          if (room < 64) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= room) v[i] = -INFINITY;
          }
          if (tgt >= col && tgt < col + room) {
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (tgt == col + i) {
                z = v[i];
                v[i] = -INFINITY;
              }
            if (live) a.zt[row] = z;
          }
          float top[4] = {mx, v[0], v[1], v[2]};
#pragma unroll
          for (int i = 3; i < 64; ++i) top[i & 3] = fmaxf(top[i & 3], v[i]);
          const float peak = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          // a row of -inf so far: any finite reference gives sums of 0
          const float ref = peak == -INFINITY ? 0.f : peak;
          // The difference first, as for G: a product of either with log2 e is
          // rounded at the size of the logit.
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            const float2 d = scaled_difference(v[i], v[i + 1], ref, LOG2E);
            s[i & 3] += ex2(d.x);
            s[(i & 3) + 1] += ex2(d.y);
          }
          // no finite maximum yet: the sum is 0, or a NaN that stays
          const float old = mx == -INFINITY ? sum : sum * ex2((mx - ref) * LOG2E);
          sum = old + ((s[0] + s[1]) + (s[2] + s[3]));
          mx = peak;
        } else if constexpr (KIND == GRAD) {
          if (c >= cols) return;
          const bool scored = tgt >= 0;
          const int64_t hit = tgt - a.v0 - col;
          // the difference first: a product of either with log2 e would round
          // by more than 1 at logits of some 10^4
#pragma unroll
          for (int i = 0; i < 64; ++i)
            v[i] = PARTS == 1 ? ex2((v[i] - lse) * LOG2E) : expf(v[i] - lse);
          if (hit >= 0 && hit < 64) {
            const float at = FEW ? a.at_target[row] : 0.f;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (hit == i) v[i] = FEW ? at : v[i] - 1.f;
          }
          // a token that is not scored has no gradient, whatever its logits are
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = scored ? v[i] * dl : 0.f;
          if (row - lane >= g.m) return;
#pragma unroll
          for (int p = 0; p < G_PARTS; ++p) {
            uint4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t u[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float &x = v[8 * i + 2 * j], &y = v[8 * i + 2 * j + 1];
                u[j] = pack_bf16(x, y);
                if (p + 1 < G_PARTS) {  // the bf16 nearest to what is left, and exactly what is left then
                  x -= __uint_as_float(u[j] << 16);
                  y -= __uint_as_float(u[j] & 0xffff0000u);
                }
              }
              w[i] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            if constexpr (PARTS == 3) {
              store_rows(w, reinterpret_cast<char *>(g.out) + ((p * a.N + row - lane) * g.out_pitch + col) * 2,
                         g.out_pitch * 2, g.m - (row - lane), 128);
            } else {
              begin_out();
#pragma unroll
              for (int i = 0; i < 8; ++i) put(i, w[i].x, w[i].y, w[i].z, w[i].w);
              send_out(&g.o, (int)col, (int)(row - lane), p);
            }
          }
        } else {
          if (c >= cols || col >= g.n || row - lane >= g.m) return;  // nothing of the warp's columns is there
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] *= unit;
          const int room = g.n - col < 64 ? (int)(g.n - col) : 64;
          if (g.wide_out) {  // what lies past the edges is not written
            if (g.out_f32) {
#pragma unroll
              for (int h = 0; h < 64; h += 32) {
                if (h >= room) break;
                if constexpr (PARTS == 3) {
                  uint4 w[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    w[i] = make_uint4(__float_as_uint(v[h + 4 * i]), __float_as_uint(v[h + 4 * i + 1]),
                                      __float_as_uint(v[h + 4 * i + 2]), __float_as_uint(v[h + 4 * i + 3]));
                  store_rows(w, reinterpret_cast<char *>(g.out) +
                                    (((int64_t)t.split * g.m + row - lane) * g.n + col + h) * 4,
                             g.n * 4, g.m - (row - lane), 4 * (room - h));
                  continue;
                }
                begin_out();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  put(i, __float_as_uint(v[h + 4 * i]), __float_as_uint(v[h + 4 * i + 1]),
                      __float_as_uint(v[h + 4 * i + 2]), __float_as_uint(v[h + 4 * i + 3]));
                send_out(&g.o, (int)col + h, (int)(row - lane), t.split);
              }
            } else {
              begin_out();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                put(i, pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                    pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
              send_out(&g.o, (int)col, (int)(row - lane), 0);
            }
            return;
          }
          if (!live) return;
          // C^T: the warp's 32 rows lie side by side.  C: rows that TMA cannot
          // address.
          const int64_t step = g.trans ? g.m : 1;
          const int64_t at = g.trans ? col * g.m + row : row * g.n + col;
          if (g.out_f32) {
            const int64_t split = beside ? 2 * t.split + half : t.split;
            float *out = reinterpret_cast<float *>(g.out) + split * g.m * g.n + at;
#pragma unroll
            for (int h = 0; h < 64; h += 16) {
              float old[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) old[i] = g.add && h + i < room ? out[(h + i) * step] : 0.f;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (h + i < room) out[(h + i) * step] = v[h + i] + old[i];
            }
          } else if (PARTS == 1) {
            __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(g.out) + at;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i < room) out[i * step] = __float2bfloat16_rn(v[i]);
          }
        }
      };
      constexpr int HALVES = PARTS == 3 ? 1 : 2;  // 64 columns each of a warp's, at most
      constexpr int SUMS = CHUNKED ? HALVES : 1;
      float acc[SUMS][64];  // the chunks so far
      if (CHUNKED)
#pragma unroll
        for (int j = 0; j < SUMS; ++j)
#pragma unroll
          for (int i = 0; i < 64; ++i) acc[j][i] = 0.f;
      for (int kb = t.kb0; kb < t.kb1; kb += min(t.kb1 - kb, CHUNK), ++hand) {
        const int buf = (int)(hand % BUFS);
        if (!mbar_wait_at(smem_u32(&acc_full[buf]), (hand / BUFS) & 1, WAIT_CYCLES)) {
          if (lane == 0) set_device_error(a.err, GLACORE_ERR_TIMEOUT);
          ok = false;
          break;
        }
        tc_fence_after();
        const bool last = t.kb1 - kb <= CHUNK;
#pragma unroll
        for (int j = 0; j < HALVES; ++j) {
          if (64 * j >= cols) break;
          float(&v)[64] = acc[CHUNKED ? j : 0];
          if constexpr (SUMS == 2) {  // few registers beside the sums
#pragma unroll
            for (int h = 0; h < 64; h += 16) {
              uint32_t r[16];
              tmem_ld16(lanes + buf * BUF_COLS + 64 * j + h, r);
              tmem_ld_wait(r);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[h + i] += __uint_as_float(r[i]);
            }
          } else {
            uint32_t r[32], q[32];
            tmem_ld32(lanes + buf * BUF_COLS + 64 * j, r);
            tmem_ld32(lanes + buf * BUF_COLS + 64 * j + 32, q);
            tmem_ld_wait32(r);
            tmem_ld_wait32(q);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[i] = (CHUNKED ? v[i] : 0.f) + __uint_as_float(r[i]);
              v[32 + i] = (CHUNKED ? v[32 + i] : 0.f) + __uint_as_float(q[i]);
            }
          }
          if (64 * j + 64 >= cols) release(buf);
          if (!CHUNKED) use(64 * j, v);
        }
        if (CHUNKED && last) {
#pragma unroll
          for (int j = 0; j < SUMS; ++j)
            if (64 * j < cols) use(64 * j, acc[j]);
        }
      }
      if (!ok) break;
      if (KIND == STATS && live && c0 < a.V)
        a.part[(int64_t)(2 * t.nt + half) * a.N + row] = make_float2(mx, sum);
    }
  }
  if (staged_out(KIND) && warp < EPI_WARPS && lane == 0) bulk_wait_all();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The logit at the target of each of few tokens, from the caller's own x and w: a
// tile's logit comes from the tensor core's truncated sum, and where p is near 1
// its error is a large part of the loss and of p - 1.
template <typename T> struct Targets {
  const T *x, *w;
  int64_t xs, D;
  // A warp's share of token n's logit at t: every `threads`-th product from
  // `first` on.  A thread's are added in A, the threads' in 64 bits.
  template <typename A> __device__ __forceinline__ double part(int64_t n, int64_t t, int first, int threads) const {
    const T *xr = x + n * xs, *wr = w + t * D;
    A f[4] = {A(0), A(0), A(0), A(0)};
    int64_t c = first;
    for (; c + 15 * threads < D; c += 16 * threads)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int64_t at = c + i * threads;
        f[i & 3] = fma((A)to_f32(xr[at]), (A)to_f32(wr[at]), f[i & 3]);
      }
    for (; c < D; c += threads) f[0] = fma((A)to_f32(xr[c]), (A)to_f32(wr[c]), f[0]);
    double s = ((double)f[0] + (double)f[1]) + ((double)f[2] + (double)f[3]);
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    return s;
  }
};

// lse and loss of 32 rows from the tiles' (maximum, sum) pairs: 32 threads per
// row take every 32nd pair, then merge in order.  The pairs are of the other
// tokens: beside the target's own 1 the sum of a well foreseen token would lose
// its digits, and its loss is nothing else.  No term of the loss is rounded at
// the size of a logit, and it is never negative.  FEW: the target's logit comes
// from `targets`, a row per warp, before the wait for the tiles: x, w and target
// were there before the call's first kernel.
constexpr int MERGE_ROWS = 32, MERGE_LANES = 32;
template <typename T, bool FEW>
__global__ void __launch_bounds__(MERGE_ROWS *MERGE_LANES)
    ce_merge_kernel(const Targets<T> targets, const float2 *__restrict__ part, int64_t slots, int64_t N, int64_t V,
                    const int64_t *__restrict__ target, const float *__restrict__ zt, float *__restrict__ loss,
                    float *__restrict__ lse, int *err) {
  __shared__ float2 red[MERGE_LANES][MERGE_ROWS];
  __shared__ float at_target[FEW ? MERGE_ROWS : 1];
  if constexpr (FEW) {
    const int64_t n = (int64_t)blockIdx.x * MERGE_ROWS + threadIdx.y, t = n < N ? target[n] : -1;
    if (t >= 0 && t < V) {
      // shares in fp32, each rounded at a small part of the logit's size: an SM's
      // few 64-bit units took 16 tokens of D = 2048 18 us longer
      const double z = targets.template part<float>(n, t, threadIdx.x, 32);
      if (threadIdx.x == 0) at_target[threadIdx.y] = (float)z;
    }
  }
  follow_wait();
  const int64_t row = (int64_t)blockIdx.x * MERGE_ROWS + threadIdx.x;
  float m = -INFINITY, s = 0.f;
  auto merge = [&](float2 p) {
    const float top = fmaxf(m, p.x), ref = top == -INFINITY ? 0.f : top;
    s = s * exp2f((m - ref) * LOG2E) + p.y * exp2f((p.x - ref) * LOG2E);
    m = top;
  };
  if (row < N) {
    int64_t i = threadIdx.y;
    for (; i + 3 * MERGE_LANES < slots; i += 4 * MERGE_LANES) {
      float2 p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = part[(i + k * MERGE_LANES) * N + row];
#pragma unroll
      for (int k = 0; k < 4; ++k) merge(p[k]);
    }
    for (; i < slots; i += MERGE_LANES) merge(part[i * N + row]);
  }
  red[threadIdx.y][threadIdx.x] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.y || row >= N) return;
  for (int i = 1; i < MERGE_LANES; ++i) merge(red[i][threadIdx.x]);
  const int64_t t = target[row];
  if (t >= V) set_device_error(err, GLACORE_ERR_INDEX);
  if (t < 0 || t >= V) {
    lse[row] = m + logf(s);
    loss[row] = 0.f;
    return;
  }
  const float z = FEW ? at_target[threadIdx.x] : zt[row];
  if (m > z) {
    const float l = logf(s + exp2f((z - m) * LOG2E));
    lse[row] = m + l;
    loss[row] = (m - z) + l;
  } else {  // the target's logit is the largest (or a NaN, or infinite: z - z)
    const float l = log1pf(s * exp2f((m - z) * LOG2E)) + (z - z);
    lse[row] = z + l;
    loss[row] = l;
  }
}

// A gradient from its splits' sums, added in order and rounded to its type.
// WIDE: n is a multiple of 4 and dx 16-byte aligned.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256)
    ce_sum_kernel(const float *__restrict__ part, int splits, int64_t n, T *__restrict__ dx) {
  follow_wait();
  follow_allow();
  if constexpr (WIDE) {
    const float4 *p = reinterpret_cast<const float4 *>(part);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n / 4; i += (int64_t)gridDim.x * 256) {
      float4 s = p[i];
#pragma unroll 4
      for (int k = 1; k < splits; ++k) {
        const float4 f = p[k * (n / 4) + i];
        s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
      }
      if constexpr (sizeof(T) == 4)
        reinterpret_cast<float4 *>(dx)[i] = s;
      else
        reinterpret_cast<uint2 *>(dx)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
  } else {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
      float s = part[i];
      for (int k = 1; k < splits; ++k) s += part[k * n + i];
      dx[i] = from_f32<T>(s);
    }
  }
}

// p - 1 at token n's target, by the CTA.
template <typename T>
__device__ __forceinline__ void find_at_target(const Targets<T> &g, int64_t n, const int64_t *target, int64_t V,
                                               const float *lse, float *at_target) {
  __shared__ double part[8];
  const int64_t t = target[n];
  if (t < 0 || t >= V) return;  // not scored: nobody reads it
  double s = g.template part<double>(n, t, threadIdx.x, 256);  // p - 1 of fp32 operands needs them all
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) s += part[i];
    at_target[n] = expm1f((float)(s - (double)lse[n]));
  }
}

// Before the products of the backward: dst [parts, cols, dpitch] = src [parts,
// rows, spitch] transposed, 64 x 64 at a time through shared memory (pitches
// are multiples of 8: two values per access); and, by one CTA beside them, the
// unit of G (null: none wanted): the largest |dloss| of a scored token, 1 if
// there is none.  With dloss one number for all tokens, the usual mean, G in
// that unit is p - [v = target] itself, and the -1 at the target of a token
// that is far from foreseen, most of its gradient, is exact in bf16.  Further
// CTAs take a token each for at_target.
template <typename T>
__global__ void __launch_bounds__(256)
    ce_prepare_kernel(const Targets<T> targets, const float *__restrict__ lse, float *__restrict__ at_target,
                      const __nv_bfloat16 *__restrict__ src, int64_t rows, int64_t cols, int64_t spitch,
                      int64_t dpitch, __nv_bfloat16 *__restrict__ dst, const float *__restrict__ dloss,
                      const int64_t *__restrict__ target, int64_t V, float *__restrict__ unit) {
  __shared__ __nv_bfloat162 tile[64][33];
  __shared__ float red[8];
  follow_wait();
  follow_allow();
  const int64_t beyond = (int64_t)blockIdx.x - (rows + 63) / 64;
  if (beyond > 0) {
    const int64_t n = (beyond - 1) * gridDim.y + blockIdx.y;
    if (blockIdx.z == 0 && n < rows) find_at_target(targets, n, target, V, lse, at_target);
    return;
  }
  if (beyond == 0) {
    if (!unit || blockIdx.y || blockIdx.z) return;
    float m = 0.f;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < rows; i += 256) {
      const int64_t t = target[i];
      const float d = fabsf(dloss[i]);
      if (t >= 0 && t < V) m = fmaxf(m, d);
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
      *unit = m > 0.f && isfinite(m) ? m : 1.f;
    }
    return;
  }
  src += blockIdx.z * rows * spitch;
  dst += blockIdx.z * cols * dpitch;
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  for (int i = y; i < 64; i += 8)
    if (r0 + i < rows && c0 + 2 * x < cols)  // an odd number of columns has its padding beside it
      tile[i][x] = *reinterpret_cast<const __nv_bfloat162 *>(src + (r0 + i) * spitch + c0 + 2 * x);
  __syncthreads();
  // columns c, c + 1 of rows 2x, 2x + 1
  for (int j = y; j < 32; j += 8) {
    const int64_t c = c0 + 2 * j;
    if (r0 + 2 * x >= rows) continue;
    const __nv_bfloat162 a = tile[2 * x][j], b = tile[2 * x + 1][j];
    if (c < cols)
      *reinterpret_cast<__nv_bfloat162 *>(dst + c * dpitch + r0 + 2 * x) = __halves2bfloat162(a.x, b.x);
    if (c + 1 < cols)
      *reinterpret_cast<__nv_bfloat162 *>(dst + (c + 1) * dpitch + r0 + 2 * x) = __halves2bfloat162(a.y, b.y);
  }
}

// Rows of x, then of w, as bf16 with a pitch that TMA can address: a copy of
// bf16 values (PARTS = 1), or the three exact parts of fp32 values.
template <int PARTS, typename T>
__global__ void __launch_bounds__(256)
    ce_pack_kernel(const T *__restrict__ x, int64_t N, int64_t xs, __nv_bfloat16 *__restrict__ xp,
                   const T *__restrict__ w, int64_t V, __nv_bfloat16 *__restrict__ wp, int64_t D, int64_t pitch) {
  follow_allow();
  const int lane = threadIdx.x & 31;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < N + V; i += (int64_t)gridDim.x * 8) {
    const int64_t r = i < N ? i : i - N, rows = i < N ? N : V;
    const T *src = i < N ? x + r * xs : w + r * D;
    __nv_bfloat16 *dst = i < N ? xp : wp;
#pragma unroll 4
    for (int64_t c = 2 * lane; c < D; c += 64) {  // two values per store (an odd row's last with a zero)
      float a = to_f32(src[c]), b = c + 1 < D ? to_f32(src[c + 1]) : 0.f;
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        uint32_t u = pack_bf16(a, b);
        if (PARTS == 3) {
          float ha = __uint_as_float(u << 16), hb = __uint_as_float(u & 0xffff0000u);
          // above bf16's largest value the nearest is cut off instead
          if (isinf(ha)) ha = __uint_as_float(__float_as_uint(a) & 0xffff0000u);
          if (isinf(hb)) hb = __uint_as_float(__float_as_uint(b) & 0xffff0000u);
          u = pack_bf16(ha, hb);
          a = isinf(ha) ? 0.f : a - ha;  // an infinity stays one, in the first part
          b = isinf(hb) ? 0.f : b - hb;
        }
        *reinterpret_cast<uint32_t *>(dst + (p * rows + r) * pitch + c) = u;
      }
    }
  }
}

// ---- host ------------------------------------------------------------------
constexpr size_t G_BYTES = (size_t)512 << 20;   // G of one piece of the vocabulary, about
// Tokens up to which the target's logit is summed apart (Targets), and the gradients
// take G in two bf16 parts (of bf16 operands).  A handful of tokens has no
// others that average an entry's error out: gradients of single tokens were up
// to 1.6e-2 off (2-norm) with neither, where rounding the result to bf16 alone
// gives 1.7e-3.  With 16 tokens of 2048 x 32000 it costs 7 of 99 us.  With 128 it
// would be 14 of 110 us, for 1.65e-3 instead of 1.9e-3: left as one bf16 there.
constexpr int64_t FEW_TOKENS = 64;
constexpr size_t SUMS_BYTES = (size_t)512 << 20;  // fp32 sums of a gradient's splits, at most (if there are several)

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Layout {
  int parts, bn, bn_z;               // bn_z: tile width of the logits
  bool few;                          // no more than FEW_TOKENS
  int g_parts;                       // of G
  bool pack;                         // x and w are copied to rows TMA can address
  int64_t pitch, xt_pitch, piece, pieces, gpitch;
  int splits, run;  // dx's K axis: `splits` runs of `run` k-blocks (in the first, longest piece)
  int splits_w, run_w;  // dw's
  bool dx_f32, dw_sums;
  int sums;  // of dx, for each of its splits
  size_t off_x, off_w, off_part, off_zt, off_unit, off_at, off_xt, off_g, off_dx, off_dw, total;
};

// Pairs of CTAs that run at once on the current device.
int64_t pair_count() {
  static std::atomic<int> cache[128];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return tc::sm_count() / 2;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tc::sm_count() / 2 * 2));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_LEAVE;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto *k = ce_product_kernel<STATS, 1, false>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();  // no device here: a size query only
      n = (int)(tc::sm_count() / 2);
    }
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// How the two gradients' units load the pairs: the time of the busiest pair,
// in k-blocks of a tile (about 0.27 us), for units of run_x and run_w
// k-blocks.  A unit takes no less than its epilogue, about EPI_KB of them, and
// 4 for its start and end.
constexpr int64_t EPI_KB = 8;
struct Deal {
  int64_t longest;
  int32_t skip;
};
Deal deal(int64_t ux, int64_t run_x, int64_t uw, int64_t run_w) {
  const int64_t P = pair_count(), cx = std::max<int64_t>(run_x, EPI_KB) + 4, cw = std::max<int64_t>(run_w, EPI_KB) + 4,
                r = ux % P, nx = ux / P;
  const int64_t skip = r ? std::min((cx + cw / 2) / cw, up(uw, P - r)) : 0;
  const int64_t rem = std::max<int64_t>(0, uw - skip * (P - r)), rounds = rem / P, rest = rem % P;
  const int64_t a = (nx + (r > 0)) * cx + (rounds + (rest > 0)) * cw;
  const int64_t b = nx * cx + (skip + rounds + (rest > r)) * cw;
  return Deal{r ? std::max(a, b) : b, (int32_t)skip};
}

// Cuts of the two gradients' K axes (dx: a piece of the vocabulary, dw: the
// tokens) for the shortest busiest pair.  A cut costs its fp32 sums' way to
// memory and back (1.8 MB per k-block's time) and a launch.
void choose_splits(Layout &L, int64_t N, int64_t D, int64_t cols) {
  static const int tries[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
  const int64_t tx = up(D, BM) * up(N, L.bn), tw = up(cols, BM) * up(D, L.bn), kx = up(cols, BK),
                kw = up(N, BK) * L.sums;
  int64_t least = -1;
  for (int sx : tries) {
    const int64_t rx = up(kx, sx), mx = up(kx, rx) * L.sums * N * D * 4;
    if (sx > 1 && (sx > kx || mx > (int64_t)SUMS_BYTES)) break;
    for (int sw : tries) {
      const int64_t rw = up(kw, sw), mw = up(kw, rw) * cols * D * 4;
      if (sw > 1 && (sw > kw || mw > (int64_t)SUMS_BYTES)) break;
      int64_t cost = deal(tx * up(kx, rx), rx, tw * up(kw, rw), rw).longest;
      if (sx > 1 || L.pieces > 1 || L.sums > 1) cost += 2 * mx / 1800000 + 8;
      if (sw > 1) cost += 2 * mw / 1800000 + 8;
      if (least < 0 || cost < least) {
        least = cost;
        L.run = (int)rx;
        L.splits = (int)up(kx, rx);
        L.run_w = (int)rw;
        L.splits_w = (int)up(kw, rw);
      }
    }
  }
}

Layout layout(int64_t N, int64_t D, int64_t V, int32_t dtype, bool backward) {
  Layout L;
  memset(&L, 0, sizeof(L));
  L.parts = dtype == GLACORE_F32 ? 3 : 1;
  L.bn = L.parts == 3 ? 128 : 256;
  L.bn_z = L.bn;
  if (L.parts == 1) {
    // The width that deals the vocabulary out most evenly: the fewest columns
    // for the busiest pair, and about 32 columns' time for a tile's start and
    // end.  It matters for few tokens, where the call is bound by reading w
    // once (16 x 2048 x 32000: 36.4 us with 256, 34.8 us with 224, 33.1 us with
    // the ring's stages no taller than the tokens, and 34.9 us now that its sums
    // are handed over every four k-blocks).
    int64_t least = -1;
    for (int bn = 256; bn >= 128; bn -= backward ? 128 : 32) {  // G leaves 64 columns of a warp at a time
      const int64_t cost = up(up(N, BM) * up(V, bn), pair_count()) * (bn + 32);
      if (least < 0 || cost < least) {
        least = cost;
        L.bn_z = bn;
      }
    }
  }
  L.pack = L.parts == 3 || D % 8 != 0;
  L.few = N <= FEW_TOKENS;
  L.pitch = up(D, 8) * 8;
  size_t off = 0;
  auto take = [&](size_t &o, size_t bytes) {
    o = off;
    off = align256(off + bytes);
  };
  if (L.pack) {
    take(L.off_x, (size_t)L.parts * N * L.pitch * 2);
    take(L.off_w, (size_t)L.parts * V * L.pitch * 2);
  }
  if (!backward) {
    take(L.off_part, (size_t)up(V, L.bn_z) * 2 * N * sizeof(float2));
    take(L.off_zt, (size_t)N * sizeof(float));
  } else {
    L.g_parts = g_parts_of(L.parts, L.few);
    L.sums = L.g_parts == 2 ? 2 : 1;
    const int64_t most = std::max<int64_t>(2048, (int64_t)(G_BYTES / (2 * L.g_parts * (size_t)N)) / 256 * 256);
    L.pieces = up(V, most);
    L.piece = up(up(V, L.pieces), 256) * 256;
    L.pieces = up(V, L.piece);
    L.gpitch = L.piece;
    L.xt_pitch = up(N, 8) * 8;
    take(L.off_unit, sizeof(float));
    if (L.few) take(L.off_at, (size_t)N * sizeof(float));
    take(L.off_xt, (size_t)L.parts * D * L.xt_pitch * 2);
    take(L.off_g, (size_t)L.g_parts * N * L.gpitch * 2);
    choose_splits(L, N, D, std::min(L.piece, V));
    L.dx_f32 = L.splits > 1 || L.pieces > 1 || L.sums > 1;
    L.dw_sums = L.splits_w > 1;
    if (L.dx_f32) take(L.off_dx, (size_t)L.splits * L.sums * N * D * sizeof(float));
    if (L.dw_sums) take(L.off_dw, (size_t)L.splits_w * std::min(L.piece, V) * D * sizeof(float));
  }
  L.total = off;
  return L;
}

// [parts, rows, cols] bf16 (or fp32), `pitch` elements between rows, part_rows
// rows between parts, box of 128 bytes x box_rows.
bool make_map3(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t parts, int64_t pitch,
               int64_t part_rows, int box_rows, bool f32 = false) {
  tc::EncodeFn enc = tc::encoder();
  if (!enc) return false;
  const int64_t es = f32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
  cuuint64_t strides[2] = {(cuuint64_t)(pitch * es), (cuuint64_t)(part_rows * pitch * es)};
  cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base),
             dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// follows: the kernel before it on the stream is one of this call's.
template <int KIND, int PARTS, bool FEW> cudaError_t launch(const Args &a, bool follows, cudaStream_t st) {
  auto *k = ce_product_kernel<KIND, PARTS, FEW>;
  const int ring = a.stages * join_of(KIND, PARTS) * block_bytes_of(PARTS, a.a_bytes, a.bn);
  const int smem = ring + extra_of(KIND, PARTS, a.a_bytes) + 1024;
  // The leave is the kernel's on this device, for every host thread: one value for
  // all calls, so that none takes it from another's launch.
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LEAVE);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(a.units, pair_count())));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = follows;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, a);
}
template <int KIND> cudaError_t launch(const Args &a, int parts, bool few, bool follows, cudaStream_t st) {
  // fp32 operands: only G's entry at the target differs
  if (parts == 3)
    return KIND == GRAD && few ? launch<KIND, 3, KIND == GRAD>(a, follows, st)
                               : launch<KIND, 3, false>(a, follows, st);
  return few ? launch<KIND, 1, true>(a, follows, st) : launch<KIND, 1, false>(a, follows, st);
}

// Rows of a K-major operand's load: a CTA's share, or what there is of it.
int box_of(int64_t rows, int share) { return (int)std::min<int64_t>(share, up(rows, 8) * 8); }

void whole_k(Gemm &g, int64_t m, int64_t n, int64_t k, int bn, int runs = 1) {
  g.a_box = box_of(m, 128);
  g.b_box = box_of(n, bn / 2);
  g.m = m;
  g.n = n;
  g.mt = (int32_t)up(m, BM);
  g.nt = (int32_t)up(n, bn);
  g.kb = g.kb_split = (int32_t)up(k, BK) * runs;
  g.splits = 1;
}

// The bf16 rows of x and w: themselves, or packed into the workspace.
struct Rows {
  const void *x, *w;
  int64_t xp, wp;  // pitches
};
cudaError_t rows_of(const Layout &L, const void *x, int64_t xs, const void *w, int64_t N, int64_t D, int64_t V,
                    char *ws, Rows &r, cudaStream_t st) {
  if (!L.pack) {
    r = Rows{x, w, xs, D};
    return cudaSuccess;
  }
  const unsigned grid = (unsigned)std::min<int64_t>(up(N + V, 8), 8 * tc::sm_count());
  __nv_bfloat16 *xp = (__nv_bfloat16 *)(ws + L.off_x), *wp = (__nv_bfloat16 *)(ws + L.off_w);
  if (L.parts == 3)
    ce_pack_kernel<3, float><<<grid, 256, 0, st>>>((const float *)x, N, xs, xp, (const float *)w, V, wp, D, L.pitch);
  else
    ce_pack_kernel<1, __nv_bfloat16><<<grid, 256, 0, st>>>((const __nv_bfloat16 *)x, N, xs, xp,
                                                           (const __nv_bfloat16 *)w, V, wp, D, L.pitch);
  mark_launch("ce_pack", st);
  r = Rows{xp, wp, L.pitch, L.pitch};
  return cudaGetLastError();
}

cudaError_t add_splits(const float *part, int splits, int64_t n, int32_t dtype, void *out, cudaStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(up(n, 1024), 16 * tc::sm_count());
  const bool wide = n % 4 == 0 && ((uintptr_t)out & 15) == 0;
  cudaError_t e;
  if (dtype == GLACORE_BF16)
    e = launch_follow(wide ? ce_sum_kernel<__nv_bfloat16, true> : ce_sum_kernel<__nv_bfloat16, false>, dim3(grid),
                      dim3(256), st, part, splits, n, (__nv_bfloat16 *)out);
  else
    e = launch_follow(wide ? ce_sum_kernel<float, true> : ce_sum_kernel<float, false>, dim3(grid), dim3(256), st, part,
                      splits, n, (float *)out);
  mark_launch("ce_sum", st);
  return e;
}

glacore_status check(const void *x, const void *w, int64_t N, int64_t D, int64_t V, int64_t xs, int32_t dtype) {
  const int64_t lim = (int64_t)1 << 30;
  if (N < 0 || D < 1 || V < 1 || N > lim || D > (1 << 22) - 64 || V > lim || (xs != 0 && xs < D) ||
      (dtype != GLACORE_BF16 && dtype != GLACORE_F32))
    return GLACORE_ERR_INVALID_ARG;
  if (N == 0) return GLACORE_OK;
  if (!x || !w || ((uintptr_t)x & 15) || ((uintptr_t)w & 15)) return GLACORE_ERR_INVALID_ARG;
  if (dtype == GLACORE_BF16 && D % 8 == 0 && xs % 8 != 0) return GLACORE_ERR_INVALID_ARG;
  return GLACORE_OK;
}

}  // namespace ce
}  // namespace glacore

using namespace glacore;
using namespace glacore::ce;

extern "C" {

size_t linear_ce_fwd_workspace_size(int64_t N, int64_t D, int64_t V, int32_t dtype) {
  if (check(nullptr, nullptr, 0, D, V, 0, dtype) || N < 1 || N > ((int64_t)1 << 30)) return 0;
  return ce::layout(N, D, V, dtype, false).total;
}
size_t linear_ce_bwd_workspace_size(int64_t N, int64_t D, int64_t V, int32_t dtype) {
  if (check(nullptr, nullptr, 0, D, V, 0, dtype) || N < 1 || N > ((int64_t)1 << 30)) return 0;
  return ce::layout(N, D, V, dtype, true).total;
}

glacore_status linear_ce_fwd(const void *x, const void *w, const int64_t *target, int64_t N, int64_t D, int64_t V,
                             int64_t x_stride, int32_t dtype, float *loss, float *lse, void *workspace,
                             size_t workspace_bytes, glacore_stream_t stream) {
  begin_marks();
  const glacore_status s = check(x, w, N, D, V, x_stride, dtype);
  if (s || N == 0) return s;
  if (!target || !loss || !lse || ((uintptr_t)target & 7) || (((uintptr_t)loss | (uintptr_t)lse) & 3))
    return GLACORE_ERR_INVALID_ARG;
  const ce::Layout L = ce::layout(N, D, V, dtype, false);
  if (!workspace || workspace_bytes < L.total || ((uintptr_t)workspace & 255)) return GLACORE_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  if (const cudaError_t be = tc::bind_context()) return status_of(be);
  char *ws = (char *)workspace;
  Rows r;
  cudaError_t e = rows_of(L, x, x_stride ? x_stride : D, w, N, D, V, ws, r, st);
  if (e != cudaSuccess) return status_of(e);
  Args a;
  memset(&a, 0, sizeof(a));
  Gemm &g = a.g[0];
  if (!make_map3(&g.a, r.x, D, N, L.parts, r.xp, N, box_of(N, 128)) ||
      !make_map3(&g.b, r.w, D, V, L.parts, r.wp, V, box_of(V, L.bn_z / 2)))
    return status_of(cudaErrorInvalidValue);
  whole_k(g, N, V, D, L.bn_z);
  a.units0 = a.units = (int64_t)g.mt * g.nt;
  a.bn = L.bn_z;
  a.a_bytes = box_of(N, 128) * BK * 2;
  a.stages = stages_of(STATS, L.parts, a.a_bytes, a.bn);
  a.N = N;
  a.V = V;
  a.target = target;
  a.part = (float2 *)(ws + L.off_part);
  a.zt = (float *)(ws + L.off_zt);
  a.err = device_error_ptr();
  e = ce::launch<STATS>(a, L.parts, L.few, L.pack, st);
  mark_launch("ce_stats", st);
  if (e != cudaSuccess) return status_of(e);
  const int64_t slots = up(V, L.bn_z / 2);  // tile halves that hold part of the vocabulary
  auto merge = [&](auto *typed, auto few) {
    typedef std::remove_const_t<std::remove_pointer_t<decltype(typed)>> T;
    const Targets<T> targets = {typed, (const T *)w, x_stride ? x_stride : D, D};
    return launch_follow(ce_merge_kernel<T, decltype(few)::value>, dim3((unsigned)up(N, MERGE_ROWS)),
                         dim3(MERGE_ROWS, MERGE_LANES), st, targets, (const float2 *)a.part, slots, N, V, target,
                         (const float *)a.zt, loss, lse, a.err);
  };
  const auto *xb = (const __nv_bfloat16 *)x;
  if (!L.few)
    e = merge(xb, std::false_type());  // reads no x
  else if (dtype == GLACORE_F32)
    e = merge((const float *)x, std::true_type());
  else
    e = merge(xb, std::true_type());
  mark_launch("ce_merge", st);
  return status_of(e);
}

glacore_status linear_ce_bwd(const void *x, const void *w, const int64_t *target, const float *lse,
                             const float *dloss, int64_t N, int64_t D, int64_t V, int64_t x_stride, int32_t dtype,
                             void *dx, void *dw, void *workspace, size_t workspace_bytes, glacore_stream_t stream) {
  begin_marks();
  const glacore_status s = check(x, w, N, D, V, x_stride, dtype);
  if (s) return s;
  const size_t es = dtype == GLACORE_F32 ? 4 : 2;
  if (!dw || ((uintptr_t)dw & 15) || ((uintptr_t)dx & 15)) return GLACORE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (N == 0) return status_of(cudaMemsetAsync(dw, 0, (size_t)V * D * es, st));
  if (!target || !lse || !dloss || !dx || ((uintptr_t)target & 7) || (((uintptr_t)lse | (uintptr_t)dloss) & 3))
    return GLACORE_ERR_INVALID_ARG;
  const ce::Layout L = ce::layout(N, D, V, dtype, true);
  if (!workspace || workspace_bytes < L.total || ((uintptr_t)workspace & 255)) return GLACORE_ERR_WORKSPACE;
  if (const cudaError_t be = tc::bind_context()) return status_of(be);
  char *ws = (char *)workspace;
  Rows r;
  cudaError_t e = rows_of(L, x, x_stride ? x_stride : D, w, N, D, V, ws, r, st);
  if (e != cudaSuccess) return status_of(e);
  int *err = device_error_ptr();
  const __nv_bfloat16 *xt = (const __nv_bfloat16 *)(ws + L.off_xt);
  float *unit = L.parts == 1 ? (float *)(ws + L.off_unit) : nullptr;  // three parts hold dloss as it is
  float *at = L.few ? (float *)(ws + L.off_at) : nullptr;
  const int64_t gy = up(D, 64), xs = x_stride ? x_stride : D;
  const dim3 grid((unsigned)(up(N, 64) + 1 + (L.few ? up(N, gy) : 0)), (unsigned)gy, (unsigned)L.parts);
  __nv_bfloat16 *to = (__nv_bfloat16 *)(ws + L.off_xt);
  const __nv_bfloat16 *rows = (const __nv_bfloat16 *)r.x;
  auto prepare = [&](auto *typed) {
    typedef std::remove_const_t<std::remove_pointer_t<decltype(typed)>> T;
    const Targets<T> targets = {typed, (const T *)w, xs, D};
    if (L.pack)
      return launch_follow(ce_prepare_kernel<T>, grid, dim3(256), st, targets, lse, at, rows, N, D, r.xp, L.xt_pitch, to,
                           dloss, target, V, unit);
    ce_prepare_kernel<T><<<grid, 256, 0, st>>>(targets, lse, at, rows, N, D, r.xp, L.xt_pitch, to, dloss, target, V,
                                               unit);
    return cudaGetLastError();
  };
  e = dtype == GLACORE_F32 ? prepare((const float *)x) : prepare((const __nv_bfloat16 *)x);
  mark_launch("ce_prepare", st);
  if (e != cudaSuccess) return status_of(e);
  for (int64_t i = 0; i < L.pieces; ++i) {
    const int64_t v0 = i * L.piece, cols = std::min(L.piece, V - v0);
    // the piece's rows of w (its parts stay V rows apart)
    const char *wp = (const char *)r.w + (size_t)v0 * r.wp * 2;
    Args a;
    memset(&a, 0, sizeof(a));
    a.bn = L.bn_z;
    a.a_bytes = box_of(N, 128) * BK * 2;
    a.stages = stages_of(GRAD, L.parts, a.a_bytes, a.bn);
    a.N = N;
    a.V = V;
    a.v0 = v0;
    a.target = target;
    a.lse = lse;
    a.dloss = dloss;
    a.unit = unit;
    a.at_target = at;
    a.err = err;
    auto w_map = [&](CUtensorMap *m, int box_rows) {
      return make_map3(m, wp, D, cols, L.parts, r.wp, V, box_rows);
    };
    auto g_map = [&](CUtensorMap *m, int box_rows) {
      return make_map3(m, ws + L.off_g, cols, N, L.g_parts, L.gpitch, N, box_rows);
    };
    if (!make_map3(&a.g[0].a, r.x, D, N, L.parts, r.xp, N, box_of(N, 128)) ||
        !w_map(&a.g[0].b, box_of(cols, L.bn_z / 2)))
      return status_of(cudaErrorInvalidValue);
    whole_k(a.g[0], N, cols, D, L.bn_z);
    // all of G's columns: the tiles' are written whole
    if (L.parts == 1 && !make_map3(&a.g[0].o, ws + L.off_g, L.gpitch, N, L.g_parts, L.gpitch, N, 32))
      return status_of(cudaErrorInvalidValue);
    a.g[0].out = ws + L.off_g;
    a.g[0].out_pitch = L.gpitch;
    a.units0 = a.units = (int64_t)a.g[0].mt * a.g[0].nt;
    e = ce::launch<GRAD>(a, L.parts, L.few, true, st);
    mark_launch("ce_grad", st);
    if (e != cudaSuccess) return status_of(e);
    // dx^T (K = the piece) and dw of the piece (K = the tokens)
    a.bn = L.bn;
    a.a_bytes = (int)A_BYTES;
    a.stages = stages_of(PRODUCT, L.parts, a.a_bytes, a.bn);
    Gemm &gx = a.g[0], &gw = a.g[1];
    if (!w_map(&gx.a, 64) || !g_map(&gx.b, box_of(N, L.bn / 2)) || !g_map(&gw.a, 64) ||
        !make_map3(&gw.b, xt, N, D, L.parts, L.xt_pitch, D, box_of(D, L.bn / 2)))
      return status_of(cudaErrorInvalidValue);
    whole_k(gx, D, N, cols, L.bn);
    gx.a_mn = 1;
    gx.kb_split = L.run;
    gx.splits = (int32_t)up(gx.kb, L.run);  // no more than the first piece's
    gx.out_f32 = L.dx_f32 || dtype == GLACORE_F32;
    gx.add = i > 0;
    gx.trans = 1;
    gx.out = L.dx_f32 ? (void *)(ws + L.off_dx) : dx;
    whole_k(gw, cols, D, N, L.bn, L.sums);  // two parts of G: one after the other
    gw.a_mn = 1;
    gw.kb_split = L.run_w;
    gw.splits = L.splits_w;
    char *dw_piece = (char *)dw + (size_t)v0 * D * es;
    gw.out_f32 = L.dw_sums || dtype == GLACORE_F32;
    gw.out = L.dw_sums ? ws + L.off_dw : dw_piece;
    gw.wide_out = D % (gw.out_f32 ? 4 : 8) == 0;
    if (L.parts == 1 && gw.wide_out && !make_map3(&gw.o, gw.out, D, cols, gw.splits, D, cols, 32, gw.out_f32))
      return status_of(cudaErrorInvalidValue);
    a.units0 = (int64_t)gx.mt * gx.nt * gx.splits;
    a.units = a.units0 + (int64_t)gw.mt * gw.nt * gw.splits;
    a.skip = deal(a.units0, gx.kb_split, a.units - a.units0, gw.kb_split).skip;
    e = ce::launch<PRODUCT>(a, L.parts, L.few, true, st);
    mark_launch("ce_product", st);
    if (e == cudaSuccess && L.dw_sums)
      e = add_splits((const float *)(ws + L.off_dw), gw.splits, cols * D, dtype, dw_piece, st);
    if (e != cudaSuccess) return status_of(e);
  }
  if (L.dx_f32) e = add_splits((const float *)(ws + L.off_dx), L.splits * L.sums, N * D, dtype, dx, st);
  return status_of(e);
}

}  // extern "C"
