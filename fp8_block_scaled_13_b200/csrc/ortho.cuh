// Orthogonalising a weight update by Newton-Schulz products, as the Muon
// optimiser does (Jordan et al., "Muon", 2024: a quintic iteration):
//   X0 = G / (|G|_F + eps);   steps times:  M = X X^T,  R = b M + c M^2,  X <- a X + R X
// on the smaller side of G: for a tall G (more rows than columns) M = X^T X
// and X <- a X + X R.
//
// Precision.  The iteration lifts small singular values by up to a = 3.4 a
// step while it cancels large terms (3.4 - 4.8 + 2.0) in the large ones, so a
// rounding of X that the next step sees as part of X comes out amplified:
// with all operands in BF16 the result is off by 1e-2 (Gaussian G) to 0.17 (a
// few strong directions over a floor, as gradients have), against 1.7e-3 for
// the rounding of the BF16 result.  Here X is held as two FP16 terms, hi + lo
// (22 significant bits), and only what enters a product is rounded to FP16,
// off the diagonal: with M = D + O and R = D' + O' (D, D' diagonal, in FP32)
//   M^2 = O O + D O + O D + D^2,      a X + R X = (a + D') X + O' X,
// the tensor cores compute X X^T, O O and O' X from FP16 operands, one product
// each, and the epilogues add the rest in FP32.  X itself is exact to 22 bits, the
// diagonals come from FP32 sums (of operands that are rounded where X X^T is long,
// see below).  Two things keep what the operands lose small for every gradient:
//  - It is rounded at random (up or down by how near the value lies), so that
//    over the long sums it averages out.  Rounded to nearest, equal entries all
//    err alike: all-equal gradients of 160 x 1342 and 640 x 5377 were 1.0e-2 and
//    1.1e-2 off, where they now are off by the rounding of the result alone.
//  - What X loses must not leave the span of X's rows and columns, since a
//    direction that X lacks is lifted by a = 3.4 in each later step.  O' (X - hi)
//    does leave it, by what the diagonal is missing; R (X - hi) does not.  So D'
//    multiplies hi alone, and all of X only in the last two steps, where
//    nothing lifts it any more and what the hi term loses would count at the
//    large directions.  (D' X throughout: a rank-1 gradient was 2e-3 to 3e-3 off at
//    sides of 130 to 300, and after ten steps by 0.2 to 0.9 of its size.)
// Off by 3e-4 to 1.1e-3 in 5 steps, before out is rounded, at sides above 128, for
// Gaussian, low-rank, all-equal, sign, block and row-repeating gradients (to
// nearest, the Gaussian ones 3e-4 to 6e-4, now 5e-4 to 9e-4).  More steps lift
// whatever is there: each takes what X's 22 bits and FP32 sums leave in a
// direction that G lacks up by a, to 2e-2 to 7e-2 in ten steps.  (Two BF16 terms
// per operand and three products each took twice as long: 2168 us against 1133
// for 12288 x 2048.)  A short sum averages less, so X X^T over up to kOrthoExactK
// takes three products, hi hi + hi lo + lo hi, and R X of up to kOrthoFewRows rows
// two, R hi + R lo, where launches and not products are the time anyway.
// Powers of two keep FP16 in range: X is stored times 2^10, M times 2^13, R
// times 2^12, which holds while |X| < 64, |M| < 8 and |R| < 16 off the
// diagonal; the iteration keeps singular values near 1.
//
// A whole call is one launch after two passes over G (its norm, and the two FP16
// terms of X0).  Its 3 * steps products D[i, j] = sum_k A[i, k] B[j, k] follow
// each other over a barrier -- of the cluster, where the grid is one, else of a
// cooperative grid's CTAs through memory: the next product's loads wait for it,
// everything else (TMEM, barriers, tensor maps) stays set up.  (One launch per product took 3.8 us each in tails and starts;
// with 128-column tiles and without the split below: 313 us against 267 for
// 2048 x 2048, 1133 against 800 to 950, by the power cap, for 12288 x 2048.)
//
// A product runs tcgen05 kind::f16 on CTA pairs, in tiles of 256 rows and 256,
// 128 or 64 columns, FP32 accumulators in TMEM (two, so that a tile's epilogue
// overlaps the next one's products), fed by TMA through a ring of 64-deep
// stages.  256 columns let the loads (64 bytes a clock and SM at the full rate)
// just follow the tensor cores; 128 columns need 96 and got 0.57 of the rate
// on all SMs, but a small product is done sooner in narrow tiles on more of
// them, each with less of an epilogue.  An operand that is stored the other way
// round ([k][i]) is read MN-major, so nothing is ever transposed in memory.  M
// and R are symmetric: only tiles that reach the diagonal's 256 x 256 blocks or
// lie below are computed, and the epilogue writes those below also to their
// mirrored place.  The tiles that do not fill a round of all CTA pairs may be
// split along k over the idle pairs; each of them leaves the FP32 partials that
// it does not own in the workspace, waits for the others' and finishes its own
// share of the columns, so the epilogue is split as well.
// The epilogue's own inputs (O, or both terms of X) come by TMA into the buffer
// that the result then leaves from, a chunk of 32 x 32 ahead.  Bound by the
// tensor cores for large G, by the 3 * steps hand-overs for small ones.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "quant.cuh"

namespace puro {

enum OrthoProduct : int { kOrthoGram = 0, kOrthoPoly = 1, kOrthoUpdate = 2 };

constexpr int kOrthoNormBlocks = 592;  // most CTAs of the passes over G, one partial sum each
constexpr int64_t kOrthoExactK = 1024; // longest X X^T sum that takes three products
constexpr int64_t kOrthoFewRows = 128; // longest R X sum that takes two
constexpr int kOrthoLate = 2;           // last steps in which all of X meets the diagonal of R
constexpr float kXScale = 1024.f, kMScale = 8192.f, kRScale = 4096.f;
constexpr int kOrthoMaxSplit = 8;

// One of the three products, as every step takes it.  Unit u < full is a whole
// tile; the units after them are the remaining tiles in `split` parts each.
struct OrthoShape {
  int32_t rows_a, rows_b;   // D is [rows_a, rows_b]
  int32_t kblocks;          // ceil(K / 64)
  int32_t passes;           // 1: hi hi; 3: hi hi, hi lo, lo hi; the update's 2: R hi, R lo
  int32_t bn;               // columns of a tile: 256, 128 or 64 (its rows are 256)
  int32_t tiles_m, tiles_n;
  int32_t full, split, units;
};

struct OrthoParams {
  OrthoShape shape[3];
  int32_t steps;
  float a, b, c;
  float* diag;              // D, the diagonal of M
  float* diag_r;            // D', the diagonal of R
  uint32_t* grid_count;     // arrivals at the grid barrier; zero before the launch
  uint32_t* tile_count;     // [3][kSplitTiles][2] arrivals of a split tile's parts; zero before the launch
  float4* partial;          // [units of split tiles][kPartial]
  __nv_bfloat16* out;       // the BF16 result, by plain stores if out_tma is 0
  int64_t ld_out;
  int32_t out_tma;
  int32_t one_cluster;      // the grid is one cluster, whose barrier separates the products
};
constexpr int kPartial = 2 * 8 * 4 * 8 * 32;  // float4 of a tile's partials: [CTA][chunk][32 rows][8][lane]
constexpr int kSplitTiles = 74;  // most tiles that can be split: fewer than CTA pairs
constexpr int kOrthoCounters = 64 + 3 * kSplitTiles * 2;

// Tensor maps.  Operands: 64-wide boxes with the 128-byte swizzle, 64 rows if
// MN-major, else 128 rows (A) or half a tile's columns (B); epilogue: boxes of
// 32 x 32 with the 64-byte swizzle.
struct OrthoMaps {
  CUtensorMap gram[2][2], gram_b[2][2];  // X as the operands of X X^T: [buffer][hi, lo]
  CUtensorMap update[2][2];              // X as an operand of the update: [buffer][hi, lo]
  CUtensorMap o, o_b;                    // O, both operands of the square
  CUtensorMap r;                         // R, an operand of the update
  CUtensorMap ex[2][2], eo, er, out;
};

struct OrthoCfg {
  static constexpr uint32_t kTile = 128 * 128;        // 128 rows x 64 FP16
  static constexpr uint32_t kStageBytes = 2 * kTile;  // A and B of one CTA
  static constexpr int kStages = 4;                   // 128 KB
  static constexpr int kEpiWarps = 8;
  static constexpr uint32_t kBuf = 4096;              // hi and lo (or mirrored), 32 rows x 64 bytes each
  static constexpr int kBufs = 3;                     // a warp's chunks in flight
  static constexpr uint32_t kEpiBytes = kEpiWarps * kBufs * kBuf;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr uint32_t kOffEpi = kStages * kStageBytes;
  static constexpr uint32_t kOffBar = kOffEpi + kEpiBytes;
  static constexpr uint32_t kNumBars = 2 * kStages + 5 + 4 + kBufs * kEpiWarps;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kOffDiag = (kOffMisc + 16 + 127) / 128 * 128;  // a diagonal at each warp's 32 columns
  static constexpr uint32_t kSmemBytes = kOffDiag + kEpiWarps * 128 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t kTmemCols = 512;          // two accumulators
};

// Shared-memory matrix descriptor of an MN-major operand tile: 128-byte
// swizzled rows of 64 elements, one row per k; 8-row groups 1024 B apart
// (stride offset), 64-element column blocks of 64 rows 8192 B apart (leading
// offset).
__device__ __forceinline__ uint64_t desc_sw128_mnmajor(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192u >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

struct OrthoUnit {
  int32_t y0, x0;       // the tile's first row and column of D
  int32_t cols;         // columns of D that it computes: a multiple of 32, bn at most
  int32_t k0, k1;       // its 64-deep blocks, of kblocks * passes
  int32_t part, parts;  // its place among the parts of a split tile
  int32_t index;        // of the split tile
};

template <bool SYM>
__device__ __forceinline__ OrthoUnit ortho_unit(const OrthoShape& s, int32_t u) {
  OrthoUnit r;
  const uint32_t total = s.kblocks * s.passes;  // (times a part fits 32 bits: 2^25 blocks at most)
  int32_t t = u;
  r.part = 0;
  r.parts = 1;
  r.index = 0;
  r.k0 = 0;
  r.k1 = (int32_t)total;
  if (s.split > 1 && u >= s.full) {
    const uint32_t split = s.split, rest = u - s.full;
    r.index = (int32_t)(rest / split);
    r.part = (int32_t)(rest % split);
    r.parts = s.split;
    t = s.full + r.index;
    r.k0 = (int32_t)(total * r.part / split);
    r.k1 = (int32_t)(total * (r.part + 1) / split);
  }
  int32_t tm, tn;
  if (SYM) {
    // row by row of tiles that reach the diagonal's 256 x 256 blocks or lie below
    const int32_t per = s.bn == 256 ? 1 : s.bn == 128 ? 2 : 4;
    for (tm = 0;; ++tm) {
      const int32_t to_diag = (tm + 1) * per, n = to_diag < s.tiles_n ? to_diag : s.tiles_n;
      if (t < n) break;
      t -= n;
    }
    tn = t;
  } else if (s.tiles_n < s.tiles_m) {
    // along the shorter side of D first, so that tiles that run at the same
    // time share their part of X
    tm = (int32_t)((uint32_t)t / (uint32_t)s.tiles_n);
    tn = t - tm * s.tiles_n;
  } else {
    tn = s.tiles_m == 1 ? t : (int32_t)((uint32_t)t / (uint32_t)s.tiles_m);
    tm = t - tn * s.tiles_m;
  }
  r.y0 = tm * 256;
  r.x0 = tn * s.bn;
  const int32_t left = s.rows_b - r.x0;
  r.cols = left >= s.bn ? s.bn : (left + 31) / 32 * 32;
  return r;
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// The same with each value rounded up or down at random, by how near it lies, on
// bits 0..12 (lo) and 16..28 (hi) of `bits`.
__device__ __forceinline__ uint32_t half_pair_random(float lo, float hi, uint32_t bits) {
  uint32_t d;
  asm("cvt.rs.f16x2.f32 %0, %1, %2, %3;" : "=r"(d) : "f"(hi), "f"(lo), "r"(bits));
  return d;
}

// Bits for the roundings of a row's pairs of columns, from column `col` on, in
// one product: for the pair n, first + n * step.  They follow from the place
// alone, so that a result repeats.  (The constants are the odd ones among the
// binary fractions of the square roots of 2, 3, 11, 17 and 19.)
struct RoundBits {
  uint32_t first, step;
};
__device__ __forceinline__ RoundBits round_bits(int32_t row, int32_t col, int32_t product) {
  uint32_t h = (uint32_t)row * 0x6A09E667u + (uint32_t)col * 0xBB67AE85u + (uint32_t)product * 0x510E527Fu;
  h = (h ^ (h >> 15)) * 0x1F83D9ABu;
  h = (h ^ (h >> 14)) * 0x5BE0CD19u;
  return {h ^ (h >> 16), h * 0x6A09E667u + 0xBB67AE85u};
}

__device__ __forceinline__ float2 half_unpack(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

__device__ __forceinline__ void count_arrive(uint32_t* c) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(c) : "memory");
}

// Waits, bounded as every wait here, until *c has reached `target`.  (The
// release of an arrival covers what the arriving thread has learned of other
// threads' writes through a shared-memory barrier.)
__device__ __forceinline__ bool count_wait(const uint32_t* c, uint32_t target, volatile int* abort) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
    if ((int32_t)(v - target) >= 0) return true;
    if ((it & 15u) == 0) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        record_error(kErrDeviceTimeout);
        *abort = 1;
        return false;
      }
    }
  }
}

struct OrthoSmem {
  uint8_t* base;
  uint64_t *full, *empty, *accf, *acce, *drain, *ready, *done, *parts_out, *parts_in, *src;
  volatile int* abort_flag;
  uint32_t pair;  // rank of the pair's first CTA, the leader, in the cluster
};

// `p` in the pair's leader.
__device__ __forceinline__ uint32_t pair_leader(const OrthoSmem& sm, const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(sm.pair));
  return a;
}

// Arrive on `bar` in both CTAs of the pair when the MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(const OrthoSmem& sm, uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          bar),
      "h"((uint16_t)(3u << sm.pair))
      : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The loops below run in one thread each: a warp that elected a lane in every
// round took 470 cycles a 64-deep block, nearly as long as the products of 256
// columns and twice as long as those of 128 (1024 x 1024: 171 us against 151).
// A single thread's time is the number of its instructions, so addresses are
// 32-bit shared-memory ones and a descriptor's upper half stays constant.

__device__ __forceinline__ void ortho_tma(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// The producer's share of one product.  `blocks` counts the 64-deep blocks so
// far: block n goes through stage n % kStages.  What can be computed before the
// operands are there comes before `arrived`, the barrier between the products.
template <bool SYM, bool AMN, bool BMN, class Barrier>
__device__ __forceinline__ bool ortho_load(const OrthoSmem& sm, const OrthoShape& s, const CUtensorMap* ah,
                                           const CUtensorMap* al, const CUtensorMap* bh, const CUtensorMap* bl,
                                           int cluster_id, int clusters, uint32_t rank, uint32_t& blocks,
                                           const Barrier& arrived) {
  using C = OrthoCfg;
  constexpr int32_t kLoA = SYM ? 2 : 1;  // the pass that takes A's lo term (of R there is none)
  // both CTAs' bytes of a stage
  const uint32_t bytes = 2 * (C::kTile + (BMN ? (s.bn == 256 ? 16384u : 8192u) : (uint32_t)s.bn * 64));
  const uint32_t full = smem_u32(sm.full), empty = smem_u32(sm.empty), base = smem_u32(sm.base);
  const uint32_t to_leader = pair_leader(sm, sm.full) - full;
  const bool wide = s.bn == 256;
  const int32_t k_end = s.kblocks * 64;
  OrthoUnit t = ortho_unit<SYM>(s, cluster_id < s.units ? cluster_id : 0);
  if (!arrived()) return false;
  auto loop = [&]() {
    for (int32_t u = cluster_id; u < s.units;) {
      const int32_t a0 = t.y0 + 128 * (int32_t)rank;
      const int32_t b0 = t.x0 + (t.cols >> 1) * (int32_t)rank;
      int32_t pass = s.passes == 1 || t.k0 == 0 ? 0 : t.k0 / s.kblocks, k = (t.k0 - pass * s.kblocks) * 64;
      const CUtensorMap* ma = pass == kLoA ? al : ah;
      const CUtensorMap* mb = pass == 1 ? bl : bh;
      for (int32_t n = t.k1 - t.k0; n > 0; --n) {
        const uint32_t stage = blocks % C::kStages, odd = blocks / C::kStages & 1, at = full + stage * 8;
        ++blocks;
        if (!mbar_try_wait(empty + stage * 8, odd ^ 1) && !mbar_wait(&sm.empty[stage], odd ^ 1, sm.abort_flag))
          return false;
        if (rank == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(at), "r"(bytes) : "memory");
        const uint32_t bar = at + to_leader, da = base + stage * C::kStageBytes, db = da + C::kTile;
        if (AMN) {
          ortho_tma(da, ma, a0, k, bar);
          ortho_tma(da + 8192, ma, a0 + 64, k, bar);
        } else {
          ortho_tma(da, ma, k, a0, bar);
        }
        if (BMN) {
          ortho_tma(db, mb, b0, k, bar);
          if (wide) ortho_tma(db + 8192, mb, b0 + 64, k, bar);
        } else {
          ortho_tma(db, mb, k, b0, bar);
        }
        k += 64;
        if (k >= k_end) {
          k = 0;
          ++pass;
          ma = pass == kLoA ? al : ah;
          mb = pass == 1 ? bl : bh;
        }
      }
      u += clusters;
      if (u < s.units) t = ortho_unit<SYM>(s, u);
    }
    return true;
  };
  const bool ok = elect_one() ? loop() : true;
  return __all_sync(0xFFFFFFFFu, ok);
}

// D[tmem] (+)= A B^T for one M = 256, K = 16 slice of FP16 operands of the CTA pair;
// a and b are the descriptors' lower halves; the upper one says the same of both
// layouts (groups 1024 bytes apart, 128-byte swizzle).
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t"
      "}" ::"r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"((1024 >> 4) | (1 << 14) | (2 << 29))
      : "memory");
}

// The MMA issuer's, in the leader CTA.
template <bool SYM, bool AMN, bool BMN>
__device__ __forceinline__ bool ortho_mma(const OrthoSmem& sm, const OrthoShape& s, uint32_t tmem, int cluster_id,
                                          int clusters, uint32_t& blocks, uint32_t& it) {
  using C = OrthoCfg;
  constexpr uint32_t kStepA = AMN ? 2048 >> 4 : 32 >> 4;  // 16 elements along k
  constexpr uint32_t kStepB = BMN ? 2048 >> 4 : 32 >> 4;
  const uint64_t a_desc0 = AMN ? desc_sw128_mnmajor(smem_u32(sm.base)) : desc_sw128_kmajor(smem_u32(sm.base));
  const uint64_t b_desc0 = BMN ? desc_sw128_mnmajor(smem_u32(sm.base) + C::kTile)
                               : desc_sw128_kmajor(smem_u32(sm.base) + C::kTile);
  const uint32_t a_lo = (uint32_t)a_desc0, b_lo = (uint32_t)b_desc0;
  const uint32_t full = smem_u32(sm.full), empty = smem_u32(sm.empty);
  for (int32_t u = cluster_id; u < s.units; u += clusters, ++it) {
    const OrthoUnit t = ortho_unit<SYM>(s, u);
    // D FP32, A and B FP16 (formats 0), MN-major flags, N, M
    const uint32_t idesc = (1u << 4) | ((AMN ? 1u : 0u) << 15) | ((BMN ? 1u : 0u) << 16) |
                           ((uint32_t)(t.cols >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
    const uint32_t acc = it & 1, d = tmem + acc * 256;
    if (!mbar_wait(&sm.acce[acc], ((it >> 1) & 1) ^ 1, sm.abort_flag)) return false;
    tc_fence_after();
    uint32_t accumulate = 0;
    for (int32_t n = t.k1 - t.k0; n > 0; --n) {
      const uint32_t stage = blocks % C::kStages, odd = blocks / C::kStages & 1;
      ++blocks;
      if (!mbar_try_wait(full + stage * 8, odd) && !mbar_wait(&sm.full[stage], odd, sm.abort_flag)) return false;
      tc_fence_after();
      const uint32_t a = a_lo + stage * (C::kStageBytes >> 4), b = b_lo + stage * (C::kStageBytes >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        tc_mma_f16(d, a + k * kStepA, b + k * kStepB, idesc, accumulate);
        accumulate = 1;
      }
      pair_commit(sm, empty + stage * 8);
    }
    pair_commit(sm, smem_u32(&sm.accf[acc]));
  }
  return true;
}

// State of an epilogue warp that outlives a product.
struct OrthoEpiState {
  uint32_t it;         // tiles so far
  uint32_t buf;        // the next chunk's buffer
  uint32_t src_phase;  // phases of the source barriers
  uint32_t splits;     // split tiles so far
};

// An epilogue warp's: 32 rows of D, every other chunk of 32 columns.  Buffers
// hold rows of 64 bytes, their 16-byte pieces XORed with bits 1..2 of the row
// (the 64-byte swizzle): lanes that each touch their own row meet no bank
// twice.
template <int EPI, bool TALL>
__device__ __forceinline__ bool ortho_epilogue(const OrthoSmem& sm, const OrthoParams& p, const CUtensorMap* src_hi,
                                               const CUtensorMap* src_lo, const CUtensorMap* dst_hi,
                                               const CUtensorMap* dst_lo, uint32_t tmem, int cluster_id, int clusters,
                                               uint32_t rank, int step, OrthoEpiState& st) {
  using C = OrthoCfg;
  constexpr bool SYM = EPI != kOrthoUpdate;
  constexpr bool kCols = EPI == kOrthoPoly || (EPI == kOrthoUpdate && TALL);  // a diagonal goes by column
  const OrthoShape& s = p.shape[EPI];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sp = warp & 3, half = (warp - 2) >> 2;
  const bool last = EPI == kOrthoUpdate && step == p.steps - 1;
  uint8_t* bufs = sm.base + C::kOffEpi + (warp - 2) * C::kBufs * C::kBuf;
  uint64_t* src_bar = sm.src + (warp - 2) * C::kBufs;
  float* cols_diag = reinterpret_cast<float*>(sm.base + C::kOffDiag) + (warp - 2) * 32;
  const int sw = (lane >> 1) & 3;  // this lane's row's swizzle
  const float* diag = EPI == kOrthoPoly ? p.diag : p.diag_r;
  for (int32_t u = cluster_id; u < s.units; u += clusters, ++st.it) {
    const OrthoUnit t = ortho_unit<SYM>(s, u);
    const uint32_t acc = st.it & 1;
    const int32_t row0 = t.y0 + 128 * (int32_t)rank + sp * 32, row = row0 + lane;
    const int32_t chunks = t.cols >> 5;
    const int32_t c0 = t.part + t.parts * half, dc = 2 * t.parts;  // this warp's chunks
    const bool rows_in = row0 < s.rows_a;
    const bool mirror = SYM && t.x0 < t.y0;
    // brings the epilogue's inputs of a chunk into a buffer
    auto prefetch = [&](int32_t c, uint32_t b) {
      uint8_t* buf = bufs + b * C::kBuf;
      const int32_t x = t.x0 + c * 32;
      mbar_arrive_expect_tx(&src_bar[b], EPI == kOrthoUpdate ? 4096 : 2048);
      tma_load_2d<1>(buf, src_hi, x, row0, smem_u32(&src_bar[b]));
      if (EPI == kOrthoUpdate) tma_load_2d<1>(buf + 2048, src_lo, x, row0, smem_u32(&src_bar[b]));
    };
    auto after = [](uint32_t b, uint32_t n) { return b + n >= C::kBufs ? b + n - C::kBufs : b + n; };
    if (EPI != kOrthoGram && rows_in && lane == 0) {
      // every buffer's last store has read it by now, or is waited for
      bulk_wait_group_read<0>();
#pragma unroll
      for (uint32_t n = 0; n < C::kBufs; ++n)
        if (c0 + (int32_t)n * dc < chunks) prefetch(c0 + (int32_t)n * dc, after(st.buf, n));
    }
    float dr = 0.f;
    if (row < s.rows_a && (EPI == kOrthoPoly || (EPI == kOrthoUpdate && !TALL))) dr = __ldcg(diag + row);
    // the diagonal at a chunk's columns, one per lane
    auto load_diag = [&](int32_t c) {
      const int32_t x = t.x0 + c * 32 + lane;
      return kCols && c < chunks && x < s.rows_b ? __ldcg(diag + x) : 0.f;
    };
    float d_next = load_diag(c0);
    // (ready before the products are: parameters and the diagonal are a miss away)
    float raw_scale = p.c / (kMScale * kMScale), c_r = p.c * (kRScale / kMScale);
    float base_r = EPI == kOrthoPoly ? fmaf(p.c, dr, p.b) * (kRScale / kMScale) : p.a + dr;
    float d_own = dr * fmaf(p.c, dr, p.b);
    // the update's factors of X's terms: a + D' for hi, for lo a, and a + D' late or
    // where R meets lo too
    const float late = s.passes == 2 || step + kOrthoLate >= p.steps ? 1.f : 0.f, k_low = fmaf(late, dr, p.a);
    if (EPI != kOrthoGram) asm volatile("" : "+f"(raw_scale), "+f"(c_r), "+f"(base_r), "+f"(d_own));
    if (!mbar_wait_warp(&sm.accf[acc], (st.it >> 1) & 1, sm.abort_flag)) return false;
    tc_fence_after();
    const uint32_t t_base = tmem + ((uint32_t)(sp * 32) << 16) + acc * 256;
    float4* part = p.partial + (int64_t)(u - s.full) * kPartial;
    if (t.parts > 1) {
      // the chunks that other parts own leave as FP32
      for (int32_t c = half; c < chunks && rows_in; c += 2) {
        if (c % t.parts == t.part) continue;
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_base + c * 32, r);
        tmem_ld_wait();
        regs_after_wait(r);
        float4* d = part + (((int)rank * 8 + c) * 4 + sp) * 256 + lane;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          d[q * 32] = make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                                  __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.parts_out);
      if (warp == 2) {
        if (!mbar_wait_warp(sm.parts_out, st.splits & 1, sm.abort_flag)) return false;
        bool ok = true;
        if (lane == 0) {
          uint32_t* count = p.tile_count + (EPI * kSplitTiles + t.index) * 2 + rank;
          count_arrive(count);
          ok = count_wait(count, (uint32_t)((step + 1) * t.parts), sm.abort_flag);
          if (ok) mbar_arrive(sm.parts_in);
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
      }
      if (!mbar_wait_warp(sm.parts_in, st.splits & 1, sm.abort_flag)) return false;
      ++st.splits;
    }
    for (int32_t c = c0, j = 0; c < chunks && rows_in; c += dc, ++j, st.buf = after(st.buf, 1)) {
      const uint32_t b = st.buf;
      uint8_t* buf_h = bufs + b * C::kBuf;
      uint8_t* buf_l = buf_h + 2048;
      uint8_t* my_h = buf_h + lane * 64;
      uint8_t* my_l = buf_l + lane * 64;
      const int32_t col0 = t.x0 + c * 32;
      uint32_t r[32];
      tmem_ld_32x32b_x32(t_base + c * 32, r);
      if (kCols) {
        // (32 shuffles instead: 4096 x 1024 in 170 us against 166)
        cols_diag[lane] = d_next;
        __syncwarp();
      }
      d_next = load_diag(c + dc);
      if (EPI == kOrthoGram) {
        if (lane == 0) bulk_wait_group_read<C::kBufs - 1>();
        __syncwarp();
      } else {
        // the next chunk's buffer, where it was not filled at the start: the
        // store from it is the last but one
        if (j + 1 >= C::kBufs && c + dc < chunks && lane == 0) {
          bulk_wait_group_read<1>();
          prefetch(c + dc, after(b, 1));
        }
        if (!mbar_wait_warp(&src_bar[b], (st.src_phase >> b) & 1, sm.abort_flag)) return false;
        st.src_phase ^= 1u << b;
      }
      tmem_ld_wait();
      regs_after_wait(r);
      float v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
      // the other parts, in an order that depends on the chunk alone (its owner)
#pragma unroll 2
      for (int32_t k = 1; k < t.parts; ++k) {
        const int32_t other = t.part + k < t.parts ? k : k - t.parts;
        const float4* d = part + (int64_t)other * kPartial + (((int)rank * 8 + c) * 4 + sp) * 256 + lane;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 f = __ldcg(d + q * 32);
          v[4 * q] += f.x;
          v[4 * q + 1] += f.y;
          v[4 * q + 2] += f.z;
          v[4 * q + 3] += f.w;
        }
      }
      const bool on_diag = SYM && row0 == col0;  // both are multiples of 32: element `lane` of the row
      if (EPI == kOrthoGram) {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= kMScale / (kXScale * kXScale);
        if (on_diag) {
          float d = 0.f;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            d = e == lane ? v[e] : d;
            v[e] = e == lane ? 0.f : v[e];
          }
          if (row < s.rows_a) p.diag[row] = d * (1.f / kMScale);
        }
      } else {
        if (EPI == kOrthoPoly && on_diag) {
          float own = 0.f;
          // on the diagonal, D' = c ((O O)_ii + D_i^2) + b D_i
#pragma unroll
          for (int e = 0; e < 32; ++e) own = e == lane ? v[e] : own;
          if (row < s.rows_a) p.diag_r[row] = fmaf(own, raw_scale, d_own);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 h4 = *reinterpret_cast<const uint4*>(my_h + ((q ^ sw) << 4));
          const uint4 l4 = EPI == kOrthoUpdate ? *reinterpret_cast<const uint4*>(my_l + ((q ^ sw) << 4)) : make_uint4(0, 0, 0, 0);
          const uint32_t hw[4] = {h4.x, h4.y, h4.z, h4.w}, lw[4] = {l4.x, l4.y, l4.z, l4.w};
          f2 dv[4] = {};
          if (kCols) {
            const float4 d0 = *reinterpret_cast<const float4*>(cols_diag + 8 * q);
            const float4 d1 = *reinterpret_cast<const float4*>(cols_diag + 8 * q + 4);
            dv[0] = f2_of(d0.x, d0.y);
            dv[1] = f2_of(d0.z, d0.w);
            dv[2] = f2_of(d1.x, d1.y);
            dv[3] = f2_of(d1.z, d1.w);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int e = 8 * q + 2 * w;
            const float2 h = half_unpack(hw[w]);
            const f2 raw = f2_of(v[e], v[e + 1]);
            f2 x;
            if (EPI == kOrthoPoly) {
              // R = c (O O + O (D_i + D_j)) + b O off the diagonal: O (c D_j + (c D_i + b)) + c O O
              x = fma2(raw, f2_both(raw_scale * kRScale), mul2(f2_of(h.x, h.y), fma2(f2_both(c_r), dv[w], f2_both(base_r))));
            } else {
              const float2 l = half_unpack(lw[w]);
              const f2 k = kCols ? fma2(dv[w], f2_both(1.f), f2_both(base_r)) : f2_both(base_r);
              const f2 k_lo = kCols ? fma2(dv[w], f2_both(late), f2_both(p.a)) : f2_both(k_low);
              x = fma2(k, f2_of(h.x, h.y), fma2(k_lo, f2_of(l.x, l.y), mul2(raw, f2_both(1.f / kRScale))));
            }
            const float2 xs = f2_get(x);
            v[e] = xs.x;
            v[e + 1] = xs.y;
          }
        }
        if (EPI == kOrthoPoly && on_diag) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = e == lane ? 0.f : v[e];
        }
      }
      if (last) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * q + 2 * e] * (1.f / kXScale), v[8 * q + 2 * e + 1] * (1.f / kXScale));
            o[e] = *reinterpret_cast<uint32_t*>(&h);
          }
          *reinterpret_cast<uint4*>(my_h + ((q ^ sw) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (!p.out_tma) {
          // rows that do not start on 16-byte boundaries: plain stores
          __syncwarp();
          for (int y = 0; y < 32 && row0 + y < s.rows_a; ++y)
            if (col0 + lane < s.rows_b)
              p.out[(int64_t)(row0 + y) * p.ld_out + col0 + lane] = *reinterpret_cast<const __nv_bfloat16*>(
                  buf_h + y * 64 + (((lane >> 3) ^ ((y >> 1) & 3)) << 4) + (lane & 7) * 2);
          fence_proxy_async_smem();
          __syncwarp();
          continue;
        }
      } else {
        RoundBits rb = round_bits(row, col0, 3 * step + EPI);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 8 * q + 2 * e;
            hi[e] = half_pair_random(v[i], v[i + 1], rb.first);
            rb.first += rb.step;
            if (EPI == kOrthoUpdate) {
              const float2 h = half_unpack(hi[e]);
              const float2 d = f2_get(fma2(f2_of(h.x, h.y), f2_both(-1.f), f2_of(v[i], v[i + 1])));
              lo[e] = half_pair(d.x, d.y);
            } else if (mirror) {
              // the transposed tile beside it: rows i and i + 1, column lane
              uint8_t* d = buf_l + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2;
              *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(hi[e]);
              *reinterpret_cast<uint16_t*>(d + 64) = static_cast<uint16_t>(hi[e] >> 16);
            }
          }
          *reinterpret_cast<uint4*>(my_h + ((q ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if (EPI == kOrthoUpdate)
            *reinterpret_cast<uint4*>(my_l + ((q ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(dst_hi, buf_h, col0, row0);
        if (EPI == kOrthoUpdate && !last) tma_store_2d(dst_lo, buf_l, col0, row0);
        if (mirror) tma_store_2d(dst_hi, buf_l, row0, col0);
        bulk_commit_group();
      }
    }
    // (every TMEM read of this warp has been waited for)
    tc_fence_before();
    __syncwarp();
    if (lane == 0)
      asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(pair_leader(sm, &sm.acce[acc])) : "memory");
  }
  return true;
}

template <bool TALL>
__global__ void __launch_bounds__(OrthoCfg::kThreads, 1)
    ortho_kernel(const __grid_constant__ OrthoMaps m, const __grid_constant__ OrthoParams p) {
  using C = OrthoCfg;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  OrthoSmem sm;
  sm.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  sm.full = reinterpret_cast<uint64_t*>(sm.base + C::kOffBar);
  sm.empty = sm.full + S;
  sm.accf = sm.empty + S;
  sm.acce = sm.accf + 2;
  sm.drain = sm.acce + 2;
  sm.ready = sm.drain + 1;
  sm.done = sm.ready + 1;
  sm.parts_out = sm.done + 1;
  sm.parts_in = sm.parts_out + 1;
  sm.src = sm.parts_in + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm.base + C::kOffMisc);
  sm.abort_flag = reinterpret_cast<volatile int*>(sm.base + C::kOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank() & 1;
  sm.pair = cluster_ctarank() & ~1u;
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int products = 3 * p.steps;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.accf[a], 1);
      mbar_init(&sm.acce[a], C::kEpiWarps * 2);
    }
    mbar_init(sm.drain, 1);
    mbar_init(sm.ready, 1);
    mbar_init(sm.done, C::kEpiWarps);
    mbar_init(sm.parts_out, C::kEpiWarps);
    mbar_init(sm.parts_in, 1);
    for (int w = 0; w < C::kBufs * C::kEpiWarps; ++w) mbar_init(&sm.src[w], 1);
    *sm.abort_flag = 0;
    fence_barrier_init();
    const CUtensorMap* maps = reinterpret_cast<const CUtensorMap*>(&m);
    for (int i = 0; i < (int)(sizeof(OrthoMaps) / sizeof(CUtensorMap)); ++i) prefetch_tmap(maps + i);
  }
  if (warp == 1) {
    tmem_alloc<2>(tmem_slot, C::kTmemCols);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_or_block_sync<2>();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // Between two products every CTA's results reach memory.  In one cluster every
  // warp arrives at the cluster's barrier when it has done its share and waits
  // there before the next (one that has given up a wait keeps doing both, so
  // that the others are not held); else the epilogues count a CTA's arrival in
  // memory and the producers wait for the count.
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t blocks = 0;  // of the elected lane, which is the same every time
    bool ok = true;
    for (int i = 0; i < products; ++i) {
      if (i > 0 && p.one_cluster) {
        __syncwarp();
        cluster_arrive();
      }
      auto arrived = [&]() {
        if (i == 0) return true;
        if (p.one_cluster) {
          cluster_wait();
          fence_proxy_async_global();
          return true;
        }
        bool here = true;
        if (lane == 0) here = count_wait(p.grid_count, (uint32_t)i * gridDim.x, sm.abort_flag);
        if (!__all_sync(0xFFFFFFFFu, here)) return false;
        fence_proxy_async_global();
        if (lane == 0) mbar_arrive(sm.ready);
        return true;
      };
      const int type = i % 3, cur = (i / 3) & 1;
      if (!ok)
        arrived();  // (one cluster: the others still wait for this warp)
      else if (type == kOrthoGram)
        ok = ortho_load<true, TALL, TALL>(sm, p.shape[kOrthoGram], &m.gram[cur][0], &m.gram[cur][1], &m.gram_b[cur][0],
                                          &m.gram_b[cur][1], cluster_id, clusters, rank, blocks, arrived);
      else if (type == kOrthoPoly)
        ok = ortho_load<true, false, false>(sm, p.shape[kOrthoPoly], &m.o, &m.o, &m.o_b, &m.o_b, cluster_id, clusters,
                                            rank, blocks, arrived);
      else if (TALL)
        ok = ortho_load<false, false, false>(sm, p.shape[kOrthoUpdate], &m.update[cur][0], &m.update[cur][1], &m.r, &m.r,
                                             cluster_id, clusters, rank, blocks, arrived);
      else
        ok = ortho_load<false, false, true>(sm, p.shape[kOrthoUpdate], &m.r, &m.r, &m.update[cur][0], &m.update[cur][1],
                                            cluster_id, clusters, rank, blocks, arrived);
      if (!ok && !p.one_cluster) break;
    }
    // let every load of the pair land before the leader can exit
    if (leader && elect_one()) {
      for (uint32_t n = blocks < S ? 0 : blocks - S; n < blocks; ++n) {
        volatile int no_abort = 0;
        mbar_wait(&sm.full[n % S], n / S & 1, &no_abort, 100000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader) {
      uint32_t blocks = 0, it = 0;  // of the elected lane
      bool ok = true;
      for (int i = 0; i < products; ++i) {
        if (i > 0 && p.one_cluster) {
          __syncwarp();
          cluster_arrive();
          cluster_wait();
        }
        if (!ok) continue;
        const int type = i % 3;
        if (elect_one()) {
          if (type == kOrthoGram)
            ok = ortho_mma<true, TALL, TALL>(sm, p.shape[kOrthoGram], tmem, cluster_id, clusters, blocks, it);
          else if (type == kOrthoPoly)
            ok = ortho_mma<true, false, false>(sm, p.shape[kOrthoPoly], tmem, cluster_id, clusters, blocks, it);
          else
            ok = ortho_mma<false, false, !TALL>(sm, p.shape[kOrthoUpdate], tmem, cluster_id, clusters, blocks, it);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok && !p.one_cluster) break;
      }
      if (elect_one()) tc_commit_local<2>(sm.drain);
      volatile int no_abort = 0;
      mbar_wait(sm.drain, 0, &no_abort, 100000000ull);
      __syncwarp();
    } else if (p.one_cluster) {
      for (int i = 1; i < products; ++i) {
        cluster_arrive();
        cluster_wait();
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    OrthoEpiState st = {0, 0, 0, 0};
    bool ok = true;
    for (int i = 0; i < products; ++i) {
      const int type = i % 3, step = i / 3, cur = step & 1;
      if (i > 0) {
        if (p.one_cluster)
          cluster_wait();
        else if (!mbar_wait_warp(sm.ready, (uint32_t)(i - 1) & 1, sm.abort_flag))
          break;
        fence_proxy_async_global();
      }
      if (!ok) {
      } else if (type == kOrthoGram)
        ok = ortho_epilogue<kOrthoGram, TALL>(sm, p, nullptr, nullptr, &m.eo, &m.eo, tmem, cluster_id, clusters, rank,
                                              step, st);
      else if (type == kOrthoPoly)
        ok = ortho_epilogue<kOrthoPoly, TALL>(sm, p, &m.eo, &m.eo, &m.er, &m.er, tmem, cluster_id, clusters, rank, step,
                                              st);
      else
        ok = ortho_epilogue<kOrthoUpdate, TALL>(sm, p, &m.ex[cur][0], &m.ex[cur][1],
                                                step == p.steps - 1 ? &m.out : &m.ex[cur ^ 1][0], &m.ex[cur ^ 1][1],
                                                tmem, cluster_id, clusters, rank, step, st);
      if (i == products - 1 || (!ok && !p.one_cluster)) break;
      // this warp's results are in memory (the wait makes its bulk stores visible to
      // this thread; the fence that orders them before TMA loads is the readers')
      if (lane == 0) bulk_wait_group<0>();
      __syncwarp();
      if (p.one_cluster) {
        cluster_arrive();
        continue;
      }
      // all of this CTA's: one arrival at the grid's barrier
      if (lane == 0) mbar_arrive(sm.done);
      if (warp == 2) {
        if (!mbar_wait_warp(sm.done, (uint32_t)i & 1, sm.abort_flag)) break;
        if (lane == 0) count_arrive(p.grid_count);
        __syncwarp();
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
    // loads of the epilogue's inputs that a given-up wait left in flight
    if (lane == 0 && *sm.abort_flag) {
      for (int b = 0; b < C::kBufs; ++b)
        for (uint32_t ph = 0; ph < 2; ++ph) {
          volatile int no_abort = 0;
          mbar_wait(&sm.src[(warp - 2) * C::kBufs + b], ph, &no_abort, 100000000ull);
        }
    }
    __syncwarp();
  }

  tc_fence_before();
  cluster_or_block_sync<2>();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, C::kTmemCols);
}

// The two passes that make X0.  The first sums the squares of G [n, k], one
// partial sum per CTA in a fixed order; the second writes 2^10 G / (|G|_F + eps)
// as FP16 hi + lo.  VEC: rows start on 16-byte boundaries.
struct OrthoSplitParams {
  const void* g;
  int64_t ld_g, ld_x;
  int32_t n, k;
  float eps;
  __half* hi;
  __half* lo;
  float* part;   // one per CTA (both passes have the same grid)
  uint32_t* counters;  // [kOrthoCounters], set to zero for the products
};

// Up to 8 values of a row from column c on, zeros past the end.
template <bool F32, bool VEC>
__device__ __forceinline__ void load_g8(const OrthoSplitParams& p, int64_t r, int32_t c, float (&v)[8]) {
  if (VEC && c + 8 <= p.k) {
    if (F32) {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.g) + r * p.ld_g + c);
      const float4 a = s[0], b = s[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.g) + r * p.ld_g + c);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = c + i >= p.k ? 0.f
           : F32        ? static_cast<const float*>(p.g)[r * p.ld_g + c + i]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.g)[r * p.ld_g + c + i]);
}

// n ceil(k / 8) pieces fit 32 bits (n, k <= 65536).
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const OrthoSplitParams p) {
  __shared__ float sm[8];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kOrthoCounters; i += 256) p.counters[i] = 0u;
  float s = 0.f;
  const uint32_t per_row = (uint32_t)(p.k + 7) / 8, total = per_row * (uint32_t)p.n;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const uint32_t r = i / per_row;
    float v[8];
    load_g8<F32, VEC>(p, r, (int32_t)(i - r * per_row) * 8, v);
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = fmaf(v[e], v[e], t);
    s += t;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) s += sm[w];
    p.part[blockIdx.x] = s;
  }
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) ortho_split_kernel(const OrthoSplitParams p) {
  pdl_wait();
  pdl_trigger();
  float s = 0.f;  // every warp adds the partial sums in the same order
  for (int i = threadIdx.x & 31; i < (int)gridDim.x; i += 32) s += p.part[i];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  const float scale = kXScale / (sqrtf(s) + p.eps);
  const uint32_t per_row = (uint32_t)(p.k + 7) / 8, total = per_row * (uint32_t)p.n;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const uint32_t r = i / per_row, c = (i - r * per_row) * 8;
    float v[8];
    load_g8<F32, VEC>(p, r, (int32_t)c, v);
    uint32_t h[4], l[4];
    const RoundBits rb = round_bits((int32_t)r, (int32_t)c, -1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[2 * e] * scale, y = v[2 * e + 1] * scale;
      h[e] = half_pair_random(x, y, rb.first + e * rb.step);
      const float2 f = half_unpack(h[e]);
      l[e] = half_pair(x - f.x, y - f.y);
    }
    // rows of X are padded to multiples of 8, so the whole piece may be written
    *reinterpret_cast<uint4*>(p.hi + (int64_t)r * p.ld_x + c) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(p.lo + (int64_t)r * p.ld_x + c) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

}  // namespace puro
