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
// each, and the epilogues add the rest in FP32 from the exact parts.  What the
// operands lose is random and averaged over the long sums, and the large,
// coherent parts -- the diagonals, and X itself -- are not rounded at all: off by
// 3e-4 to 8e-4 for Gaussian, low-rank, power-law and geometric spectra.  (Two
// BF16 terms per operand and three products each were as exact and took twice
// as long: 2168 us against 1133 for 12288 x 2048.)  A short sum averages
// less, so X X^T over up to kOrthoExactK takes three products, hi hi + hi lo +
// lo hi, where launches and not products are the time anyway.
// Powers of two keep FP16 in range: X is stored times 2^10, M times 2^13, R
// times 2^12, which holds while |X| < 64, |M| < 8 and |R| < 16 off the
// diagonal; the iteration keeps singular values near 1.
//
// All three products of a step are one kernel, D[i, j] = sum_k P[i, k] Q[j, k]:
// tcgen05 kind::f16 on CTA pairs (256-row tiles), FP32 accumulators in TMEM,
// fed by TMA.  An operand that is stored the other way round ([k][i]) is read
// MN-major, so nothing is ever transposed in memory.  M and R are symmetric:
// only tiles on or below the diagonal are computed and the epilogue writes
// each one also to its mirrored place; with 256 x 128 tiles a 2048-wide M is 72
// units, one wave of the 74 CTA pairs.  Bound by the tensor cores for large G, by launches
// (2 + 3 steps, overlapped by programmatic dependent launch) for small ones.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace puro {

enum OrthoEpilogue : int { kOrthoGram = 0, kOrthoPoly = 1, kOrthoUpdate = 2 };

constexpr int kOrthoNormBlocks = 592;  // CTAs of the norm pass, one partial sum each
constexpr int64_t kOrthoExactK = 1024; // longest X X^T sum that takes three products
constexpr float kXScale = 1024.f, kMScale = 8192.f, kRScale = 4096.f;

struct OrthoParams {
  int32_t rows_a, rows_b;   // D is [rows_a, rows_b]
  int32_t kblocks;          // ceil(K / 64)
  int32_t passes;           // 1: hi hi; 3: hi hi, hi lo, lo hi
  int32_t tiles_m, tiles_n;
  int32_t units;            // tiles; kOrthoGram / kOrthoPoly: those on or below the diagonal
  float a, b, c;
  float* diag;              // Gram: D written; Poly: D read
  float* diag_r;            // Poly: D' written; Update: D' read
  const __half* src_hi;     // Poly: O (times 2^13); Update: X hi
  const __half* src_lo;     // Update: X lo
  int64_t ld_src;
  __nv_bfloat16* out;       // last step: the BF16 result
  int64_t ld_out;
  int32_t col_diag;         // Update: D' goes by column (tall G)
  int32_t last, out_tma;    // last step; the result goes out by TMA (else by plain stores)
};

template <int BN>
struct OrthoCfg {
  static constexpr int kBM = 256;              // tile rows (a CTA pair)
  static constexpr int kBNC = BN / 2;          // rows of Q in each CTA
  static constexpr uint32_t kTileA = 128 * 128;       // 128 rows x 64 FP16
  static constexpr uint32_t kTileB = kBNC * 128;
  static constexpr uint32_t kStageBytes = kTileA + kTileB;
  static constexpr int kStages = BN == 256 ? 6 : 8;   // 192 KB
  static constexpr int kEpiWarps = 8;
  static constexpr int kEpiCols = BN / 2;
  static constexpr uint32_t kEpiBytes = kEpiWarps * 4096;  // hi and lo, 32 rows x 64 bytes each
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr uint32_t kOffEpi = kStages * kStageBytes;
  static constexpr uint32_t kOffBar = kOffEpi + kEpiBytes;
  static constexpr uint32_t kNumBars = 2 * kStages + 5;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t kTmemCols = 2 * BN;       // two accumulators
};

// D[tmem] (+)= A B^T for one M = 256, K = 16 slice of FP16 operands of the CTA pair.
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory matrix descriptor of an MN-major operand tile: 128-byte
// swizzled rows of 64 elements, one row per k; 8-row groups 1024 B apart
// (stride offset), 64-element column blocks of 64 rows 8192 B apart (leading
// offset).
__device__ __forceinline__ uint64_t desc_sw128_mnmajor(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192u >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// Tile (tm, tn) of unit u.  Symmetric results count the 128-column tiles on or
// below the diagonal row block by row block (2 I + 2 of them in row block I).
template <bool SYM>
__device__ __forceinline__ void ortho_tile(const OrthoParams& p, int u, int& tm, int& tn) {
  if (SYM) {
    int i = 0;
    for (;; ++i) {
      const int n = 2 * i + 2 < p.tiles_n ? 2 * i + 2 : p.tiles_n;
      if (u < n) break;
      u -= n;
    }
    tm = i;
    tn = u;
  } else {
    tn = u / p.tiles_m;
    tm = u - tn * p.tiles_m;
  }
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float2 half_unpack(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

template <int BN, bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(OrthoCfg<BN>::kThreads, 1)
    ortho_gemm_kernel(const __grid_constant__ CUtensorMap tm_ah, const __grid_constant__ CUtensorMap tm_al,
                      const __grid_constant__ CUtensorMap tm_bh, const __grid_constant__ CUtensorMap tm_bl,
                      const __grid_constant__ CUtensorMap tm_dh, const __grid_constant__ CUtensorMap tm_dl,
                      const __grid_constant__ OrthoParams p) {
  using C = OrthoCfg<BN>;
  constexpr int S = C::kStages;
  constexpr bool SYM = EPI != kOrthoUpdate;
  // D FP32, A and B FP16 (formats 0), MN-major flags, N, M
  constexpr uint32_t kIdesc = (1u << 4) | ((AMN ? 1u : 0u) << 15) | ((BMN ? 1u : 0u) << 16) |
                              ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(C::kBM >> 4) << 24);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + S;
  uint64_t* accf = empty + S;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1, clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf[a], 1);
      mbar_init(&acce[a], C::kEpiWarps * 2);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_ah);
    prefetch_tmap(&tm_al);
    prefetch_tmap(&tm_bh);
    prefetch_tmap(&tm_bl);
    prefetch_tmap(&tm_dh);
    prefetch_tmap(&tm_dl);
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
  pdl_trigger();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
    bool ok = true;
    for (int u = cluster_id; u < p.units && ok; u += clusters) {
      int tm, tn;
      ortho_tile<SYM>(p, u, tm, tn);
      const int a0 = tm * C::kBM + 128 * (int)rank;
      const int b0 = tn * BN + C::kBNC * (int)rank;
      for (int i = 0; i < p.kblocks * p.passes; ++i) {
        const int pass = i / p.kblocks, k0 = (i - pass * p.kblocks) * 64;
        if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
          const uint32_t bar = leader_addr<2>(&full[stage]);
          uint8_t* da = smem + stage * C::kStageBytes;
          uint8_t* db = da + C::kTileA;
          const CUtensorMap* ma = pass == 2 ? &tm_al : &tm_ah;
          const CUtensorMap* mb = pass == 1 ? &tm_bl : &tm_bh;
          if (AMN) {
            tma_load_2d<2>(da, ma, a0, k0, bar);
            tma_load_2d<2>(da + 8192, ma, a0 + 64, k0, bar);
          } else {
            tma_load_2d<2>(da, ma, k0, a0, bar);
          }
          if (BMN) {
#pragma unroll
            for (int h = 0; h < C::kBNC / 64; ++h) tma_load_2d<2>(db + 8192 * h, mb, b0 + 64 * h, k0, bar);
          } else {
            tma_load_2d<2>(db, mb, k0, b0, bar);
          }
        }
        issued_mask |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == S) { stage = 0; phase ^= 1; }
      }
    }
    // let every load of the pair land before the leader can exit
    if (lane == 0 && leader) {
      for (int s = 0; s < S; ++s)
        if (issued_mask & (1u << s)) {
          volatile int no_abort = 0;
          mbar_wait(&full[s], (issued_phase >> s) & 1u, &no_abort, 100000000ull);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader) {
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t base = smem_u32(smem);
      const uint64_t a_desc0 = AMN ? desc_sw128_mnmajor(base) : desc_sw128_kmajor(base);
      const uint64_t b_desc0 = BMN ? desc_sw128_mnmajor(base + C::kTileA) : desc_sw128_kmajor(base + C::kTileA);
      constexpr uint32_t kStepA = AMN ? 2048 >> 4 : 32 >> 4;  // 16 elements along k
      constexpr uint32_t kStepB = BMN ? 2048 >> 4 : 32 >> 4;
      for (int u = cluster_id; u < p.units && ok; u += clusters, ++it) {
        const int acc = it & 1;
        if (!mbar_wait_warp(&acce[acc], ((it >> 1) & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int i = 0; i < p.kblocks * p.passes; ++i) {
          if (!mbar_wait_warp(&full[stage], phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = a_desc0 + (uint64_t)(stage * (C::kStageBytes >> 4));
            const uint64_t bd = b_desc0 + (uint64_t)(stage * (C::kStageBytes >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_f16(d, ad + k * kStepA, bd + k * kStepB, kIdesc, (i | k) != 0 ? 1u : 0u);
            tc_commit_all<2>(&empty[stage]);
          }
          if (++stage == S) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_all<2>(&accf[acc]);
      }
      if (elect_one()) tc_commit_local<2>(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort, 100000000ull);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int sp = warp & 3, half = (warp - 2) >> 2;
    uint8_t* buf_h = smem + C::kOffEpi + (warp - 2) * 4096;
    uint8_t* buf_l = buf_h + 2048;
    constexpr int kChunks = C::kEpiCols / 32;
    constexpr int kSrc = EPI == kOrthoUpdate ? 8 : 4;  // 16-byte words of the source per thread and chunk
    // hands a staged pair of 32 x 32 tiles to TMA
    auto store = [&](int x, int y, bool low) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&tm_dh, buf_h, x, y);
        if (low) tma_store_2d(&tm_dl, buf_l, x, y);
        bulk_commit_group();
      }
    };
    // waits until the buffers may be written once more
    auto again = [&]() {
      if (lane == 0) bulk_wait_group_read<0>();
      __syncwarp();
    };
    // this thread's row of a chunk of the source: O, or X hi and X lo
    auto load_src = [&](int row, int col0, uint4 (&v)[8]) {
      if (EPI == kOrthoGram) return;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool in = row < p.rows_a && col0 + 8 * q < p.rows_b;
        const int64_t at = (int64_t)row * p.ld_src + col0 + 8 * q;
        v[q] = in ? *reinterpret_cast<const uint4*>(p.src_hi + at) : make_uint4(0, 0, 0, 0);
        if (kSrc == 8) v[4 + q] = in ? *reinterpret_cast<const uint4*>(p.src_lo + at) : make_uint4(0, 0, 0, 0);
      }
    };
    int it = 0;
    for (int u = cluster_id; u < p.units; u += clusters, ++it) {
      int tm, tn;
      ortho_tile<SYM>(p, u, tm, tn);
      const int acc = it & 1;
      const int row0 = tm * C::kBM + 128 * (int)rank + sp * 32;
      const int row = row0 + lane;
      const int colh = tn * BN + half * C::kEpiCols;
      const bool mirror = SYM && (tn >> 1) < tm;
      uint4 src[8];
      load_src(row, colh, src);
      const float dr = row < p.rows_a ? (EPI == kOrthoPoly ? p.diag[row] : EPI == kOrthoUpdate && !p.col_diag ? p.diag_r[row] : 0.f) : 0.f;
      if (!mbar_wait_warp(&accf[acc], (it >> 1) & 1, abort_flag)) break;
      tc_fence_after();
      const uint32_t t_base = tmem + ((uint32_t)(sp * 32) << 16) + acc * BN + half * C::kEpiCols;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int col0 = colh + c * 32;
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_base + c * 32, r);
        uint4 cur[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) cur[q] = src[q];
        if (c + 1 < kChunks) load_src(row, col0 + 32, src);
        tmem_ld_wait();
        regs_after_wait(r);
        if (c == kChunks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader<2>(&acce[acc]);
        }
        if (row0 >= p.rows_a || col0 >= p.rows_b) continue;
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
        if (EPI == kOrthoGram) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            v[e] *= kMScale / (kXScale * kXScale);
            if (row == col0 + e) {
              if (row < p.rows_a) p.diag[row] = v[e] * (1.f / kMScale);
              v[e] = 0.f;
            }
          }
        }
        if (EPI != kOrthoGram) {
          // D or D' of the columns
          const float* dp = EPI == kOrthoPoly ? p.diag : p.diag_r;
          const float dc = (EPI == kOrthoPoly || p.col_diag) && col0 + lane < p.rows_b ? dp[col0 + lane] : 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t hw[4] = {cur[q].x, cur[q].y, cur[q].z, cur[q].w};
            const uint32_t lw[4] = {cur[4 + q].x, cur[4 + q].y, cur[4 + q].z, cur[4 + q].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int e = 8 * q + 2 * w;
              const float2 h = half_unpack(hw[w]);
              const float d0 = __shfl_sync(0xFFFFFFFFu, dc, e), d1 = __shfl_sync(0xFFFFFFFFu, dc, e + 1);
              if (EPI == kOrthoPoly) {
                // R = c (O O + O (D_i + D_j)) + b O off the diagonal
                v[e] = fmaf(v[e], p.c * (kRScale / (kMScale * kMScale)), h.x * (kRScale / kMScale) * fmaf(p.c, dr + d0, p.b));
                v[e + 1] = fmaf(v[e + 1], p.c * (kRScale / (kMScale * kMScale)), h.y * (kRScale / kMScale) * fmaf(p.c, dr + d1, p.b));
              } else {
                const float2 l = half_unpack(lw[w]);
                v[e] = fmaf(p.a + dr + d0, h.x + l.x, v[e] * (1.f / kRScale));
                v[e + 1] = fmaf(p.a + dr + d1, h.y + l.y, v[e + 1] * (1.f / kRScale));
              }
            }
          }
          if (EPI == kOrthoPoly) {
            // on it, D' = c ((O O)_ii + D_i^2) + b D_i
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (row == col0 + e) {
                if (row < p.rows_a)
                  p.diag_r[row] = fmaf(__uint_as_float(r[e]), p.c / (kMScale * kMScale), dr * fmaf(p.c, dr, p.b));
                v[e] = 0.f;
              }
          }
        }
        if (EPI == kOrthoUpdate && p.last) {
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e] * (1.f / kXScale), v[2 * e + 1] * (1.f / kXScale));
            o[e] = *reinterpret_cast<uint32_t*>(&h);
          }
          again();
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(buf_h + lane * 64 + 16 * q) = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          if (p.out_tma) {
            store(col0, row0, false);
          } else {
            // rows that do not start on 16-byte boundaries: plain stores
            __syncwarp();
            for (int y = 0; y < 32 && row0 + y < p.rows_a; ++y)
              if (col0 + lane < p.rows_b)
                p.out[(int64_t)(row0 + y) * p.ld_out + col0 + lane] = reinterpret_cast<const __nv_bfloat16*>(buf_h)[y * 32 + lane];
            __syncwarp();
          }
          continue;
        }
        uint32_t hi[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) hi[e] = half_pair(v[2 * e], v[2 * e + 1]);
        again();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          *reinterpret_cast<uint4*>(buf_h + lane * 64 + 16 * q) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
          if (EPI == kOrthoUpdate) {
            uint32_t lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 h = half_unpack(hi[4 * q + e]);
              lo[e] = half_pair(v[8 * q + 2 * e] - h.x, v[8 * q + 2 * e + 1] - h.y);
            }
            *reinterpret_cast<uint4*>(buf_l + lane * 64 + 16 * q) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (SYM && mirror) {
          // the transposed tile beside it, in the second buffer
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            uint16_t* t = reinterpret_cast<uint16_t*>(buf_l) + 64 * e + lane;
            t[0] = static_cast<uint16_t>(hi[e]);
            t[32] = static_cast<uint16_t>(hi[e] >> 16);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_dh, buf_h, col0, row0);
            tma_store_2d(&tm_dh, buf_l, row0, col0);
            bulk_commit_group();
          }
        } else {
          store(col0, row0, EPI == kOrthoUpdate);
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
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
  float* part;   // [kOrthoNormBlocks]
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
  for (int i = threadIdx.x & 31; i < kOrthoNormBlocks; i += 32) s += p.part[i];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  const float scale = kXScale / (sqrtf(s) + p.eps);
  const uint32_t per_row = (uint32_t)(p.k + 7) / 8, total = per_row * (uint32_t)p.n;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const uint32_t r = i / per_row, c = (i - r * per_row) * 8;
    float v[8];
    load_g8<F32, VEC>(p, r, (int32_t)c, v);
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[2 * e] * scale, y = v[2 * e + 1] * scale;
      h[e] = half_pair(x, y);
      const float2 f = half_unpack(h[e]);
      l[e] = half_pair(x - f.x, y - f.y);
    }
    // rows of X are padded to multiples of 8, so the whole piece may be written
    *reinterpret_cast<uint4*>(p.hi + (int64_t)r * p.ld_x + c) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(p.lo + (int64_t)r * p.ld_x + c) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

}  // namespace puro
