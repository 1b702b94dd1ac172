// Orthogonalising a weight update by Newton-Schulz products, as the Muon
// optimiser does (Jordan et al., "Muon", 2024: a quintic iteration):
//   X0 = G / (|G|_F + eps);   steps times:  M = X X^T,  P = a I + b M + c M^2,  X <- P X
// on the smaller side of G: for a tall G (more rows than columns) M = X^T X
// and X <- X P.
//
// Precision.  The iteration multiplies small singular values by up to a = 3.4
// a step while it cancels large terms (3.4 - 4.8 + 2.0) in the large ones, so
// operand roundings come out amplified: with BF16 operands the result is off
// by 1e-2 (Gaussian G) to 0.17 (a few strong directions over a floor, as
// gradients have), with FP16 ones by 2e-3 to 2e-2, against 1.7e-3 for the
// rounding of the BF16 result.  So every operand is held as two BF16 terms,
// hi + lo (16 significant bits), and each product takes three tensor-core
// products, hi hi + hi lo + lo hi, into one FP32 accumulator: off by 1.5e-5
// to 2.5e-4.  A BF16 G is exact in one term and takes fewer products.
//
// All three products of a step are one kernel, D[i, j] = sum_k P[i, k] Q[j, k]:
// tcgen05 kind::f16 on CTA pairs (256-row tiles), fed by TMA through a ring of
// 64-deep stages that hold the hi and lo tiles of both operands -- four tiles
// loaded for three products.  An operand that is stored the other way round
// ([k][i]) is read MN-major, so nothing is ever transposed in memory.  M and
// P are symmetric: only tiles on or below the diagonal are computed and the
// epilogue writes each one also to its mirrored place; with 256 x 128 tiles a
// 2048-wide M is 72 units, one wave of the 74 CTA pairs.  The norm of G
// scales the first M (by its square) and the first X in the epilogue, so G is
// read once to split it.  Bound by the tensor cores for large G, by launches
// (1 + 3 steps, overlapped by programmatic dependent launch) for small ones.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace puro {

enum OrthoEpilogue : int { kOrthoGram = 0, kOrthoPoly = 1, kOrthoUpdate = 2 };

constexpr int kOrthoNormBlocks = 592;  // CTAs of the splitting pass, one partial sum each

struct OrthoParams {
  int32_t rows_a, rows_b;   // D is [rows_a, rows_b]
  int32_t kblocks;          // ceil(K / 64)
  int32_t tiles_m, tiles_n;
  int32_t units;            // tiles; kOrthoGram / kOrthoPoly: those on or below the diagonal
  int32_t terms_a, terms_b; // 2: hi and lo, 1: hi only (lo is zero)
  float alpha, beta, diag;  // kOrthoPoly: alpha acc + beta M + diag I
  const __nv_bfloat16* m_hi;
  const __nv_bfloat16* m_lo;
  int64_t ld_m;
  const float* norm_part;   // kOrthoNormBlocks sums of squares of G, or null (already normalised)
  float eps;
  __nv_bfloat16* out;       // last step: the BF16 result, by plain stores if out_tma is 0
  int64_t ld_out;
  int32_t last, out_tma;
};

template <int BN>
struct OrthoCfg {
  static constexpr int kBM = 256;              // tile rows (a CTA pair)
  static constexpr int kBNC = BN / 2;          // rows of Q in each CTA
  static constexpr uint32_t kTileA = 128 * 128;       // 128 rows x 64 BF16
  static constexpr uint32_t kTileB = kBNC * 128;
  static constexpr uint32_t kStageBytes = 2 * (kTileA + kTileB);
  static constexpr int kStages = BN == 256 ? 3 : 4;   // 192 KB
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

// D[tmem] (+)= A B^T for one M = 256, K = 16 slice of BF16 operands of the CTA pair.
__device__ __forceinline__ void tc_mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
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

// 1 / (|G|_F + eps) from the partial sums, by a converged warp.
__device__ __forceinline__ float ortho_scale(const OrthoParams& p, int lane) {
  if (!p.norm_part) return 1.f;
  float s = 0.f;
  for (int i = lane; i < kOrthoNormBlocks; i += 32) s += p.norm_part[i];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  return 1.f / (sqrtf(s) + p.eps);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
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
  // D FP32, A and B BF16, MN-major flags, N, M
  constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((AMN ? 1u : 0u) << 15) | ((BMN ? 1u : 0u) << 16) |
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
    const uint32_t tx = 2 * (p.terms_a * C::kTileA + p.terms_b * C::kTileB);
    bool ok = true;
    for (int u = cluster_id; u < p.units && ok; u += clusters) {
      int tm, tn;
      ortho_tile<SYM>(p, u, tm, tn);
      const int a0 = tm * C::kBM + 128 * (int)rank;
      const int b0 = tn * BN + C::kBNC * (int)rank;
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], tx);
          const uint32_t bar = leader_addr<2>(&full[stage]);
          uint8_t* st = smem + stage * C::kStageBytes;
          const int k0 = kb * 64;
          for (int t = 0; t < p.terms_a; ++t) {
            const CUtensorMap* m = t ? &tm_al : &tm_ah;
            uint8_t* d = st + t * C::kTileA;
            if (AMN) {
              tma_load_2d<2>(d, m, a0, k0, bar);
              tma_load_2d<2>(d + 8192, m, a0 + 64, k0, bar);
            } else {
              tma_load_2d<2>(d, m, k0, a0, bar);
            }
          }
          for (int t = 0; t < p.terms_b; ++t) {
            const CUtensorMap* m = t ? &tm_bl : &tm_bh;
            uint8_t* d = st + 2 * C::kTileA + t * C::kTileB;
            if (BMN) {
              for (int h = 0; h < C::kBNC / 64; ++h) tma_load_2d<2>(d + 8192 * h, m, b0 + 64 * h, k0, bar);
            } else {
              tma_load_2d<2>(d, m, k0, b0, bar);
            }
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
      const uint64_t b_desc0 = BMN ? desc_sw128_mnmajor(base + 2 * C::kTileA) : desc_sw128_kmajor(base + 2 * C::kTileA);
      constexpr uint32_t kStepA = AMN ? 2048 >> 4 : 32 >> 4;  // 16 elements along k
      constexpr uint32_t kStepB = BMN ? 2048 >> 4 : 32 >> 4;
      for (int u = cluster_id; u < p.units && ok; u += clusters, ++it) {
        const int acc = it & 1;
        if (!mbar_wait_warp(&acce[acc], ((it >> 1) & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!mbar_wait_warp(&full[stage], phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ah = a_desc0 + (uint64_t)(stage * (C::kStageBytes >> 4));
            const uint64_t bh = b_desc0 + (uint64_t)(stage * (C::kStageBytes >> 4));
            const uint64_t al = ah + (C::kTileA >> 4), bl = bh + (C::kTileB >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_bf16(d, ah + k * kStepA, bh + k * kStepB, kIdesc, (kb | k) != 0 ? 1u : 0u);
            if (p.terms_b > 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) tc_mma_bf16(d, ah + k * kStepA, bl + k * kStepB, kIdesc, 1u);
            }
            if (p.terms_a > 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) tc_mma_bf16(d, al + k * kStepA, bh + k * kStepB, kIdesc, 1u);
            }
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
    float scale = 1.f;
    if (EPI != kOrthoPoly) scale = ortho_scale(p, lane);
    if (EPI == kOrthoGram) scale *= scale;
    // hands a staged 32 x 32 pair of tiles to TMA; `again` waits until the
    // buffers may be written once more
    auto store = [&](int x, int y, bool low) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&tm_dh, buf_h, x, y);
        if (low) tma_store_2d(&tm_dl, buf_l, x, y);
        bulk_commit_group();
      }
    };
    auto again = [&]() {
      if (lane == 0) bulk_wait_group_read<0>();
      __syncwarp();
    };
    int it = 0;
    for (int u = cluster_id; u < p.units; u += clusters, ++it) {
      int tm, tn;
      ortho_tile<SYM>(p, u, tm, tn);
      const int acc = it & 1;
      const int row0 = tm * C::kBM + 128 * (int)rank + sp * 32;
      const int row = row0 + lane;
      const bool mirror = SYM && (tn >> 1) < tm;
      if (!mbar_wait_warp(&accf[acc], (it >> 1) & 1, abort_flag)) break;
      tc_fence_after();
      const uint32_t t_base = tmem + ((uint32_t)(sp * 32) << 16) + acc * BN + half * C::kEpiCols;
      for (int c = 0; c < C::kEpiCols / 32; ++c) {
        const int col0 = tn * BN + half * C::kEpiCols + c * 32;
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_base + c * 32, r);
        tmem_ld_wait();
        regs_after_wait(r);
        if (c == C::kEpiCols / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader<2>(&acce[acc]);
        }
        if (row0 >= p.rows_a || col0 >= p.rows_b) continue;
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]) * (EPI == kOrthoPoly ? p.alpha : scale);
        if (EPI == kOrthoPoly) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (row < p.rows_a && col0 + 8 * q < p.rows_b) {
              const uint4 h = *reinterpret_cast<const uint4*>(p.m_hi + (int64_t)row * p.ld_m + col0 + 8 * q);
              const uint4 l = *reinterpret_cast<const uint4*>(p.m_lo + (int64_t)row * p.ld_m + col0 + 8 * q);
              const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float m0 = __uint_as_float(hw[e] << 16) + __uint_as_float(lw[e] << 16);
                const float m1 = __uint_as_float(hw[e] & 0xFFFF0000u) + __uint_as_float(lw[e] & 0xFFFF0000u);
                v[8 * q + 2 * e] = fmaf(p.beta, m0, v[8 * q + 2 * e]);
                v[8 * q + 2 * e + 1] = fmaf(p.beta, m1, v[8 * q + 2 * e + 1]);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (row == col0 + e) v[e] += p.diag;
        }
        // hi and lo of each pair of columns
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          hi[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
          lo[e] = bf16_pair(v[2 * e] - __uint_as_float(hi[e] << 16),
                            v[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
        }
        if (EPI == kOrthoUpdate && p.last && !p.out_tma) {
          // a result whose rows do not start on 16-byte boundaries: plain
          // stores, a row at a time through shared memory
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(buf_h + lane * 64 + 16 * q) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
          __syncwarp();
          for (int y = 0; y < 32 && row0 + y < p.rows_a; ++y)
            if (col0 + lane < p.rows_b)
              p.out[(int64_t)(row0 + y) * p.ld_out + col0 + lane] = reinterpret_cast<const __nv_bfloat16*>(buf_h)[y * 32 + lane];
          continue;
        }
        const bool low = !(EPI == kOrthoUpdate && p.last);
        again();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          *reinterpret_cast<uint4*>(buf_h + lane * 64 + 16 * q) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
          *reinterpret_cast<uint4*>(buf_l + lane * 64 + 16 * q) = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
        }
        store(col0, row0, low);
        if (mirror) {
          again();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            uint16_t* h = reinterpret_cast<uint16_t*>(buf_h) + 64 * e + lane;
            uint16_t* l = reinterpret_cast<uint16_t*>(buf_l) + 64 * e + lane;
            h[0] = static_cast<uint16_t>(hi[e]);
            h[32] = static_cast<uint16_t>(hi[e] >> 16);
            l[0] = static_cast<uint16_t>(lo[e]);
            l[32] = static_cast<uint16_t>(lo[e] >> 16);
          }
          store(row0, col0, true);
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

// Splits G [n, k] into BF16 hi + lo (F32) or copies it (BF16, COPY), and sums
// its squares: one partial sum per CTA, in a fixed order.
struct OrthoSplitParams {
  const void* g;
  int64_t ld_g, n, k, ld_x;
  __nv_bfloat16* hi;
  __nv_bfloat16* lo;
  float* part;   // [kOrthoNormBlocks]
};

template <bool F32, bool COPY>
__global__ void __launch_bounds__(256) ortho_split_kernel(const OrthoSplitParams p) {
  __shared__ float sm[8];
  pdl_wait();
  pdl_trigger();
  float s = 0.f;
  const int64_t total = p.n * p.k, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / p.k, c = i - r * p.k;
    const float v = F32 ? static_cast<const float*>(p.g)[r * p.ld_g + c]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.g)[r * p.ld_g + c]);
    s = fmaf(v, v, s);
    if (F32 || COPY) {
      const __nv_bfloat16 h = __float2bfloat16_rn(v);
      p.hi[r * p.ld_x + c] = h;
      if (F32) p.lo[r * p.ld_x + c] = __float2bfloat16_rn(v - __bfloat162float(h));
    }
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

}  // namespace puro
