// The Newton-Schulz iteration of ortho.cuh for gradients with a side of at most
// 128 and another of at most 2048, in one launch of one cluster.
//
// In small products everything but the arithmetic costs: the general kernel
// spends 8000 to 10000 cycles on each of the 3 * steps hand-overs through
// global memory.  Here the matrix never leaves the SMs.  With m the shorter side,
// X is [m, w] (a tall gradient is read and written transposed, which changes
// nothing else), and each CTA of the cluster keeps 128 of its columns: in FP32
// in registers, thread (row, half of the columns) 64 of them, and as FP16 hi +
// lo in shared memory as the operand of the products.  One copy in
// shared memory serves both: X X^T reads it K-major, the update R X reads the
// same rows MN-major.  O (the off-diagonal part of M) and then R take one
// [128, 128] tile.
//   per step: M_p = X_p X_p^T (hi hi, hi lo, lo hi)        tensor cores
//             M = sum over the cluster, through distributed shared memory: CTA p
//               adds the rows of its band in a fixed order and hands them to all
//             S = O O;  R = c (S + O D + D O) + b O          tensor cores, epilogue
//             X_p <- (a + D') X_p + R X_p (R hi, R lo)       tensor cores, epilogue
// (scales, D, D' as in ortho.cuh; only the operands of products are rounded, X to
// 22 bits, O and R off their diagonals at random to 11, and X itself is FP32 from
// step to step: what the products of few rows lost of X with hi alone left a rank-1
// gradient 3e-2 off).  Every CTA forms the whole of S and R for itself:
// that is less than handing them over would take.  Bound by latency.
#pragma once

#include "ortho.cuh"

namespace puro {

constexpr int kSmallSide = 128;      // longest shorter side
constexpr int kSmallSlice = 128;     // columns of X per CTA
constexpr int kSmallMaxCluster = 16;
constexpr int kSmallThreads = 256;

struct OrthoSmallParams {
  const void* g;
  int64_t ld_g;
  __nv_bfloat16* out;
  int64_t ld_out;
  int32_t m, w;             // X is [m, w]
  int32_t tall, g_f32;      // G is [w, m]; FP32, else BF16
  int32_t vec_g, vec_out;   // rows of G start on boundaries of four elements, of out on 16 bytes
  int32_t steps;
  float a, b, c, eps;
};

struct OrthoSmallCfg {
  static constexpr uint32_t kTile = 128 * 128;              // [128][64] FP16, 128-byte swizzle
  static constexpr uint32_t kOffLo = 2 * kTile;             // X hi: two tiles, X lo: two
  static constexpr uint32_t kOffO = 4 * kTile;              // O, then R
  static constexpr uint32_t kOffSum = 6 * kTile;            // partial M, two buffers: [32 column quads][128 rows] float4
  static constexpr uint32_t kOffDiag = kOffSum + 2 * 65536; // D, D'
  static constexpr uint32_t kOffRed = kOffDiag + 1024;      // sums of squares: 8 warps, the CTA's
  static constexpr uint32_t kOffMisc = kOffRed + 64;        // barrier, TMEM address, abort flag
  static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ void tc_mma_f16_1(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_peer(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_peer_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float ld_peer_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_peer_f1(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Eight values as FP16, rounded at random.
__device__ __forceinline__ uint4 half_row8(const float* v, const RoundBits& b) {
  return make_uint4(half_pair_random(v[0], v[1], b.first), half_pair_random(v[2], v[3], b.first + b.step),
                    half_pair_random(v[4], v[5], b.first + 2 * b.step), half_pair_random(v[6], v[7], b.first + 3 * b.step));
}

// Byte of a 16-byte piece (8 columns from c on) of row r in two [128][64] tiles.
__device__ __forceinline__ uint32_t small_piece(int r, int c) {
  return (uint32_t)((c >> 6) * 16384 + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4));
}

__global__ void __launch_bounds__(kSmallThreads, 1) ortho_small_kernel(const OrthoSmallParams p) {
  using C = OrthoSmallCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* tile_o = smem + C::kOffO;
  float4* sums = reinterpret_cast<float4*>(smem + C::kOffSum);
  float* diag = reinterpret_cast<float*>(smem + C::kOffDiag);
  float* diag_r = diag + 128;
  float* red = reinterpret_cast<float*>(smem + C::kOffRed);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = 32 * (warp & 3) + lane, half = warp >> 2, col0 = 64 * half;  // this thread's part of the slice
  const uint32_t rank = cluster_ctarank();
  uint32_t peers;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(peers));
  const int32_t j0 = (int32_t)rank * kSmallSlice;           // the slice's first column of X
  const int32_t m16 = (p.m + 15) / 16 * 16;                 // rows that products see
  const int32_t slice = p.w - j0 < kSmallSlice ? p.w - j0 : kSmallSlice;  // <= 0: an empty slice

  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc<1>(tmem_slot, 256);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_row = (uint32_t)(32 * (warp & 3)) << 16;
  pdl_wait();
  pdl_trigger();

  // X0 = G / (|G| + eps)
  float x[64];
  const int32_t live = row < p.m ? (slice - col0 < 64 ? slice - col0 : 64) : 0;  // columns of this thread that exist
  if (p.tall) {
    const int64_t first = (int64_t)(j0 + col0) * p.ld_g + row;
#pragma unroll
    for (int e = 0; e < 64; ++e) {
      x[e] = 0.f;
      if (e < live)
        x[e] = p.g_f32 ? static_cast<const float*>(p.g)[first + e * p.ld_g]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(p.g)[first + e * p.ld_g]);
    }
  } else {
    // a warp reads 16 rows, 4 columns a lane; rows lie in `sums` with their
    // pieces XORed by the row, so that both sides meet no bank twice
    const int32_t c = 4 * lane, n = slice - c < 4 ? slice - c : 4;  // columns that exist
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int r = 16 * warp + i;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < p.m) {
        const int64_t at = (int64_t)r * p.ld_g + j0 + c;
        if (p.vec_g && n == 4) {
          if (p.g_f32) {
            const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p.g) + at);
            v[0] = f.x;
            v[1] = f.y;
            v[2] = f.z;
            v[3] = f.w;
          } else {
            const uint2 f = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.g) + at);
            v[0] = __uint_as_float(f.x << 16);
            v[1] = __uint_as_float(f.x & 0xFFFF0000u);
            v[2] = __uint_as_float(f.y << 16);
            v[3] = __uint_as_float(f.y & 0xFFFF0000u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < n)
              v[e] = p.g_f32 ? static_cast<const float*>(p.g)[at + e]
                             : __bfloat162float(static_cast<const __nv_bfloat16*>(p.g)[at + e]);
        }
      }
      sums[r * 32 + (lane ^ (r & 31))] = make_float4(v[0], v[1], v[2], v[3]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const float4 f = sums[row * 32 + ((col0 / 4 + u) ^ (row & 31))];
      x[4 * u] = f.x;
      x[4 * u + 1] = f.y;
      x[4 * u + 2] = f.z;
      x[4 * u + 3] = f.w;
    }
  }
  {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 64; ++e) s = fmaf(x[e], x[e], s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    if (tid == 0) {
      s = red[0];
      for (int w = 1; w < 8; ++w) s += red[w];
      red[8] = s;
    }
    cluster_or_block_sync<2>();
    s = 0.f;
    for (uint32_t q = 0; q < peers; ++q) s += ld_peer_f1(cluster_peer(smem_u32(red + 8), q));
    const float scale = 1.f / (sqrtf(s) + p.eps);
#pragma unroll
    for (int e = 0; e < 64; ++e) x[e] *= scale;
  }
  auto write_x = [&]() {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v0 = x[8 * u + 2 * e] * kXScale, v1 = x[8 * u + 2 * e + 1] * kXScale;
        hi[e] = half_pair(v0, v1);
        const float2 h = half_unpack(hi[e]);
        lo[e] = half_pair(v0 - h.x, v1 - h.y);
      }
      const uint32_t at = small_piece(row, col0 + 8 * u);
      *reinterpret_cast<uint4*>(smem + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(smem + C::kOffLo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };
  // what the threads have written is seen by the tensor cores after this, and
  // their TMEM reads come before the next products' writes
  auto hand_over = [&]() {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  uint32_t phase = 0;
  // the products issued by warp 0 are done (a wait that gives up has set the
  // error word; the CTA goes on, so that the cluster's barriers stay in step)
  auto finish = [&]() {
    mbar_wait_warp(bar, phase, abort_flag);
    phase ^= 1;
    tc_fence_after();
  };
  const uint32_t sb = smem_u32(smem);
  // D FP32, A and B FP16, M = 128; B MN-major: bit 16
  auto idesc = [](int32_t n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
  };
  auto kmajor = [&](uint32_t offset, int k) { return desc_sw128_kmajor(sb + offset + (k >> 2) * 16384) + (k & 3) * 2; };

  write_x();
  hand_over();
  for (int step = 0; step < p.steps; ++step) {
    // ---- M_p = X_p X_p^T
    const int kx = slice > 0 ? (slice + 15) / 16 : 1;  // (an empty slice holds zeros)
    if (warp == 0) {
      if (elect_one()) {
        uint32_t accumulate = 0;
        for (int pass = 0; pass < 3; ++pass)
          for (int k = 0; k < kx; ++k) {
            tc_mma_f16_1(tmem, kmajor(pass == 2 ? C::kOffLo : 0, k), kmajor(pass == 1 ? C::kOffLo : 0, k), idesc(m16, false),
                         accumulate);
            accumulate = 1;
          }
        tc_commit_local<1>(bar);
      }
      __syncwarp();
    }
    finish();
    // ---- O and D
    float4* mine = sums + (step & 1) * 4096;  // (alternating, so that no barrier has to follow the reads)
    if (peers > 1) {
#pragma unroll 1
      for (int c = col0; c < col0 + 64 && c < m16; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + t_row + c, r);
        tmem_ld_wait();
        regs_after_wait(r);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          mine[(c / 4 + q) * 128 + row] = make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                                                      __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
      }
      cluster_or_block_sync<2>();
    }
    constexpr float kToM = kMScale / (kXScale * kXScale);
    if (peers <= 2) {
#pragma unroll 1
      for (int c = col0; c < col0 + 64 && c < m16; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + t_row + c, r);
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0.f;
        if (peers == 2) {
          const uint32_t from = cluster_peer(smem_u32(mine + (c / 4) * 128 + row), rank ^ 1);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 f = ld_peer_f4(from + q * 2048);
            v[4 * q] = f.x;
            v[4 * q + 1] = f.y;
            v[4 * q + 2] = f.z;
            v[4 * q + 3] = f.w;
          }
        }
        tmem_ld_wait();
        regs_after_wait(r);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = (__uint_as_float(r[e]) + v[e]) * kToM;
        if ((row & ~31) == c) {
          float d = 0.f;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e == lane) {
              d = v[e];
              v[e] = 0.f;
            }
          diag[row] = d * (1.f / kMScale);
        }
        const RoundBits rb = round_bits(row, c, 3 * step);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(tile_o + small_piece(row, c + 8 * q)) =
              half_row8(v + 8 * q, {rb.first + 4 * q * rb.step, rb.step});
      }
      hand_over();
    } else {
      // the band of rows that this CTA adds, 8 columns at a time
      const int band = 128 / (int)peers, first = (int)rank * band;
      for (int i = tid; i < band * (m16 / 8); i += kSmallThreads) {
        const int r = first + i % band, c = i / band * 8;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        const uint32_t at = smem_u32(mine + (c / 4) * 128 + r);
        for (uint32_t q = 0; q < peers; q += 4) {  // (four or more: eight loads in flight)
          float4 f[4], g[4];
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t from = cluster_peer(at, q + k);
            f[k] = ld_peer_f4(from);
            g[k] = ld_peer_f4(from + 128 * 16);
          }
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            v[0] += f[k].x;
            v[1] += f[k].y;
            v[2] += f[k].z;
            v[3] += f[k].w;
            v[4] += g[k].x;
            v[5] += g[k].y;
            v[6] += g[k].z;
            v[7] += g[k].w;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= kToM;
        float d = 0.f;
        const bool on_diag = (r & ~7) == c;
        if (on_diag) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e == (r & 7)) {
              d = v[e] * (1.f / kMScale);
              v[e] = 0.f;
            }
        }
        const uint4 o = half_row8(v, round_bits(r, c, 3 * step));
        const uint32_t to = smem_u32(tile_o + small_piece(r, c)), to_d = smem_u32(diag + r);
        for (uint32_t q = 0; q < peers; ++q) {
          st_peer_v4(cluster_peer(to, q), o);
          if (on_diag) st_peer_f1(cluster_peer(to_d, q), d);
        }
      }
      fence_proxy_async_all();
      tc_fence_before();
      cluster_or_block_sync<2>();
      tc_fence_after();
      fence_proxy_async_all();
    }
    // ---- S = O O
    if (warp == 0) {
      if (elect_one()) {
        for (int k = 0; k < m16 / 16; ++k)
          tc_mma_f16_1(tmem, kmajor(C::kOffO, k), kmajor(C::kOffO, k), idesc(m16, false), k > 0);
        tc_commit_local<1>(bar);
      }
      __syncwarp();
    }
    finish();
    // ---- R in O's place, D'
    const float dr = diag[row];
#pragma unroll 1
    for (int c = col0; c < col0 + 64 && c < m16; c += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem + t_row + c, r);
      tmem_ld_wait();
      regs_after_wait(r);
      const bool on_diag = (row & ~31) == c;
      const float raw = p.c / (kMScale * kMScale);
      RoundBits rb = round_bits(row, c, 3 * step + 1);
      float d_new = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4* at = reinterpret_cast<uint4*>(tile_o + small_piece(row, c + 8 * q));
        const uint4 h4 = *at;
        const uint32_t hw[4] = {h4.x, h4.y, h4.z, h4.w};
        const float4 da = *reinterpret_cast<const float4*>(diag + c + 8 * q), db = *reinterpret_cast<const float4*>(diag + c + 8 * q + 4);
        const float dc[8] = {da.x, da.y, da.z, da.w, db.x, db.y, db.z, db.w};
        uint32_t o[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int e = 8 * q + 2 * w;
          const float2 h = half_unpack(hw[w]);
          const float s0 = __uint_as_float(r[e]), s1 = __uint_as_float(r[e + 1]);
          float v0 = fmaf(s0, raw * kRScale, h.x * (kRScale / kMScale) * fmaf(p.c, dr + dc[2 * w], p.b));
          float v1 = fmaf(s1, raw * kRScale, h.y * (kRScale / kMScale) * fmaf(p.c, dr + dc[2 * w + 1], p.b));
          if (on_diag && e == lane) {
            d_new = fmaf(s0, raw, dr * fmaf(p.c, dr, p.b));
            v0 = 0.f;
          }
          if (on_diag && e + 1 == lane) {
            d_new = fmaf(s1, raw, dr * fmaf(p.c, dr, p.b));
            v1 = 0.f;
          }
          o[w] = half_pair_random(v0, v1, rb.first);
          rb.first += rb.step;
        }
        *at = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (on_diag) diag_r[row] = d_new;
    }
    hand_over();
    // ---- R X_p: B is X hi, then X lo, read MN-major, its 64-column tiles 16 KB apart
    if (warp == 0) {
      if (elect_one()) {
        uint32_t accumulate = 0;
        for (uint32_t term = 0; term < 2 * C::kOffLo; term += C::kOffLo)
          for (int k = 0; k < m16 / 16; ++k) {
            const uint64_t b = (uint64_t)(((sb + term + k * 2048) & 0x3FFFFu) >> 4) | ((uint64_t)(16384u >> 4) << 16) |
                               ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
            tc_mma_f16_1(tmem + 128, kmajor(C::kOffO, k), b, idesc(128, true), accumulate);
            accumulate = 1;
          }
        tc_commit_local<1>(bar);
      }
      __syncwarp();
    }
    finish();
    const float keep = p.a + (row < m16 ? diag_r[row] : 0.f);
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem + t_row + 128 + col0 + c, r);
      tmem_ld_wait();
      regs_after_wait(r);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        x[c + e] = fmaf(keep, x[c + e], __uint_as_float(r[e]) * (1.f / (kRScale * kXScale)));
    }
    if (step + 1 < p.steps) {
      // rows past m stay zero (R has no such rows, but TMEM may hold anything there)
      if (row >= p.m) {
#pragma unroll
        for (int e = 0; e < 64; ++e) x[e] = 0.f;
      }
      write_x();
      hand_over();
    }
  }
  if (p.tall) {
    const int64_t first = (int64_t)(j0 + col0) * p.ld_out + row;
#pragma unroll
    for (int e = 0; e < 64; ++e)
      if (e < live) p.out[first + e * p.ld_out] = __float2bfloat16_rn(x[e]);
  } else {
    // through the tiles of X hi (no product reads them any more), so that lanes
    // write along rows
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __nv_bfloat162 f = __floats2bfloat162_rn(x[8 * u + 2 * e], x[8 * u + 2 * e + 1]);
        o[e] = *reinterpret_cast<uint32_t*>(&f);
      }
      *reinterpret_cast<uint4*>(smem + small_piece(row, col0 + 8 * u)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    __syncthreads();
    const int c = 8 * (tid & 15);
    const int32_t n = slice - c < 8 ? slice - c : 8;
    for (int r = tid >> 4; r < p.m; r += kSmallThreads / 16) {
      const uint8_t* at = smem + small_piece(r, c);
      __nv_bfloat16* to = p.out + (int64_t)r * p.ld_out + j0 + c;
      if (p.vec_out && n == 8) {
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(at);
      } else {
        for (int e = 0; e < n; ++e) to[e] = reinterpret_cast<const __nv_bfloat16*>(at)[e];
      }
    }
  }
  tc_fence_before();
  cluster_or_block_sync<2>();  // no CTA leaves while a peer still reads from it
  tc_fence_after();
  if (warp == 0) tmem_dealloc<1>(tmem, 256);
}

}  // namespace puro
