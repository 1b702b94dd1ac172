// The norms around a block, fused with the block's gate, the residual sum and
// the FP8 quantization of the next (or, backward, the previous) linear layer.
//
// Forward, for each token (row of D columns):
//   hh = h * r1,  r1 = rsqrt(mean(h^2) + eps)      (hh = h without a norm after the block)
//   y  = bf16(x + scale * ((hh * w_post) * gate))  (y = x without a block output)
//   n  = bf16(y * r2 * w_pre),  r2 = rsqrt(mean(y^2) + eps)
// n leaves as E4M3 codes with one scale per 1x128 group, row-wise, transposed
// or both, exactly as the activation quantizer encodes a BF16 tensor; or as
// BF16.  r2 is taken from the stored (BF16) y, so that the backward pass and a
// recomputation from y see the same numbers.  That makes r2 follow y's rounding:
// in a strong channel (|y| of 32 or more in a row of 2048 with a mean square of
// 3) a y that rounds the other way moves r2 by 1e-3.  So y is formed in just
// this order, each operation rounded to FP32 by itself as separate operations
// on tensors are: nothing is multiplied ahead and nothing fused.  (The mean and
// its sum with eps too: fused, r1 of 1920 columns differed in its last bit from
// that of separate operations in 30% of the rows instead of 17%.)
//
// Backward, with t = dn * w_pre, nh = y * r2, e = scale * gate * w_post:
//   dY = dy + r2 * (t - nh * mean(t nh))     -> dx = bf16(dY)
//   dh = r1 * (e dY - hh * mean(e dY hh))    -> codes or BF16 (rounded to BF16 first)
//   dw_pre = sum_t dn nh,  S = sum_t gate dY hh,  dw_post = scale S,
//   dgate  = scale w_post dY hh, summed to the gate's shape.
// mean(e dY hh) is taken in the same pass over the row as mean(t nh): with
// base = dy + r2 t it is mean(e hh base) - r2 mean(t nh) mean(e hh nh), so one
// block-wide reduction of three sums serves both norms.  All sums are FP32.
//
// Both are bound by HBM.  A norm needs whole rows and the transposed codes 128
// of them, more than an SM holds, so the work is split in two passes: one over
// rows, which leaves y (or dh) in BF16, and, where transposed codes are asked
// for, the tile quantizer over that result (forward with the product by r2 and
// w_pre in its first step).  The second pass reads 2 bytes per element more
// than one pass would have to, but each streams without a pause: a single
// kernel on clusters of 8 CTAs x 16 rows, which held the rows in shared memory
// and exchanged column maxima, spent most of its time in barriers with no load
// in flight (32768 x 2048 on both norms: 227 us forward with a gate per token and
// 347 us backward with one per element, against 117 us and 230 us now).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "quant.cuh"

namespace puro {

enum GateKind : int { kGateNone = 0, kGateToken = 1, kGateChannel = 2, kGateFull = 3 };

// Where the quantized result goes.  q, qt or bf may be null.
struct CodeOut {
  uint8_t* q;
  int64_t ld_q;
  uint8_t* s;      // blocked, rows x cols/128 groups
  int64_t s_g4;
  uint8_t* qt;
  int64_t ld_qt;
  uint8_t* st;     // blocked, cols x ceil(rows/128) groups
  int64_t st_g4;
  __nv_bfloat16* bf;  // BF16 result instead of codes
  int64_t ld_bf;
};

struct NormParams {
  int64_t rows;
  int32_t cols;
  int32_t rpc;                 // backward: rows per CTA
  const __nv_bfloat16* x;      // forward: x; backward: y (the residual stream after the sum)
  int64_t ld_x;
  const __nv_bfloat16* h;      // block output, or null
  int64_t ld_h;
  const void* w_pre;
  const void* w_post;          // or null
  const void* gate;            // or null
  int64_t ld_gate;             // kGateFull
  int32_t w_f32, gate_f32, gate_kind;
  int32_t wide;                // w_pre, w_post and a channel gate start on 16-byte boundaries
  int32_t scale_pow2;          // forward: scale is a power of two
  uint32_t* ctr;               // a tile counter to set to zero for the pass after this one, or null
  float scale, eps;
  // forward
  __nv_bfloat16* y;
  int64_t ld_y;
  float* rstd;                 // written forward, read backward
  float* rstd_post;
  // backward
  const __nv_bfloat16* dn;
  int64_t ld_dn;
  const __nv_bfloat16* dy;     // or null
  int64_t ld_dy;
  __nv_bfloat16* dx;
  int64_t ld_dx;
  void* dgate;                 // FP32 [rows] (token), BF16 [rows][ld_dgate] (full)
  int64_t ld_dgate;
  float* part;                 // [CTAs][2][cols] column sums of dn nh and gate dY hh
  CodeOut out;
};

constexpr int kNormMaxCols = 8192;

__device__ __forceinline__ uint4 ldg_stream(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}

// Sums the three values of each of ROWS = 2 or 1 rows over the block; every
// thread gets the same result, added in the same order.  Lanes first share the values out
// among themselves (each ends with one of up to eight, 8 shuffles instead of
// 5 for every value), and every warp adds the warps' shares.  `red` holds
// [2][32][8] floats; the caller flips `buf` from call to call, which one
// barrier per call makes safe.
template <int ROWS>
__device__ __forceinline__ void row_sums(float (&v)[3 * ROWS], float* red, int& buf) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  float a[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const float other = ROWS == 2 ? v[3 * ROWS - 3 + k] : v[k];  // of the second row
    const float keep = ROWS == 2 && b4 ? other : v[k], give = ROWS == 2 && b4 ? v[k] : other;
    a[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
  }
  const float k0 = (b3 ? a[2] : a[0]) + __shfl_xor_sync(0xFFFFFFFFu, b3 ? a[0] : a[2], 8);
  const float k1 = (b3 ? 0.f : a[1]) + __shfl_xor_sync(0xFFFFFFFFu, b3 ? a[1] : 0.f, 8);
  float t = (b2 ? k1 : k0) + __shfl_xor_sync(0xFFFFFFFFu, b2 ? k0 : k1, 4);
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 2);
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 1);
  float* r = red + buf * 256;
  buf ^= 1;
  if ((lane & 3) == 0) r[(threadIdx.x >> 5) * 8 + (lane >> 2)] = t;
  __syncthreads();
  t = 0.f;
  for (int w = lane & 3; w < warps; w += 4) t += r[w * 8 + (lane >> 2)];
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 1);
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 2);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = __shfl_sync(0xFFFFFFFFu, t, 4 * k);
    if (ROWS == 2) v[3 * ROWS - 3 + k] = __shfl_sync(0xFFFFFFFFu, t, 16 + 4 * k);
  }
}

// Sums one value of each of B = 4 or 2 rows over the block, in the same way.
template <int B>
__device__ __forceinline__ void one_sum(float (&v)[B], float* red, int& buf) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const bool b4 = lane & 16, b3 = lane & 8;
  const float u2 = B == 4 ? v[B - 2] : 0.f, u3 = B == 4 ? v[B - 1] : 0.f;
  const float k0 = (b4 ? u2 : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, b4 ? v[0] : u2, 16);
  const float k1 = (b4 ? u3 : v[1]) + __shfl_xor_sync(0xFFFFFFFFu, b4 ? v[1] : u3, 16);
  float t = (b3 ? k1 : k0) + __shfl_xor_sync(0xFFFFFFFFu, b3 ? k0 : k1, 8);
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, off);
  float* r = red + buf * 256;
  buf ^= 1;
  if ((lane & 7) == 0) r[(threadIdx.x >> 5) * 4 + (lane >> 3)] = t;
  __syncthreads();
  t = 0.f;
  for (int w = lane & 7; w < warps; w += 8) t += r[w * 4 + (lane >> 3)];
#pragma unroll
  for (int off = 1; off <= 4; off <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, off);
#pragma unroll
  for (int k = 0; k < B; ++k) v[k] = __shfl_sync(0xFFFFFFFFu, t, 8 * k);
}

// Codes and scale bytes of two 16-lane groups of 128 columns: (r0, c0) and
// (r1, c1) are the places of this thread's 8 columns v0 and v1; in0 and in1 say
// whether they exist (the same for all lanes of a group).
__device__ __forceinline__ void emit_groups(const CodeOut& o, int64_t r0, int32_t c0, bool in0, const uint4& v0,
                                            int64_t r1, int32_t c1, bool in1, const uint4& v1) {
  uint32_t a = amax2(amax2(v0.x, v0.y), amax2(v0.z, v0.w)), b = amax2(amax2(v1.x, v1.y), amax2(v1.z, v1.w));
  uint32_t m = amax2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)) & 0x7FFF7FFFu;
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  const uint32_t k2 = scale_k2(m), bytes = scale_bytes2(m, k2);
  auto emit = [&](int64_t r, int32_t c, const uint4& v, float scale, uint8_t byte) {
    const int32_t g = c >> 7;
    if ((threadIdx.x & 15) == 0)
      o.s[((r >> 7) * o.s_g4 + (g >> 2)) * 512 + (g & 3) + blocked_in_chunk((int)(r & 127))] = byte;
    *reinterpret_cast<uint2*>(o.q + r * o.ld_q + c) = encode_row8(v, bf16_bits(scale));
  };
  if (in0) emit(r0, c0, v0, scale_lo(k2), static_cast<uint8_t>(bytes));
  if (in1) emit(r1, c1, v1, scale_hi(k2), static_cast<uint8_t>(bytes >> 16));
}

// Scale bytes 127 for the rows that pad the last 128, by one CTA.
__device__ __forceinline__ void pad_row_scales(const CodeOut& o, int64_t rows, int32_t cols) {
  const int64_t last = (rows + 127) / 128 * 128;
  const int32_t groups = cols >> 7;
  for (int64_t i = threadIdx.x; i < (last - rows) * groups; i += blockDim.x) {
    const int64_t r = rows + i / groups;
    const int32_t g = (int32_t)(i % groups);
    o.s[((r >> 7) * o.s_g4 + (g >> 2)) * 512 + (g & 3) + blocked_in_chunk((int)(r & 127))] = 127;
  }
}

// 16-byte copy global -> shared that does not pass through registers; bytes = 0
// writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Both row passes: a thread keeps 8 fixed columns of the CTA's p.rpc rows (so
// weights and column sums stay in registers), and the next rows' tensors are
// copied to shared memory, two stages of a few rows each, while the present
// ones are worked on.  A thread reads only what it copied itself, so the copies
// need no barrier, and 80 KB per CTA stay in flight.  (A forward pass with a
// warp to a row, loading into registers, kept the memory busy for two thirds
// of the time: 84 us for 32768 x 2048 against 76.)

constexpr uint32_t kNormRedBytes = 2 * 32 * 8 * 4;

// Shared memory of a row pass: the sums' scratch and two stages of `rows` rows
// of up to three (forward) or five (backward) tensors.
__host__ __device__ constexpr uint32_t norm_pass_smem(int rows, int32_t threads, int tensors) {
  return kNormRedBytes + 2u * rows * tensors * threads * 16;
}

// The forward row pass: y, the norms' factors and, if asked for, n as row-wise
// codes or BF16.  POST: with a norm of h; GATE: its kind of gate (without h
// neither is looked at).  (One kernel that looks at run time, with branches in
// every row, took 121 us for 32768 x 2048 with a norm of h, against 110.)
template <int MAXT, int B, bool POST, int GATE>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : MAXT == 512 ? 2 : 1) norm_forward_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t nsmem[];
  float* red = reinterpret_cast<float*>(nsmem);
  const uint8_t* ring = nsmem + kNormRedBytes;
  const int tensors = 1 + (p.h != nullptr) + (GATE == kGateFull);
  const uint32_t pitch = blockDim.x * 16;  // one row of one tensor
  const int32_t col = threadIdx.x * 8;
  const bool active = col < p.cols;
  const int64_t row0 = (int64_t)blockIdx.x * p.rpc;
  const int32_t nrows = (int32_t)(p.rows - row0 < p.rpc ? p.rows - row0 : p.rpc);
  const float inv_d = 1.f / (float)p.cols;
  pdl_wait();
  pdl_trigger();
  if (p.ctr && blockIdx.x == 0 && threadIdx.x == 0) *p.ctr = 0u;

  // copies rows rb .. rb + B - 1 into stage (rb / B) & 1; rows past the end become zeros
  auto fetch = [&](int32_t rb) {
    if (rb < nrows) {
      uint32_t dst = smem_u32(ring) + ((rb / B) & 1) * B * tensors * pitch + threadIdx.x * 16;
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int64_t r = row0 + (rb + k < nrows ? rb + k : rb);
        const uint32_t bytes = active && rb + k < nrows ? 16 : 0;
        const int32_t c = active ? col : 0;
        auto copy = [&](const __nv_bfloat16* t, int64_t ld) {
          cp_async16(dst, t + r * ld + c, bytes);
          dst += pitch;
        };
        copy(p.x, p.ld_x);
        if (p.h) copy(p.h, p.ld_h);
        if (GATE == kGateFull) copy(static_cast<const __nv_bfloat16*>(p.gate), p.ld_gate);
      }
    }
    cp_async_commit();
  };
  fetch(0);
  fetch(B);

  f2 w[4], wp[4], gc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = wp[i] = gc[i] = 0;
  const bool emits = p.out.bf || p.out.q;
  if (active) {
    if (emits) load_param8(p.w_pre, p.w_f32, p.wide, col, w);
    if (POST) load_param8(p.w_post, p.w_f32, p.wide, col, wp);
    if (GATE == kGateChannel) load_param8(p.gate, p.gate_f32, p.wide, col, gc);
  }
  const float last = p.scale_pow2 ? p.scale : 1.f;
  int buf = 0;
#pragma unroll 1
  for (int32_t rb = 0; rb < nrows; rb += B) {
    cp_async_wait<1>();
    const uint8_t* src = ring + ((rb / B) & 1) * B * tensors * pitch + threadIdx.x * 16;
    uint4 yv[B];
    float sum[B];
    if (p.h) {
      uint4 hv[B];
      float f[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const uint8_t* s = src + k * tensors * pitch;
        yv[k] = lds_v4(s);
        hv[k] = lds_v4(s + pitch);
      }
      if (POST) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
          f2 h[4], s = 0;
          unpack8(hv[k], h);
#pragma unroll
          for (int i = 0; i < 4; ++i) s = fma2(h[i], h[i], s);
          sum[k] = f2_sum(s);
        }
        one_sum<B>(sum, red, buf);
#pragma unroll
        for (int k = 0; k < B; ++k) {
          f[k] = rsqrtf(__fadd_rn(__fmul_rn(sum[k], inv_d), p.eps));
          if (threadIdx.x == 0 && rb + k < nrows) p.rstd_post[row0 + rb + k] = f[k];
        }
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int64_t r = row0 + rb + k;
        f2 x[4], h[4];
        unpack8(yv[k], x);
        unpack8(hv[k], h);
        if (POST) {
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = mul2(mul2(h[i], f2_both(f[k])), wp[i]);
        }
        if (GATE != kGateNone) {
          f2 g[4];
          if (GATE == kGateFull) {
            unpack8(lds_v4(src + (k * tensors + 2) * pitch), g);
          } else {
            const f2 t = f2_both(GATE == kGateToken && rb + k < nrows ? load_param(p.gate, p.gate_f32, r) : 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = GATE == kGateToken ? t : gc[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = mul2(h[i], g[i]);
        }
        // (a product with one, or with a power of two, is exact, so that the fused
        // form rounds as an addition does; a plain packed sum the compiler would fuse
        // with the product before it, in spite of the roundings that both name)
        if (!p.scale_pow2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = mul2(h[i], f2_both(p.scale));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fma2(h[i], f2_both(last), x[i]);
        yv[k] = pack8(x);
        if (active && rb + k < nrows) *reinterpret_cast<uint4*>(p.y + r * p.ld_y + col) = yv[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < B; ++k) yv[k] = lds_v4(src + k * pitch);
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      f2 y[4], s = 0;
      unpack8(yv[k], y);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(y[i], y[i], s);
      sum[k] = f2_sum(s);
    }
    one_sum<B>(sum, red, buf);
    // (every load from this stage has been used in the sums by now)
    fetch(rb + 2 * B);
    float r2[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      r2[k] = rsqrtf(__fadd_rn(__fmul_rn(sum[k], inv_d), p.eps));
      if (threadIdx.x == 0 && rb + k < nrows) p.rstd[row0 + rb + k] = r2[k];
    }
    if (emits) {
#pragma unroll
      for (int k = 0; k < B; ++k) yv[k] = normed8(yv[k], r2[k], w);
      if (p.out.bf && active) {
#pragma unroll
        for (int k = 0; k < B; ++k)
          if (rb + k < nrows) *reinterpret_cast<uint4*>(p.out.bf + (row0 + rb + k) * p.out.ld_bf + col) = yv[k];
      }
      if (p.out.q) {
#pragma unroll
        for (int k = 0; k < B; k += 2)
          emit_groups(p.out, row0 + rb + k, col, active && rb + k < nrows, yv[k], row0 + rb + k + 1, col,
                      active && rb + k + 1 < nrows, yv[k + 1]);
      }
    }
  }
  cp_async_wait<0>();
  if (p.out.q && blockIdx.x == gridDim.x - 1) pad_row_scales(p.out, p.rows, p.cols);
}

// The backward row pass: dx, the gate's gradient, dh as BF16 or row-wise codes,
// and the CTA's column sums.
template <int MAXT, int ROWS>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) norm_backward_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t nsmem[];
  const int tensors = 2 + (p.dy != nullptr) + (p.h != nullptr) + (p.gate_kind == kGateFull);
  const uint32_t pitch = blockDim.x * 16;  // one row of one tensor
  float* red = reinterpret_cast<float*>(nsmem);
  const uint8_t* ring = nsmem + kNormRedBytes;
  const int32_t col = threadIdx.x * 8;
  const bool active = col < p.cols;
  const int64_t row0 = (int64_t)blockIdx.x * p.rpc;
  const int32_t nrows = (int32_t)(p.rows - row0 < p.rpc ? p.rows - row0 : p.rpc);
  const float inv_d = 1.f / (float)p.cols;
  pdl_wait();
  pdl_trigger();
  if (p.ctr && blockIdx.x == 0 && threadIdx.x == 0) *p.ctr = 0u;

  // copies rows rb .. rb + ROWS - 1 into stage (rb / ROWS) & 1; rows past the end become zeros
  auto fetch = [&](int32_t rb) {
    if (rb < nrows) {
      uint32_t dst = smem_u32(ring) + ((rb / ROWS) & 1) * ROWS * tensors * pitch + threadIdx.x * 16;
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int64_t r = row0 + (rb + k < nrows ? rb + k : rb);
        const uint32_t bytes = active && rb + k < nrows ? 16 : 0;
        const int32_t c = active ? col : 0;
        auto copy = [&](const __nv_bfloat16* t, int64_t ld) {
          cp_async16(dst, t + r * ld + c, bytes);
          dst += pitch;
        };
        copy(p.dn, p.ld_dn);
        copy(p.x, p.ld_x);
        if (p.dy) copy(p.dy, p.ld_dy);
        if (p.h) copy(p.h, p.ld_h);
        if (p.gate_kind == kGateFull) copy(static_cast<const __nv_bfloat16*>(p.gate), p.ld_gate);
      }
    }
    cp_async_commit();
  };
  fetch(0);
  fetch(ROWS);

  f2 w[4], e[4], acc_w[4], acc_s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = acc_w[i] = acc_s[i] = 0;
    e[i] = f2_both(p.scale);
  }
  if (active) {
    f2 v[4];
    load_param8(p.w_pre, p.w_f32, p.wide, col, w);
    if (p.w_post) {
      load_param8(p.w_post, p.w_f32, p.wide, col, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = mul2(e[i], v[i]);
    }
    if (p.gate_kind == kGateChannel) {
      load_param8(p.gate, p.gate_f32, p.wide, col, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = mul2(e[i], v[i]);
    }
  }
  int buf = 0;
#pragma unroll 1
  for (int32_t rb = 0; rb < nrows; rb += ROWS) {
    uint4 nv[ROWS], yv[ROWS], gv[ROWS], hv[ROWS], tv[ROWS], out[ROWS];
    float r1[ROWS], r2[ROWS], gt[ROWS];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t r = row0 + rb + k;
      const bool row_in = rb + k < nrows;
      r2[k] = row_in ? p.rstd[r] : 0.f;
      r1[k] = row_in && p.w_post ? p.rstd_post[r] : 1.f;
      gt[k] = row_in && p.gate_kind == kGateToken ? load_param(p.gate, p.gate_f32, r) : 1.f;
    }
    cp_async_wait<1>();
    const uint8_t* stage = ring + ((rb / ROWS) & 1) * ROWS * tensors * pitch + threadIdx.x * 16;
    auto read = [&](int k) {
      const uint8_t* src = stage + k * tensors * pitch;
      nv[k] = lds_v4(src);
      yv[k] = lds_v4(src += pitch);
      gv[k] = p.dy ? lds_v4(src += pitch) : zero;
      hv[k] = p.h ? lds_v4(src += pitch) : zero;
      tv[k] = p.gate_kind == kGateFull ? lds_v4(src += pitch) : zero;
    };
#pragma unroll
    for (int k = 0; k < ROWS; ++k) read(k);
    float sum[3 * ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      f2 dn[4], y[4], g[4];
      unpack8(nv[k], dn);
      unpack8(yv[k], y);
      unpack8(gv[k], g);
      const f2 rr = f2_both(r2[k]);
      f2 s1 = 0, sp = 0, sq = 0;
      if (p.h) {
        f2 h[4], t[4];
        unpack8(hv[k], h);
        unpack8(tv[k], t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 nh = mul2(y[i], rr), tt = mul2(dn[i], w[i]), base = fma2(rr, tt, g[i]);
          f2 eh = mul2(e[i], mul2(h[i], f2_both(r1[k])));
          if (p.gate_kind == kGateFull) eh = mul2(eh, t[i]);
          s1 = fma2(tt, nh, s1);
          sp = fma2(eh, base, sp);
          sq = fma2(eh, nh, sq);
          acc_w[i] = fma2(dn[i], nh, acc_w[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 nh = mul2(y[i], rr);
          s1 = fma2(mul2(dn[i], w[i]), nh, s1);
          acc_w[i] = fma2(dn[i], nh, acc_w[i]);
        }
      }
      sum[3 * k] = f2_sum(s1);
      sum[3 * k + 1] = f2_sum(sp);
      sum[3 * k + 2] = f2_sum(sq);
    }
    row_sums<ROWS>(sum, red, buf);
    // (1024 threads have 64 registers each, too few to keep the rows over the
    // barrier: they read them again, 8192 x 8192 in 267 us against 298)
    if (MAXT == 1024) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        asm volatile("" ::: "memory");
        read(k);
      }
    } else {
      // (every load from this stage has been used in the sums by now)
      fetch(rb + 2 * ROWS);
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t r = row0 + rb + k;
      const bool in = active && rb + k < nrows;
      const float m1 = sum[3 * k] * inv_d;
      const float dot = fmaf(-r2[k] * m1, sum[3 * k + 2], sum[3 * k + 1]);  // sum of e dY hh
      const float m2 = gt[k] * dot * inv_d;
      if (p.gate_kind == kGateToken && threadIdx.x == 0 && rb + k < nrows) static_cast<float*>(p.dgate)[r] = dot;
      f2 dn[4], y[4], g[4], h[4];
      unpack8(nv[k], dn);
      unpack8(yv[k], y);
      unpack8(gv[k], g);
      const f2 rr = f2_both(r2[k]), neg_m1 = f2_both(-m1);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // dY
        g[i] = fma2(rr, fma2(mul2(y[i], rr), neg_m1, mul2(dn[i], w[i])), g[i]);
      if (in) *reinterpret_cast<uint4*>(p.dx + r * p.ld_dx + col) = pack8(g);
      if (!p.h) continue;
      unpack8(hv[k], h);
      f2 t[4];
      unpack8(tv[k], t);
      const f2 ra = f2_both(r1[k]), gate = f2_both(gt[k]), neg_m2 = f2_both(-m2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 hh = mul2(h[i], ra);
        const f2 gd = mul2(p.gate_kind == kGateFull ? t[i] : gate, g[i]);
        acc_s[i] = fma2(gd, hh, acc_s[i]);
        t[i] = mul2(mul2(e[i], g[i]), hh);  // the gate's own gradient (full)
        const f2 v = mul2(e[i], gd);
        h[i] = p.w_post ? mul2(ra, fma2(hh, neg_m2, v)) : v;
      }
      if (p.gate_kind == kGateFull && in)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dgate) + r * p.ld_dgate + col) = pack8(t);
      out[k] = pack8(h);
      if (p.out.bf && in) *reinterpret_cast<uint4*>(p.out.bf + r * p.out.ld_bf + col) = out[k];
    }
    if (MAXT == 1024) fetch(rb + 2 * ROWS);  // (the rows read again have been used)
    if (p.out.q) {
#pragma unroll
      for (int k = 0; k < ROWS; k += 2)
        emit_groups(p.out, row0 + rb + k, col, active && rb + k < nrows, out[k], row0 + rb + k + 1, col,
                    active && k + 1 < ROWS && rb + k + 1 < nrows, k + 1 < ROWS ? out[(k + 1) % ROWS] : zero);
    }
  }
  cp_async_wait<0>();
  if (active) {
    ulonglong2* d = reinterpret_cast<ulonglong2*>(p.part + (int64_t)blockIdx.x * 2 * p.cols + col);
    d[0] = make_ulonglong2(acc_w[0], acc_w[1]);
    d[1] = make_ulonglong2(acc_w[2], acc_w[3]);
    d += p.cols / 4;
    d[0] = make_ulonglong2(acc_s[0], acc_s[1]);
    d[1] = make_ulonglong2(acc_s[2], acc_s[3]);
  }
  if (p.out.q && blockIdx.x == gridDim.x - 1) pad_row_scales(p.out, p.rows, p.cols);
}

// Column gradients from the CTAs' partial sums [parts][2][cols], in a fixed
// order: a block takes 32 columns of one of the two sums, its 16 warps every
// sixteenth partial.  Added in 64 bits and rounded once, so that the error does
// not grow with the rows (in FP32, 2^20 rows alike were off by 2^-15).
struct NormColumnParams {
  const float* part;
  int64_t parts;
  int32_t cols;
  const void* w_post;
  const void* gate;  // channel gate or null
  int32_t w_f32, gate_f32;
  float scale;
  int32_t accumulate;
  int32_t early;      // see below
  float* dw_pre;
  float* dw_post;     // or null
  float* dgate;       // channel gate's gradient or null
};

__global__ void __launch_bounds__(512) norm_column_kernel(const NormColumnParams p) {
  __shared__ double sm[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t c = blockIdx.x * 32 + lane;  // cols is a multiple of 128
  // early: the quantizer runs between the row pass and this one.  Its CTAs let
  // this kernel start only once they have seen the row pass complete, so the
  // sums may be read while it still works; the wait for it comes at the end,
  // so that whatever waits for this kernel has waited for both.
  if (!p.early) pdl_wait();
  pdl_trigger();
  double sum = 0.;
  const float* src = p.part + (int64_t)blockIdx.y * p.cols + c;
#pragma unroll 8
  for (int64_t i = warp; i < p.parts; i += 16) sum += __ldcg(src + i * 2 * p.cols);
  sm[warp][lane] = sum;
  __syncthreads();
  if (p.early) pdl_wait();
  if (warp) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) sum += sm[k][lane];
  const float a = (float)sum;
  // (explicit adds: fused into the product before them, they would round
  // differently from the call that overwrites)
  const bool add = p.accumulate != 0;
  if (blockIdx.y == 0) {
    p.dw_pre[c] = add ? __fadd_rn(p.dw_pre[c], a) : a;
    return;
  }
  if (p.dw_post) {
    const float v = p.scale * (p.gate ? load_param(p.gate, p.gate_f32, c) : 1.f) * a;
    p.dw_post[c] = add ? __fadd_rn(p.dw_post[c], v) : v;
  }
  if (p.dgate) {
    const float v = p.scale * (p.w_post ? load_param(p.w_post, p.w_f32, c) : 1.f) * a;
    p.dgate[c] = add ? __fadd_rn(p.dgate[c], v) : v;
  }
}

}  // namespace puro
