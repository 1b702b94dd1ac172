// The norms around a block, fused with the block's gate, the residual sum and
// the FP8 quantization of the next (or, backward, the previous) linear layer.
//
// Forward, for each token (row of D columns):
//   hh = h * r1,  r1 = rsqrt(mean(h^2) + eps)      (hh = h without a norm after the block)
//   y  = bf16(x + scale * gate * hh * w_post)      (y = x without a block output)
//   n  = bf16(y * r2 * w_pre),  r2 = rsqrt(mean(y^2) + eps)
// n leaves as E4M3 codes with one scale per 1x128 group, row-wise, transposed
// or both, exactly as the activation quantizer encodes a BF16 tensor; or as
// BF16.  r2 is taken from the stored (BF16) y, so that the backward pass and a
// recomputation from y see the same numbers.
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
// Both are bound by HBM.  A CTA takes RPC rows and all D columns, each thread
// 8 fixed columns, so column sums stay in registers and every load is 16
// bytes.  The transposed codes need the amax of 128 rows: a cluster of 128 /
// RPC CTAs covers them and exchanges only the column maxima through
// distributed shared memory; the rows themselves wait in the CTA's own shared
// memory as BF16 (32 D bytes for 16 rows) and never go out and come back.
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
  int32_t rpc;                 // rows per CTA
  const __nv_bfloat16* x;      // forward: x; backward: y (the residual stream after the sum)
  int64_t ld_x;
  const __nv_bfloat16* h;      // block output, or null
  int64_t ld_h;
  const void* w_pre;
  const void* w_post;          // or null
  const void* gate;            // or null
  int64_t ld_gate;             // kGateFull
  int32_t w_f32, gate_f32, gate_kind;
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
  float* part;                 // [clusters][2][cols] column sums of dn nh and gate dY hh
  CodeOut out;
};

constexpr int kNormMaxCols = 8192;

__device__ __forceinline__ uint4 ldg_stream(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}

// The 8 BF16 values of a 16-byte word as FP32.
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ float load_param(const void* p, int32_t f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Sums K values over the block; every thread gets the same result, added in
// the same order.  `red` holds [2][32] rows of K floats; the caller flips
// `buf` from call to call, which one barrier per call makes safe.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float* red, int& buf) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], off);
  const int warps = blockDim.x >> 5;
  float* r = red + buf * 32 * K;
  buf ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) r[(threadIdx.x >> 5) * K + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += r[w * K + k];
}

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t local, uint32_t rank) {
  uint32_t a;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}

__device__ __forceinline__ void cluster_sync_all() { cluster_or_block_sync<2>(); }

// Codes and scale bytes of one pair of rows (row r in m's low half, row r + 1
// in the high half; v0, v1 their 8 columns in this thread).  Rows at or past
// `rows` get the scale byte 127 and no codes.
__device__ __forceinline__ void emit_row_pair(const CodeOut& o, int64_t r, int64_t rows, int32_t col,
                                              bool active, const uint4& v0, const uint4& v1, bool second) {
  uint32_t a = amax2(amax2(v0.x, v0.y), amax2(v0.z, v0.w)), b = amax2(amax2(v1.x, v1.y), amax2(v1.z, v1.w));
  uint32_t m = amax2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)) & 0x7FFF7FFFu;
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  const uint32_t k2 = scale_k2(m);
  if (!active) return;
  if ((threadIdx.x & 15) == 0) {
    const uint32_t bytes = scale_bytes2(m, k2);
    const int32_t g = col >> 7;
    uint8_t* s = o.s + ((r >> 7) * o.s_g4 + (g >> 2)) * 512 + (g & 3);
    s[blocked_in_chunk((int)(r & 127))] = static_cast<uint8_t>(bytes);
    if (second) s[blocked_in_chunk((int)((r + 1) & 127))] = static_cast<uint8_t>(bytes >> 16);
  }
  uint8_t* q = o.q + r * o.ld_q + col;
  if (r < rows) *reinterpret_cast<uint2*>(q) = encode_row8(v0, bf16_bits(scale_lo(k2)));
  if (second && r + 1 < rows) *reinterpret_cast<uint2*>(q + o.ld_q) = encode_row8(v1, bf16_bits(scale_hi(k2)));
}

// The transposed codes of this CTA's RPC rows.  hold: [RPC][cols] BF16 rows in
// shared memory (each thread reads back only its own columns); cm: this
// thread's column maxima over the CTA's rows; xch: [threads] 16-byte words.
// `sync` runs the cluster barrier after which every peer's maxima are readable.
template <int RPC>
__device__ __forceinline__ void emit_columns(const CodeOut& o, const uint8_t* hold, const uint4* xch, int64_t row0,
                                             int64_t rows, int32_t cols, int32_t col, bool active, uint32_t rank) {
  if (!active) return;
  const uint32_t cs = 128 / RPC;
  uint32_t m[4] = {0, 0, 0, 0};
  const uint32_t mine = smem_u32(xch + threadIdx.x);
#pragma unroll
  for (uint32_t p = 0; p < cs; ++p) {
    const uint4 v = ld_cluster_v4(mine, p);
    m[0] = __vmaxu2(m[0], v.x);
    m[1] = __vmaxu2(m[1], v.y);
    m[2] = __vmaxu2(m[2], v.z);
    m[3] = __vmaxu2(m[3], v.w);
  }
  uint32_t k2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) k2[i] = scale_k2(m[i]);
  if ((threadIdx.x & (cs - 1)) == rank) {
    // columns col .. col + 7 are rows of the transposed scale array
    const int64_t tr = row0 >> 7;
    uint8_t* s = o.st + ((int64_t)(col >> 7) * o.st_g4 + (tr >> 2)) * 512 + (tr & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = scale_bytes2(m[i], k2[i]);
      s[blocked_in_chunk((col + 2 * i) & 127)] = static_cast<uint8_t>(b);
      s[blocked_in_chunk((col + 2 * i + 1) & 127)] = static_cast<uint8_t>(b >> 16);
    }
  }
  if (row0 >= (rows + 15) / 16 * 16) return;
  uint2 c[RPC / 8][8];
#pragma unroll
  for (int p = 0; p < RPC / 8; ++p) {
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = lds_v4(hold + ((int64_t)(p * 8 + k) * cols + col) * 2);
    c[p][0] = encode_col8<0>(v, bf16_bits(scale_lo(k2[0])));
    c[p][1] = encode_col8<1>(v, bf16_bits(scale_hi(k2[0])));
    c[p][2] = encode_col8<2>(v, bf16_bits(scale_lo(k2[1])));
    c[p][3] = encode_col8<3>(v, bf16_bits(scale_hi(k2[1])));
    c[p][4] = encode_col8<4>(v, bf16_bits(scale_lo(k2[2])));
    c[p][5] = encode_col8<5>(v, bf16_bits(scale_hi(k2[2])));
    c[p][6] = encode_col8<6>(v, bf16_bits(scale_lo(k2[3])));
    c[p][7] = encode_col8<7>(v, bf16_bits(scale_hi(k2[3])));
  }
  uint8_t* dst = o.qt + (int64_t)col * o.ld_qt + row0;
#pragma unroll
  for (int l = 0; l < 8; ++l, dst += o.ld_qt) {
    if constexpr (RPC == 16)
      *reinterpret_cast<uint4*>(dst) = make_uint4(c[0][l].x, c[0][l].y, c[1][l].x, c[1][l].y);
    else
      *reinterpret_cast<uint2*>(dst) = c[0][l];
  }
}

// Shared memory: [RPC][cols] BF16 held rows (COL), [threads] column maxima
// (COL), the block sums' scratch, and backward the CTA's column sums.
template <int RPC, bool COL, bool BWD>
__host__ __device__ inline uint32_t norm_smem_bytes(int32_t cols) {
  return (COL ? (uint32_t)RPC * cols * 2 + (uint32_t)cols * 2 : 0u) + 2 * 32 * 8 * 4 +
         (BWD ? (uint32_t)cols * 8 : 0u);
}

template <int MAXT, int RPC, bool COL>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) norm_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t nsmem[];
  uint8_t* hold = nsmem;
  uint4* xch = reinterpret_cast<uint4*>(nsmem + (COL ? RPC * p.cols * 2 : 0));
  float* red = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(xch) + (COL ? p.cols * 2 : 0));
  const int32_t col = threadIdx.x * 8;
  const bool active = col < p.cols;
  const int64_t row0 = (int64_t)blockIdx.x * p.rpc;
  const int64_t nrows = p.rows - row0 < p.rpc ? p.rows - row0 : p.rpc;  // may be <= 0
  const float inv_d = 1.f / (float)p.cols;
  pdl_wait();
  pdl_trigger();

  float w[8], e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = active ? load_param(p.w_pre, p.w_f32, col + i) : 0.f;
    e[i] = p.scale;
    if (p.w_post && active) e[i] *= load_param(p.w_post, p.w_f32, col + i);
    if (p.gate_kind == kGateChannel && active) e[i] *= load_param(p.gate, p.gate_f32, col + i);
  }
  uint32_t cm[4] = {0, 0, 0, 0};
  int buf = 0;
  constexpr int B = 4;  // rows in flight
  for (int rb = 0; rb < p.rpc; rb += B) {
    uint4 yv[B];
    if (rb < nrows) {
      uint4 hv[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int64_t r = row0 + rb + k;
        const bool in = active && rb + k < nrows;
        yv[k] = in ? ldg_stream(p.x + r * p.ld_x + col) : make_uint4(0, 0, 0, 0);
        hv[k] = in && p.h ? ldg_stream(p.h + r * p.ld_h + col) : make_uint4(0, 0, 0, 0);
      }
      float sum[B];
      if (p.h) {
        float r1[B];
        if (p.w_post) {
#pragma unroll
          for (int k = 0; k < B; ++k) {
            float f[8];
            unpack8(hv[k], f);
            sum[k] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[k] = fmaf(f[i], f[i], sum[k]);
          }
          block_sum(sum, red, buf);
#pragma unroll
          for (int k = 0; k < B; ++k) {
            r1[k] = rsqrtf(fmaf(sum[k], inv_d, p.eps));
            if (threadIdx.x == 0 && rb + k < nrows) p.rstd_post[row0 + rb + k] = r1[k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < B; ++k) r1[k] = 1.f;
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
          const int64_t r = row0 + rb + k;
          const bool in = active && rb + k < nrows;
          if (p.gate_kind == kGateToken && rb + k < nrows) r1[k] *= load_param(p.gate, p.gate_f32, r);
          float x[8], h[8], g[8];
          unpack8(yv[k], x);
          unpack8(hv[k], h);
          if (p.gate_kind == kGateFull) {
            unpack8(in ? ldg_stream(static_cast<const __nv_bfloat16*>(p.gate) + r * p.ld_gate + col)
                       : make_uint4(0, 0, 0, 0), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] *= g[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = fmaf(h[i] * r1[k], e[i], x[i]);
          yv[k] = pack8(x);
          if (in) *reinterpret_cast<uint4*>(p.y + r * p.ld_y + col) = yv[k];
        }
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        float f[8];
        unpack8(yv[k], f);
        sum[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[k] = fmaf(f[i], f[i], sum[k]);
      }
      block_sum(sum, red, buf);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const float r2 = rsqrtf(fmaf(sum[k], inv_d, p.eps));
        if (threadIdx.x == 0 && rb + k < nrows) p.rstd[row0 + rb + k] = r2;
        float f[8];
        unpack8(yv[k], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * r2 * w[i];
        // rows past the end hold zeros (an exact zero, whatever the weights)
        yv[k] = rb + k < nrows ? pack8(f) : make_uint4(0, 0, 0, 0);
        if (p.out.bf && active && rb + k < nrows)
          *reinterpret_cast<uint4*>(p.out.bf + (row0 + rb + k) * p.out.ld_bf + col) = yv[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < B; ++k) yv[k] = make_uint4(0, 0, 0, 0);
    }
    if (p.out.q) {
#pragma unroll
      for (int k = 0; k < B; k += 2)
        if (rb + k < p.rpc)
          emit_row_pair(p.out, row0 + rb + k, p.rows, col, active, yv[k], yv[k + 1], rb + k + 1 < p.rpc);
    }
    if (COL) {
#pragma unroll
      for (int k = 0; k < B; ++k) {
        cm[0] = amax2(cm[0], yv[k].x);
        cm[1] = amax2(cm[1], yv[k].y);
        cm[2] = amax2(cm[2], yv[k].z);
        cm[3] = amax2(cm[3], yv[k].w);
        if (active) *reinterpret_cast<uint4*>(hold + ((int64_t)(rb + k) * p.cols + col) * 2) = yv[k];
      }
    }
  }
  if (COL) {
    if (active)
      xch[threadIdx.x] = make_uint4(cm[0] & 0x7FFF7FFFu, cm[1] & 0x7FFF7FFFu, cm[2] & 0x7FFF7FFFu, cm[3] & 0x7FFF7FFFu);
    cluster_sync_all();
    emit_columns<RPC>(p.out, hold, xch, row0, p.rows, p.cols, col, active, cluster_ctarank());
    cluster_sync_all();  // no CTA leaves while a peer still reads its maxima
  }
  // the scale bytes of the rows that pad the last 128 (a cluster covers them itself)
  if (!COL && p.out.q && blockIdx.x == gridDim.x - 1) {
    const int64_t first = row0 + p.rpc, last = (p.rows + 127) / 128 * 128;
    const int32_t groups = p.cols >> 7;
    for (int64_t i = threadIdx.x; i < (last - first) * groups; i += blockDim.x) {
      const int64_t r = first + i / groups;
      const int32_t g = (int32_t)(i % groups);
      p.out.s[((r >> 7) * p.out.s_g4 + (g >> 2)) * 512 + (g & 3) + blocked_in_chunk((int)(r & 127))] = 127;
    }
  }
}

// Always launched in clusters of 128 / RPC CTAs (the column sums are joined
// over the cluster before they leave); COL adds the transposed codes.
template <int MAXT, int RPC, bool COL>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) norm_backward_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t nsmem[];
  uint8_t* hold = nsmem;
  uint4* xch = reinterpret_cast<uint4*>(nsmem + (COL ? RPC * p.cols * 2 : 0));
  float* red = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(xch) + (COL ? p.cols * 2 : 0));
  float* csum = red + 2 * 32 * 8;  // [2][cols]
  const int32_t col = threadIdx.x * 8;
  const bool active = col < p.cols;
  const int64_t row0 = (int64_t)blockIdx.x * RPC;
  const int64_t nrows = p.rows - row0 < RPC ? p.rows - row0 : RPC;  // may be <= 0
  const float inv_d = 1.f / (float)p.cols;
  const uint32_t rank = cluster_ctarank();
  pdl_wait();
  pdl_trigger();

  float w[8], e[8], acc_w[8], acc_s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = active ? load_param(p.w_pre, p.w_f32, col + i) : 0.f;
    e[i] = p.scale;
    if (p.w_post && active) e[i] *= load_param(p.w_post, p.w_f32, col + i);
    if (p.gate_kind == kGateChannel && active) e[i] *= load_param(p.gate, p.gate_f32, col + i);
    acc_w[i] = acc_s[i] = 0.f;
  }
  uint32_t cm[4] = {0, 0, 0, 0};
  int buf = 0;
  constexpr int B = 2;  // rows in flight
#pragma unroll 1
  for (int rb = 0; rb < RPC; rb += B) {
    uint4 out[B];
    if (rb < nrows) {
      uint4 nv[B], yv[B], gv[B], hv[B], tv[B];
      float r1[B], r2[B], gt[B];
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int64_t r = row0 + rb + k;
        const bool in = active && rb + k < nrows;
        nv[k] = in ? ldg_stream(p.dn + r * p.ld_dn + col) : zero;
        yv[k] = in ? ldg_stream(p.x + r * p.ld_x + col) : zero;
        gv[k] = in && p.dy ? ldg_stream(p.dy + r * p.ld_dy + col) : zero;
        hv[k] = in && p.h ? ldg_stream(p.h + r * p.ld_h + col) : zero;
        tv[k] = in && p.gate_kind == kGateFull
                    ? ldg_stream(static_cast<const __nv_bfloat16*>(p.gate) + r * p.ld_gate + col) : zero;
        const bool row_in = rb + k < nrows;
        r2[k] = row_in ? p.rstd[r] : 0.f;
        r1[k] = row_in && p.w_post ? p.rstd_post[r] : 1.f;
        gt[k] = row_in && p.gate_kind == kGateToken ? load_param(p.gate, p.gate_f32, r) : 1.f;
      }
      float sum[3 * B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        float dn[8], y[8], g[8], h[8], t[8];
        unpack8(nv[k], dn);
        unpack8(yv[k], y);
        unpack8(gv[k], g);
        unpack8(hv[k], h);
        unpack8(tv[k], t);
        float s1 = 0.f, sp = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float nh = y[i] * r2[k], tt = dn[i] * w[i];
          const float base = fmaf(r2[k], tt, g[i]);
          float eh = e[i] * (h[i] * r1[k]);
          if (p.gate_kind == kGateFull) eh *= t[i];
          s1 = fmaf(tt, nh, s1);
          sp = fmaf(eh, base, sp);
          sq = fmaf(eh, nh, sq);
          acc_w[i] = fmaf(dn[i], nh, acc_w[i]);
        }
        sum[3 * k] = s1;
        sum[3 * k + 1] = sp;
        sum[3 * k + 2] = sq;
      }
      block_sum(sum, red, buf);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int64_t r = row0 + rb + k;
        const bool in = active && rb + k < nrows;
        const float m1 = sum[3 * k] * inv_d;
        const float dot = fmaf(-r2[k] * m1, sum[3 * k + 2], sum[3 * k + 1]);  // sum of e dY hh
        const float m2 = gt[k] * dot * inv_d;
        if (p.gate_kind == kGateToken && threadIdx.x == 0 && rb + k < nrows) static_cast<float*>(p.dgate)[r] = dot;
        float dn[8], y[8], g[8], h[8], t[8];
        unpack8(nv[k], dn);
        unpack8(yv[k], y);
        unpack8(gv[k], g);
        unpack8(hv[k], h);
        unpack8(tv[k], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float nh = y[i] * r2[k];
          const float d = fmaf(r2[k], dn[i] * w[i] - nh * m1, g[i]);  // dY
          g[i] = d;
          const float hh = h[i] * r1[k];
          float gg = gt[k];
          if (p.gate_kind == kGateFull) gg = t[i];
          acc_s[i] = fmaf(gg * d, hh, acc_s[i]);
          t[i] = e[i] * d * hh;  // the gate's own gradient (full)
          const float v = e[i] * gg * d;
          h[i] = p.w_post ? r1[k] * (v - hh * m2) : v;
        }
        if (in) {
          *reinterpret_cast<uint4*>(p.dx + r * p.ld_dx + col) = pack8(g);
          if (p.gate_kind == kGateFull)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dgate) + r * p.ld_dgate + col) = pack8(t);
        }
        out[k] = in ? pack8(h) : zero;
        if (p.out.bf && in) *reinterpret_cast<uint4*>(p.out.bf + r * p.out.ld_bf + col) = out[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < B; ++k) out[k] = make_uint4(0, 0, 0, 0);
    }
    if (p.out.q) emit_row_pair(p.out, row0 + rb, p.rows, col, active, out[0], out[1], true);
    if (COL) {
#pragma unroll
      for (int k = 0; k < B; ++k) {
        cm[0] = amax2(cm[0], out[k].x);
        cm[1] = amax2(cm[1], out[k].y);
        cm[2] = amax2(cm[2], out[k].z);
        cm[3] = amax2(cm[3], out[k].w);
        if (active) *reinterpret_cast<uint4*>(hold + ((int64_t)(rb + k) * p.cols + col) * 2) = out[k];
      }
    }
  }
  if (active) {
    if (COL)
      xch[threadIdx.x] = make_uint4(cm[0] & 0x7FFF7FFFu, cm[1] & 0x7FFF7FFFu, cm[2] & 0x7FFF7FFFu, cm[3] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      csum[col + i] = acc_w[i];
      csum[p.cols + col + i] = acc_s[i];
    }
  }
  cluster_sync_all();
  if (COL) emit_columns<RPC>(p.out, hold, xch, row0, p.rows, p.cols, col, active, rank);
  // column sums of the cluster's 128 rows: each CTA joins its share of the columns
  constexpr int kCs = 128 / RPC;
  const int32_t quads = 2 * p.cols / 4;  // 4-float pieces of [2][cols]
  for (int32_t i = (int32_t)rank * (int32_t)blockDim.x + threadIdx.x; i < quads; i += kCs * blockDim.x) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kCs; ++c) {
      const uint4 v = ld_cluster_v4(smem_u32(csum + 4 * i), c);
      a.x += __uint_as_float(v.x);
      a.y += __uint_as_float(v.y);
      a.z += __uint_as_float(v.z);
      a.w += __uint_as_float(v.w);
    }
    *reinterpret_cast<float4*>(p.part + (int64_t)(blockIdx.x / kCs) * 2 * p.cols + 4 * i) = a;
  }
  cluster_sync_all();  // no CTA leaves while a peer still reads from it
}

// Column gradients from the clusters' partial sums [parts][2][cols], in a
// fixed order: a block takes 32 columns, its 8 warps every eighth partial.
struct NormColumnParams {
  const float* part;
  int64_t parts;
  int32_t cols;
  const void* w_post;
  const void* gate;  // channel gate or null
  int32_t w_f32, gate_f32;
  float scale;
  int32_t accumulate;
  float* dw_pre;
  float* dw_post;     // or null
  float* dgate;       // channel gate's gradient or null
};

__global__ void __launch_bounds__(256) norm_column_kernel(const NormColumnParams p) {
  __shared__ float sm[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t c = blockIdx.x * 32 + lane;  // cols is a multiple of 128
  pdl_wait();
  pdl_trigger();
  float a = 0.f, b = 0.f;
  for (int64_t i = warp; i < p.parts; i += 8) {
    a += p.part[i * 2 * p.cols + c];
    b += p.part[i * 2 * p.cols + p.cols + c];
  }
  sm[0][warp][lane] = a;
  sm[1][warp][lane] = b;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    a += sm[0][k][lane];
    b += sm[1][k][lane];
  }
  // (an explicit add: fused into the product before it, it would round
  // differently from the call that overwrites)
  const bool add = p.accumulate != 0;
  p.dw_pre[c] = add ? __fadd_rn(p.dw_pre[c], a) : a;
  if (p.dw_post) {
    const float v = p.scale * (p.gate ? load_param(p.gate, p.gate_f32, c) : 1.f) * b;
    p.dw_post[c] = add ? __fadd_rn(p.dw_post[c], v) : v;
  }
  if (p.dgate) {
    const float v = p.scale * (p.w_post ? load_param(p.w_post, p.w_f32, c) : 1.f) * b;
    p.dgate[c] = add ? __fadd_rn(p.dgate[c], v) : v;
  }
}

}  // namespace puro
