// The gated activation between the two projections of an FFN, fused with the
// FP8 quantization of the linear layer beside it.
//
//   forward : a = bf16(g * sigmoid(g) * u)                        -> codes of a
//   backward: dg = bf16(da u s (1 + g (1 - s))),  du = bf16(da g s) -> codes of [dg | du]
// with s = sigmoid(g), for gu = [g | u], the BF16 output of the fused
// gate+up projection.  The codes are those the activation quantizer gives
// for the BF16 tensor.
//
// Bound by HBM: 4 bytes read and 2 written per element forward, 6 and 4
// backward.  A CTA of 256 threads takes one 128 x 128 tile -- the unit in
// which both groupings (1x128 along a row, 128x1 along a column) close, so
// nothing is exchanged between CTAs -- and thread (i, j) holds rows 8i..8i+7,
// columns 8j..8j+7, as the quantizer's threads do.  Backward, one CTA writes
// the tile of dg and that of du from one read of the three inputs.
#pragma once

#include "common.cuh"
#include "norm.cuh"
#include "quant.cuh"

namespace puro {

struct GatedParams {
  int64_t rows;
  int32_t f;                    // columns of g, of u and of da
  int32_t tiles_c;              // f / 128
  const __nv_bfloat16* gu;      // [rows][2f]
  int64_t ld_gu;
  const __nv_bfloat16* da;      // backward: [rows][f]
  int64_t ld_da;
  CodeOut out;                  // forward [rows][f], backward [rows][2f]
};

constexpr uint32_t kGatedSmemBytes = kQtTileBytes + 8 * 64 * 4 + 128 * 4 + 1024;

// Quantizes the 128 x 128 tile (tr, tc) that the block holds in v (rows past
// the end zero) and writes its codes and scales, or stores it as BF16.
// Shared memory: qt_s 16 KB (1024-byte aligned), col_part [8][16][4],
// col_scale [128]; free for reuse after the caller's next barrier, qt_s once
// the tensor store has read it.
template <bool ROW, bool COL, bool BF>
__device__ __forceinline__ void emit_tile(const uint4 (&v)[8], const CodeOut& o, const CUtensorMap* tm_qt,
                                          int64_t rows, int32_t tr, int32_t tc, uint8_t* qt_s,
                                          uint32_t* col_part, float* col_scale) {
  const int tid = threadIdx.x, i = tid >> 4, j = tid & 15, warp = tid >> 5;
  const int64_t r0 = (int64_t)tr * 128 + 8 * i;
  const int32_t c0 = tc * 128 + 8 * j;
  const int32_t nrow = (int32_t)(rows - r0 < 8 ? rows - r0 : 8);  // rows of this thread that exist
  if (BF) {
    __nv_bfloat16* d = o.bf + r0 * o.ld_bf + c0;
#pragma unroll
    for (int k = 0; k < 8; ++k, d += o.ld_bf)
      if (k < nrow) *reinterpret_cast<uint4*>(d) = v[k];
  }
  if (COL) {
    uint32_t cm[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      cm[0] = amax2(cm[0], v[k].x);
      cm[1] = amax2(cm[1], v[k].y);
      cm[2] = amax2(cm[2], v[k].z);
      cm[3] = amax2(cm[3], v[k].w);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cm[q] &= 0x7FFF7FFFu;
      cm[q] = __vmaxu2(cm[q], __shfl_xor_sync(0xFFFFFFFFu, cm[q], 16));
    }
    if ((tid & 16) == 0)
      *reinterpret_cast<uint4*>(&col_part[(warp * 16 + j) * 4]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
    __syncthreads();
    if (tid < 64) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = __vmaxu2(m, col_part[(w * 16 + (tid >> 2)) * 4 + (tid & 3)]);
      const uint32_t k2 = scale_k2(m);
      const uint32_t b2 = scale_bytes2(m, k2);
      uint8_t* s = o.st + ((int64_t)tc * o.st_g4 + (tr >> 2)) * 512 + (tr & 3) + blocked_in_chunk(2 * tid);
      s[0] = static_cast<uint8_t>(b2);
      s[16] = static_cast<uint8_t>(b2 >> 16);
      *reinterpret_cast<float2*>(&col_scale[2 * tid]) = make_float2(scale_lo(k2), scale_hi(k2));
    }
  }
  if (ROW) {
    uint8_t* q = o.q + r0 * o.ld_q + c0;
    uint8_t* s = o.s + ((int64_t)tr * o.s_g4 + (tc >> 2)) * 512 + (tc & 3);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const uint4 &x = v[k], &y = v[k + 1];
      const uint32_t a = amax2(amax2(x.x, x.y), amax2(x.z, x.w)), b = amax2(amax2(y.x, y.y), amax2(y.z, y.w));
      uint32_t m = amax2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)) & 0x7FFF7FFFu;
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
      const uint32_t k2 = scale_k2(m);
      if (j == k) {
        const uint32_t bytes = scale_bytes2(m, k2);
        s[blocked_in_chunk(8 * i + k)] = static_cast<uint8_t>(bytes);
        s[blocked_in_chunk(8 * i + k + 1)] = static_cast<uint8_t>(bytes >> 16);
      }
      if (k < nrow) *reinterpret_cast<uint2*>(q) = encode_row8(x, bf16_bits(scale_lo(k2)));
      if (k + 1 < nrow) *reinterpret_cast<uint2*>(q + o.ld_q) = encode_row8(y, bf16_bits(scale_hi(k2)));
      q += 2 * o.ld_q;
    }
  }
  if (COL) {
    __syncthreads();  // column scales published
    const float4 a = *reinterpret_cast<const float4*>(&col_scale[8 * j]);
    const float4 b = *reinterpret_cast<const float4*>(&col_scale[8 * j + 4]);
    // staging layout of the tensor store: transposed row 8j + l at staging row
    // 16 l + j, 8-byte chunk i ^ 2 (j & 7) (see quant_kernel)
    uint8_t* dst = qt_s + j * 128 + ((i ^ (2 * (j & 7))) << 3);
    *reinterpret_cast<uint2*>(dst + 0 * 2048) = encode_col8<0>(v, bf16_bits(a.x));
    *reinterpret_cast<uint2*>(dst + 1 * 2048) = encode_col8<1>(v, bf16_bits(a.y));
    *reinterpret_cast<uint2*>(dst + 2 * 2048) = encode_col8<2>(v, bf16_bits(a.z));
    *reinterpret_cast<uint2*>(dst + 3 * 2048) = encode_col8<3>(v, bf16_bits(a.w));
    *reinterpret_cast<uint2*>(dst + 4 * 2048) = encode_col8<4>(v, bf16_bits(b.x));
    *reinterpret_cast<uint2*>(dst + 5 * 2048) = encode_col8<5>(v, bf16_bits(b.y));
    *reinterpret_cast<uint2*>(dst + 6 * 2048) = encode_col8<6>(v, bf16_bits(b.z));
    *reinterpret_cast<uint2*>(dst + 7 * 2048) = encode_col8<7>(v, bf16_bits(b.w));
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tma_store_3d(tm_qt, qt_s, tr * 128, tc * 16, 0);
      bulk_commit_group();
    }
  }
}

// sigmoid(g); exp(-g) = inf for very negative g gives 0.
__device__ __forceinline__ float sigmoid_f(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

template <bool BWD, bool ROW, bool COL, bool BF>
__global__ void __launch_bounds__(256, 2) gated_kernel(const __grid_constant__ CUtensorMap tm_qt, const GatedParams p) {
  extern __shared__ uint8_t gsmem_raw[];
  uint8_t* qt_s = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint32_t* col_part = reinterpret_cast<uint32_t*>(qt_s + kQtTileBytes);
  float* col_scale = reinterpret_cast<float*>(col_part + 8 * 64);
  const int tid = threadIdx.x, i = tid >> 4, j = tid & 15;
  if (COL && tid == 0) prefetch_tmap(&tm_qt);
  const int32_t tr = blockIdx.x / p.tiles_c, tc = blockIdx.x - tr * p.tiles_c;
  const int64_t r0 = (int64_t)tr * 128 + 8 * i;
  const int32_t nrow = (int32_t)(p.rows - r0 < 8 ? p.rows - r0 : 8);
  const __nv_bfloat16* gp = p.gu + r0 * p.ld_gu + tc * 128 + 8 * j;
  pdl_wait();
  pdl_trigger();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 g[8], u[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    g[k] = k < nrow ? ldg_stream(gp + k * p.ld_gu) : zero;
    u[k] = k < nrow ? ldg_stream(gp + k * p.ld_gu + p.f) : zero;
  }
  if (!BWD) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a[8], b[8];
      unpack8(g[k], a);
      unpack8(u[k], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = a[e] * sigmoid_f(a[e]) * b[e];
      g[k] = pack8(a);
    }
    emit_tile<ROW, COL, BF>(g, p.out, &tm_qt, p.rows, tr, tc, qt_s, col_part, col_scale);
  } else {
    const __nv_bfloat16* dp = p.da + r0 * p.ld_da + tc * 128 + 8 * j;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 dv = k < nrow ? ldg_stream(dp + k * p.ld_da) : zero;
      float a[8], b[8], d[8];
      unpack8(g[k], a);
      unpack8(u[k], b);
      unpack8(dv, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = sigmoid_f(a[e]);
        const float ds = d[e] * s;
        d[e] = ds * a[e];                                  // du
        a[e] = ds * b[e] * fmaf(a[e], 1.f - s, 1.f);       // dg
      }
      g[k] = pack8(a);
      u[k] = pack8(d);
    }
    emit_tile<ROW, COL, BF>(g, p.out, &tm_qt, p.rows, tr, tc, qt_s, col_part, col_scale);
    if (COL) {
      if (tid == 0) bulk_wait_group_read<0>();
      __syncthreads();
    }
    emit_tile<ROW, COL, BF>(u, p.out, &tm_qt, p.rows, tr, tc + p.tiles_c, qt_s, col_part, col_scale);
  }
  if (COL && tid == 0) bulk_wait_group<0>();
}

}  // namespace puro
