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
// backward.  A CTA of 256 threads works on 128 x 128 tiles -- the unit in
// which both groupings (1x128 along a row, 128x1 along a column) close, so
// nothing is exchanged between CTAs -- and thread (i, j) holds rows 8i..8i+7,
// columns 8j..8j+7, as the quantizer's threads do.  Backward, one CTA writes
// the tile of dg and that of du from one read of the three inputs.  While a
// tile is encoded, TMA brings the next one into the stage that its values have
// left: two CTAs per SM keep 128 KB (backward 192 KB) in flight.  The grid has
// one CTA per tile, and a CTA that is done takes over the tile of one that has
// not been launched yet (cluster launch control), so that SMs that stream
// faster take more tiles without a counter to set up.  (One tile per CTA,
// loaded into registers, left the memory idle while it was encoded:
// 32768 x 6144 took 300 us, 16384 x 6144 backward 261 us, against 204 and 178;
// at the copy rate the bytes alone take 184 and 154.)
#pragma once

#include "common.cuh"
#include "norm.cuh"
#include "quant.cuh"

namespace puro {

struct GatedParams {
  int64_t rows;
  int32_t f;                    // columns of g, of u and of da
  int32_t tiles_c;              // f / 128
  CodeOut out;                  // forward [rows][f], backward [rows][2f]
};

// The input stage, the transposed codes' staging tile (1024-byte aligned; the
// column maxima live in it before), the column scales, two barriers, the
// answer of the launch control and two words.
template <bool BWD>
constexpr uint32_t gated_smem_bytes() {
  return (BWD ? 3 : 2) * kQTileBytes + kQtTileBytes + 128 * 4 + 16 + 16 + 16;
}

// Asks for the tile of a CTA that has not been launched yet; the answer
// completes 16 bytes on the barrier.
__device__ __forceinline__ void request_tile(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}

// The tile of the answer, or -1.
__device__ __forceinline__ int32_t requested_tile(const void* answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return got ? (int32_t)x : -1;
}

// Quantizes the 128 x 128 tile (tr, tc) that the block holds in v (rows past
// the end zero) and writes its codes and scales, or stores it as BF16.
template <bool ROW, bool COL, bool BF>
__device__ __forceinline__ void emit_tile(const uint4 (&v)[8], const CodeOut& o, const CUtensorMap* tm_qt,
                                          int64_t rows, int32_t tr, int32_t tc, uint8_t* qt_s,
                                          float* col_scale) {
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
  if (ROW) {
    uint32_t rowmax[4];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const uint4 &x = v[k], &y = v[k + 1];
      const uint32_t a = amax2(amax2(x.x, x.y), amax2(x.z, x.w)), b = amax2(amax2(y.x, y.y), amax2(y.z, y.w));
      rowmax[k >> 1] = amax2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)) & 0x7FFF7FFFu;
    }
    uint8_t byte;
    const float s_mine = share_row_scales(rowmax, j, &byte);
    if ((j & 1) == 0)
      o.s[((int64_t)tr * o.s_g4 + (tc >> 2)) * 512 + (tc & 3) + blocked_in_chunk(8 * i + (j >> 1))] = byte;
    uint8_t* q = o.q + r0 * o.ld_q + c0;
#pragma unroll
    for (int k = 0; k < 8; ++k, q += o.ld_q) {
      const uint2 c = encode_row8(v[k], bf16_bits(__shfl_sync(0xFFFFFFFFu, s_mine, (tid & 16) + 2 * k)));
      if (k < nrow) *reinterpret_cast<uint2*>(q) = c;
    }
  }
  if (COL) {
    uint32_t* col_part = reinterpret_cast<uint32_t*>(qt_s);  // [8 warps][16][4]
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
    // the tensor store before has read the staging tile
    if (tid == 0) bulk_wait_group_read<0>();
    __syncthreads();
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
    __syncthreads();  // column scales published, maxima read
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

// sigmoid(g) = 1 / (1 + exp(-g)) = 2^-22 / (2^-22 + 2^(-g log2(e) - 22)).  The
// scaled denominator stays below 2^126 down to g = -102, past which the sigmoid
// is below FP32's subnormal range (-inf gives 0); unscaled it leaves the range of
// a reciprocal at g = -87.3, and products with a large u lost what is left there.
// The exponent is rounded to 2^-24 of itself, so the sigmoid is off by 2^-19 +
// |g| 2^-22 of itself, against the half step of 2^-9 when a result is rounded to
// BF16.  (32768 x 6144: 204 us; 201 unscaled; 212 with exp(-|g|) and a choice of
// the numerator; 239 with expf.)
__device__ __forceinline__ float sigmoid1(float g) {
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(fmaf(g, -1.4426950408889634f, -22.f)));
  return __fdividef(0x1p-22f, e + 0x1p-22f);
}
__device__ __forceinline__ f2 sigmoid2(f2 g) {
  const float2 v = f2_get(g);
  return f2_of(sigmoid1(v.x), sigmoid1(v.y));
}

template <bool BWD, bool ROW, bool COL, bool BF>
__global__ void __launch_bounds__(256, 2)
    gated_kernel(const __grid_constant__ CUtensorMap tm_gu, const __grid_constant__ CUtensorMap tm_da,
                 const __grid_constant__ CUtensorMap tm_qt, const GatedParams p) {
  constexpr uint32_t kTensors = BWD ? 3 : 2;
  extern __shared__ __align__(1024) uint8_t gsmem[];
  uint8_t* stage = gsmem;                                   // g, u, da: [128][128] BF16 each
  uint8_t* qt_s = gsmem + kTensors * kQTileBytes;
  float* col_scale = reinterpret_cast<float*>(qt_s + kQtTileBytes);
  uint8_t* answer = reinterpret_cast<uint8_t*>(col_scale + 128);
  uint64_t* full = reinterpret_cast<uint64_t*>(answer + 16);
  uint64_t* asked = full + 1;
  volatile int32_t* next_tile = reinterpret_cast<volatile int32_t*>(full + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + 2) + 1;
  const int tid = threadIdx.x, i = tid >> 4, j = tid & 15;
  if (tid == 0) {
    mbar_init(full, 1);
    mbar_init(asked, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_gu);
    if (BWD) prefetch_tmap(&tm_da);
    if (COL) prefetch_tmap(&tm_qt);
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  // thread 0: the loads of a tile, and the request for the one after it
  auto load = [&](int32_t t) {
    const int32_t r = t / p.tiles_c, c = t - r * p.tiles_c;
    mbar_arrive_expect_tx(full, kTensors * kQTileBytes);
    tma_load_2d<1>(stage, &tm_gu, c * 128, r * 128, smem_u32(full));
    tma_load_2d<1>(stage + kQTileBytes, &tm_gu, p.f + c * 128, r * 128, smem_u32(full));
    if (BWD) tma_load_2d<1>(stage + 2 * kQTileBytes, &tm_da, c * 128, r * 128, smem_u32(full));
    mbar_arrive_expect_tx(asked, 16);
    request_tile(answer, asked);
  };
  int32_t tile = (int32_t)blockIdx.x;
  if (tid == 0) load(tile);

  for (uint32_t it = 0;; ++it) {
    const bool ok = mbar_wait(full, it & 1, abort_flag);
    const int32_t tr = tile / p.tiles_c, tc = tile - tr * p.tiles_c;
    // this thread's 8 rows x 8 columns; rows past the end came as zeros and give zeros
    const uint8_t* src = stage + (8 * i) * 256 + 16 * j;
    uint4 v[8], w[BWD ? 8 : 1];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f2 g[4], u[4];
      unpack8(lds_v4(src + k * 256), g);
      unpack8(lds_v4(src + kQTileBytes + k * 256), u);
      if (!BWD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = mul2(mul2(g[e], sigmoid2(g[e])), u[e]);
      } else {
        f2 d[4];
        unpack8(lds_v4(src + 2 * kQTileBytes + k * 256), d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (the small factor s last: a product with it first could leave FP32's range)
          const f2 s = sigmoid2(g[e]), one = f2_both(1.f), du = mul2(mul2(d[e], g[e]), s);
          g[e] = mul2(mul2(mul2(d[e], u[e]), s), fma2(g[e], fma2(s, f2_both(-1.f), one), one));  // dg
          d[e] = du;
        }
        w[BWD ? k : 0] = pack8(d);
      }
      v[k] = pack8(g);
      // (keeps the compiler from loading all rows at once, which spills)
      if (BWD) __syncwarp();
    }
    // every thread has read the stage; if any wait gave up, all stop here
    if (__syncthreads_or(!ok)) break;
    if (tid == 0) {
      int32_t next = -1;
      if (mbar_wait(asked, it & 1, abort_flag)) next = requested_tile(answer);
      if (next >= 0) {
        fence_proxy_async_smem();  // the stage's and the answer's reads come before their next writes
        load(next);
      }
      *next_tile = next;
    }
    // (one copy of the code for both tiles: two spill more and are slower)
#pragma unroll 1
    for (int half = 0;;) {
      emit_tile<ROW, COL, BF>(v, p.out, &tm_qt, p.rows, tr, tc + half * p.tiles_c, qt_s, col_scale);
      if (!BWD || ++half == 2) break;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = w[BWD ? k : 0];
    }
    if (!COL) __syncthreads();  // next_tile is published (the tile's other barriers do it otherwise)
    tile = *next_tile;
    if (tile < 0) break;
  }
  if (COL && tid == 0) bulk_wait_group<0>();
  // Every copy and request was waited for above, unless a wait gave up; then
  // let those in flight land (bounded) before the block exits.
  if (tid == 0 && *abort_flag) {
    for (uint32_t phase = 0; phase < 2; ++phase) {
      volatile int no_abort = 0;
      mbar_wait(full, phase, &no_abort, 100000000ull);
      mbar_wait(asked, phase, &no_abort, 100000000ull);
    }
  }
}

}  // namespace puro
