// C ABI of the block-scaled FP8 linear layer (declared in include/puro_fp8.h).
//
// Host side: argument validation (before any CUDA call), device check
// (sm_100 only), TMA tensor-map encoding through the driver entry point
// (no link against libcuda), and kernel launches on the caller's stream.
// All kernels live in this one translation unit so that they share the
// device error word.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <functional>
#include <mutex>
#include <queue>
#include <type_traits>
#include <vector>

#include "../../include/puro_fp8.h"
#include "common.cuh"
#include "gated.cuh"
#include "gemm.cuh"
#include "norm.cuh"
#include "ortho.cuh"
#include "ortho_small.cuh"
#include "quant.cuh"

namespace {

constexpr int kMaxDevices = 64;

#ifndef PURO_GEMM_BN
#define PURO_GEMM_BN 256
#endif
#ifndef PURO_GEMM_CG
#define PURO_GEMM_CG 2
#endif

struct DeviceInfo {
  bool checked = false;
  bool supported = false;
  int index = 0;  // CUDA device ordinal (index into the per-device caches)
  int sms = 0;
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Current device: must be compute capability 10.0 (B200, sm_100a).
int current_device(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PURO_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.checked) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PURO_ERR_CUDA;
    d.supported = (major == 10 && minor == 0);
    d.index = dev;
    d.sms = sms;
    d.checked = true;
  }
  if (!d.supported) return PURO_ERR_UNSUPPORTED_DEVICE;
  *out = &d;
  return PURO_OK;
}

int get_encoder() {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_encode) return PURO_OK;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr)
    return PURO_ERR_CUDA;
  g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  return PURO_OK;
}

// 2-D byte tensor [outer, inner] with row stride `ld` bytes; box {box_inner,
// box_outer} stored with the given shared-memory swizzle; out-of-range reads
// return zero.
int make_map_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PURO_OK : PURO_ERR_CUDA;
}

// Blocked scale array of `rows` rows x `groups` groups seen as a 3-D tensor
// of 32-bit words {128 words per chunk, ceil(groups/4) chunks, ceil(rows/128)
// row blocks}; a box of {128, 1, nblk} loads nblk consecutive row blocks of
// one group quadruple.
int make_map_scales(CUtensorMap* m, const void* base, int64_t rows, int64_t groups, uint32_t nblk) {
  const uint64_t g4 = (uint64_t)((groups + 3) / 4), rb = (uint64_t)((rows + 127) / 128);
  cuuint64_t dims[3] = {128, g4, rb};
  cuuint64_t strides[2] = {512, g4 * 512};
  cuuint32_t box[3] = {128, 1, nblk};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PURO_OK : PURO_ERR_CUDA;
}

// The transposed codes qt [cols][ld_qt] as a 3-D tensor {qt_cols, cols/8,
// 8} with strides {1, 8 ld_qt, ld_qt} bytes and 128-byte swizzle: a 128 x
// 16 x 8 box is one tile, its transposed row 8 c_hi + c_lo at staging row
// 16 c_lo + c_hi, which is how the kernels stage it.  qt_cols: the bytes of
// a transposed row that are written (rows rounded up to 16 for
// activations, whose padding codes are 0; n for weights).
int make_map_qt(CUtensorMap* m, void* qt, int64_t qt_cols, int64_t cols, int64_t ld_qt) {
  cuuint64_t dims[3] = {(cuuint64_t)qt_cols, (cuuint64_t)(cols / 8), 8};
  cuuint64_t strides[2] = {(cuuint64_t)ld_qt * 8, (cuuint64_t)ld_qt};
  cuuint32_t box[3] = {128, 16, 8};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, qt, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PURO_OK : PURO_ERR_CUDA;
}

// [outer, inner] 16-bit matrix, boxes of box_inner x box_outer elements.
int make_map_16(CUtensorMap* m, const void* base, int64_t inner, int64_t outer, int64_t ld, uint32_t box_inner,
                uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PURO_OK : PURO_ERR_CUDA;
}

int64_t g4_of(int64_t groups) { return (groups + 3) / 4; }

int launch_status() {
  return cudaGetLastError() == cudaSuccess ? PURO_OK : PURO_ERR_CUDA;
}

// ------------------------------------------------------------------ quant

template <bool ROW, bool COL, bool BLOCK, bool RSHFL, int STAGES, bool NORM = false>
int launch_quant_cfg(const void* x, int64_t ld_x, const puro::QuantParams& p, const DeviceInfo& dev,
                     cudaStream_t stream) {
  int st = get_encoder();
  if (st != PURO_OK) return st;
  CUtensorMap m;
  if ((st = make_map_16(&m, x, p.cols, p.rows, ld_x, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE)) != PURO_OK) return st;
  CUtensorMap mqt = m;
  if (COL) {
    if ((st = make_map_qt(&mqt, p.qt, BLOCK ? p.rows : (p.rows + 15) / 16 * 16, p.cols, p.ld_qt)) != PURO_OK)
      return st;
  }
  auto kern = puro::quant_kernel<ROW, COL, BLOCK, RSHFL, STAGES, NORM>;
  constexpr uint32_t smem = puro::quant_smem_bytes<STAGES>();
  // per device, once (threads racing on the first call both set the same value)
  static std::atomic<bool> attr_done[kMaxDevices] = {};
  if (!attr_done[dev.index].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return PURO_ERR_CUDA;
    attr_done[dev.index].store(true, std::memory_order_release);
  }
  constexpr int64_t kPerSm = STAGES == 1 ? 3 : 2;  // resident CTAs per SM (shared memory)
  const int64_t grid = p.tiles < kPerSm * dev.sms ? p.tiles : kPerSm * dev.sms;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(puro::kQThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, m, mqt, p) != cudaSuccess) return PURO_ERR_CUDA;
  return launch_status();
}

// A B200's SMs (fixed, so that what depends on them does not depend on the
// device's state).
constexpr int64_t kSms = 148;

bool quant_short_stream(int64_t tiles) { return tiles <= 8 * 2 * kSms; }

// Short tile streams (up to about 8 tiles per CTA at two CTAs per SM): two
// stages, two CTAs per SM, a static tile schedule.  Longer streams: one
// stage, three CTAs per SM, and the tiles after each CTA's first handed out
// by ticket when the caller gave a tile counter (SMs stream at different
// rates, up to ~35% apart on a B200; with a static split the launch lasts as
// long as its slowest SM: 32768 x 12288 BOTH took 298 us static and 255 us by
// ticket).  Activations share their row scales by shuffles in both forms
// (7% fewer instructions than every lane deriving its own; with three CTAs
// per SM there are warps enough to hide the shuffles' latency).  Weights (at
// most a few thousand tiles) take two stages and the static schedule.  Each
// form was measured faster in its own range.
template <bool ROW, bool COL, bool BLOCK, bool NORM = false>
int launch_quant(const void* x, int64_t ld_x, const puro::QuantParams& p, const DeviceInfo& dev,
                 cudaStream_t stream) {
  const bool short_stream = quant_short_stream(p.tiles);
  puro::QuantParams ps = p;
  if (BLOCK || short_stream) ps.ctr = nullptr;
  // the kernel's division-free tile decode (tiles_c >= 1 here; < 2^24)
  ps.tc_magic = 0;
  ps.tc_shift = 0;
  if (ps.tiles_c > 1) {
    int l = 0;
    while ((int64_t(1) << l) < ps.tiles_c) ++l;
    ps.tc_magic = (uint32_t)(((uint64_t(1) << (31 + l)) + (uint64_t)ps.tiles_c - 1) / (uint64_t)ps.tiles_c);
    ps.tc_shift = l - 1;
  }
  if constexpr (BLOCK) {
    return launch_quant_cfg<ROW, COL, BLOCK, false, 2>(x, ld_x, ps, dev, stream);
  } else {
    if (short_stream) return launch_quant_cfg<ROW, COL, BLOCK, ROW, 2, NORM>(x, ld_x, ps, dev, stream);
    return launch_quant_cfg<ROW, COL, BLOCK, ROW, 1, NORM>(x, ld_x, ps, dev, stream);
  }
}

// ------------------------------------------------------------------ gemm

struct GemmArgs {
  const void* a;    int64_t lda;   // E4M3 [rows_a, K]
  const void* sfa;                 // blocked, rows_a x ceil(K/128) groups
  const void* b;    int64_t ldb;   // E4M3 [rows_b, K]
  const void* sfb;                 // blocked, rows_b x ceil(K/128) groups
  void* d; int64_t ldd;             // output [rows_a, rows_b], ldd elements per row
  int64_t rows_a, rows_b, k;
  int out;                          // puro::GemmOut
};

// Tensor maps of one GEMM: A, B, the scales of A and B, the output, and B
// again with half-height boxes (m[0..5]).
template <int CG, int BN, int BK, int OUT>
int make_gemm_maps(const GemmArgs& g, CUtensorMap* m) {
  using C = puro::GemmCfg<CG, BN, BK>;
  const int64_t kb = (g.k + 127) / 128;
  int st;
  const CUtensorMapSwizzle sw = BK == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if ((st = make_map_u8(&m[0], g.a, g.k, g.rows_a, g.lda, BK, 128, sw)) != PURO_OK) return st;
  if ((st = make_map_u8(&m[1], g.b, g.k, g.rows_b, g.ldb, BK, C::kBNC, sw)) != PURO_OK) return st;
  // B in half-height boxes, for half-width tiles
  if ((st = make_map_u8(&m[5], g.b, g.k, g.rows_b, g.ldb, BK, C::kBNC / 2, sw)) != PURO_OK) return st;
  if ((st = make_map_scales(&m[2], g.sfa, g.rows_a, kb, 1)) != PURO_OK) return st;
  if ((st = make_map_scales(&m[3], g.sfb, g.rows_b, kb, C::kNB)) != PURO_OK) return st;
  // output [rows_a, rows_b], row stride ldd elements; store boxes of 32 rows
  // x 64 bytes (32 BF16 or 16 FP32 columns)
  const bool f32 = OUT != puro::kOutBf16;
  cuuint64_t dims[2] = {(cuuint64_t)g.rows_b, (cuuint64_t)g.rows_a};
  cuuint64_t strides[1] = {(cuuint64_t)g.ldd * (f32 ? 4 : 2)};
  cuuint32_t box[2] = {f32 ? 16u : 32u, 32};
  cuuint32_t estr[2] = {1, 1};
  if (g_encode(&m[4], f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.d,
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return PURO_ERR_CUDA;
  return PURO_OK;
}

// Longest-processing-time-first assignment of the two problems' tiles to
// `clusters` clusters: tiles in order of decreasing cost (K blocks plus a
// fixed per-tile share for the epilogue), each to the least-loaded cluster;
// every cluster runs its tiles in the order they were assigned.
void make_schedule(puro::GemmParams& p, int clusters) {
  const int units = p.units;
  std::vector<int> order(units);
  for (int u = 0; u < units; ++u) order[u] = u;
  auto cost = [&](int u) { return p.prob[u >= p.tiles0 ? 1 : 0].kblocks + 2; };  // no split units here
  std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return cost(x) > cost(y); });
  using Slot = std::pair<int64_t, int>;  // (load, cluster), least load first, then lowest index
  std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>> heap;
  for (int c = 0; c < clusters; ++c) heap.push({0, c});
  std::vector<std::vector<int>> lists(clusters);
  for (int u : order) {
    Slot s = heap.top();
    heap.pop();
    lists[s.second].push_back(u);
    heap.push({s.first + cost(u), s.second});
  }
  int off = 0;
  for (int c = 0; c < clusters; ++c) {
    p.sched_off[c] = (uint16_t)off;
    for (int u : lists[c]) p.sched_unit[off++] = (uint16_t)u;
  }
  p.sched_off[clusters] = (uint16_t)off;
  p.sched = 1;
}

// One launch of the GEMM kernel over one problem (g1 == nullptr) or two
// independent problems that share the launch.
template <int CG, int BN, int BK, int OUT0, int OUT1>
int launch_gemm_cfg(const GemmArgs& g0, const GemmArgs* g1, DeviceInfo* dev, cudaStream_t stream) {
  using C = puro::GemmCfg<CG, BN, BK>;
  CUtensorMap m0[6], m1[6];
  int st;
  if ((st = make_gemm_maps<CG, BN, BK, OUT0>(g0, m0)) != PURO_OK) return st;
  if (g1) {
    if ((st = make_gemm_maps<CG, BN, BK, OUT1>(*g1, m1)) != PURO_OK) return st;
  } else {
    memcpy(m1, m0, sizeof(m0));  // unused by a one-problem launch
  }
  auto kern = puro::gemm_block_scaled_kernel<CG, BN, BK, OUT0, OUT1>;
  // per device, once (threads racing on the first call both store the same value)
  static std::atomic<int> max_clusters[kMaxDevices] = {};
  const int dev_id = dev->index;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // the occupancy query below uses the cluster attribute only
  if (max_clusters[dev_id].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) !=
        cudaSuccess)
      return PURO_ERR_CUDA;
    int n = 0;
    cfg.gridDim = dim3(CG * (dev->sms / CG));
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) n = dev->sms / CG;
    max_clusters[dev_id].store(n < puro::kMaxSchedClusters ? n : puro::kMaxSchedClusters,
                               std::memory_order_release);
  }
  static thread_local puro::GemmParams p;  // ~4.5 KB: kept off the stack
  memset(&p, 0, sizeof(p));
  const GemmArgs* gs[2] = {&g0, g1};
  p.nprob = g1 ? 2 : 1;
  for (int i = 0; i < p.nprob; ++i) {
    const GemmArgs& g = *gs[i];
    p.prob[i].rows_a = (int32_t)g.rows_a;
    p.prob[i].rows_b = (int32_t)g.rows_b;
    p.prob[i].kblocks = (int32_t)((g.k + BK - 1) / BK);
    p.prob[i].tiles_m = (int32_t)((g.rows_a + C::kBM - 1) / C::kBM);
    p.prob[i].tiles_n = (int32_t)((g.rows_b + BN - 1) / BN);
    // the larger operand is walked in the slower index, so that the tiles
    // running at the same time share its rows and L2 keeps them
    p.prob[i].n_fastest = g.rows_a > g.rows_b ? 1 : 0;
  }
  const int C_max = max_clusters[dev_id].load(std::memory_order_acquire);
  for (int i = 0; i < p.nprob; ++i) {
    const int64_t t = (int64_t)p.prob[i].tiles_m * p.prob[i].tiles_n;
    p.prob[i].split_from = (int32_t)t;
    p.prob[i].units = (int32_t)t;
  }
  if (!g1 && BN == 256) {
    // one GEMM: if the last wave of tiles would fill at most half the clusters,
    // split its tiles into half-width tiles, which then all run at once
    const int64_t t = p.prob[0].split_from;
    const int64_t full = (t / C_max) * C_max, rest = t - full;
    if (rest > 0 && 2 * rest <= C_max) {
      p.prob[0].split_from = (int32_t)full;
      p.prob[0].units = (int32_t)(full + 2 * rest);
    }
  }
  p.tiles0 = p.prob[0].units;
  p.units = p.prob[0].units + (g1 ? p.prob[1].units : 0);
  const int clusters = p.units < C_max ? p.units : C_max;
  if (g1 && p.units <= puro::kMaxSchedUnits) make_schedule(p, clusters);
  cfg.gridDim = dim3(CG * clusters);
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, m0[0], m0[1], m0[2], m0[3], m0[4], m1[0], m1[1], m1[2], m1[3],
                         m1[4], m0[5], m1[5], p) != cudaSuccess)
    return PURO_ERR_CUDA;
  return launch_status();
}

int launch_gemm(const GemmArgs& g, cudaStream_t stream) {
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != PURO_OK) return st;
  if ((st = get_encoder()) != PURO_OK) return st;
  if (g.rows_a == 0 || g.rows_b == 0) return PURO_OK;
  if (g.k == 0) {
    // empty reduction: the product is exactly zero (nothing to add when accumulating)
    if (g.out == puro::kOutF32Add) return PURO_OK;
    const size_t es = g.out == puro::kOutBf16 ? 2 : 4;
    if (cudaMemset2DAsync(g.d, (size_t)g.ldd * es, 0, (size_t)g.rows_b * es, (size_t)g.rows_a,
                          stream) != cudaSuccess)
      return PURO_ERR_CUDA;
    return PURO_OK;
  }
  constexpr int CG = PURO_GEMM_CG, BN = PURO_GEMM_BN, BK = PURO_GEMM_BK;
  switch (g.out) {
    case puro::kOutBf16:
      return launch_gemm_cfg<CG, BN, BK, puro::kOutBf16, puro::kOutBf16>(g, nullptr, dev, stream);
    case puro::kOutF32:
      return launch_gemm_cfg<CG, BN, BK, puro::kOutF32, puro::kOutF32>(g, nullptr, dev, stream);
    case puro::kOutF32Add:
      return launch_gemm_cfg<CG, BN, BK, puro::kOutF32Add, puro::kOutF32Add>(g, nullptr, dev, stream);
    default:
      return PURO_ERR_LAYOUT;
  }
}

// Two independent GEMMs in one launch: g0 with a BF16 output (the data
// gradient) and g1 with any output kind (the weight gradient).  A problem
// that is empty, or has an empty reduction, is run on its own.
int launch_gemm_pair(const GemmArgs& g0, const GemmArgs& g1, cudaStream_t stream) {
  const bool e0 = g0.rows_a == 0 || g0.rows_b == 0 || g0.k == 0;
  const bool e1 = g1.rows_a == 0 || g1.rows_b == 0 || g1.k == 0;
  if (e0 || e1) {
    int st = launch_gemm(g0, stream);
    if (st != PURO_OK) return st;
    return launch_gemm(g1, stream);
  }
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != PURO_OK) return st;
  if ((st = get_encoder()) != PURO_OK) return st;
  constexpr int CG = PURO_GEMM_CG, BN = PURO_GEMM_BN, BK = PURO_GEMM_BK;
  if (g0.out != puro::kOutBf16) return PURO_ERR_LAYOUT;
  switch (g1.out) {
    case puro::kOutBf16:
      return launch_gemm_cfg<CG, BN, BK, puro::kOutBf16, puro::kOutBf16>(g0, &g1, dev, stream);
    case puro::kOutF32:
      return launch_gemm_cfg<CG, BN, BK, puro::kOutBf16, puro::kOutF32>(g0, &g1, dev, stream);
    case puro::kOutF32Add:
      return launch_gemm_cfg<CG, BN, BK, puro::kOutBf16, puro::kOutF32Add>(g0, &g1, dev, stream);
    default:
      return PURO_ERR_LAYOUT;
  }
}

// Shape/alignment checks shared by the three GEMMs.
int check_mat(const void* p, int64_t ld, int64_t min_ld, int64_t elem_bytes) {
  if (!p) return PURO_ERR_NULL;
  if (!aligned16(p)) return PURO_ERR_ALIGN;
  if (ld < min_ld) return PURO_ERR_SHAPE;
  if ((ld * elem_bytes) % 16) return PURO_ERR_ALIGN;
  return PURO_OK;
}

constexpr int64_t kMaxDim = (int64_t)1 << 31;

}  // namespace

// Argument checks and GEMM mapping of the gradient GEMMs.  They return
// PURO_OK with *g filled in, kNothingToDo when the output is empty, or an
// error status; nothing is launched.
constexpr int kNothingToDo = 1;

int dgrad_args(const void* qdy, int64_t ld_qdy, const void* sdy, const void* qwt, int64_t ld_qwt,
               const void* sw_bwd, void* dx, int64_t ld_dx, int64_t m, int64_t n, int64_t k,
               GemmArgs* g) {
  if (m < 0 || n < 0 || k < 0 || m >= kMaxDim || n >= kMaxDim || k >= kMaxDim) return PURO_ERR_SHAPE;
  if (n % 128 || k % 128) return PURO_ERR_SHAPE;
  if (m == 0 || k == 0) return kNothingToDo;
  int r;
  if ((r = check_mat(dx, ld_dx, k, 2)) != PURO_OK) return r;
  if (n > 0) {
    if ((r = check_mat(qdy, ld_qdy, n, 1)) != PURO_OK) return r;
    if ((r = check_mat(qwt, ld_qwt, n, 1)) != PURO_OK) return r;
    if (!sdy || !sw_bwd) return PURO_ERR_NULL;
    if (!aligned16(sdy) || !aligned16(sw_bwd)) return PURO_ERR_ALIGN;
  }
  *g = GemmArgs{qdy, ld_qdy, sdy, qwt, ld_qwt, sw_bwd, dx, ld_dx, m, k, n, puro::kOutBf16};
  return PURO_OK;
}

int wgrad_args(const void* qdyt, int64_t ld_qdyt, const void* sdyt, const void* qxt, int64_t ld_qxt,
               const void* sxt, void* dw, int64_t ld_dw, int64_t m, int64_t n, int64_t k, int out,
               GemmArgs* g) {
  if (m < 0 || n < 0 || k < 0 || m >= kMaxDim || n >= kMaxDim || k >= kMaxDim) return PURO_ERR_SHAPE;
  if (n % 128 || k % 128) return PURO_ERR_SHAPE;
  if (n == 0 || k == 0) return kNothingToDo;
  int r;
  if ((r = check_mat(dw, ld_dw, k, out == puro::kOutBf16 ? 2 : 4)) != PURO_OK) return r;
  if (m > 0) {
    if ((r = check_mat(qdyt, ld_qdyt, (m + 15) / 16 * 16, 1)) != PURO_OK) return r;
    if ((r = check_mat(qxt, ld_qxt, (m + 15) / 16 * 16, 1)) != PURO_OK) return r;
    if (!sdyt || !sxt) return PURO_ERR_NULL;
    if (!aligned16(sdyt) || !aligned16(sxt)) return PURO_ERR_ALIGN;
  }
  *g = GemmArgs{qdyt, ld_qdyt, sdyt, qxt, ld_qxt, sxt, dw, ld_dw, n, k, m, out};
  return PURO_OK;
}

extern "C" {

const char* puro_fp8_status_string(int status) {
  switch (status) {
    case PURO_OK: return "PURO_OK";
    case PURO_ERR_NULL: return "PURO_ERR_NULL: a required pointer is NULL";
    case PURO_ERR_ALIGN: return "PURO_ERR_ALIGN: pointer or leading dimension not 16-byte aligned";
    case PURO_ERR_SHAPE: return "PURO_ERR_SHAPE: size or leading dimension out of range";
    case PURO_ERR_LAYOUT: return "PURO_ERR_LAYOUT: unknown layout flag";
    case PURO_ERR_CUDA: return "PURO_ERR_CUDA: a CUDA call failed";
    case PURO_ERR_UNSUPPORTED_DEVICE: return "PURO_ERR_UNSUPPORTED_DEVICE: needs sm_100 (B200)";
    case PURO_ERR_DEVICE_TIMEOUT: return "PURO_ERR_DEVICE_TIMEOUT: a bounded device wait expired";
    default: return "unknown puro_status";
  }
}

int64_t puro_fp8_blocked_scale_bytes(int64_t rows, int64_t groups) {
  if (rows <= 0 || groups <= 0) return 0;
  return ((rows + 127) / 128) * g4_of(groups) * 512;
}

int puro_fp8_quant_act(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int layout,
                       void* q, int64_t ld_q, void* s, void* qt, int64_t ld_qt, void* st,
                       uint32_t* tile_counter, void* stream) {
  if (layout != PURO_ROWWISE && layout != PURO_COLWISE && layout != PURO_BOTH)
    return PURO_ERR_LAYOUT;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim) return PURO_ERR_SHAPE;
  if (cols % 128) return PURO_ERR_SHAPE;
  if (rows == 0 || cols == 0) return PURO_OK;
  if ((cols / 128) * ((rows + 127) / 128) >= kMaxDim) return PURO_ERR_SHAPE;
  int r;
  if ((r = check_mat(x, ld_x, cols, 2)) != PURO_OK) return r;
  const bool row = layout & PURO_ROWWISE, col = layout & PURO_COLWISE;
  if (row) {
    if ((r = check_mat(q, ld_q, cols, 1)) != PURO_OK) return r;
    if (!s) return PURO_ERR_NULL;
    if (!aligned16(s)) return PURO_ERR_ALIGN;
  }
  if (col) {
    if ((r = check_mat(qt, ld_qt, (rows + 15) / 16 * 16, 1)) != PURO_OK) return r;
    if (!st) return PURO_ERR_NULL;
    if (!aligned16(st)) return PURO_ERR_ALIGN;
  }
  if (reinterpret_cast<uintptr_t>(tile_counter) % 8) return PURO_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((r = current_device(&dev)) != PURO_OK) return r;
  puro::QuantParams p{};
  p.ctr = tile_counter;
  p.rows = rows;
  p.cols = cols;
  p.q = static_cast<uint8_t*>(q);
  p.ld_q = ld_q;
  p.s = static_cast<uint8_t*>(s);
  p.s_g4 = g4_of(cols / 128);
  p.qt = static_cast<uint8_t*>(qt);
  p.ld_qt = ld_qt;
  p.st = static_cast<uint8_t*>(st);
  p.st_g4 = g4_of((rows + 127) / 128);
  p.tiles_c = (int32_t)(cols / 128);
  p.tiles = (int32_t)(p.tiles_c * ((rows + 127) / 128));
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  if (row && col) return launch_quant<true, true, false>(x, ld_x, p, *dev, sm);
  if (row) return launch_quant<true, false, false>(x, ld_x, p, *dev, sm);
  return launch_quant<false, true, false>(x, ld_x, p, *dev, sm);
}

int puro_fp8_quant_weight(const void* w, int64_t n, int64_t k, int64_t ld_w, void* q, int64_t ld_q,
                          void* s, void* qt, int64_t ld_qt, void* s_fwd, void* s_bwd,
                          void* stream) {
  if (n < 0 || k < 0 || n >= kMaxDim || k >= kMaxDim || n % 128 || k % 128) return PURO_ERR_SHAPE;
  if (n == 0 || k == 0) return PURO_OK;
  if ((k / 128) * (n / 128) >= kMaxDim) return PURO_ERR_SHAPE;
  int r;
  if ((r = check_mat(w, ld_w, k, 2)) != PURO_OK) return r;
  if ((r = check_mat(q, ld_q, k, 1)) != PURO_OK) return r;
  if (!s) return PURO_ERR_NULL;
  if (qt && (r = check_mat(qt, ld_qt, n, 1)) != PURO_OK) return r;
  if ((s_fwd && !aligned16(s_fwd)) || (s_bwd && !aligned16(s_bwd))) return PURO_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((r = current_device(&dev)) != PURO_OK) return r;
  puro::QuantParams p{};
  p.rows = n;
  p.cols = k;
  p.q = static_cast<uint8_t*>(q);
  p.ld_q = ld_q;
  p.qt = static_cast<uint8_t*>(qt);
  p.ld_qt = ld_qt;
  p.sw = static_cast<uint8_t*>(s);
  p.sw_fwd = static_cast<uint8_t*>(s_fwd);
  p.fwd_g4 = g4_of(k / 128);
  p.sw_bwd = static_cast<uint8_t*>(s_bwd);
  p.bwd_g4 = g4_of(n / 128);
  p.tiles_c = (int32_t)(k / 128);
  p.tiles = (int32_t)(p.tiles_c * (n / 128));
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  if (qt) return launch_quant<true, true, true>(w, ld_w, p, *dev, sm);
  return launch_quant<true, false, true>(w, ld_w, p, *dev, sm);
}

int puro_fp8_gemm_fprop(const void* qx, int64_t ld_qx, const void* sx, const void* qw,
                        int64_t ld_qw, const void* sw_fwd, void* y, int64_t ld_y, int64_t m,
                        int64_t n, int64_t k, void* stream) {
  if (m < 0 || n < 0 || k < 0 || m >= kMaxDim || n >= kMaxDim || k >= kMaxDim) return PURO_ERR_SHAPE;
  if (n % 128 || k % 128) return PURO_ERR_SHAPE;
  if (m == 0 || n == 0) return PURO_OK;
  int r;
  if ((r = check_mat(y, ld_y, n, 2)) != PURO_OK) return r;
  if (k > 0) {
    if ((r = check_mat(qx, ld_qx, k, 1)) != PURO_OK) return r;
    if ((r = check_mat(qw, ld_qw, k, 1)) != PURO_OK) return r;
    if (!sx || !sw_fwd) return PURO_ERR_NULL;
    if (!aligned16(sx) || !aligned16(sw_fwd)) return PURO_ERR_ALIGN;
  }
  GemmArgs g{qx, ld_qx, sx, qw, ld_qw, sw_fwd, y, ld_y, m, n, k, puro::kOutBf16};
  return launch_gemm(g, static_cast<cudaStream_t>(stream));
}

int puro_fp8_gemm_dgrad(const void* qdy, int64_t ld_qdy, const void* sdy, const void* qwt,
                        int64_t ld_qwt, const void* sw_bwd, void* dx, int64_t ld_dx, int64_t m,
                        int64_t n, int64_t k, void* stream) {
  GemmArgs g;
  const int r = dgrad_args(qdy, ld_qdy, sdy, qwt, ld_qwt, sw_bwd, dx, ld_dx, m, n, k, &g);
  if (r != PURO_OK) return r == kNothingToDo ? PURO_OK : r;
  return launch_gemm(g, static_cast<cudaStream_t>(stream));
}

int puro_fp8_gemm_wgrad(const void* qdyt, int64_t ld_qdyt, const void* sdyt, const void* qxt,
                        int64_t ld_qxt, const void* sxt, void* dw, int64_t ld_dw, int64_t m,
                        int64_t n, int64_t k, void* stream) {
  GemmArgs g;
  const int r = wgrad_args(qdyt, ld_qdyt, sdyt, qxt, ld_qxt, sxt, dw, ld_dw, m, n, k, puro::kOutBf16, &g);
  if (r != PURO_OK) return r == kNothingToDo ? PURO_OK : r;
  return launch_gemm(g, static_cast<cudaStream_t>(stream));
}

int puro_fp8_gemm_wgrad_f32(const void* qdyt, int64_t ld_qdyt, const void* sdyt, const void* qxt,
                            int64_t ld_qxt, const void* sxt, void* dw, int64_t ld_dw, int64_t m,
                            int64_t n, int64_t k, int accumulate, void* stream) {
  if (accumulate != 0 && accumulate != 1) return PURO_ERR_LAYOUT;
  GemmArgs g;
  const int r = wgrad_args(qdyt, ld_qdyt, sdyt, qxt, ld_qxt, sxt, dw, ld_dw, m, n, k,
                           accumulate ? puro::kOutF32Add : puro::kOutF32, &g);
  if (r != PURO_OK) return r == kNothingToDo ? PURO_OK : r;
  return launch_gemm(g, static_cast<cudaStream_t>(stream));
}

int puro_fp8_gemm_dgrad_wgrad(const void* qdy, int64_t ld_qdy, const void* sdy, const void* qwt,
                              int64_t ld_qwt, const void* sw_bwd, void* dx, int64_t ld_dx,
                              const void* qdyt, int64_t ld_qdyt, const void* sdyt, const void* qxt,
                              int64_t ld_qxt, const void* sxt, void* dw, int64_t ld_dw, int64_t m,
                              int64_t n, int64_t k, int dw_kind, void* stream) {
  if (dw_kind < PURO_DW_BF16 || dw_kind > PURO_DW_F32_ACCUMULATE) return PURO_ERR_LAYOUT;
  const int out = dw_kind == PURO_DW_BF16 ? puro::kOutBf16
                  : dw_kind == PURO_DW_F32 ? puro::kOutF32 : puro::kOutF32Add;
  GemmArgs gd, gw;
  const int rd = dgrad_args(qdy, ld_qdy, sdy, qwt, ld_qwt, sw_bwd, dx, ld_dx, m, n, k, &gd);
  if (rd != PURO_OK && rd != kNothingToDo) return rd;
  const int rw = wgrad_args(qdyt, ld_qdyt, sdyt, qxt, ld_qxt, sxt, dw, ld_dw, m, n, k, out, &gw);
  if (rw != PURO_OK && rw != kNothingToDo) return rw;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rd == kNothingToDo) return rw == kNothingToDo ? PURO_OK : launch_gemm(gw, s);
  if (rw == kNothingToDo) return launch_gemm(gd, s);
  return launch_gemm_pair(gd, gw, s);
}

int puro_fp8_device_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return PURO_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, puro::g_status, sizeof(int)) != cudaSuccess) return PURO_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(puro::g_status, &zero, sizeof(int)) != cudaSuccess) return PURO_ERR_CUDA;
  }
  return v;
}

}  // extern "C"

// ------------------------------------------------------------------ self-test

namespace puro {
__global__ void bounded_wait_selftest_kernel(uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);  // nothing ever arrives
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait(&bar, 0, &abort_flag, limit_ns);
}
}  // namespace puro

extern "C" int puro_fp8_test_schedule(int32_t units0, int32_t kblocks0, int32_t units1,
                                      int32_t kblocks1, int32_t clusters, int32_t* offsets,
                                      int32_t* units) {
  if (!offsets || !units) return PURO_ERR_NULL;
  if (clusters < 1 || clusters > puro::kMaxSchedClusters || units0 < 0 || units1 < 0 ||
      kblocks0 < 0 || kblocks1 < 0 || (int64_t)units0 + units1 > puro::kMaxSchedUnits)
    return PURO_ERR_SHAPE;
  static puro::GemmParams p;  // a few KB: kept off the caller's stack
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  memset(&p, 0, sizeof(p));
  p.nprob = 2;
  p.prob[0].kblocks = kblocks0;
  p.prob[0].units = units0;
  p.prob[1].kblocks = kblocks1;
  p.prob[1].units = units1;
  p.tiles0 = units0;
  p.units = units0 + units1;
  make_schedule(p, clusters);
  for (int c = 0; c <= clusters; ++c) offsets[c] = p.sched_off[c];
  for (int u = 0; u < p.units; ++u) units[u] = p.sched_unit[u];
  return PURO_OK;
}

extern "C" int puro_fp8_test_bounded_wait(int64_t limit_ns, void* stream) {
  if (limit_ns < 1000) limit_ns = 1000;
  if (limit_ns > 5000000000ll) limit_ns = 5000000000ll;
  DeviceInfo* dev = nullptr;
  int r = current_device(&dev);
  if (r != PURO_OK) return r;
  puro::bounded_wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
      (uint64_t)limit_ns);
  return launch_status();
}

// ---------------------------------------------------------------- static-scratch entry point
//
// Some callers cannot hand this library any device memory beyond their inputs
// and outputs: an engine that reserves the GPU's memory for its own pool at
// start-up leaves nothing for cudaMalloc (which then fails, or stalls the
// device while the pool gives memory back), and a C caller that only holds
// the buffers it was given has no allocator to ask.  For them, the
// quantizer's tile counter lives in this file-scope array instead: 256
// bytes (one counter pair is used) in the library's own device memory, held
// by every GPU that loads the library until the process exits.  Host code
// needs its device address, which cudaGetSymbolAddress gives once per device
// (the symbol's name is only a host-side stand-in).
namespace {

constexpr size_t kStaticScratchBytes = 256;
static __device__ __align__(256) uint32_t g_static_scratch[kStaticScratchBytes / 4];
uint32_t* g_static_scratch_addr[kMaxDevices] = {};

}  // namespace

extern "C" int puro_fp8_quant_act_static_scratch(const void* x, int64_t rows, int64_t cols,
                                                 int64_t ld_x, int layout, void* q, int64_t ld_q,
                                                 void* s, void* qt, int64_t ld_qt, void* st,
                                                 void* stream) {
  // the sizes this entry point takes (the rest is checked by the common path)
  if (layout != PURO_ROWWISE && layout != PURO_COLWISE && layout != PURO_BOTH)
    return PURO_ERR_LAYOUT;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim || cols % 128) return PURO_ERR_SHAPE;
  if (rows == 0 || cols == 0) return PURO_OK;
  // the counter's 32-bit tickets: at most one per tile plus one per CTA
  if ((cols / 128) * ((rows + 127) / 128) >= kMaxDim) return PURO_ERR_SHAPE;
  DeviceInfo* dev = nullptr;
  int r = current_device(&dev);
  if (r != PURO_OK) return r;
  uint32_t* ctr = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_static_scratch_addr[dev->index]) {
      void* a = nullptr;
      if (cudaGetSymbolAddress(&a, g_static_scratch) != cudaSuccess || a == nullptr)
        return PURO_ERR_CUDA;
      g_static_scratch_addr[dev->index] = static_cast<uint32_t*>(a);
    }
    ctr = g_static_scratch_addr[dev->index];
  }
  // The counter must start at zero.  Each call clears it on its stream before
  // its kernel (the kernel also leaves it zero), so a call that ended early
  // leaves nothing behind; calls that overlap on the GPU share it and race.
  if (cudaMemsetAsync(ctr, 0, 2 * sizeof(uint32_t), static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return PURO_ERR_CUDA;
  return puro_fp8_quant_act(x, rows, cols, ld_x, layout, q, ld_q, s, qt, ld_qt, st, ctr, stream);
}

// ---------------------------------------------------------------- norms and gated activation

namespace {

// Checks the outputs of a kernel that leaves a BF16 result [rows, cols] as
// codes or as it is, and fills in where they go.
int code_out_args(int layout, int64_t rows, int64_t cols, void* q, int64_t ld_q, void* s, void* qt,
                  int64_t ld_qt, void* st, void* bf, int64_t ld_bf, puro::CodeOut* o) {
  *o = puro::CodeOut{};
  int r;
  if (layout == PURO_BF16) {
    if ((r = check_mat(bf, ld_bf, cols, 2)) != PURO_OK) return r;
    o->bf = static_cast<__nv_bfloat16*>(bf);
    o->ld_bf = ld_bf;
    return PURO_OK;
  }
  if (layout & PURO_ROWWISE) {
    if ((r = check_mat(q, ld_q, cols, 1)) != PURO_OK) return r;
    if (!s) return PURO_ERR_NULL;
    if (!aligned16(s)) return PURO_ERR_ALIGN;
    o->q = static_cast<uint8_t*>(q);
    o->ld_q = ld_q;
    o->s = static_cast<uint8_t*>(s);
    o->s_g4 = g4_of(cols / 128);
  }
  if (layout & PURO_COLWISE) {
    if ((r = check_mat(qt, ld_qt, (rows + 15) / 16 * 16, 1)) != PURO_OK) return r;
    if (!st) return PURO_ERR_NULL;
    if (!aligned16(st)) return PURO_ERR_ALIGN;
    o->qt = static_cast<uint8_t*>(qt);
    o->ld_qt = ld_qt;
    o->st = static_cast<uint8_t*>(st);
    o->st_g4 = g4_of((rows + 127) / 128);
  }
  return PURO_OK;
}

bool known_layout(int layout) {
  return layout == PURO_ROWWISE || layout == PURO_COLWISE || layout == PURO_BOTH || layout == PURO_BF16;
}

bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Sizes and parameters that both directions of the norms take.
int norm_common_args(const void* w_pre, const void* w_post, int w_f32, const void* gate, int64_t ld_gate,
                     int gate_kind, int gate_f32, float scale, const void* h, int64_t rows, int64_t cols,
                     puro::NormParams* p) {
  if (!w_pre) return PURO_ERR_NULL;
  const uintptr_t wa = w_f32 ? 4 : 2;
  if (!aligned_to(w_pre, wa) || !aligned_to(w_post, wa)) return PURO_ERR_ALIGN;
  if (gate_kind != PURO_GATE_NONE) {
    if (!gate) return PURO_ERR_NULL;
    if (gate_kind == PURO_GATE_FULL) {
      int r;
      if ((r = check_mat(gate, ld_gate, cols, 2)) != PURO_OK) return r;
    } else if (!aligned_to(gate, gate_f32 ? 4 : 2)) {
      return PURO_ERR_ALIGN;
    }
  }
  p->rows = rows;
  p->cols = (int32_t)cols;
  p->w_pre = w_pre;
  p->w_post = h ? w_post : nullptr;
  p->w_f32 = w_f32;
  p->gate = h ? gate : nullptr;
  p->ld_gate = ld_gate;
  p->gate_kind = h ? gate_kind : PURO_GATE_NONE;
  p->gate_f32 = gate_f32;
  p->scale = scale;
  p->wide = aligned16(w_pre) && aligned16(p->w_post) && (gate_kind != PURO_GATE_CHANNEL || aligned16(gate));
  return PURO_OK;
}

int norm_flags(int w_f32, int gate_kind, int gate_f32, int64_t rows, int64_t cols, int layout) {
  if (!known_layout(layout)) return PURO_ERR_LAYOUT;
  if (gate_kind < PURO_GATE_NONE || gate_kind > PURO_GATE_FULL || (w_f32 & ~1) || (gate_f32 & ~1) ||
      (gate_kind == PURO_GATE_FULL && gate_f32))
    return PURO_ERR_LAYOUT;
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols % 128 || cols > puro::kNormMaxCols) return PURO_ERR_SHAPE;
  return PURO_OK;
}

// Launches `kern` on `grid` CTAs; it may start while the kernel before it on
// the stream still runs.
template <class Kern, class Params>
int launch_chained(Kern kern, const Params& p, dim3 grid, int threads, uint32_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return PURO_ERR_CUDA;
  }
  return PURO_OK;
}

// Quantizer parameters of a BF16 tensor [rows, cols] that the kernel before
// this one leaves, its tile counter included.
puro::QuantParams quant_params(const puro::CodeOut& o, int64_t rows, int64_t cols, uint32_t* ctr) {
  puro::QuantParams p{};
  p.ctr = ctr;
  p.rows = rows;
  p.cols = cols;
  p.q = o.q;
  p.ld_q = o.ld_q;
  p.s = o.s;
  p.s_g4 = o.s_g4;
  p.qt = o.qt;
  p.ld_qt = o.ld_qt;
  p.st = o.st;
  p.st_g4 = o.st_g4;
  p.tiles_c = (int32_t)(cols / 128);
  p.tiles = (int32_t)(p.tiles_c * ((rows + 127) / 128));
  return p;
}

// Rows that a CTA of a row pass takes: `most`, or fewer, down to `least`, where
// that would leave an SM without its `resident` CTAs.  (The split, and with it
// the order in which the backward pass adds its sums over tokens, depends on
// the sizes alone.)
int norm_rpc(int64_t rows, int64_t resident, int most, int least) {
  int rpc = most;
  while (rpc > least && rows < rpc * resident * kSms) rpc /= 2;
  return rpc;
}
// 32 backward: each CTA leaves 8 bytes per column for the column pass
// (32768 x 2048: 230 us with 32 rows, 243 with 16, 235 with 64).
int norm_backward_rpc(int64_t rows, int64_t cols) {
  return norm_rpc(rows, cols <= 2048 ? 2 : 1, 32, cols <= 4096 ? 4 : 2);
}

int64_t norm_backward_parts(int64_t rows, int64_t cols) {
  const int rpc = norm_backward_rpc(rows, cols);
  return (rows + rpc - 1) / rpc;
}

// The workspace: the tile counter of the quantizing pass, the partial column
// sums and, where transposed codes are asked for, dh in BF16.
constexpr int64_t kNormCounterBytes = 256;
int64_t norm_part_bytes(int64_t rows, int64_t cols) {
  return norm_backward_parts(rows, cols) * 2 * cols * (int64_t)sizeof(float);
}

template <class Kern>
int launch_norm_pass(Kern kern, std::atomic<bool>* done, uint32_t max_smem, const puro::NormParams& p, uint32_t smem,
                     const DeviceInfo& dev, cudaStream_t stream) {
  if (!done[dev.index].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)max_smem) != cudaSuccess)
      return PURO_ERR_CUDA;
    done[dev.index].store(true, std::memory_order_release);
  }
  return launch_chained(kern, p, dim3((unsigned)((p.rows + p.rpc - 1) / p.rpc)), (p.cols / 8 + 31) / 32 * 32, smem,
                        stream);
}

template <int MAXT, int ROWS, bool POST, int GATE>
int launch_norm_forward_as(puro::NormParams p, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevices] = {};
  // 16 forward, for an even end (32768 x 2048, both norms and a gate per token: 117
  // us; 124 with 32 rows, 122 with 8), but 32 where one CTA fills an SM (8192 x
  // 8192: 142 us against 145)
  p.rpc = norm_rpc(p.rows, MAXT == 256 ? 3 : MAXT == 512 ? 2 : 1, MAXT == 1024 ? 32 : 16, ROWS);
  const int threads = (p.cols / 8 + 31) / 32 * 32;
  const int tensors = 1 + (p.h != nullptr) + (GATE == PURO_GATE_FULL);
  return launch_norm_pass(puro::norm_forward_kernel<MAXT, ROWS, POST, GATE>, done, puro::norm_pass_smem(ROWS, MAXT, 3), p,
                          puro::norm_pass_smem(ROWS, threads, tensors), dev, stream);
}

template <int MAXT, int ROWS>
int launch_norm_forward(const puro::NormParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  auto with_gate = [&](auto post) {
    constexpr bool kPost = decltype(post)::value;
    switch (p.gate_kind) {
      case PURO_GATE_TOKEN: return launch_norm_forward_as<MAXT, ROWS, kPost, PURO_GATE_TOKEN>(p, dev, stream);
      case PURO_GATE_CHANNEL: return launch_norm_forward_as<MAXT, ROWS, kPost, PURO_GATE_CHANNEL>(p, dev, stream);
      case PURO_GATE_FULL: return launch_norm_forward_as<MAXT, ROWS, kPost, PURO_GATE_FULL>(p, dev, stream);
      default: return launch_norm_forward_as<MAXT, ROWS, kPost, PURO_GATE_NONE>(p, dev, stream);
    }
  };
  return p.w_post ? with_gate(std::true_type{}) : with_gate(std::false_type{});
}

template <int MAXT, int ROWS>
int launch_norm_backward(const puro::NormParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevices] = {};
  const int threads = (p.cols / 8 + 31) / 32 * 32;
  const int tensors = 2 + (p.dy != nullptr) + (p.h != nullptr) + (p.gate_kind == PURO_GATE_FULL);
  return launch_norm_pass(puro::norm_backward_kernel<MAXT, ROWS>, done, puro::norm_pass_smem(ROWS, MAXT, 5), p,
                          puro::norm_pass_smem(ROWS, threads, tensors), dev, stream);
}

template <bool BWD, bool ROW, bool COL, bool BF>
int launch_gated_cfg(const puro::GatedParams& p, const void* gu, int64_t ld_gu, const void* da, int64_t ld_da,
                     const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap mgu, mda, mqt;
  int st;
  if ((st = get_encoder()) != PURO_OK) return st;
  if ((st = make_map_16(&mgu, gu, 2 * (int64_t)p.f, p.rows, ld_gu, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE)) != PURO_OK)
    return st;
  mda = mqt = mgu;
  if (BWD &&
      (st = make_map_16(&mda, da, p.f, p.rows, ld_da, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE)) != PURO_OK)
    return st;
  if (COL &&
      (st = make_map_qt(&mqt, p.out.qt, (p.rows + 15) / 16 * 16, (BWD ? 2 : 1) * (int64_t)p.f, p.out.ld_qt)) != PURO_OK)
    return st;
  auto kern = puro::gated_kernel<BWD, ROW, COL, BF>;
  constexpr uint32_t smem = puro::gated_smem_bytes<BWD>();
  static std::atomic<bool> done[kMaxDevices] = {};
  if (!done[dev.index].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return PURO_ERR_CUDA;
    done[dev.index].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((p.rows + 127) / 128 * p.tiles_c));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, mgu, mda, mqt, p) != cudaSuccess) {
    cudaGetLastError();
    return PURO_ERR_CUDA;
  }
  return PURO_OK;
}

template <bool BWD>
int gated(const void* da, int64_t ld_da, const void* gu, int64_t ld_gu, int64_t rows, int64_t f, int layout,
          void* q, int64_t ld_q, void* s, void* qt, int64_t ld_qt, void* st, void* bf, int64_t ld_bf,
          void* stream) {
  if (!known_layout(layout)) return PURO_ERR_LAYOUT;
  if (rows < 0 || f < 0 || rows >= kMaxDim || f >= kMaxDim / 2 || f % 128) return PURO_ERR_SHAPE;
  if (rows == 0 || f == 0) return PURO_OK;
  if ((f / 128) * ((rows + 127) / 128) >= kMaxDim / 2) return PURO_ERR_SHAPE;
  int r;
  if ((r = check_mat(gu, ld_gu, 2 * f, 2)) != PURO_OK) return r;
  if (BWD && (r = check_mat(da, ld_da, f, 2)) != PURO_OK) return r;
  puro::GatedParams p{};
  if ((r = code_out_args(layout, rows, (BWD ? 2 : 1) * f, q, ld_q, s, qt, ld_qt, st, bf, ld_bf, &p.out)) != PURO_OK)
    return r;
  DeviceInfo* dev = nullptr;
  if ((r = current_device(&dev)) != PURO_OK) return r;
  p.rows = rows;
  p.f = (int32_t)f;
  p.tiles_c = (int32_t)(f / 128);
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  switch (layout) {
    case PURO_ROWWISE: return launch_gated_cfg<BWD, true, false, false>(p, gu, ld_gu, da, ld_da, *dev, sm);
    case PURO_COLWISE: return launch_gated_cfg<BWD, false, true, false>(p, gu, ld_gu, da, ld_da, *dev, sm);
    case PURO_BOTH: return launch_gated_cfg<BWD, true, true, false>(p, gu, ld_gu, da, ld_da, *dev, sm);
    default: return launch_gated_cfg<BWD, false, false, true>(p, gu, ld_gu, da, ld_da, *dev, sm);
  }
}

}  // namespace

extern "C" {

int puro_fp8_residual_norm(const void* x, int64_t ld_x, const void* h, int64_t ld_h, const void* w_pre,
                           const void* w_post, int w_f32, const void* gate, int64_t ld_gate, int gate_kind,
                           int gate_f32, float scale, float eps, int64_t rows, int64_t cols, void* y, int64_t ld_y,
                           float* rstd, float* rstd_post, int layout, void* q, int64_t ld_q, void* s, void* qt,
                           int64_t ld_qt, void* st, void* n, int64_t ld_n, void* workspace, void* stream) {
  int r;
  if ((r = norm_flags(w_f32, gate_kind, gate_f32, rows, cols, layout)) != PURO_OK) return r;
  if (!(eps > 0.f)) return PURO_ERR_SHAPE;
  if (rows == 0 || cols == 0) return PURO_OK;
  puro::NormParams p{};
  if ((r = check_mat(x, ld_x, cols, 2)) != PURO_OK) return r;
  if (h) {
    if ((r = check_mat(h, ld_h, cols, 2)) != PURO_OK) return r;
    if ((r = check_mat(y, ld_y, cols, 2)) != PURO_OK) return r;
  }
  if ((r = norm_common_args(w_pre, w_post, w_f32, gate, ld_gate, gate_kind, gate_f32, scale, h, rows, cols, &p)) !=
      PURO_OK)
    return r;
  if (!rstd || (p.w_post && !rstd_post)) return PURO_ERR_NULL;
  if (!aligned_to(rstd, 4) || !aligned_to(rstd_post, 4)) return PURO_ERR_ALIGN;
  if ((r = code_out_args(layout, rows, cols, q, ld_q, s, qt, ld_qt, st, n, ld_n, &p.out)) != PURO_OK) return r;
  // Row-wise codes and BF16 come from the row pass; transposed codes, and the
  // row-wise ones beside them, from the tile pass over y.
  const bool col = p.out.qt != nullptr;
  const puro::CodeOut out = p.out;
  if (col) {
    if (puro_fp8_residual_norm_workspace_bytes(rows, cols, layout, 0)) {
      if (!workspace) return PURO_ERR_NULL;
      if (!aligned16(workspace)) return PURO_ERR_ALIGN;
      p.ctr = static_cast<uint32_t*>(workspace);
    }
    p.out = puro::CodeOut{};
  }
  DeviceInfo* dev = nullptr;
  if ((r = current_device(&dev)) != PURO_OK) return r;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.ld_x = ld_x;
  p.h = static_cast<const __nv_bfloat16*>(h);
  p.ld_h = ld_h;
  p.eps = eps;
  int exponent;
  p.scale_pow2 = std::fabs(std::frexp(scale, &exponent)) == 0.5f;
  p.y = static_cast<__nv_bfloat16*>(y);
  p.ld_y = ld_y;
  p.rstd = rstd;
  p.rstd_post = rstd_post;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  r = cols <= 2048   ? launch_norm_forward<256, 4>(p, *dev, sm)
      : cols <= 4096 ? launch_norm_forward<512, 2>(p, *dev, sm)
                     : launch_norm_forward<1024, 2>(p, *dev, sm);
  if (r != PURO_OK || !col) return r;
  puro::QuantParams qp = quant_params(out, rows, cols, p.ctr);
  qp.rstd = rstd;
  qp.w = w_pre;
  qp.w_f32 = w_f32;
  qp.w_wide = aligned16(w_pre);
  const void* src = h ? y : x;
  const int64_t ld = h ? ld_y : ld_x;
  return out.q ? launch_quant<true, true, false, true>(src, ld, qp, *dev, sm)
               : launch_quant<false, true, false, true>(src, ld, qp, *dev, sm);
}

int64_t puro_fp8_residual_norm_workspace_bytes(int64_t rows, int64_t cols, int layout, int backward) {
  if (rows <= 0 || cols <= 0) return 0;
  const bool col = layout == PURO_COLWISE || layout == PURO_BOTH;
  if (!backward) return col && !quant_short_stream((rows + 127) / 128 * (cols / 128)) ? kNormCounterBytes : 0;
  return kNormCounterBytes + norm_part_bytes(rows, cols) + (col ? rows * cols * 2 : 0);
}

int puro_fp8_residual_norm_backward(const void* dn, int64_t ld_dn, const void* dy, int64_t ld_dy, const void* y,
                                    int64_t ld_y, const float* rstd, const void* h, int64_t ld_h,
                                    const float* rstd_post, const void* w_pre, const void* w_post, int w_f32,
                                    const void* gate, int64_t ld_gate, int gate_kind, int gate_f32, float scale,
                                    int64_t rows, int64_t cols, void* dx, int64_t ld_dx, float* dw_pre,
                                    float* dw_post, void* dgate, int64_t ld_dgate, int accumulate, int layout,
                                    void* q, int64_t ld_q, void* s, void* qt, int64_t ld_qt, void* st, void* dh,
                                    int64_t ld_dh, void* workspace, void* stream) {
  int r;
  if ((r = norm_flags(w_f32, gate_kind, gate_f32, rows, cols, layout)) != PURO_OK) return r;
  if (accumulate != 0 && accumulate != 1) return PURO_ERR_LAYOUT;
  if (cols == 0) return PURO_OK;
  puro::NormParams p{};
  if ((r = norm_common_args(w_pre, w_post, w_f32, gate, ld_gate, rows ? gate_kind : PURO_GATE_NONE, gate_f32, scale,
                            h, rows, cols, &p)) != PURO_OK)
    return r;
  // (an empty h has no address: without rows, the weights and the gate alone
  // say which gradients there are)
  if (rows == 0) p.w_post = w_post;
  const bool channel = (h || rows == 0) && gate_kind == PURO_GATE_CHANNEL;
  if (!dw_pre || (p.w_post && !dw_post) || (channel && (!dgate || !gate))) return PURO_ERR_NULL;
  if (!aligned_to(dw_pre, 4) || !aligned_to(dw_post, 4) || (channel && !aligned_to(dgate, 4))) return PURO_ERR_ALIGN;
  if (rows > 0) {
    if ((r = check_mat(dn, ld_dn, cols, 2)) != PURO_OK) return r;
    if (dy && (r = check_mat(dy, ld_dy, cols, 2)) != PURO_OK) return r;
    if ((r = check_mat(y, ld_y, cols, 2)) != PURO_OK) return r;
    if ((r = check_mat(dx, ld_dx, cols, 2)) != PURO_OK) return r;
    if (!rstd || !workspace) return PURO_ERR_NULL;
    if (!aligned_to(rstd, 4) || !aligned16(workspace)) return PURO_ERR_ALIGN;
    if (h) {
      if ((r = check_mat(h, ld_h, cols, 2)) != PURO_OK) return r;
      if (p.w_post && !rstd_post) return PURO_ERR_NULL;
      if (!aligned_to(rstd_post, 4)) return PURO_ERR_ALIGN;
      if (p.gate_kind == PURO_GATE_FULL && (r = check_mat(dgate, ld_dgate, cols, 2)) != PURO_OK) return r;
      if (p.gate_kind == PURO_GATE_TOKEN) {
        if (!dgate) return PURO_ERR_NULL;
        if (!aligned_to(dgate, 4)) return PURO_ERR_ALIGN;
      }
      if ((r = code_out_args(layout, rows, cols, q, ld_q, s, qt, ld_qt, st, dh, ld_dh, &p.out)) != PURO_OK) return r;
    }
  }
  DeviceInfo* dev = nullptr;
  if ((r = current_device(&dev)) != PURO_OK) return r;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  if (rows > 0) {
    p.dn = static_cast<const __nv_bfloat16*>(dn);
    p.ld_dn = ld_dn;
    p.dy = static_cast<const __nv_bfloat16*>(dy);
    p.ld_dy = ld_dy;
    p.x = static_cast<const __nv_bfloat16*>(y);
    p.ld_x = ld_y;
    p.h = static_cast<const __nv_bfloat16*>(h);
    p.ld_h = ld_h;
    p.rstd = const_cast<float*>(rstd);
    p.rstd_post = const_cast<float*>(rstd_post);
    p.dx = static_cast<__nv_bfloat16*>(dx);
    p.ld_dx = ld_dx;
    p.dgate = dgate;
    p.ld_dgate = ld_dgate;
    char* ws = static_cast<char*>(workspace);
    p.part = reinterpret_cast<float*>(ws + kNormCounterBytes);
    p.rpc = norm_backward_rpc(rows, cols);
    const bool col = p.out.qt != nullptr;
    const puro::CodeOut out = p.out;
    if (col) {
      // dh in BF16 first; the quantizer makes both kinds of codes from it
      p.ctr = reinterpret_cast<uint32_t*>(ws);
      p.out = puro::CodeOut{};
      p.out.bf = reinterpret_cast<__nv_bfloat16*>(ws + kNormCounterBytes + norm_part_bytes(rows, cols));
      p.out.ld_bf = cols;
    }
    r = cols <= 2048   ? launch_norm_backward<256, 2>(p, *dev, sm)
        : cols <= 4096 ? launch_norm_backward<512, 2>(p, *dev, sm)
                       : launch_norm_backward<1024, 1>(p, *dev, sm);
    if (r != PURO_OK) return r;
    if (col) {
      const puro::QuantParams qp = quant_params(out, rows, cols, p.ctr);
      r = out.q ? launch_quant<true, true, false>(p.out.bf, cols, qp, *dev, sm)
                : launch_quant<false, true, false>(p.out.bf, cols, qp, *dev, sm);
      if (r != PURO_OK) return r;
    }
  }
  puro::NormColumnParams c{};
  c.part = reinterpret_cast<const float*>(static_cast<char*>(workspace) + kNormCounterBytes);
  c.parts = rows ? norm_backward_parts(rows, cols) : 0;
  c.cols = (int32_t)cols;
  c.w_post = p.w_post;
  c.gate = channel ? gate : nullptr;
  c.w_f32 = w_f32;
  c.gate_f32 = gate_f32;
  c.scale = scale;
  c.accumulate = accumulate;
  c.early = rows > 0 && h && (layout & PURO_COLWISE) && layout != PURO_BF16;
  c.dw_pre = dw_pre;
  c.dw_post = p.w_post ? dw_post : nullptr;
  c.dgate = channel ? static_cast<float*>(dgate) : nullptr;
  return launch_chained(puro::norm_column_kernel, c, dim3((unsigned)(cols / 32), c.dw_post || c.dgate ? 2 : 1), 512, 0,
                        sm);
}

int puro_fp8_swiglu(const void* gu, int64_t ld_gu, int64_t rows, int64_t f, int layout, void* q, int64_t ld_q,
                    void* s, void* qt, int64_t ld_qt, void* st, void* a, int64_t ld_a, void* stream) {
  return gated<false>(nullptr, 0, gu, ld_gu, rows, f, layout, q, ld_q, s, qt, ld_qt, st, a, ld_a, stream);
}

int puro_fp8_swiglu_backward(const void* da, int64_t ld_da, const void* gu, int64_t ld_gu, int64_t rows, int64_t f,
                             int layout, void* q, int64_t ld_q, void* s, void* qt, int64_t ld_qt, void* st,
                             void* dgu, int64_t ld_dgu, void* stream) {
  return gated<true>(da, ld_da, gu, ld_gu, rows, f, layout, q, ld_q, s, qt, ld_qt, st, dgu, ld_dgu, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- orthogonalisation

namespace {

constexpr int kOrthoMaxSteps = 64;
constexpr int64_t kOrthoMaxDim = 65536;

// How the three products of a step are cut into units for 74 CTA pairs (see
// ortho.cuh): the tile width, and for the tiles beyond the last full round of
// pairs a split along k, that together should take the least time.  In cycles,
// measured on a B200: a 64-deep block of a tile, by its width; 32 columns of an
// epilogue, which two sets of warps share; a split tile's hand-over, and writing
// and reading 32 columns of partials.  (200 x 333: 74 us against 118 with 256
// columns throughout, 512 x 512: 97 against 146, 2048 x 2048: 219 against 239,
// and 327 with 64 throughout; without splits 900 x 900 takes 142 against 133.)
constexpr int64_t kOrthoPairs = kSms / 2;
constexpr int64_t kOrthoBlockCycles[3] = {510, 380, 280};  // 256, 128, 64 columns
constexpr int64_t kOrthoChunkCycles = 1500;
constexpr int64_t kOrthoSplitCycles = 2500, kOrthoWriteCycles = 300, kOrthoReadCycles = 350;
constexpr int64_t kOrthoLeast = 4;  // blocks that a part keeps
constexpr int64_t kOrthoClusterPairs = 8;      // CTA pairs of the largest cluster
constexpr int64_t kOrthoGridBarrier = 600;    // what the grid's barrier takes more than a cluster's
static_assert(kOrthoPairs <= puro::kSplitTiles, "counters for every split tile");

struct OrthoPlan {
  puro::OrthoShape shape[3];
  int64_t pairs;        // CTA pairs of the launch
  int64_t cost;         // estimated cycles of a step
  int64_t split_units;  // most units of split tiles in one product
  bool one_cluster;     // the pairs are one cluster
};

// The plan for at most `pairs` CTA pairs.
OrthoPlan ortho_plan_for(int64_t n, int64_t k, int64_t pairs) {
  OrthoPlan plan{};
  const int64_t m = n < k ? n : k, w = n < k ? k : n;
  const int64_t rows[3] = {m, m, n}, cols[3] = {m, m, k}, sums[3] = {w, m, m};
  for (int i = 0; i < 3; ++i) {
    puro::OrthoShape& s = plan.shape[i];
    s.rows_a = (int32_t)rows[i];
    s.rows_b = (int32_t)cols[i];
    s.kblocks = (int32_t)((sums[i] + 63) / 64);
    s.passes = i == puro::kOrthoGram && w <= puro::kOrthoExactK ? 3 : i == puro::kOrthoUpdate && m <= puro::kOrthoFewRows ? 2 : 1;
    const int64_t tm = (rows[i] + 255) / 256, total = (int64_t)s.kblocks * s.passes;
    int64_t best = INT64_MAX;
    for (int j = 0; j < 3; ++j) {
      const int64_t bn = 256 >> j, tn = (cols[i] + bn - 1) / bn, block = kOrthoBlockCycles[j];
      int64_t tiles = tm * tn;
      if (i != puro::kOrthoUpdate) {
        tiles = 0;
        for (int64_t t = 0; t < tm; ++t) tiles += std::min(tn, (t + 1) * (256 / bn));
      }
      const int64_t chunks = std::min(bn, (cols[i] + 31) / 32 * 32) / 32;
      for (int64_t split = 1; split <= puro::kOrthoMaxSplit; ++split) {
        const int64_t rest = tiles % pairs;
        if (split > 1 && (rest == 0 || rest * split > pairs || total / split < kOrthoLeast)) break;
        const int64_t rounds = split > 1 ? tiles / pairs : (tiles + pairs - 1) / pairs;
        int64_t cost = rounds * total * block;
        const int64_t own = (chunks + split - 1) / split;  // chunks that a part of the last tile finishes
        if (split > 1)
          cost += (total + split - 1) / split * block + kOrthoSplitCycles + (chunks - own) * kOrthoWriteCycles +
                  own * (split - 1) * kOrthoReadCycles;
        cost += (own + 1) / 2 * kOrthoChunkCycles;
        if (cost >= best) continue;
        best = cost;
        s.bn = (int32_t)bn;
        s.tiles_m = (int32_t)tm;
        s.tiles_n = (int32_t)tn;
        s.split = (int32_t)split;
        s.full = (int32_t)(split > 1 ? tiles - rest : tiles);
        s.units = (int32_t)(split > 1 ? s.full + rest * split : tiles);
      }
    }
    if (s.split > 1) plan.split_units = std::max<int64_t>(plan.split_units, s.units - s.full);
    plan.pairs = std::max(plan.pairs, std::min<int64_t>(s.units, pairs));
    plan.cost += best;
  }
  return plan;
}

// On the whole device, or, where that is estimated to be faster, in one cluster
// (plan.pairs is then the cluster's, a power of two).
// (200 x 333: 74 us in one cluster, 82 on the device; 512 x 512: 109 and 97.)
OrthoPlan ortho_plan(int64_t n, int64_t k) {
  const OrthoPlan device = ortho_plan_for(n, k, kOrthoPairs);
  OrthoPlan cluster = ortho_plan_for(n, k, kOrthoClusterPairs);
  if (cluster.cost > device.cost + 3 * kOrthoGridBarrier) return device;
  int64_t pairs = 1;
  while (pairs < cluster.pairs) pairs *= 2;
  cluster.pairs = pairs;
  cluster.one_cluster = true;
  return cluster;
}

// Where the workspace of an n x k problem keeps its matrices, in bytes, each
// from a multiple of 256 on.  Rows start on multiples of 128 bytes: the 128-byte
// rows that TMA reads would else each touch two lines of L2 (900 x 900: 133 us
// against 155).
struct OrthoLayout {
  int64_t ld_x, ld_m;
  int64_t x[2][2], o, r, diag, diag_r, part, counters, partial;
  int64_t bytes;
};

OrthoLayout ortho_layout(int64_t n, int64_t k, const OrthoPlan& plan) {
  OrthoLayout l{};
  const int64_t m = n < k ? n : k;
  l.ld_x = (k + 63) / 64 * 64;
  l.ld_m = (m + 63) / 64 * 64;
  auto take = [&](int64_t bytes) {
    const int64_t at = l.bytes;
    l.bytes += (bytes + 255) / 256 * 256;
    return at;
  };
  for (int i = 0; i < 2; ++i)
    for (int t = 0; t < 2; ++t) l.x[i][t] = take(n * l.ld_x * 2);
  l.o = take(m * l.ld_m * 2);
  l.r = take(m * l.ld_m * 2);
  l.diag = take(m * 4);
  l.diag_r = take(m * 4);
  l.part = take(puro::kOrthoNormBlocks * 4);
  l.counters = take(puro::kOrthoCounters * 4);
  l.partial = take(plan.split_units * puro::kPartial * 16);
  return l;
}

// Whether the FP16 form holds the iteration with these coefficients: from
// singular values in [0, 1], X stays below 2, so that |M| <= 4, and |R| <= 15.
// A step maps the values in [0, h] onto just [0, max |x p(x)|], and the maximum is
// at h or where the quintic's slope a + 3 b q + 5 c q^2 (q = x^2) is zero.  (Points
// of a grid don't do: a chaotic quintic takes the values between them elsewhere.)
// 2^-9 a step is left for the roundings.
bool ortho_in_range(int steps, double a, double b, double c) {
  double h = 1.;
  for (int s = 0; s < steps; ++s) {
    h *= 1. + 0x1p-9;
    const double q_h = h * h, d = 9. * b * b - 20. * c * a;
    double top = 0., r_top = 0.;
    auto visit = [&](double q) {  // (a NaN is no place in the interval)
      if (!(q >= 0. && q <= q_h)) return;
      const double r = q * (b + c * q);
      top = std::max(top, std::fabs(std::sqrt(q) * (a + r)));
      r_top = std::max(r_top, std::fabs(r));
    };
    visit(q_h);
    visit(-b / (2. * c));  // the extreme of r
    visit(-a / (3. * b));  // a slope without its quadratic term
    if (d >= 0.) {
      // the two roots without cancellation: one from the sum of like signs, the other from their product
      const double t = -(3. * b + std::copysign(std::sqrt(d), b));
      visit(t / (10. * c));
      visit(2. * a / t);
    }
    if (!(top < 2. && r_top < 15.)) return false;
    h = top;
  }
  return true;
}

template <bool TALL>
int launch_ortho(const puro::OrthoMaps& m, const puro::OrthoParams& p, int64_t pairs, const DeviceInfo& dev,
                 cudaStream_t stream) {
  using C = puro::OrthoCfg;
  auto kern = puro::ortho_kernel<TALL>;
  static std::atomic<bool> done[kMaxDevices] = {};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * (unsigned)kOrthoPairs);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!done[dev.index].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      cudaGetLastError();
      return PURO_ERR_CUDA;
    }
    done[dev.index].store(true, std::memory_order_release);
  }
  // (asked for every launch: a context may have only some of the device's SMs)
  int resident = 0;
  if (cudaOccupancyMaxActiveClusters(&resident, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return PURO_ERR_CUDA;
  }
  if (resident < pairs) return PURO_ERR_UNSUPPORTED_DEVICE;
  cfg.gridDim = dim3(2 * (unsigned)pairs);
  cfg.numAttrs = 2;
  if (p.one_cluster) {
    attr[0].val.clusterDim.x = 2 * (unsigned)pairs;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
  } else {
    attr[1].id = cudaLaunchAttributeCooperative;  // its CTAs wait for one another
    attr[1].val.cooperative = 1;
  }
  if (cudaLaunchKernelEx(&cfg, kern, m, p) != cudaSuccess) {
    cudaGetLastError();
    return PURO_ERR_CUDA;
  }
  return PURO_OK;
}

// One cluster's shared memory and registers hold it: up to 128 on a side.
// (128 x 128: 33 us against 54 by the general kernel, 100 x 1800: 59 against 84.)
bool ortho_small(int64_t n, int64_t k) {
  return std::min(n, k) <= puro::kSmallSide && std::max(n, k) <= puro::kSmallSlice * puro::kSmallMaxCluster;
}

int launch_ortho_small(const puro::OrthoSmallParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  auto kern = puro::ortho_small_kernel;
  constexpr int smem = (int)puro::OrthoSmallCfg::kSmemBytes;
  static std::atomic<bool> done[kMaxDevices] = {};
  if (!done[dev.index].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return PURO_ERR_CUDA;
    done[dev.index].store(true, std::memory_order_release);
  }
  unsigned cluster = 1;
  while (cluster * puro::kSmallSlice < (unsigned)p.w) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(puro::kSmallThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return PURO_ERR_CUDA;
  }
  return PURO_OK;
}

template <bool F32, bool VEC>
int launch_ortho_split(const puro::OrthoSplitParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t pieces = (int64_t)p.n * ((p.k + 7) / 8);
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(puro::kOrthoNormBlocks, (pieces + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, puro::ortho_norm_kernel<F32, VEC>, p) != cudaSuccess ||
      cudaLaunchKernelEx(&cfg, puro::ortho_split_kernel<F32, VEC>, p) != cudaSuccess) {
    cudaGetLastError();
    return PURO_ERR_CUDA;
  }
  return PURO_OK;
}

}  // namespace

extern "C" int64_t puro_fp8_orthogonalize_workspace_bytes(int64_t n, int64_t k) {
  if (n <= 0 || k <= 0 || n > kOrthoMaxDim || k > kOrthoMaxDim) return 0;
  return ortho_small(n, k) ? 256 : ortho_layout(n, k, ortho_plan(n, k)).bytes;
}

extern "C" int puro_fp8_orthogonalize(const void* g, int64_t ld_g, int g_f32, int64_t n, int64_t k, int steps,
                                      float a, float b, float c, float eps, void* out, int64_t ld_out,
                                      void* workspace, void* stream) {
  if (g_f32 & ~1) return PURO_ERR_LAYOUT;
  if (n < 0 || k < 0 || n > kOrthoMaxDim || k > kOrthoMaxDim || steps < 1 || steps > kOrthoMaxSteps || !(eps >= 0.f))
    return PURO_ERR_SHAPE;
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !ortho_in_range(steps, a, b, c)) return PURO_ERR_SHAPE;
  if (n == 0 || k == 0) return PURO_OK;
  if (!g || !out || !workspace) return PURO_ERR_NULL;
  if (!aligned_to(g, g_f32 ? 4 : 2) || !aligned_to(out, 2) || !aligned_to(workspace, 256)) return PURO_ERR_ALIGN;
  if (ld_g < k || ld_out < k) return PURO_ERR_SHAPE;
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != PURO_OK) return st;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  if (ortho_small(n, k)) {
    puro::OrthoSmallParams p{};
    p.g = g;
    p.ld_g = ld_g;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ld_out = ld_out;
    p.tall = n > k;
    p.m = (int32_t)std::min(n, k);
    p.w = (int32_t)std::max(n, k);
    p.g_f32 = g_f32;
    p.vec_g = aligned_to(g, g_f32 ? 16 : 8) && ld_g % 4 == 0;
    p.vec_out = aligned16(out) && ld_out % 8 == 0;
    p.steps = steps;
    p.a = a;
    p.b = b;
    p.c = c;
    p.eps = eps;
    return launch_ortho_small(p, *dev, sm);
  }
  if ((st = get_encoder()) != PURO_OK) return st;

  const OrthoPlan plan = ortho_plan(n, k);
  const OrthoLayout l = ortho_layout(n, k, plan);
  const bool tall = n > k;
  const int64_t m = tall ? k : n;
  char* ws = static_cast<char*>(workspace);
  auto at = [&](int64_t offset) { return static_cast<void*>(ws + offset); };

  // X as an operand whose sum runs along a row (K-major) or down a column
  // (MN-major), and everything as the epilogue reads and writes it
  puro::OrthoMaps maps;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B, sw_e = CU_TENSOR_MAP_SWIZZLE_64B;
  auto half = [&](int product) { return (uint32_t)plan.shape[product].bn / 2; };
  for (int i = 0; i < 2; ++i) {
    for (int t = 0; t < 2; ++t) {
      if ((st = make_map_16(&maps.gram[i][t], at(l.x[i][t]), k, n, l.ld_x, 64, tall ? 64 : 128, sw)) != PURO_OK ||
          (st = make_map_16(&maps.update[i][t], at(l.x[i][t]), k, n, l.ld_x, 64, tall ? 128 : 64, sw)) != PURO_OK ||
          (st = make_map_16(&maps.gram_b[i][t], at(l.x[i][t]), k, n, l.ld_x, 64, tall ? 64 : half(0), sw)) != PURO_OK ||
          (st = make_map_16(&maps.ex[i][t], at(l.x[i][t]), k, n, l.ld_x, 32, 32, sw_e)) != PURO_OK)
        return st;
    }
  }
  if ((st = make_map_16(&maps.o, at(l.o), m, m, l.ld_m, 64, 128, sw)) != PURO_OK ||
      (st = make_map_16(&maps.o_b, at(l.o), m, m, l.ld_m, 64, half(1), sw)) != PURO_OK ||
      (st = make_map_16(&maps.r, at(l.r), m, m, l.ld_m, 64, tall ? half(2) : 128, sw)) != PURO_OK ||
      (st = make_map_16(&maps.eo, at(l.o), m, m, l.ld_m, 32, 32, sw_e)) != PURO_OK ||
      (st = make_map_16(&maps.er, at(l.r), m, m, l.ld_m, 32, 32, sw_e)) != PURO_OK)
    return st;
  const bool out_tma = aligned16(out) && ld_out % 8 == 0;
  maps.out = maps.er;  // not used when the result leaves by plain stores
  if (out_tma && (st = make_map_16(&maps.out, out, k, n, ld_out, 32, 32, sw_e)) != PURO_OK) return st;

  puro::OrthoParams p{};
  for (int i = 0; i < 3; ++i) p.shape[i] = plan.shape[i];
  p.steps = steps;
  p.a = a;
  p.b = b;
  p.c = c;
  p.diag = static_cast<float*>(at(l.diag));
  p.diag_r = static_cast<float*>(at(l.diag_r));
  p.grid_count = static_cast<uint32_t*>(at(l.counters));
  p.tile_count = p.grid_count + 64;
  p.partial = static_cast<float4*>(at(l.partial));
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ld_out = ld_out;
  p.out_tma = out_tma;
  p.one_cluster = plan.one_cluster;

  const bool vec = aligned16(g) && ld_g % (g_f32 ? 4 : 8) == 0;
  const puro::OrthoSplitParams sp{g, ld_g, l.ld_x, (int32_t)n, (int32_t)k, eps, static_cast<__half*>(at(l.x[0][0])),
                                  static_cast<__half*>(at(l.x[0][1])), static_cast<float*>(at(l.part)), p.grid_count};
  if (g_f32)
    st = vec ? launch_ortho_split<true, true>(sp, sm) : launch_ortho_split<true, false>(sp, sm);
  else
    st = vec ? launch_ortho_split<false, true>(sp, sm) : launch_ortho_split<false, false>(sp, sm);
  if (st != PURO_OK) return st;
  return tall ? launch_ortho<true>(maps, p, plan.pairs, *dev, sm) : launch_ortho<false>(maps, p, plan.pairs, *dev, sm);
}
