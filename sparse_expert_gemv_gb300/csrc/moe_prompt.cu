// Host side of the C ABI declared in include/moe_prompt.h: argument checks,
// launch shapes, tensor maps and the product handle.
#include "moe_prompt.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <new>

#include "moe_host.cuh"
#include "moe_product.cuh"
#include "moe_prompt_rows.cuh"

struct moe_product : moe::Handle {
  moe_product_config_t cfg;
  int num_sms;
  int mt;             // weight tiles of an expert
  CUtensorMap tm_w;
  uint8_t* sfa;       // the weights' scales in tile order
  std::atomic<bool> armed;   // the next run's waits run out (moe_product_arm_timeout)
};

namespace {

using moe::aligned;
using moe::encode;
using moe::launch;

// ---- norm --------------------------------------------------------------------

template <int V>
moe_status_t norm_launch(const moe::NormParams& p, int T, void* stream) {
  const int nv = p.H / V;
  // One vector a thread while few rows are under way, two from 2048 rows or 512
  // vectors on (smaller blocks, more rows an SM), of single values up to 16 on
  // 1024 threads (us with one and with two: 1 row of 2048 1.9 / 2.3, 1024 rows 3.3
  // / 3.5, 4096 rows of 4096 20.1 / 16.7, 16384 of 2048 39.7 / 37.2, MXFP8 rows out).
  const bool two = nv > 512 || (nv > 128 && T >= 2048);
  const int threads = nv > 1024 ? 1024 : ((two ? (nv + 1) / 2 : nv) + 31) / 32 * 32;
  const int per = (nv + threads - 1) / threads;
  if (per <= 1) return launch(moe::moe_add_rms_norm_rows<V, 1>, T, threads, 0, stream, 1, p);
  static_assert(moe::kNormMaxH <= 2 * 1024 * 8, "at most two vectors of eight a thread");
  if (V > 1 || per <= 2)
    return launch(moe::moe_add_rms_norm_rows<V, 2>, T, threads, 0, stream, 1, p);
  if (per <= 4) return launch(moe::moe_add_rms_norm_rows<1, 4>, T, threads, 0, stream, 1, p);
  return launch(moe::moe_add_rms_norm_rows<1, 16>, T, threads, 0, stream, 1, p);
}

// ---- combine -----------------------------------------------------------------

template <int V>
moe_status_t combine_launch(const moe::CombineParams& p, unsigned grid, unsigned threads,
                            void* stream) {
  if (p.k == 1) return launch(moe::moe_combine_rows<V, 1>, grid, threads, 0, stream, 1, p);
  if (p.k == 2) return launch(moe::moe_combine_rows<V, 2>, grid, threads, 0, stream, 1, p);
  if (p.k <= 4) return launch(moe::moe_combine_rows<V, 4>, grid, threads, 0, stream, 1, p);
  return launch(moe::moe_combine_rows<V, moe::kCombineBatch>, grid, threads, 0, stream, 1, p);
}

// ---- group -------------------------------------------------------------------

using GroupKernel = void (*)(const moe::GroupParams);
constexpr GroupKernel kGroupKernels[3] = {moe::moe_group_slots<7>, moe::moe_group_slots<8>,
                                          moe::moe_group_slots<10>};

// The most CTAs a group cluster may have on the current device: 16 where its
// GPCs take such a cluster, else the portable 8; 0 when a CUDA call failed.
// Asked once a device (the attributes it sets stay).
int group_cluster_limit() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kMaxDevices && known[dev].load(std::memory_order_acquire))
    return known[dev].load(std::memory_order_relaxed);
  int limit = 16;
  for (GroupKernel k : kGroupKernels) {
    const size_t smem = moe::group_smem(moe::kGroupThreads / 32, moe::kProdMaxE,
                                        moe::kGroupThreads * moe::kGroupBatch);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(moe::kGroupThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
      return 0;
    int n = 0;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      limit = 8;
    }
  }
  if (dev < kMaxDevices) known[dev].store(limit, std::memory_order_release);
  return limit;
}

// ---- product -----------------------------------------------------------------

bool is_fp4(const moe_product_config_t& c) { return (c.flags & MOE_FLAG_MXFP4) != 0; }
bool is_silu(const moe_product_config_t& c) { return (c.flags & MOE_PRODUCT_SILU_MUL) != 0; }

// The weights as [E][N][K] in boxes of 128 rows, or with SILU_MUL as
// [groups of 16 rows][gate, up][odd][8][K] in boxes of four groups' gate rows
// and the up rows I further on, even neurons before odd ones. There the groups
// of all experts lie in one row, and the last I/16 (up rows whose own up rows
// would lie past the end) are left out: a tile that runs past its expert's
// last neuron reads other rows or zeros, and its surplus is not stored. MXFP4 codes are spread to a byte each on the way (16 codes and 8
// bytes of padding in 16 bytes of shared memory).
bool encode_weights(moe_product* m, const uint8_t* w) {
  const moe_product_config_t& c = m->cfg;
  const CUtensorMapDataType type =
      is_fp4(c) ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const cuuint64_t row = is_fp4(c) ? c.K / 2 : c.K, N = c.N, K = c.K, E = c.E;
  if (is_silu(c)) {
    const cuuint64_t I = N / 2, groups = E * (N / 16) - I / 16;
    const cuuint64_t dims[5] = {K, 8, 2, 2, groups};
    const cuuint64_t strides[4] = {2 * row, row, I * row, 16 * row};
    const cuuint32_t box[5] = {moe::kProdK, 8, 2, 2, 4};
    return encode(&m->tm_w, type, 5, w, dims, strides, box);
  }
  const cuuint64_t dims[3] = {K, N, E};
  const cuuint64_t strides[2] = {row, N * row};
  const cuuint32_t box[3] = {moe::kProdK, moe::kProdRows, 1};
  return encode(&m->tm_w, type, 3, w, dims, strides, box);
}

constexpr size_t kProductSmem = (size_t)moe::ProductSmem::total + 1024;

void free_product(moe_product* m) {
  m->release();
  cudaFree(m->sfa);
  delete m;
}

}  // namespace

extern "C" {

moe_status_t moe_add_rms_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual,
                              const uint16_t* weight, float eps, uint16_t* sum, uint16_t* y,
                              uint8_t* codes, uint8_t* scales, void* stream) {
  if (T < 0 || H < 1 || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (H > moe::kNormMaxH || (codes && H % 32)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!x || !weight || (!y && !codes) || (codes == nullptr) != (scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(sum, 2) ||
      !aligned(y, 2))
    return MOE_ERR_MISALIGNED;
  const moe::NormParams p{x, residual, weight, sum, y, codes, scales, H, eps};
  const bool vec = H % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) &&
                   aligned(sum, 16) && aligned(y, 16) && aligned(codes, 8);
  return vec ? norm_launch<8>(p, T, stream) : norm_launch<1>(p, T, stream);
}

moe_status_t moe_group(int32_t T, int32_t k, int32_t E, const int32_t* topk_ids, int32_t* offsets,
                       int32_t* rows, int32_t* slots, void* stream) {
  if (T < 0 || k < 1 || E < 1) return MOE_ERR_INVALID_ARG;
  if (E > moe::kProdMaxE || (int64_t)T * k > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
    return MOE_ERR_MISALIGNED;
  const int S = T * k;
  if (S == 0) {   // every group is empty
    return cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  if (!topk_ids || !rows || !slots) return MOE_ERR_INVALID_ARG;
  // As many CTAs as keep 512 slots each, so that a warp walks few of them (2048
  // slots of 256 experts: 7.8 us with one CTA, 6.2 with two, 5.0 with four).
  const int limit = group_cluster_limit();
  if (!limit) return MOE_ERR_CUDA;
  int C = 1;
  while (C < limit && S > 512 * C) C *= 2;
  const int warps = std::min(moe::kGroupThreads / 32, (S + 32 * C - 1) / (32 * C));
  const int per = ((S + C * warps - 1) / (C * warps) + 31) / 32 * 32;
  // division by k: 2^(31 + l) / k rounded up, 2^l the power of two at or above
  // k, is off by less than 2^-(l + 31) of a quotient, too little to reach the
  // next whole number for any s <= 2^30
  int l = 0;
  while ((int64_t)1 << l < k) ++l;
  const unsigned inverse = (unsigned)((((uint64_t)1 << (31 + l)) + k - 1) / k);
  // from 2048 slots a CTA on, while a warp's range is one batch (us staged and
  // stored directly, 256 experts: 512 slots a CTA 5.4 / 5.2, 1024 6.5 / 6.4, 2048
  // 7.4 / 7.5, 4096 9.1 / 9.6, 8192 12.6 / 13.8)
  const int staged = per <= 32 * moe::kGroupBatch && warps * per >= 2048 ? warps * per : 0;
  const moe::GroupParams p{topk_ids, offsets, rows, slots, S, E, per, inverse, l, staged};
  return launch(kGroupKernels[E <= 128 ? 0 : E <= 256 ? 1 : 2], C, warps * 32,
                moe::group_smem(warps, E, staged), stream, C, p);
}

moe_status_t moe_combine(int32_t T, int32_t k, int32_t H, int32_t R, const uint16_t* y,
                         const int32_t* slots, const float* w, const uint16_t* residual,
                         uint16_t* out, void* stream) {
  if (T < 0 || k < 1 || H < 1 || R < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if ((!y && R > 0) || !slots || !w || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(y, 2) || !aligned(slots, 4) || !aligned(w, 4) || !aligned(residual, 2) ||
      !aligned(out, 2))
    return MOE_ERR_MISALIGNED;
  const bool vec = H % 8 == 0 && aligned(y, 16) && aligned(residual, 16) && aligned(out, 16);
  const int nv = vec ? H / 8 : H;
  const int nb = (nv + moe::kCombineThreads - 1) / moe::kCombineThreads;
  if ((int64_t)T * nb > 0x7fffffff) return MOE_ERR_UNSUPPORTED_SHAPE;
  const moe::CombineParams p{y, slots, w, residual, out, k, H, R, nb};
  // a token's vectors in equal parts over its CTAs
  const unsigned threads = ((nv + nb - 1) / nb + 31) / 32 * 32;
  return vec ? combine_launch<8>(p, T * nb, threads, stream)
             : combine_launch<1>(p, T * nb, threads, stream);
}

moe_status_t moe_product_create(const moe_product_config_t* cfg, const uint8_t* w,
                                const uint8_t* w_scales, moe_product_t* out, void* stream) {
  if (out) *out = nullptr;
  if (!cfg || !out || !w || !w_scales) return MOE_ERR_INVALID_ARG;
  const moe_product_config_t c = *cfg;
  if (c.E < 1 || c.N < 1 || c.K < 1 || (c.flags & ~(MOE_FLAG_MXFP4 | MOE_PRODUCT_SILU_MUL)))
    return MOE_ERR_INVALID_ARG;
  if (c.E > moe::kProdMaxE || c.N % (is_silu(c) ? 64 : 8) || c.K % (is_fp4(c) ? 128 : 32))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(w, 32)) return MOE_ERR_MISALIGNED;
  moe_product* m = new (std::nothrow) moe_product();
  if (!m) return MOE_ERR_CUDA;
  m->cfg = c;
  m->mt = is_silu(c) ? (c.N / 2 + 63) / 64 : (c.N + moe::kProdRows - 1) / moe::kProdRows;
  const int nk = (c.K + moe::kProdK - 1) / moe::kProdK;
  const int mt2 = (m->mt + 1) / 2 * 2;   // a pair of CTAs takes two tiles
  const int64_t blocks = (int64_t)c.E * mt2 * nk;
  const bool ok =
      blocks <= 0x7fffffff && cudaGetDevice(&m->device) == cudaSuccess &&
      cudaDeviceGetAttribute(&m->num_sms, cudaDevAttrMultiProcessorCount, m->device) ==
          cudaSuccess &&
      cudaMalloc(&m->sfa, (size_t)blocks * moe::kProdSfaBytes) == cudaSuccess &&
      m->acquire(static_cast<cudaStream_t>(stream)) &&
      encode_weights(m, w) &&
      cudaFuncSetAttribute(moe::moe_product_tiles<false>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kProductSmem) == cudaSuccess &&
      cudaFuncSetAttribute(moe::moe_product_tiles<true>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kProductSmem) == cudaSuccess;
  if (ok) {
    moe::moe_product_lay_scales<<<(unsigned)blocks, 128, 0, static_cast<cudaStream_t>(stream)>>>(
        w_scales, m->sfa, c.N, c.K, mt2, is_silu(c));
  }
  // the scales are laid out once this returns: calls may come on any stream
  if (!ok || cudaGetLastError() != cudaSuccess ||
      cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    (void)cudaGetLastError();
    free_product(m);
    return MOE_ERR_CUDA;
  }
  *out = m;
  return MOE_OK;
}

moe_status_t moe_product_destroy(moe_product_t m) {
  if (m) free_product(m);
  return MOE_OK;
}

moe_status_t moe_product_run(moe_product_t m, int32_t R, int32_t A, const uint8_t* a,
                             const uint8_t* a_scales, const int32_t* offsets, const int32_t* rows,
                             uint16_t* y, uint8_t* codes, uint8_t* scales, void* stream) {
  if (!m || R < 0 || A < 0) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  const moe_product_config_t& c = m->cfg;
  const bool silu = is_silu(c);
  if (A < 1 || (!rows && A != R) || !a || !a_scales || !offsets) return MOE_ERR_INVALID_ARG;
  if (silu ? (!codes || !scales || y) : (!y || codes || scales)) return MOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(y, 16) ||
      !aligned(codes, 16))
    return MOE_ERR_MISALIGNED;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return MOE_ERR_CUDA;
  if (device != m->device) return MOE_ERR_INVALID_ARG;
  moe::ProductParams p;
  p.tm_w = m->tm_w;
  if (!rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)c.K, (cuuint64_t)A};
    const cuuint64_t strides[1] = {(cuuint64_t)c.K};
    for (int b = 0; b < 3; ++b) {
      const cuuint32_t box[2] = {moe::kProdK, 16u << b};
      if (!encode(&p.tm_a[b], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a, dims, strides, box))
        return MOE_ERR_CUDA;
    }
  }
  p.a = a;
  p.sfa = m->sfa;
  p.a_scales = a_scales;
  p.offsets = offsets;
  p.rows = rows;
  p.y = y;
  p.codes = codes;
  p.scales = scales;
  p.err = m->d_err;
  p.E = c.E;
  p.N = c.N;
  p.K = c.K;
  p.R = R;
  p.A = A;
  p.mt = m->mt;
  const int ks = c.K / 32;
  p.sf_vec = ks % 16 == 0 && aligned(a_scales, 16) ? 16 : ks % 4 == 0 && aligned(a_scales, 4) ? 4 : 1;
  p.w_bytes = is_fp4(c) ? moe::kProdABytes / 2 : moe::kProdABytes;
  p.a_format = is_fp4(c) ? 5 : 0;
  const bool armed = m->armed.exchange(false, std::memory_order_relaxed);
  p.polls = armed ? 50 : moe::kMbarPolls;   // a millisecond
  p.withheld = armed;
  // one pair of CTAs a pair of SMs, and no more than there can be tiles
  const int64_t most = ((int64_t)std::min(c.E, R) + R / moe::kProdCols) * ((m->mt + 1) / 2);
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(std::max(1, m->num_sms / 2), most);
  const moe_status_t st =
      launch(silu ? moe::moe_product_tiles<true> : moe::moe_product_tiles<false>, grid,
             moe::kProdThreads, kProductSmem, stream, 2, p);
  if (st == MOE_OK) m->mark_done(static_cast<cudaStream_t>(stream));
  return st;
}

moe_status_t moe_product_arm_timeout(moe_product_t m) {
  if (!m) return MOE_ERR_INVALID_ARG;
  m->armed.store(true, std::memory_order_relaxed);
  return MOE_OK;
}

moe_status_t moe_product_get_error_latest(moe_product_t m, uint32_t* device_flags) {
  if (device_flags) *device_flags = 0;
  if (!m || !device_flags) return MOE_ERR_INVALID_ARG;
  return m->read_error(device_flags);
}

moe_status_t moe_product_get_error(moe_product_t m, void* stream, uint32_t* device_flags) {
  if (device_flags) *device_flags = 0;
  if (!m || !device_flags) return MOE_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return MOE_ERR_CUDA;
  return m->read_error(device_flags);
}

}  // extern "C"
