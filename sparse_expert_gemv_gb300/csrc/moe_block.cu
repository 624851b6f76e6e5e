// Host side of the C ABI declared in include/moe_block.h: argument checks,
// launch shapes and the dense product's handle.
#include "moe_block.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <new>

#include "moe_block_rows.cuh"
#include "moe_dense.cuh"
#include "moe_host.cuh"

struct moe_dense : moe::Handle {
  moe_dense_config_t cfg;
  const uint16_t* weight;
  const uint16_t* bias;
};

namespace {

using moe::aligned;
using moe::launch;

// ---- routing -----------------------------------------------------------------

template <int R>
moe_status_t route_launch(const moe::RouteParams& p, void* stream) {
  const size_t smem = p.groups > 1 ? (size_t)moe::kRouteWarps * p.E * sizeof(double) : 0;
  return launch(moe::moe_route_experts_rows<R>, (p.T + moe::kRouteWarps - 1) / moe::kRouteWarps,
                moe::kRouteWarps * 32, smem, stream, 1, p);
}

// ---- norms -------------------------------------------------------------------

template <int V>
moe_status_t norm_pair_launch(const moe::NormPairParams& p, int T, void* stream) {
  const int nv = p.H / V;
  const bool two = nv > 512 || (nv > 128 && T >= 2048);
  const int threads = nv > 1024 ? 1024 : ((two ? (nv + 1) / 2 : nv) + 31) / 32 * 32;
  const int per = (nv + threads - 1) / threads;
  if (per <= 1) return launch(moe::moe_norm_add_norm_rows<V, 1>, T, threads, 0, stream, 1, p);
  static_assert(moe::kNormMaxH <= 2 * 1024 * 8, "at most two vectors of eight a thread");
  if (V > 1 || per <= 2)
    return launch(moe::moe_norm_add_norm_rows<V, 2>, T, threads, 0, stream, 1, p);
  if (per <= 4) return launch(moe::moe_norm_add_norm_rows<1, 4>, T, threads, 0, stream, 1, p);
  return launch(moe::moe_norm_add_norm_rows<1, 16>, T, threads, 0, stream, 1, p);
}

void free_dense(moe_dense* m) {
  m->release();
  delete m;
}

}  // namespace

extern "C" {

moe_status_t moe_route_experts(const moe_route_config_t* cfg, int32_t T, const void* logits,
                               const float* bias, int32_t* ids, float* w, void* stream) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  const moe_route_config_t c = *cfg;
  constexpr uint32_t known =
      MOE_ROUTE_BF16 | MOE_ROUTE_SIGMOID | MOE_ROUTE_GROUP_TOP2 | MOE_ROUTE_RENORMALIZE;
  if (T < 0 || c.E < 1 || c.k < 1 || c.groups < 1 || c.top_groups < 1 ||
      c.top_groups > c.groups || !std::isfinite(c.scale) || (c.flags & ~known))
    return MOE_ERR_INVALID_ARG;
  if (c.E > moe::kRouteMaxE || c.k > 32 || c.groups > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c.E % c.groups || c.k > c.top_groups * (c.E / c.groups)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !w) return MOE_ERR_INVALID_ARG;
  const bool bf16 = (c.flags & MOE_ROUTE_BF16) != 0;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(w, 4))
    return MOE_ERR_MISALIGNED;
  moe::RouteParams p;
  p.logits = logits;
  p.bias = bias;
  p.ids = ids;
  p.w = w;
  p.T = T;
  p.E = c.E;
  p.k = c.k;
  // every group kept: the groups decide nothing
  p.groups = c.top_groups == c.groups ? 1 : c.groups;
  p.per = c.E / p.groups;
  p.top_groups = c.top_groups;
  p.scale = c.scale;
  p.bf16 = bf16;
  p.sigmoid = (c.flags & MOE_ROUTE_SIGMOID) != 0;
  p.top2 = (c.flags & MOE_ROUTE_GROUP_TOP2) != 0;
  p.renormalize = (c.flags & MOE_ROUTE_RENORMALIZE) != 0;
  if (c.E <= 64) return route_launch<2>(p, stream);
  if (c.E <= 128) return route_launch<4>(p, stream);
  if (c.E <= 256) return route_launch<8>(p, stream);
  return route_launch<32>(p, stream);
}

moe_status_t moe_norm_add_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual,
                               const uint16_t* post_weight, const uint16_t* pre_weight,
                               const uint16_t* gate, float scale, float residual_scale, float eps,
                               uint32_t flags, uint16_t* sum, uint16_t* y, uint8_t* codes,
                               uint8_t* scales, void* stream) {
  constexpr uint32_t shape = MOE_NORM_GATE_ROW | MOE_NORM_GATE_FULL;
  constexpr uint32_t func = MOE_NORM_GATE_SIGMOID | MOE_NORM_GATE_TANH;
  if (T < 0 || H < 1 || !(eps >= 0.f) || !std::isfinite(scale) || !std::isfinite(residual_scale) ||
      (flags & ~(shape | func | MOE_NORM_UNIT_OFFSET)) || (flags & shape) == shape ||
      (flags & func) == func || ((flags & (shape | func)) && !gate && T > 0))
    return MOE_ERR_INVALID_ARG;
  if (H > moe::kNormMaxH || (codes && H % 32)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!x || !residual || !sum || (pre_weight == nullptr) != (!y && !codes) ||
      (codes == nullptr) != (scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  for (const uint16_t* a : {x, residual, post_weight, pre_weight, gate,
                            const_cast<const uint16_t*>(sum), const_cast<const uint16_t*>(y)})
    if (!aligned(a, 2)) return MOE_ERR_MISALIGNED;
  moe::NormPairParams p;
  p.x = x;
  p.residual = residual;
  p.post = post_weight;
  p.pre = pre_weight;
  p.gate = gate;
  p.sum = sum;
  p.y = y;
  p.codes = codes;
  p.scales = scales;
  p.H = H;
  p.scale = scale;
  p.residual_scale = residual_scale;
  p.eps = eps;
  p.offset = flags & MOE_NORM_UNIT_OFFSET ? 1.f : 0.f;
  p.gate_row = (flags & MOE_NORM_GATE_ROW) != 0;
  p.gate_full = (flags & MOE_NORM_GATE_FULL) != 0;
  p.gate_sigmoid = (flags & MOE_NORM_GATE_SIGMOID) != 0;
  p.gate_tanh = (flags & MOE_NORM_GATE_TANH) != 0;
  bool vec = H % 8 == 0 && aligned(codes, 8) && (p.gate_row || aligned(gate, 16));
  for (const uint16_t* a : {x, residual, post_weight, pre_weight, const_cast<const uint16_t*>(sum),
                            const_cast<const uint16_t*>(y)})
    vec = vec && aligned(a, 16);
  return vec ? norm_pair_launch<8>(p, T, stream) : norm_pair_launch<1>(p, T, stream);
}

moe_status_t moe_dense_create(const moe_dense_config_t* cfg, const uint16_t* weight,
                              const uint16_t* bias, moe_dense_t* out) {
  if (out) *out = nullptr;
  if (!cfg || !out || !weight) return MOE_ERR_INVALID_ARG;
  const moe_dense_config_t c = *cfg;
  if (c.N < 1 || c.K < 1 || c.activation < MOE_ACT_NONE || c.activation > MOE_ACT_SILU_MUL)
    return MOE_ERR_INVALID_ARG;
  if (c.K % 8 || (c.activation == MOE_ACT_SILU_MUL && c.N % 2)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(weight, 16) || !aligned(bias, 2)) return MOE_ERR_MISALIGNED;
  moe_dense* m = new (std::nothrow) moe_dense();
  if (!m) return MOE_ERR_CUDA;
  m->cfg = c;
  m->weight = weight;
  m->bias = bias;
  const bool ok = cudaGetDevice(&m->device) == cudaSuccess && m->acquire(nullptr) &&
                  cudaStreamSynchronize(nullptr) == cudaSuccess;
  if (!ok) {
    (void)cudaGetLastError();
    free_dense(m);
    return MOE_ERR_CUDA;
  }
  *out = m;
  return MOE_OK;
}

moe_status_t moe_dense_destroy(moe_dense_t m) {
  if (m) free_dense(m);
  return MOE_OK;
}

moe_status_t moe_dense_run(moe_dense_t m, int32_t R, const uint16_t* x, const uint16_t* residual,
                           void* out, int32_t out_float, void* stream) {
  if (!m || R < 0) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!x || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 2) || !aligned(out, out_float ? 4 : 2))
    return MOE_ERR_MISALIGNED;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return MOE_ERR_CUDA;
  if (device != m->device) return MOE_ERR_INVALID_ARG;
  const moe_dense_config_t& c = m->cfg;
  moe::DenseParams p;
  p.x = x;
  p.w = m->weight;
  p.bias = m->bias;
  p.residual = residual;
  p.out = out;
  p.R = R;
  p.N = c.N;
  p.K = c.K;
  p.M = c.activation == MOE_ACT_SILU_MUL ? c.N / 2 : c.N;
  p.act = c.activation;
  p.out_float = out_float != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  moe::moe_dense_simple<<<dim3((p.M + 63) / 64, (R + 63) / 64), 256, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  m->mark_done(s);
  return MOE_OK;
}

moe_status_t moe_dense_get_error(moe_dense_t m, void* stream, uint32_t* device_flags) {
  if (device_flags) *device_flags = 0;
  if (!m || !device_flags) return MOE_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return MOE_ERR_CUDA;
  return m->read_error(device_flags);
}

}  // extern "C"
