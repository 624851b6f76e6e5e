// Dense matrix products of bf16 rows with bias, activation and residual in the
// epilogue.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_block.h"
#include "moe_device.cuh"

namespace moe {

// SiLU with e = exp(-|v|) <= 1: nothing overflows.
__device__ __forceinline__ float dense_silu(float v) {
  const float e = expf(-fabsf(v));
  return (v < 0.f ? v * e : v) / (1.f + e);
}

__device__ __forceinline__ float dense_act(int act, float v) {
  switch (act) {
    case MOE_ACT_RELU: return v > 0.f ? v : v != v ? v : 0.f;
    case MOE_ACT_SILU: return dense_silu(v);
    case MOE_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH:
      return 0.5f * v * (1.f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
    default: return v;
  }
}

struct DenseParams {
  const uint16_t* x;         // [R, K]
  const uint16_t* w;         // [N, K]
  const uint16_t* bias;      // or null
  const uint16_t* residual;  // or null
  void* out;                 // [R, M]
  int R, N, K, M, act, out_float;
};

// The plain form: tiles of 64 x 64 outputs, FP32 FMAs from shared memory.
__global__ void __launch_bounds__(256) moe_dense_simple(const DenseParams p) {
  __shared__ float xs[16][65], ws[2][16][65];
  const int silu_mul = p.act == MOE_ACT_SILU_MUL;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int m0 = blockIdx.x * 64, r0 = blockIdx.y * 64;
  float acc[2][4][4] = {};
  pdl_wait();
  for (int k0 = 0; k0 < p.K; k0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int k = i & 15, r = i >> 4;
      const bool in = k0 + k < p.K;
      auto get = [&](const uint16_t* a, int row, int rows) {
        return in && row < rows ? __uint_as_float((uint32_t)a[(size_t)row * p.K + k0 + k] << 16) : 0.f;
      };
      xs[k][r] = get(p.x, r0 + r, p.R);
      ws[0][k][r] = get(p.w, m0 + r, p.M);
      if (silu_mul) ws[1][k][r] = m0 + r < p.M ? get(p.w, p.M + m0 + r, p.N) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
      for (int h = 0; h <= silu_mul; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[h][i][j] = fmaf(xs[k][ty + 16 * i], ws[h][k][tx + 16 * j], acc[h][i][j]);
    __syncthreads();
  }
  auto bf16 = [](uint16_t v) { return __uint_as_float((uint32_t)v << 16); };
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + ty + 16 * i, m = m0 + tx + 16 * j;
      if (r >= p.R || m >= p.M) continue;
      float v = acc[0][i][j] + (p.bias ? bf16(p.bias[m]) : 0.f);
      if (silu_mul) {
        const float up = acc[1][i][j] + (p.bias ? bf16(p.bias[p.M + m]) : 0.f);
        v = dense_silu(v) * up;
      } else {
        v = dense_act(p.act, v);
      }
      const size_t at = (size_t)r * p.M + m;
      if (p.residual) v += bf16(p.residual[at]);
      if (p.out_float)
        static_cast<float*>(p.out)[at] = v;
      else
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rn(v);
    }
}

}  // namespace moe
