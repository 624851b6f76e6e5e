// The row operators between routed experts: the router's choice and the norms
// around a block's end.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_device.cuh"
#include "moe_prompt_rows.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// moe_route_experts_rows: one warp a token.
// ---------------------------------------------------------------------------
struct RouteParams {
  const void* logits;
  const float* bias;   // or null
  int32_t* ids;
  float* w;
  int T, E, k, groups, per, top_groups;   // per: experts of a group
  float scale;
  int bf16, sigmoid, top2, renormalize;
};

constexpr int kRouteWarps = 4;
constexpr int kRouteMaxE = 1024;

__device__ __forceinline__ float route_off() { return -__int_as_float(0x7f800000); }

__device__ __forceinline__ float route_logit(const RouteParams& p, size_t at) {
  const float l = p.bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.logits)[at] << 16)
                         : static_cast<const float*>(p.logits)[at];
  return l > route_off() ? l : route_off();   // NaN too
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

template <int R>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_experts_rows(const RouteParams p) {
  extern __shared__ double route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRouteWarps + warp;
  pdl_wait();
  if (t >= p.T) return;
  const double off = route_off();
  float l[R], mx = route_off();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int e = lane + 32 * r;
    l[r] = e < p.E ? route_logit(p, (size_t)t * p.E + e) : route_off();
    mx = fmaxf(mx, l[r]);
  }
  mx = warp_max(mx);
  const bool infinite = mx == -route_off();
  // scores, and what experts are compared by
  double s[R], key[R], z = 0.0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (p.sigmoid) {
      s[r] = 1.0 / (1.0 + exp(-(double)l[r]));
    } else {
      s[r] = infinite ? (l[r] == mx ? 1.0 : 0.0) : l[r] > route_off() ? exp((double)l[r] - mx) : 0.0;
      z += s[r];
    }
  }
  if (!p.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] /= z;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int e = lane + 32 * r;
    key[r] = l[r];
    if (p.bias && e < p.E) {
      key[r] = s[r] + (double)p.bias[e];
      if (!(key[r] > off) || !(l[r] > route_off())) key[r] = off;
    }
  }
  if (p.groups > 1) {
    double* sm = route_smem + (size_t)warp * p.E;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = lane + 32 * r;
      if (e < p.E) sm[e] = p.top2 && key[r] > off ? (p.bias ? key[r] : s[r]) : key[r];
    }
    __syncwarp();
    double score = off;
    if (lane < p.groups) {
      double m1 = off, m2 = off;
      for (int i = 0; i < p.per; ++i) {
        const double v = sm[lane * p.per + i];
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
      score = p.top2 && m2 > off ? m1 + m2 : m1;
    }
    int rank = 0;
    for (int j = 0; j < p.groups; ++j) {
      const double other = __shfl_sync(kFull, score, j);
      rank += other > score || (other == score && j < lane);
    }
    const unsigned kept = __ballot_sync(kFull, lane < p.groups && rank < p.top_groups);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = lane + 32 * r;
      if (e < p.E && !((kept >> (e / p.per)) & 1u)) key[r] = off;
    }
  }
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    double best = off;
    int at = 0x7fffffff;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (key[r] > best) best = key[r], at = lane + 32 * r;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(kFull, best, o);
      const int oa = __shfl_xor_sync(kFull, at, o);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (at == 0x7fffffff) break;   // none is left
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (lane + 32 * r == at) key[r] = off;
    if (lane == j) mine = at;
  }
  // the chosen experts' weights, in FP32
  const float lm = mine >= 0 ? route_logit(p, (size_t)t * p.E + mine) : route_off();
  float v = 0.f;
  if (p.sigmoid) {
    if (mine >= 0) v = 1.f / (1.f + expf(-lm));
  } else {
    // relative to the largest chosen logit where the sum is that of the chosen
    const float top = p.renormalize ? warp_max(lm) : mx;
    if (mine >= 0) v = top == -route_off() ? (lm == top ? 1.f : 0.f) : expf(lm - top);
    if (!p.renormalize && mine >= 0) v /= (float)z;
  }
  if (p.renormalize) {
    const float sum = warp_sum(v);
    v = sum > 0.f ? v / sum : 0.f;
  }
  if (lane < p.k) {
    p.ids[(size_t)t * p.k + lane] = mine;
    p.w[(size_t)t * p.k + lane] = v * p.scale;
  }
}

// ---------------------------------------------------------------------------
// moe_norm_add_norm_rows: one CTA a row, whose values stay in registers between
// the two reductions and the outputs (NV vectors of V values a thread), so that
// every operand is read once and every output written once. Bound by HBM.
// ---------------------------------------------------------------------------
struct NormPairParams {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* post;   // or null
  const uint16_t* pre;    // or null
  const uint16_t* gate;   // or null
  uint16_t* sum;          // may be x or residual
  uint16_t* y;            // or null
  uint8_t* codes;         // or null (then scales too)
  uint8_t* scales;
  int H;
  float scale, residual_scale, eps;
  float offset;           // added to norm weights
  int gate_row, gate_full, gate_sigmoid, gate_tanh;
};

// Sum of `v` over the CTA, in every thread; `part` is not used before or after
// by another sum without a barrier between.
__device__ __forceinline__ float cta_sum(float v, float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum(v);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return warp_sum(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f);
}

__device__ __forceinline__ float gate_value(const NormPairParams& p, float g) {
  if (p.gate_sigmoid) return 1.f / (1.f + expf(-g));
  if (p.gate_tanh) return tanhf(g);
  return g;
}

template <int V, int NV>
__global__ void __launch_bounds__(1024) moe_norm_add_norm_rows(const NormPairParams p) {
  __shared__ float part[2][32];
  const int H = p.H, nv = H / V;
  const size_t base = (size_t)blockIdx.x * H;
  pdl_wait();
  // every load of the row in flight before the first is used
  typename RowVec<V>::Raw x[NV], res[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nv) x[i] = RowVec<V>::once(p.x + base + (size_t)v * V);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nv) res[i] = RowVec<V>::once(p.residual + base + (size_t)v * V);
  }
  float r = 1.f;
  if (p.post) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * blockDim.x + threadIdx.x < nv) {
        float f[V];
        RowVec<V>::values(x[i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(f[j], f[j], ss);
      }
    r = rsqrtf(cta_sum(ss, part[0]) / (float)H + p.eps);
  }
  float row_gate = p.scale;
  if (p.gate && p.gate_row) {
    float g[1];
    RowVec<1>::load(p.gate + blockIdx.x, g);
    row_gate *= gate_value(p, g[0]);
  }
  float f[NV][V], ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nv) {
      float b[V], g[V];
      RowVec<V>::values(x[i], f[i]);
      if (p.post) {
        float w[V];
        RowVec<V>::load(p.post + (size_t)v * V, w);
#pragma unroll
        for (int j = 0; j < V; ++j) f[i][j] = f[i][j] * r * (w[j] + p.offset);
      }
      if (p.gate && !p.gate_row) {
        RowVec<V>::load(p.gate + (p.gate_full ? base : 0) + (size_t)v * V, g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[i][j] *= gate_value(p, g[j]);
      }
      RowVec<V>::values(res[i], b);
      // the residual stream is kept in bf16, and what is kept is normalised
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float s = fmaf(f[i][j], row_gate, b[j] * p.residual_scale);
        f[i][j] = __uint_as_float((uint32_t)f32_to_bf16_rn(s) << 16);
        ss = fmaf(f[i][j], f[i][j], ss);
      }
      RowVec<V>::store(p.sum + base + (size_t)v * V, f[i]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] = 0.f;
    }
  }
  if (!p.pre) return;
  r = rsqrtf(cta_sum(ss, part[1]) / (float)H + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    float n[V];
    uint32_t amax = 0u;
    if (v < nv) {
      RowVec<V>::load(p.pre + (size_t)v * V, n);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        n[j] = f[i][j] * r * (n[j] + p.offset);
        amax = max(amax, __float_as_uint(n[j]) & 0x7fffffffu);
      }
      if (p.y) RowVec<V>::store(p.y + base + (size_t)v * V, n);
    }
    if (p.codes) {   // H is a multiple of 32: a block's lanes are all in or all out
#pragma unroll
      for (int o = 16 / V; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, o));
      if (v < nv) {
        const uint32_t s = mx_scale_code(amax);
        const float inv = mx_inverse(s);
#pragma unroll
        for (int j = 0; j < V; ++j) n[j] *= inv;
        RowVec<V>::store_codes(p.codes + base + (size_t)v * V, n);
        if (v % (32 / V) == 0) p.scales[(base + (size_t)v * V) / 32] = (uint8_t)s;
      }
    }
  }
}

}  // namespace moe
