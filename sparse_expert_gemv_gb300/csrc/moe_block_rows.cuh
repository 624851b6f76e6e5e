// The row operators between routed experts: the router's choice and the norms
// around a block's end.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_device.cuh"
#include "moe_prompt_rows.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// moe_route_experts_rows: one warp a token, lane l with the R experts from R l on.
//
// Experts are ordered by 32-bit keys: the bits of the compared value (its
// logit, or in FP32 its score plus bias) made monotone, with the expert's
// place in the lowest bits; 0 is an expert that is off. A lane sorts its keys
// once by a network, and a round of the choice is one warp-wide maximum of the
// lanes' first keys.
//
// The choice has to be that of FP64 arithmetic. bf16 logits leave 16 bits for
// the place, so without a bias their keys are exact and all different. Other
// keys lose the low bits and carry the FP32 score's error: where two values that
// decide something lie closer than that (the next one chosen, the first one
// left out, the last group kept and the first dropped), the experts in question
// are compared again in FP64, one a lane. That is 0.2 % of rows of 256 sigmoid
// scores with a bias. More than 32 in question, as in rows of equal logits,
// take the choice by scans (route_slow).
// ---------------------------------------------------------------------------
struct RouteParams {
  const void* logits;
  const float* bias;   // or null
  int32_t* ids;
  float* w;
  int T, E, k, groups, per, top_groups;   // per: experts of a group
  // log2 of the lanes a group's experts lie in, where that is a whole power of
  // two; else -1
  int lane_shift;
  int packed_shift;   // the same of moe_route_experts_packed's lanes
  float scale;
  int bf16, sigmoid, top2, renormalize;
  int vec;        // a lane's logits are one aligned piece of the row
  int bias_vec;   // and its biases
  int smem;       // bytes a warp has
};

constexpr int kRouteWarps = 4;
constexpr int kRouteMaxE = 1024;

__device__ __forceinline__ float route_off() { return __int_as_float(0xff800000); }

// NaN as -inf
__device__ __forceinline__ float route_clean(float l) { return fmaxf(l, route_off()); }

__device__ __forceinline__ float route_logit(const RouteParams& p, size_t at) {
  return route_clean(p.bf16 ? bf16_lo(static_cast<const uint16_t*>(p.logits)[at])
                            : static_cast<const float*>(p.logits)[at]);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// The choice in FP64, by plain scans: lane j's j-th expert or -1. `key` is the
// warp's, E values.
__device__ __forceinline__ int route_slow(const RouteParams& p, int t, double* key) {
  const int lane = threadIdx.x & 31;
  const size_t row = (size_t)t * p.E;
  const double off = route_off();
  float mx = route_off();
  for (int e = lane; e < p.E; e += 32) mx = fmaxf(mx, route_logit(p, row + e));
  mx = warp_max(mx);
  const bool infinite = mx == -route_off();
  auto raw = [&](float l) {   // a softmax's numerator, or a sigmoid
    if (p.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
    if (infinite) return l == mx ? 1.0 : 0.0;
    return l > route_off() ? exp((double)l - mx) : 0.0;
  };
  double z = 1.0;
  if (!p.sigmoid) {
    z = 0.0;
    for (int e = lane; e < p.E; e += 32) z += raw(route_logit(p, row + e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
  }
  const bool sums = p.groups > 1 && p.top2;
  // what experts compare by; without a bias first the scores where groups add them
  for (int pass = sums && !p.bias ? 0 : 1; pass < 2; ++pass) {
    for (int e = lane; e < p.E; e += 32) {
      const float l = route_logit(p, row + e);
      double v = l;
      if (p.bias || pass == 0) v = l > route_off() ? raw(l) / z + (p.bias ? (double)p.bias[e] : 0.0) : off;
      v = v > off ? v : off;
      // a group dropped in the first pass stays dropped
      key[e] = pass == 1 && sums && !p.bias && key[e] == off ? off : v;
    }
    __syncwarp();
    if (p.groups > 1 && (pass == 0 || !sums || p.bias)) {
      double score = off;
      if (lane < p.groups) {
        double m1 = off, m2 = off;
        for (int i = 0; i < p.per; ++i) {
          const double v = key[lane * p.per + i];
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
      for (int e = lane; e < p.E; e += 32)
        if (!((kept >> (e / p.per)) & 1u)) key[e] = off;
      __syncwarp();
    }
  }
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    double best = off;
    int at = 0x7fffffff;
    for (int e = lane; e < p.E; e += 32)
      if (key[e] > best) best = key[e], at = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(kFull, best, o);
      const int oa = __shfl_xor_sync(kFull, at, o);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (at == 0x7fffffff) break;   // none is left
    if ((at & 31) == lane) key[at] = off;
    __syncwarp();
    if (lane == j) mine = at;
  }
  return mine;
}

// A chosen expert's score but for a factor of the row: the softmax's term relative to
// `top`, or the sigmoid, relative to e^top where that is below 1, so that weights
// keep their digits where all scores are tiny.
__device__ __forceinline__ float route_weight(bool sigmoid, float l, float top) {
  if (sigmoid) return (l < 0.f ? expf(l - fminf(top, 0.f)) : 1.f) / (1.f + expf(-fabsf(l)));
  return top == -route_off() ? (l == top ? 1.f : 0.f) : expf(l - top);
}

// What expert e compares by, in FP64: its score plus bias, or with `plain` its
// logit. -inf where it is off.
__device__ __forceinline__ double route_exact(const RouteParams& p, int t, int e, bool plain, float mx,
                                              double z) {
  const float l = route_logit(p, (size_t)t * p.E + e);
  if (plain || !(l > route_off())) return l;
  double v = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - mx) / z;
  if (p.bias) v += (double)p.bias[e];
  return v > (double)route_off() ? v : (double)route_off();
}

// The sum of a softmax in FP64.
template <int R>
__device__ __forceinline__ double route_sum(const float (&l)[R], float mx) {
  double z = 0.0;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (__any_sync(kFull, l[r] > route_off())) z += l[r] > route_off() ? exp((double)l[r] - mx) : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
  return z;
}

// FP64 values are compared as order-preserving integers: comparisons in FP64 take
// tens of cycles each. (No NaN comes here; -0 as 0.)
__device__ __forceinline__ int64_t route_order(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double route_unorder(int64_t b) {
  return __longlong_as_double(b ^ ((b >> 63) & 0x7fffffffffffffffll));
}
__device__ __forceinline__ int64_t warp_max(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, (int64_t)__shfl_xor_sync(kFull, (long long)v, o));
  return v;
}

// Appends the experts of the lanes with `in` to a warp's list of at most 32 and
// counts them in any case.
__device__ __forceinline__ void route_append(int* list, int& n, bool in, int e) {
  const unsigned all = __ballot_sync(kFull, in);
  const int at = n + __popc(all & ((1u << (threadIdx.x & 31)) - 1u));
  if (in && at < 32) list[at] = e;
  n += __popc(all);
}

// Order-preserving bits of a float, and back.
__device__ __forceinline__ uint32_t route_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
// (`mask`: low bits that hold a place; they read as a bf16's or as cut off)
__device__ __forceinline__ float route_value(uint32_t key, uint32_t mask) {
  return __uint_as_float((int32_t)key < 0 ? (key & ~mask) ^ 0x80000000u : ~(key | mask));
}

// The R logits of a lane, cleaned; -inf past the last expert.
template <int R>
__device__ __forceinline__ void route_load(const RouteParams& p, int t, int lane, float (&l)[R]) {
  const size_t row = (size_t)t * p.E;
  const int e0 = lane * R;
  if (p.vec) {   // all of a lane's or none
    uint32_t w[R];
    if (e0 < p.E) {
      if (p.bf16) {
        constexpr int N = R < 2 ? 1 : R / 2;
        uint32_t h[N];
        const uint16_t* src = static_cast<const uint16_t*>(p.logits) + row + e0;
        if constexpr (R == 1) {
          h[0] = *src;
        } else if constexpr (R == 2) {
          h[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
        } else if constexpr (R == 4) {
          const uint2 a = __ldg(reinterpret_cast<const uint2*>(src));
          h[0] = a.x, h[1] = a.y;
        } else {
#pragma unroll
          for (int i = 0; i < R / 8; ++i) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(src) + i);
            h[4 * i] = a.x, h[4 * i + 1] = a.y, h[4 * i + 2] = a.z, h[4 * i + 3] = a.w;
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = r & 1 ? h[r / 2] & 0xffff0000u : h[r / 2] << 16;
      } else {
        const float* src = static_cast<const float*>(p.logits) + row + e0;
        if constexpr (R == 1) {
          w[0] = __float_as_uint(__ldg(src));
        } else if constexpr (R == 2) {
          const uint2 a = __ldg(reinterpret_cast<const uint2*>(src));
          w[0] = a.x, w[1] = a.y;
        } else {
#pragma unroll
          for (int i = 0; i < R / 4; ++i) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(src) + i);
            w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      l[r] = e0 < p.E ? route_clean(__uint_as_float(w[r])) : route_off();
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) l[r] = e0 + r < p.E ? route_logit(p, row + e0 + r) : route_off();
  }
}

// Keys in descending order by Batcher's odd-even merge sort, in templates so that
// every index is a constant.
template <int R, int LO, int N, int S>
__device__ __forceinline__ void route_merge(uint32_t (&k)[R]) {
  if constexpr (2 * S < N) {
    route_merge<R, LO, N, 2 * S>(k);
    route_merge<R, LO + S, N, 2 * S>(k);
  }
#pragma unroll
  for (int i = 2 * S < N ? LO + S : LO; i + S < LO + N; i += 2 * S) {
    const uint32_t a = k[i], b = k[i + S];
    k[i] = max(a, b);
    k[i + S] = min(a, b);
  }
}
template <int R, int LO = 0, int N = R>
__device__ __forceinline__ void route_sort(uint32_t (&k)[R]) {
  if constexpr (N > 1) {
    route_sort<R, LO, N / 2>(k);
    route_sort<R, LO + N / 2, N / 2>(k);
    route_merge<R, LO, N, 1>(k);
  }
}

// e^x and 1 / x in one instruction each after a multiplication: off by 2 + 1.2 |x|
// and by one unit of 2^-23; results below 2^-126 are 0, and so is 1 / infinity.
__device__ __forceinline__ float route_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float route_inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The bias of experts e0.. added to v.
template <int R>
__device__ __forceinline__ void route_add_bias(const RouteParams& p, int e0, float (&v)[R]) {
  if (R >= 4 && p.bias_vec) {
    if (e0 < p.E) {
#pragma unroll
      for (int r = 0; r + 3 < R; r += 4) {
        const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + e0 + r));
        v[r] += b.x, v[r + 1] += b.y, v[r + 2] += b.z, v[r + 3] += b.w;
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (e0 + r < p.E) v[r] += __ldg(p.bias + e0 + r);
  }
}

// Token t by a whole warp, which has `own`, p.smem bytes of shared memory. EXACT:
// bf16 logits without a bias.
template <int R, bool EXACT>
__device__ __forceinline__ void route_row(const RouteParams& p, const int t, uint8_t* const own) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kMask = EXACT ? 1023u : (uint32_t)R - 1u;
  const int e0 = lane * R;
  float l[R];
  route_load<R>(p, t, lane, l);
  const bool sums = p.groups > 1 && p.top2;
  const bool scored = p.bias != nullptr || (sums && !EXACT);   // keys are scores, not logits
  float mx = 0.f, z = 1.f;
  bool flag = false;   // FP32 does not decide this row
  if (!p.sigmoid && (scored || sums || !p.renormalize)) {
    mx = route_off();
#pragma unroll
    for (int r = 0; r < R; ++r) mx = fmaxf(mx, l[r]);
    mx = route_value(__reduce_max_sync(kFull, route_key(mx)), 0u);
    flag = mx == -route_off();
    z = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      z += flag ? (l[r] == mx ? 1.f : 0.f) : route_exp(l[r] - mx);   // (off: 0)
    z = warp_sum(z);
  }
  const float inv_z = route_inverse(z);
  auto score = [&](float v) {
    return p.sigmoid ? route_inverse(1.f + route_exp(-v)) : route_exp(v - mx) * inv_z;
  };
  // Errors of two such scores: the short exp is off by 2 + 1.2 |x| units of 2^-23
  // and its argument by |x| 2^-23; times a sigmoid's slope or a softmax's
  // e^-|x| that is below 2^-22 and 2^-20 of the largest score, the sum's and the
  // division's errors included.
  const float tol = !(scored || sums) ? 0.f : p.sigmoid ? 0x1p-20f : 0x1p-18f * inv_z;
  // and of the rest, relative: the bias's addition, the bits cut off
  constexpr float kCut = (float)R * 0x1p-22f;
  auto make_keys = [&](const float (&logit)[R], uint32_t (&key)[R]) {
    float v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = logit[r];
    if constexpr (!EXACT) {
      if (scored) {
        if (p.sigmoid) {
#pragma unroll
          for (int r = 0; r < R; ++r) v[r] = route_inverse(1.f + route_exp(-v[r]));
        } else {
#pragma unroll
          for (int r = 0; r < R; ++r) v[r] = route_exp(v[r] - mx) * inv_z;
        }
        if (p.bias) route_add_bias<R>(p, e0, v);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t place = EXACT ? 1023u - (uint32_t)(e0 + r) : (uint32_t)(R - 1 - r);
      // (-0 as 0)
      key[r] = logit[r] > route_off() && v[r] > route_off()
                   ? (route_key(v[r] + 0.f) & ~kMask) | place
                   : 0u;
    }
  };
  uint32_t key[R];
  make_keys(l, key);
  int* list = reinterpret_cast<int*>(own);
  // ---- groups
  const int shift = max(p.lane_shift, 0);
  int g = lane;             // the group whose score this lane has
  bool keep = true;         // whether it is kept
  unsigned kept = kFull;    // the same of group j in bit j << shift
  // group of expert e0 + r where a lane's experts lie in several
  auto group_of = [&](int r) { return p.lane_shift >= 0 ? g : min((e0 + r) / p.per, 31); };
  if (p.groups > 1) {
    uint32_t h1 = 0u, h2 = 0u;   // its two largest keys
    if (p.lane_shift >= 0) {
      route_sort<R>(key);
      h1 = key[0];
      if constexpr (R > 1) h2 = key[1];
      g = lane >> p.lane_shift;
      for (int o = 1; o < 1 << p.lane_shift; o <<= 1) {
        const uint32_t a1 = __shfl_xor_sync(kFull, h1, o), a2 = __shfl_xor_sync(kFull, h2, o);
        h2 = max(min(h1, a1), max(h2, a2));
        h1 = max(h1, a1);
      }
    } else {
      uint32_t* sm = reinterpret_cast<uint32_t*>(list);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (e0 + r < p.E) sm[e0 + r] = key[r];
      __syncwarp();
      if (lane < p.groups) {
#pragma unroll 4
        for (int i = 0; i < p.per; ++i) {
          const uint32_t a = sm[lane * p.per + i];
          h2 = max(h2, min(h1, a));
          h1 = max(h1, a);
        }
      }
      __syncwarp();
    }
    uint32_t mine = h1;   // the group's score, as a key
    float size = 0.f;     // the magnitudes in a sum
    if (sums && h1) {
      float v = route_value(h1, kMask), u = route_value(h2, kMask);
      v = scored ? v : score(v);
      u = !h2 ? 0.f : scored ? u : score(u);
      size = fabsf(v) + fabsf(u);
      mine = route_key(v + u);
    }
    const bool real = g < p.groups;
    if (!real) mine = 0u;
    int rank = 0;   // the lanes of a group share the groups it is compared with
    const int lanes = 1 << shift;
    for (int j0 = 0; j0 < p.groups; j0 += lanes) {
      const int j = j0 + (lane & (lanes - 1));
      const uint32_t other = __shfl_sync(kFull, mine, j << shift);   // (of lane j * lanes mod 32)
      rank += j < p.groups && (other > mine || (other == mine && j < g));
    }
    for (int o = 1; o < lanes; o <<= 1) rank += __shfl_xor_sync(kFull, rank, o);
    keep = real && rank < p.top_groups;
    if (sums || !EXACT) {
      const uint32_t mask = sums ? 0u : kMask;
      const uint32_t next = __reduce_max_sync(kFull, keep ? 0u : mine);
      const float last = route_value(__reduce_min_sync(kFull, keep ? mine : 0xffffffffu), mask);
      const float first = route_value(next, mask);
      size = sums ? __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(size)))
                  : scored ? fmaxf(fabsf(last), fabsf(first)) : 0.f;
      // (a sum holds two scores, and what it is rounded by itself)
      const float gap = 2.f * (tol + kCut * size);
      if (__builtin_expect(next && !flag && !(last - first > gap), 0)) {
        // Groups near the border are compared by exact scores. Of their experts
        // those matter that may be among a group's two largest.
        const float v = route_value(mine, mask);
        const bool near = mine && (keep ? !(v > first + gap) : !(v < last - gap));
        const float least = h2 ? route_value(h2, kMask) - gap : route_off();
        const unsigned nears = __ballot_sync(kFull, near);
        int n = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int gr = group_of(r) << shift;
          const float bound = __shfl_sync(kFull, least, gr);
          const int e = EXACT ? 1023 - (int)(key[r] & kMask) : e0 + R - 1 - (int)(key[r] & kMask);
          route_append(list, n, key[r] && ((nears >> gr) & 1u) && route_value(key[r], kMask) >= bound, e);
        }
        __syncwarp();
        // (an infinite bias leaves no bounds: the bound of a group's second infinity is NaN)
        flag = n > 32 || !(gap < -route_off());
        if (!flag) {
          const double zd = p.sigmoid || !(sums || p.bias) ? 1.0 : route_sum<R>(l, mx);
          const int e = lane < n ? list[lane] : 0;
          const int64_t none = route_order(route_off());
          const int64_t x =
              lane < n ? route_order(route_exact(p, t, e, !(sums || p.bias), mx, zd)) : none;
          const int ge = lane < n ? e / p.per : -1;
          int64_t exact = none;
          for (int j = 0; j < p.groups; ++j) {
            if (!((nears >> (j << shift)) & 1u)) continue;
            int64_t sum = warp_max(ge == j ? x : none);
            if (sums) {
              const int at = __ffs(__ballot_sync(kFull, ge == j && x == sum)) - 1;
              const int64_t m2 = warp_max(ge == j && lane != at ? x : none);
              if (m2 > none) sum = route_order(route_unorder(sum) + route_unorder(m2));
            }
            if (g == j) exact = sum;
          }
          const unsigned sure = __ballot_sync(kFull, keep && !near && (lane & ((1 << shift) - 1)) == 0);
          int place = __popc(sure);
#pragma unroll 4
          for (int j = 0; j < p.groups; ++j) {
            const int64_t other = __shfl_sync(kFull, (long long)exact, j << shift);
            if ((nears >> (j << shift)) & 1u) place += other > exact || (other == exact && j < g);
          }
          if (near) keep = place < p.top_groups;
          __syncwarp();
        }
      }
    }
    kept = __ballot_sync(kFull, keep);
    if (p.lane_shift >= 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) key[r] = keep ? key[r] : 0u;
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (!((kept >> group_of(r)) & 1u)) key[r] = 0u;
      route_sort<R>(key);
    }
  } else {
    route_sort<R>(key);
  }
  // ---- experts
  // Lane j keeps the j-th key and who had it. A lane's next key comes from
  // registers, or of long lists from shared memory (one load a round, not R moves).
  constexpr bool kListed = R > 4;
  uint32_t* keys = reinterpret_cast<uint32_t*>(own) + lane;
  if constexpr (kListed) {
#pragma unroll
    for (int r = 1; r < R; ++r) keys[32 * r] = key[r];
    keys[32 * R] = 0u;
  }
  uint32_t got = 0u, next = 0u;
  unsigned who = 0u;
  const int rounds = EXACT ? p.k : p.k + 1;   // and the first one left out
#pragma unroll 1
  for (int j = 0; j < rounds; ++j) {
    next = __reduce_max_sync(kFull, key[0]);
    const bool win = next && key[0] == next;
    if constexpr (!EXACT) {
      const unsigned all = __ballot_sync(kFull, win);
      if (lane == j) who = all;
    }
    if (lane == j) got = next;
    if (win) {
      if constexpr (kListed) {
        keys += 32;
        key[0] = *keys;
      } else {
#pragma unroll
        for (int r = 0; r + 1 < R; ++r) key[r] = key[r + 1];
        key[R - 1] = 0u;
      }
    }
  }
  int mine = -1;
  if constexpr (EXACT) {
    if (got) mine = 1023 - (int)(got & kMask);
  } else {
    if (got) mine = __ffs(who) * R - 1 - (int)(got & kMask);
    // whether each is clearly larger than the next one
    const float v = route_value(got, kMask);
    uint32_t after = __shfl_down_sync(kFull, got, 1);
    if (lane == p.k - 1) after = next;
    const float u = route_value(after, kMask);
    const float gap = tol + (scored ? kCut * fmaxf(fabsf(v), fabsf(u)) : 0.f);
    // (equal keys of several lanes leave in one round)
    const bool close =
        __any_sync(kFull, lane < p.k && (__popc(who) > 1 || (after && !(v - u > gap))));
    if (__builtin_expect(close && !flag, 0)) {
      const uint32_t last = __shfl_sync(kFull, got, p.k - 1);
      const float least = last ? route_value(last, kMask) : route_off();
      const float slack = 2.f * (tol + kCut * fabsf(least) * (scored && last));
      __syncwarp();
      // every expert that may be among the k, in exact order (all of them where no
      // k are left)
      int n = 0;
      route_load<R>(p, t, lane, l);
      uint32_t c[R];
      make_keys(l, c);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool in = c[r] && (p.groups == 1 || ((kept >> (group_of(r) << shift)) & 1u));
        route_append(list, n, in && !(route_value(c[r], kMask) < least - slack), e0 + r);
      }
      __syncwarp();
      flag = n > 32;
      if (!flag) {
        const double zd = p.sigmoid || !p.bias ? 1.0 : route_sum<R>(l, mx);
        const int e = lane < n ? list[lane] : p.E;
        const int64_t x =
            route_order(lane < n ? route_exact(p, t, e, !p.bias, mx, zd) : (double)route_off());
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const int64_t other = __shfl_sync(kFull, (long long)x, j);
          const int oe = __shfl_sync(kFull, e, j);
          rank += other > x || (other == x && oe < e);
        }
        __syncwarp();
        if (lane < n) list[rank] = e;
        __syncwarp();
        mine = lane < n ? list[lane] : -1;
      }
    }
  }
  if (__builtin_expect(flag, 0)) {
    __syncwarp();
    mine = route_slow(p, t, reinterpret_cast<double*>(own));
  }
  if (lane >= p.k) mine = -1;
  // ---- the chosen experts' weights
  const float lm = mine >= 0 ? route_logit(p, (size_t)t * p.E + mine) : route_off();
  // Relative to the largest chosen logit where the sum is that of the chosen (and
  // to infinite ones where there are any, which a bias may pass over).
  const float top = p.renormalize && mx < -route_off() ? warp_max(lm) : p.sigmoid ? 0.f : mx;
  float v = mine >= 0 ? route_weight(p.sigmoid, lm, top) : 0.f;
  if (p.renormalize) {
    const float sum = warp_sum(v);
    v = sum > 0.f ? v / sum : 0.f;
  } else if (!p.sigmoid && mine >= 0) {
    v /= z;
  }
  if (lane < p.k) {
    p.ids[(size_t)t * p.k + lane] = mine;
    p.w[(size_t)t * p.k + lane] = v * p.scale;
  }
}

template <int R, bool EXACT>
__global__ void __launch_bounds__(kRouteWarps * 32, R <= 8 ? 9 : 4) moe_route_experts_rows(
    const __grid_constant__ RouteParams p) {
  extern __shared__ double route_smem[];
  const int warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRouteWarps + warp;
  pdl_wait();
  pdl_trigger();
  if (t < p.T) route_row<R, EXACT>(p, t, reinterpret_cast<uint8_t*>(route_smem) + warp * p.smem);
}

// ---------------------------------------------------------------------------
// moe_route_experts_packed: many tokens of up to 256 experts, W lanes each with 32
// experts (E = 32 W), at most 8 experts a token, groups of whole lanes. What a warp
// does once a token in moe_route_experts_rows it does here for 32 / W tokens at once
// (us of 16384 tokens, one way and the other: 64 experts 8.9 / 5.5, 128 in bf16 8.6 /
// 5.3, with groups, a bias and sigmoids 13.5 / 12; 256 12.5 / 10.8, with a bias 17 / 19,
// which therefore stay there, as do calls of fewer tokens: 4096 3.9 / 3.0, 1024 2.4 /
// 2.9).
//
// Keys are signed fixed-point numbers of 27 bits (2^-24 of a score plus bias, 2^-20 of
// a logit) over the expert's place in the lane, or a bf16's bits over its place of
// all. A lane sorts its nine largest. Rows that this does not decide go to
// route_row.
// ---------------------------------------------------------------------------
constexpr int kRouteListed = 9;   // 8 chosen and the first one left out
constexpr int kRouteOff = INT32_MIN;

// Keys in descending order, by the same network as route_sort.
template <int R, int LO, int N, int S>
__device__ __forceinline__ void key_merge(int (&k)[R]) {
  if constexpr (2 * S < N) {
    key_merge<R, LO, N, 2 * S>(k);
    key_merge<R, LO + S, N, 2 * S>(k);
  }
#pragma unroll
  for (int i = 2 * S < N ? LO + S : LO; i + S < LO + N; i += 2 * S) {
    const int a = k[i], b = k[i + S];
    k[i] = max(a, b);
    k[i + S] = min(a, b);
  }
}
template <int R, int LO, int N>
__device__ __forceinline__ void key_sort(int (&k)[R]) {
  if constexpr (N > 1) {
    key_sort<R, LO, N / 2>(k);
    key_sort<R, LO + N / 2, N / 2>(k);
    key_merge<R, LO, N, 1>(k);
  }
}
// k[A..A + 7] = the eight largest of the descending k[A..] and k[B..], in order;
// `ninth` = the largest of those left over, or what it was.
template <int A, int B>
__device__ __forceinline__ void key_top8(int (&k)[32], int& ninth) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = k[A + i], b = k[B + 7 - i];
    k[A + i] = max(a, b);
    ninth = max(ninth, min(a, b));
  }
#pragma unroll
  for (int s = 4; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & s)) {
        const int a = k[A + i], b = k[A + i + s];
        k[A + i] = max(a, b);
        k[A + i + s] = min(a, b);
      }
}

// Nearest whole number, saturated.
__device__ __forceinline__ int to_fixed(float v) {
  int r;
  asm("cvt.rni.s32.f32 %0, %1;" : "=r"(r) : "f"(v));
  return r;
}

template <int W, bool EXACT>
__global__ void __launch_bounds__(kRouteWarps * 32, 5) moe_route_experts_packed(
    const __grid_constant__ RouteParams p) {
  extern __shared__ double route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (W - 1), base = lane & ~(W - 1);
  const int first = (blockIdx.x * kRouteWarps + warp) * (32 / W);
  const int t = first + lane / W;
  pdl_wait();
  pdl_trigger();
  if (first >= p.T) return;
  const bool sums = p.groups > 1 && p.top2;
  const bool scored = p.bias != nullptr || (sums && !EXACT);
  auto sub_max = [&](int v) {
#pragma unroll
    for (int o = 1; o < W; o <<= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
  };
  auto sub_sum = [&](float v) {
#pragma unroll
    for (int o = 1; o < W; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
  };
  // ---- logits, in their order
  float l[32];
  if (t < p.T) {
    const size_t at = (size_t)t * (32 * W) + 32 * sub;
    if (p.bf16) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.logits) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 a = __ldg(src + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) l[8 * i + j] = j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
      }
    } else {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 a = __ldg(src + i);
        l[4 * i] = a.x, l[4 * i + 1] = a.y, l[4 * i + 2] = a.z, l[4 * i + 3] = a.w;
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < 32; ++r) l[r] = route_off();
  }
  // ---- softmax
  float mx = 0.f, z = 1.f;
  bool flag = false;   // this does not decide the token's row
  if (!p.sigmoid && (scored || sums || !p.renormalize)) {
    mx = route_off();
#pragma unroll
    for (int r = 0; r < 32; ++r) mx = fmaxf(mx, l[r]);
#pragma unroll
    for (int o = 1; o < W; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    flag = mx == -route_off();
    z = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) z += route_exp(route_clean(l[r]) - mx);
    z = sub_sum(z);
  }
  const float inv_z = route_inverse(z);
  auto score = [&](float v) {
    return p.sigmoid ? route_inverse(1.f + route_exp(-v)) : route_exp(v - mx) * inv_z;
  };
  // ---- keys
  int key[32];
  constexpr float kUnit = 0x1p29f;   // of a score plus bias, below 4
  if constexpr (EXACT) {
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const int b = __float_as_int(l[r] + 0.f);   // (-0 as 0)
      key[r] = l[r] > route_off() ? (b ^ ((b >> 31) & 0x7fff0000)) | (1023 - 32 * sub - r) : kRouteOff;
    }
  } else {
    float v[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r] = l[r];
    if (scored) {
      if (p.sigmoid) {
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r] = route_inverse(1.f + route_exp(-v[r]));
      } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r] = route_exp(v[r] - mx) * inv_z;
      }
      if (p.bias) {
        const float4* src = reinterpret_cast<const float4*>(p.bias + 32 * sub);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 b = __ldg(src + i);
          v[4 * i] += b.x, v[4 * i + 1] += b.y, v[4 * i + 2] += b.z, v[4 * i + 3] += b.w;
        }
      }
    }
    const float unit = scored ? kUnit : 0x1p25f;
#pragma unroll
    for (int r = 0; r < 32; ++r)   // (cut off above kRouteOff's neighbours)
      key[r] = l[r] > route_off() && v[r] > route_off()
                   ? (to_fixed(fmaxf(v[r] * unit, -0x1.fffffep30f)) & ~31) | (31 - r)
                   : kRouteOff;
  }
  int ninth = kRouteOff;
  key_sort<32, 0, 8>(key);
  key_sort<32, 8, 8>(key);
  key_sort<32, 16, 8>(key);
  key_sort<32, 24, 8>(key);
  key_top8<0, 8>(key, ninth);
  key_top8<16, 24>(key, ninth);
  key_top8<0, 16>(key, ninth);
  // units by which keys of values that FP32 tells apart differ: the scores' errors (as
  // in route_row), the sum's rounding below 4, place bits
  const float tol = !(scored || sums) ? 0.f : p.sigmoid ? 0x1p-20f : 0x1p-18f * inv_z;
  const uint32_t gap = scored ? (uint32_t)(tol * kUnit) + 256u + 64u : 31u;
  // ---- groups
  bool keep = true;
  if (p.groups > 1) {
    int h1 = key[0], h2 = key[1];
    for (int o = 1; o < 1 << p.packed_shift; o <<= 1) {
      const int a1 = __shfl_xor_sync(kFull, h1, o), a2 = __shfl_xor_sync(kFull, h2, o);
      h2 = max(min(h1, a1), max(h2, a2));
      h1 = max(h1, a1);
    }
    int mine = h1;
    uint32_t apart = gap;
    if (sums) {
      if constexpr (EXACT) {   // scores in units of 2^-28
        auto part = [&](int k) {
          const int b = k & 0xffff0000;
          const float s = score(__int_as_float(b ^ ((b >> 31) & 0x7fff0000)));
          return k == kRouteOff ? 0 : to_fixed(s * (0.5f * kUnit));
        };
        if (h1 != kRouteOff) mine = part(h1) + part(h2);
        apart = (uint32_t)(tol * kUnit) + 8u;
      } else {
        // halves, so that two below 4 add up; what was cut off at 4 decides nothing
        if (h2 != kRouteOff) mine = (h1 >> 1) + (h2 >> 1);
        else if (h1 != kRouteOff) mine = h1 >> 1;
        flag |= h1 >= INT32_MAX - 64 || (h2 != kRouteOff && h2 < -INT32_MAX + 256);
      }
    }
    const int g = sub >> p.packed_shift;
    int rank = 0;
    unsigned near = 0u;   // groups too close to this one, in bits as lanes are
    for (int j = 0; j < p.groups; ++j) {
      const int other = __shfl_sync(kFull, mine, base | (j << p.packed_shift));
      rank += other > mine || (other == mine && j < g);
      const uint32_t d = (uint32_t)max(other, mine) - (uint32_t)min(other, mine);
      near |= (unsigned)(d <= apart) << (j << p.packed_shift);
    }
    keep = rank < p.top_groups;
    const unsigned kept = __ballot_sync(kFull, keep) >> base;
    // (two groups with nothing left are not told apart, and need not be)
    if (sums || !EXACT) flag |= mine != kRouteOff && (near & (keep ? ~kept : kept)) != 0u;
    if (!keep) {
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = kRouteOff;
      ninth = kRouteOff;
    }
  }
  // ---- experts: slot j is the lane's with sub = j mod W
  constexpr int kSlots = W >= 8 ? 1 : 8 / W;
  int got[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) got[i] = -1;
  int before = 0;
#pragma unroll
  for (int j = 0; j < kRouteListed; ++j) {
    if (EXACT ? j >= p.k : j > p.k) break;
    const int top = sub_max(key[0]);
    const bool some = top != kRouteOff, win = some && key[0] == top;
    int id;
    if constexpr (EXACT) {
      id = 1023 - (top & 1023);
    } else {
      const unsigned who = (__ballot_sync(kFull, win) >> base) & (unsigned)((1ull << W) - 1);
      id = 32 * (__ffs(who) - 1) + 31 - (top & 31);
      flag |= some && ((j > 0 && (uint32_t)before - (uint32_t)top <= gap) ||
                       (j < p.k && (who & (who - 1u)) != 0u));
      before = top;
    }
    if (j < p.k && sub == (j & (W - 1)) && some) got[j / W < kSlots ? j / W : 0] = id;
    if (win) {
#pragma unroll
      for (int i = 0; i < 7; ++i) key[i] = key[i + 1];
      key[7] = ninth;
      ninth = kRouteOff;
    }
  }
  // ---- the chosen experts' weights
  const bool mine = t < p.T;
  float lm[kSlots], v[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    lm[i] = mine && got[i] >= 0 ? route_logit(p, (size_t)t * (32 * W) + got[i]) : route_off();
  float top = p.sigmoid ? 0.f : mx;
  if (p.renormalize) {
    const bool infinite = mx == -route_off();   // (as in route_row)
    float best = route_off();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) best = fmaxf(best, lm[i]);
#pragma unroll
    for (int o = 1; o < W; o <<= 1) best = fmaxf(best, __shfl_xor_sync(kFull, best, o));
    if (!infinite) top = best;
  }
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    v[i] = got[i] >= 0 ? route_weight(p.sigmoid, lm[i], top) : 0.f;
    total += v[i];
  }
  if (p.renormalize)
    total = sub_sum(total);
  else
    total = p.sigmoid ? 1.f : z;
  const unsigned flags = __ballot_sync(kFull, flag) >> base;
  const bool again = mine && (flags & (unsigned)((1ull << W) - 1)) != 0u;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int j = sub + W * i;
    if (mine && !again && j < p.k) {
      p.ids[(size_t)t * p.k + j] = got[i];
      p.w[(size_t)t * p.k + j] = (total > 0.f ? v[i] / total : 0.f) * p.scale;
    }
  }
  unsigned todo = __ballot_sync(kFull, again && sub == 0);
  while (__builtin_expect(todo != 0u, 0)) {
    route_row<W, EXACT>(p, first + (__ffs(todo) - 1) / W,
                        reinterpret_cast<uint8_t*>(route_smem) + warp * p.smem);
    __syncwarp();
    todo &= todo - 1u;
  }
}

// ---------------------------------------------------------------------------
// moe_norm_add_norm_rows: one CTA (of short rows one warp) a row, whose values stay in registers between
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
  int T, H;
  float scale, residual_scale, eps;
  float inv_h;            // 1 / H
  float offset;           // added to norm weights
  int gate_row, gate_full, gate_sigmoid, gate_tanh;
};

// Sum of `v` over the CTA, in every thread; `part` is not used before or after
// by another sum without a barrier between.
__device__ __forceinline__ float cta_sum(float v, float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = warp_sum(v);
  if (warps == 1) return v;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  if (warps > 4) return warp_sum(lane < warps ? part[lane] : 0.f);
  v = part[0] + part[1];
  if (warps > 2) v += part[2];
  if (warps > 3) v += part[3];
  return v;
}

__device__ __forceinline__ float gate_value(const NormPairParams& p, float g) {
  if (p.gate_sigmoid) return 1.f / (1.f + expf(-g));
  if (p.gate_tanh) return tanhf(g);
  return g;
}

// What a row's gate and the scale multiply its branch by.
__device__ __forceinline__ float norm_row_gate(const NormPairParams& p, int row) {
  return p.gate && p.gate_row ? p.scale * gate_value(p, bf16_lo(p.gate[row])) : p.scale;
}

// Two FP32 values in one register pair, for the packed FP32 instructions, each of
// which rounds both as the single one would: the norms are bound by instructions as
// much as by HBM (4096 rows of 7168: 33.3 million, 27.3 with these, 21.8 with four
// vectors a thread, at 92, 89 and 71 us for 8191 rows).
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ static F2 of(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
  }
  __device__ __forceinline__ static F2 both(float a) { return of(a, a); }
  __device__ __forceinline__ static F2 bf16(uint32_t w) { return of(bf16_lo(w), bf16_hi(w)); }
  __device__ __forceinline__ void get(float& lo, float& hi) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// A row's vector as pairs: 16 bytes are four, a single value is one with a zero.
template <int V>
struct Pairs {
  static constexpr int N = V == 8 ? 4 : 1;
  F2 f[N];
  __device__ __forceinline__ explicit Pairs(typename RowVec<V>::Raw raw) {
    if constexpr (V == 8) {
      f[0] = F2::bf16(raw.x), f[1] = F2::bf16(raw.y), f[2] = F2::bf16(raw.z), f[3] = F2::bf16(raw.w);
    } else {
      f[0] = F2::bf16(raw);
    }
  }
  __device__ __forceinline__ typename RowVec<V>::Raw packed() const {
    float lo[N], hi[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i].get(lo[i], hi[i]);
    if constexpr (V == 8)
      return make_uint4(RowVec<8>::pack(lo[0], hi[0]), RowVec<8>::pack(lo[1], hi[1]),
                        RowVec<8>::pack(lo[2], hi[2]), RowVec<8>::pack(lo[3], hi[3]));
    else
      return f32_to_bf16_rn(lo[0]);
  }
};

// The new residual stream of one vector, as it is kept (and what is kept is
// normalised): from the branch x, its norm's factor r and weights w, the gate's
// values (of the vector `gate`, with GATE) and the stream before.
template <int V, bool GATE>
__device__ __forceinline__ typename RowVec<V>::Raw norm_stream(
    const NormPairParams& p, typename RowVec<V>::Raw x, typename RowVec<V>::Raw res,
    typename RowVec<V>::Raw w, typename RowVec<V>::Raw gate, float r, float row_gate) {
  constexpr int N = Pairs<V>::N;
  Pairs<V> f(x);
  const Pairs<V> b(res);
  if (p.post) {
    Pairs<V> ww(w);
    if (p.offset != 0.f) {
#pragma unroll
      for (int i = 0; i < N; ++i) ww.f[i] = ww.f[i] + F2::both(p.offset);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) f.f[i] = f.f[i] * F2::both(r) * ww.f[i];
  }
  if constexpr (GATE) {
    Pairs<V> g(gate);
    if (p.gate_sigmoid || p.gate_tanh) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float lo, hi;
        g.f[i].get(lo, hi);
        g.f[i] = F2::of(gate_value(p, lo), gate_value(p, hi));
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) f.f[i] = f.f[i] * g.f[i];
  }
  const F2 rg = F2::both(row_gate);
  if (p.residual_scale == 1.f) {
#pragma unroll
    for (int i = 0; i < N; ++i) f.f[i] = fma2(f.f[i], rg, b.f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      f.f[i] = fma2(f.f[i], rg, b.f[i] * F2::both(p.residual_scale));
  }
  return f.packed();
}

// The sum of squares, in two halves.
template <int V>
__device__ __forceinline__ F2 norm_squares(typename RowVec<V>::Raw x, F2 ss) {
  const Pairs<V> f(x);
#pragma unroll
  for (int i = 0; i < Pairs<V>::N; ++i) ss = fma2(f.f[i], f.f[i], ss);
  return ss;
}
__device__ __forceinline__ float norm_factor(const NormPairParams& p, F2 ss, float* part) {
  float lo, hi;
  ss.get(lo, hi);
  return rsqrtf(cta_sum(lo + hi, part) * p.inv_h + p.eps);
}

// The outputs of vector v of a row that begins at `base`: the stream s times r
// and the weights. All lanes of a warp take part.
template <int V>
__device__ __forceinline__ void norm_outputs(const NormPairParams& p, size_t base, int v, bool in,
                                             typename RowVec<V>::Raw s, typename RowVec<V>::Raw w,
                                             float r) {
  using Row = RowVec<V>;
  constexpr int N = Pairs<V>::N;
  Pairs<V> n(s);
  if (in) {
    Pairs<V> ww(w);
    if (p.offset != 0.f) {
#pragma unroll
      for (int i = 0; i < N; ++i) ww.f[i] = ww.f[i] + F2::both(p.offset);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) n.f[i] = n.f[i] * F2::both(r) * ww.f[i];
    if (p.y) *reinterpret_cast<typename Row::Raw*>(p.y + base + (size_t)v * V) = n.packed();
  }
  if (p.codes) {   // H is a multiple of 32: a block's lanes are all in or all out
    float f[2 * N];
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) n.f[i].get(f[2 * i], f[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < V; ++j) amax = max(amax, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
    for (int o = 16 / V; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, o));
    if (in) {
      const uint32_t sc = mx_scale_code(amax);
      const float inv = mx_inverse(sc);
      float q[V];
#pragma unroll
      for (int j = 0; j < V; ++j) q[j] = f[j] * inv;
      Row::store_codes(p.codes + base + (size_t)v * V, q);
      if (v % (32 / V) == 0) p.scales[(base + (size_t)v * V) / 32] = (uint8_t)sc;
    }
  }
}

// GATE: a gate with a value per channel or element. (An instance of its own: with
// the gate's functions in every instance the code outgrew the instruction cache,
// 8191 rows of 7168 without a gate took 100 us instead of 71.)
template <int V, int NV, bool GATE>
__global__ void __launch_bounds__(V == 8 && NV > 2 ? 256 : 1024) moe_norm_add_norm_rows(
    const __grid_constant__ NormPairParams p) {
  __shared__ float part[2][32];
  using Row = RowVec<V>;
  using Raw = typename Row::Raw;
  const int nv = p.H / V;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.T) return;   // (only where a row is a warp's: no barrier follows)
  const size_t base = (size_t)row * p.H;
  auto at = [&](int i) { return i * (int)blockDim.x + (int)threadIdx.x; };
  pdl_wait();
  pdl_trigger();
  // every load of the row in flight before the first is used (but for rows of
  // many single values, whose registers would not hold them)
  constexpr bool kAhead = V == 8 || NV <= 4;
  Raw x[NV], res[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (at(i) < nv) x[i] = Row::once(p.x + base + (size_t)at(i) * V);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (kAhead && at(i) < nv) res[i] = Row::once(p.residual + base + (size_t)at(i) * V);
  const float row_gate = norm_row_gate(p, row);
  float r = 1.f;
  F2 ss = F2::both(0.f);
  if (p.post) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at(i) < nv) ss = norm_squares<V>(x[i], ss);
    r = norm_factor(p, ss, part[0]);
    ss = F2::both(0.f);
  }
  // weights and gates a few vectors ahead of their use
  constexpr int B = !kAhead ? 1 : NV < 4 ? NV : 4;
#pragma unroll
  for (int i0 = 0; i0 < NV; i0 += B) {
    Raw w[B], g[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      w[i] = g[i] = Raw();
      if (at(i0 + i) >= nv) continue;
      const size_t v = (size_t)at(i0 + i) * V;
      if (!kAhead) res[i0 + i] = Row::once(p.residual + base + v);
      if (p.post) w[i] = Row::raw(p.post + v);
      if (GATE) g[i] = Row::raw(p.gate + (p.gate_full ? base : 0) + v);
    }
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (at(i0 + i) < nv) {
        Raw& s = x[i0 + i];
        s = norm_stream<V, GATE>(p, s, res[i0 + i], w[i], g[i], r, row_gate);
        ss = norm_squares<V>(s, ss);
        *reinterpret_cast<Raw*>(p.sum + base + (size_t)at(i0 + i) * V) = s;
      }
  }
  if (!p.pre) return;
  r = norm_factor(p, ss, part[1]);
#pragma unroll
  for (int i0 = 0; i0 < NV; i0 += B) {
    Raw w[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      w[i] = Raw();
      if (at(i0 + i) < nv) w[i] = Row::raw(p.pre + (size_t)at(i0 + i) * V);
    }
#pragma unroll
    for (int i = 0; i < B; ++i)
      norm_outputs<V>(p, base, at(i0 + i), at(i0 + i) < nv, x[i0 + i], w[i], r);
  }
}

}  // namespace moe
