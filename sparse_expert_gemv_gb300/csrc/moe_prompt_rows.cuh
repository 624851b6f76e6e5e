// The row operators of the layer's prompt form: the residual addition with
// its root-mean-square norm and MXFP8 output, the grouping of routed slots by
// expert, and the routing-weighted combination of expert rows.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_device.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// MXFP8 quantisation
// ---------------------------------------------------------------------------

// Scale code of a block whose largest magnitude has the bits `amax`
// (sign cleared): floor(log2 amax) - 8 + 127, i.e. the biased exponent less 8,
// at least 0; 127 for a block of zeros; 255 (NaN) when a value of the block
// is infinite or NaN (their bits compare above every finite value's).
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax) {
  const uint32_t b = amax >> 23;
  uint32_t s = b > 8u ? b - 8u : 0u;
  s = amax == 0u ? 127u : s;
  return b == 255u ? 255u : s;
}

// 2^(127 - s), what a block's values are multiplied by before they round to
// E4M3: a normal number for every code mx_scale_code gives (s <= 246); NaN
// for 255, so that every code of such a block is NaN.
__device__ __forceinline__ float mx_inverse(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - s) << 23);
}

// Two values -> two E4M3 codes (a in the low byte), rounded to nearest even
// and saturated to 448; NaN -> 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// ---------------------------------------------------------------------------
// rows in vectors: V = 8 bf16 values (16 bytes) or single values
// ---------------------------------------------------------------------------
template <int V>
struct RowVec;

template <>
struct RowVec<8> {
  using Raw = uint4;   // as stored: half the registers of the values
  __device__ __forceinline__ static Raw raw(const uint16_t* p) {
    return *reinterpret_cast<const uint4*>(p);
  }
  // of rows that are read once: out of the caches first
  __device__ __forceinline__ static Raw once(const uint16_t* p) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ static void load(const uint16_t* p, float (&f)[8]) {
    values(raw(p), f);
  }
  __device__ __forceinline__ static void values(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
  }
  __device__ __forceinline__ static uint32_t pack(float a, float b) {
    return (uint32_t)f32_to_bf16_rn(a) | ((uint32_t)f32_to_bf16_rn(b) << 16);
  }
  __device__ __forceinline__ static void store(uint16_t* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
  }
  __device__ __forceinline__ static void store_codes(uint8_t* p, const float (&f)[8]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16),
                                              e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
  }
};

template <>
struct RowVec<1> {
  using Raw = uint16_t;
  __device__ __forceinline__ static Raw raw(const uint16_t* p) { return *p; }
  __device__ __forceinline__ static Raw once(const uint16_t* p) { return __ldcs(p); }
  __device__ __forceinline__ static void load(const uint16_t* p, float (&f)[1]) {
    values(raw(p), f);
  }
  __device__ __forceinline__ static void values(uint16_t v, float (&f)[1]) {
    f[0] = __uint_as_float((uint32_t)v << 16);
  }
  __device__ __forceinline__ static void store(uint16_t* p, const float (&f)[1]) {
    *p = f32_to_bf16_rn(f[0]);
  }
  __device__ __forceinline__ static void store_codes(uint8_t* p, const float (&f)[1]) {
    *p = (uint8_t)e4m3x2(f[0], f[0]);
  }
};

// ---------------------------------------------------------------------------
// moe_add_rms_norm_rows: one CTA a row. The row's sums stay in registers
// (NV vectors of V values a thread) between the reduction and the outputs, so
// every operand is read once and every output written once. A quantisation
// block is 32 / V neighbouring lanes, whose largest magnitude is a butterfly
// over them. Bound by HBM: all of a row's loads are issued before the first is
// used, and as loads of what is read once (8191 rows of 7168, MXFP8 out: 68 us
// with a vector's loads behind the one before, 63 so, 6.6 TB/s; 4096 rows of
// 4096 22.1 and 20.1 us with the cached and the read-once form).
// ---------------------------------------------------------------------------
struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;   // or null
  const uint16_t* weight;
  uint16_t* sum;              // or null; may be x or residual
  uint16_t* y;                // or null
  uint8_t* codes;             // or null (then scales too)
  uint8_t* scales;
  int H;
  float eps;
};

constexpr int kNormMaxH = 16384;   // 1024 threads hold 16 values each

template <int V, int NV>
__global__ void __launch_bounds__(1024) moe_add_rms_norm_rows(const NormParams p) {
  __shared__ float part[32];
  const int H = p.H, nv = H / V;
  const size_t base = (size_t)blockIdx.x * H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  // every load of the row in flight before the first is used
  typename RowVec<V>::Raw x[NV], res[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nv) x[i] = RowVec<V>::once(p.x + base + (size_t)v * V);
  }
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v < nv) res[i] = RowVec<V>::once(p.residual + base + (size_t)v * V);
    }
  }
  float f[NV][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nv) {
      RowVec<V>::values(x[i], f[i]);
      if (p.residual) {
        float r[V];
        RowVec<V>::values(res[i], r);
        // the residual stream is kept in bf16, and what is kept is normalised
#pragma unroll
        for (int j = 0; j < V; ++j)
          f[i][j] = __uint_as_float((uint32_t)f32_to_bf16_rn(f[i][j] + r[j]) << 16);
      }
      if (p.sum) RowVec<V>::store(p.sum + base + (size_t)v * V, f[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(f[i][j], f[i][j], ss);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] = 0.f;
    }
  }
  ss = warp_sum(ss);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  ss = warp_sum(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f);
  const float r = rsqrtf(ss / (float)H + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    float n[V];
    uint32_t amax = 0u;
    if (v < nv) {
      RowVec<V>::load(p.weight + (size_t)v * V, n);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        n[j] = f[i][j] * r * n[j];
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

// ---------------------------------------------------------------------------
// moe_group_slots: stable counting sort of S = T * k slots by expert, one
// cluster of C CTAs (1 to 16). The slots are cut into one contiguous range per
// warp of the cluster. Each warp counts its range into a table of its own
// (lanes of equal id find one another by ballots over the id's bits, so no
// atomics and a fixed order) and keeps each slot's rank there; the CTAs
// exchange their totals through distributed shared memory; each slot's place is
// then its expert's start, what lower warps hold of it, and its rank. Bound by
// latency up to some 8192 slots (2.7 us for 256 of them, 5.5 for 8192), by the
// ballots and counts of 16 SMs beyond (12.9 for 131072).
// ---------------------------------------------------------------------------
constexpr int kGroupThreads = 1024;
constexpr int kGroupBatch = 8;

struct GroupParams {
  const int32_t* ids;
  int32_t* offsets;
  int32_t* rows;
  int32_t* slots;
  int S, E;
  int per_warp;   // slots a warp takes, a multiple of 32
  // s / k = (2 s * k_inverse) >> (32 + k_shift) for s <= 2^30
  unsigned k_inverse;
  int k_shift;
  // slots of a CTA that go to `rows` through shared memory, in the order of
  // their places there, so that a warp's stores are a few runs and not 32
  // single words; 0 to store directly
  int staged;
};

// `staged`: places of the CTA's slots before they are written (see below).
__host__ __device__ constexpr size_t group_smem(int warps, int E, int staged) {
  return (size_t)((warps + 3) * E + 1 + 2 * staged) * sizeof(int);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Word `p` of this CTA's shared memory, read from CTA `rank` of the cluster.
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.b32 %0, [a];\n\t}"
      : "=r"(v)
      : "r"(smem_addr(p)), "r"(rank)
      : "memory");
  return v;
}

// The lanes whose value (of BITS bits) is this lane's, where `in` holds.
template <int BITS>
__device__ __forceinline__ unsigned same_value(unsigned v, bool in) {
  unsigned same = __ballot_sync(kFull, in);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool one = (v >> b) & 1u;
    const unsigned ones = __ballot_sync(kFull, one);
    same &= one ? ones : ~ones;
  }
  return same;
}

// BITS: of the largest expert id, E - 1.
template <int BITS>
__global__ void __launch_bounds__(kGroupThreads) moe_group_slots(const GroupParams p) {
  extern __shared__ int sm_group[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E, C = gridDim.x, rank = blockIdx.x;
  int* mine = sm_group;              // [E] this CTA's slots of each expert
  int* start = mine + E;             // [E] all CTAs' slots, then the groups' starts
  int* local = start + E;            // [E] starts of the experts among this CTA's slots
  int* tab = local + E;              // [warps][E] each warp's count, then its next place
  int* stage = tab + warps * E + 1;  // [staged] tokens, then [staged] places
  int* cnt = tab + warp * E;
  pdl_wait();
  pdl_trigger();   // the next kernel's prologue may run beside this one
  for (int e = lane; e < E; e += 32) cnt[e] = 0;
  __syncwarp();
  const long long w0 = (long long)(rank * warps + warp) * p.per_warp;
  const int lo = (int)min((long long)p.S, w0), hi = (int)min((long long)p.S, w0 + p.per_warp);
  const unsigned below = (1u << lane) - 1u;
  // A warp's range is one batch up to kGroupBatch * 32 slots: its ids and
  // ranks then stay in registers, else the ranks wait in `slots`.
  const bool one = p.per_warp <= 32 * kGroupBatch;
  int id[kGroupBatch], rank_in[kGroupBatch];
  for (int s0 = lo; s0 < hi; s0 += 32 * kGroupBatch) {
#pragma unroll
    for (int i = 0; i < kGroupBatch; ++i) {
      const int s = s0 + 32 * i + lane;
      id[i] = s < hi ? p.ids[s] : -1;
      if (id[i] >= E) id[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < kGroupBatch; ++i) {
      if (s0 + 32 * i >= hi) break;
      const int s = s0 + 32 * i + lane, e = id[i];
      const bool in = e >= 0;
      const unsigned same = same_value<BITS>(e, in);
      const int before = in ? cnt[e] : 0;
      __syncwarp();
      if (in && (same & below) == 0u) cnt[e] = before + __popc(same);
      __syncwarp();
      rank_in[i] = before + __popc(same & below);
      if (!one && s < hi) p.slots[s] = rank_in[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int c = tab[w * E + e];
      tab[w * E + e] = sum;
      sum += c;
    }
    mine[e] = sum;
  }
  if (C > 1) cluster_sync(); else __syncthreads();
  // experts' totals, and what lower CTAs place before this one's slots
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int total = 0, before = 0;
    for (int c = 0; c < C; ++c) {
      const int v = C > 1 ? ld_cluster(mine + e, c) : mine[e];
      if (c < rank) before += v;
      total += v;
    }
    start[e] = total;
    local[e] = before;
  }
  // no CTA leaves (or changes `mine`) while another still reads it
  if (C > 1) cluster_sync(); else __syncthreads();
  // exclusive prefixes over the experts: where a group starts (then where this
  // CTA's part of it does), and where an expert starts among this CTA's slots
  if (warp == 0) {
    int carry = 0, mine_carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int v = e < E ? start[e] : 0, m = e < E ? mine[e] : 0;
      int incl = v, mi = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, incl, o), w = __shfl_up_sync(kFull, mi, o);
        if (lane >= o) incl += u, mi += w;
      }
      if (e < E) {
        start[e] = carry + incl - v + local[e];
        if (rank == 0) p.offsets[e] = carry + incl - v;
        local[e] = mine_carry + mi - m;
      }
      carry += __shfl_sync(kFull, incl, 31);
      mine_carry += __shfl_sync(kFull, mi, 31);
    }
    if (lane == 0) {
      stage[-1] = carry;   // rows in all groups
      if (rank == 0) p.offsets[E] = carry;
    }
    mine[0] = mine_carry;  // this CTA's slots that join a group
  }
  __syncthreads();
  for (int s0 = lo; s0 < hi; s0 += 32 * kGroupBatch) {
    if (!one) {
#pragma unroll
      for (int i = 0; i < kGroupBatch; ++i) {
        const int s = s0 + 32 * i + lane;
        id[i] = s < hi ? p.ids[s] : -1;
        if (id[i] >= E) id[i] = -1;
        rank_in[i] = s < hi ? p.slots[s] : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < kGroupBatch; ++i) {
      const int s = s0 + 32 * i + lane, e = id[i];
      if (s >= hi) break;
      const int in_cta = e >= 0 ? cnt[e] + rank_in[i] : 0;
      const int q = e >= 0 ? start[e] + in_cta : -1;
      p.slots[s] = q;
      if (e < 0) continue;
      const int token = (int)(__umulhi(2u * s, p.k_inverse) >> p.k_shift);
      if (p.staged) {
        stage[local[e] + in_cta] = token;
        stage[p.staged + local[e] + in_cta] = q;
      } else {
        p.rows[q] = token;
      }
    }
  }
  if (p.staged) {
    __syncthreads();
    for (int i = threadIdx.x; i < mine[0]; i += blockDim.x) p.rows[stage[p.staged + i]] = stage[i];
  }
  // rows past the last group
  const int used = stage[-1];
  for (long long r = (long long)used + rank * blockDim.x + threadIdx.x; r < p.S;
       r += (long long)C * blockDim.x)
    p.rows[r] = -1;
}

// ---------------------------------------------------------------------------
// moe_combine_rows: a thread owns V neighbouring values of one token's output
// and adds that token's rows in slot order (no atomics, a fixed order). Bound
// by HBM: eight rows' loads in flight, as loads of what is read once (8192
// tokens of 8 rows of 2048: 58 us row by row, 49.9 with eight in flight, 46.0
// with read-once loads, 7.3 TB/s). It lets no dependent launch start early: the
// next one's CTAs would take this one's places (49.9 us then). With few rows a
// token the writes and the residual are most of the traffic: 16384 tokens of one
// row of 2592 50 to 59 us, 5 TB/s (83 with registers for eight rows and an uneven
// second CTA); two or four tokens a thread are no faster (50, 53).
// ---------------------------------------------------------------------------
struct CombineParams {
  const uint16_t* y;
  const int32_t* slots;
  const float* w;
  const uint16_t* residual;   // or null
  uint16_t* out;
  int k, H, R;
  int nb;                     // CTAs a token
};

constexpr int kCombineThreads = 256;
constexpr int kCombineBatch = 8;

// B: rows in flight at once, the power of two at or above k up to
// kCombineBatch: few rows then take few registers (64 at B = 8, 40 at 1) and
// more threads share an SM.
template <int V, int B>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_rows(const CombineParams p) {
  const int t = blockIdx.x / p.nb;
  const int v = (blockIdx.x % p.nb) * blockDim.x + threadIdx.x;
  pdl_wait();
  if (v >= p.H / V) return;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  const int32_t* slots = p.slots + (size_t)t * p.k;
  const float* w = p.w + (size_t)t * p.k;
  const size_t at = (size_t)t * p.H + (size_t)v * V;
  typename RowVec<V>::Raw res{};
  if (p.residual) res = RowVec<V>::once(p.residual + at);
  for (int j0 = 0; j0 < p.k; j0 += B) {
    // a batch of rows in flight at once; absent ones weigh nothing
    int q[B];
    float wj[B];
    typename RowVec<V>::Raw y[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      q[j] = j0 + j < p.k ? slots[j0 + j] : -1;
      if (q[j] >= p.R) q[j] = -1;
      wj[j] = q[j] >= 0 ? w[j0 + j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (q[j] >= 0) y[j] = RowVec<V>::once(p.y + (size_t)q[j] * p.H + (size_t)v * V);
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (q[j] >= 0) {
        float f[V];
        RowVec<V>::values(y[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(wj[j], f[i], acc[i]);
      }
  }
  float r[V];
  RowVec<V>::values(res, r);
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] += r[i];
  RowVec<V>::store(p.out + at, acc);
}

}  // namespace moe
