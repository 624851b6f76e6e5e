// Dense matrix products of bf16 rows with bias, activation and residual in the
// epilogue, on the tensor cores (tcgen05.mma kind::f16, FP32 accumulators in
// tensor memory, operands staged by TMA).
//
// Operands are swapped, as in the grouped product: weight rows are the MMA's M
// dimension and the caller's rows its N dimension, so that a handful of rows
// still fills a tile and a call's rows can be cut to any multiple of 16.
//
//   moe_dense_tiles  many rows: a persistent pair of CTAs (cta_group::2) a pair
//                    of SMs over tiles of 256 weight rows by up to 256 rows
//   moe_dense_split  few rows: a cluster of CTAs (cta_group::1) a tile of 128
//                    weight rows, each over a part of K; the parts meet in
//                    distributed shared memory and are added in a fixed order
#pragma once

#include <cuda.h>

#include <cstdint>

#include "moe_block.h"
#include "moe_device.cuh"
#include "moe_product.cuh"
#include "moe_tcgen05.cuh"

namespace moe {

constexpr int kDenseRows = 128;   // weight rows a CTA
constexpr int kDenseK = 64;       // K elements a stage: one 128-byte swizzle row
constexpr int kDenseABytes = kDenseRows * kDenseK * 2;
constexpr int kDenseCols = 256;   // rows of x a tile of moe_dense_tiles, at most

struct DenseParams {
  // boxes of 128 rows; with SILU_MUL of 64 (split), or (tiles) [groups of 16][gate,
  // up][16 rows] in boxes of four groups, or where I is no multiple of 16, of 16 rows
  CUtensorMap tm_w;
  CUtensorMap tm_x;          // boxes of nt / 2 rows (tiles), nt rows (split)
  // out and residual in boxes of 32 rows by 64 (tiles with bf16 outputs and vec)
  CUtensorMap tm_out, tm_res;
  const uint16_t* bias;      // [N] or null
  const uint16_t* residual;  // [R, M] or null
  void* out;                 // [R, M]
  uint32_t* err;
  int R, M, nk;              // nk: stages K takes
  int act, out_float;        // (out_float: split)
  int vec;                   // rows of out and residual take 16-byte accesses
  int nt;                    // rows of x a tile
  int mt, tt;                // tiles along M and R
  int stages;                // of the ring
  int groups;                // tm_w has the groups of 16 (tiles, SILU_MUL)
  uint32_t polls;            // of a bounded wait: kMbarPolls
  uint32_t withheld;         // 1: stages lack an arrival, so that waits run out (tests)
};

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------

// SiLU with e = exp(-|v|) <= 1: nothing overflows, and the divisor stays where
// the short division is good to two units. The short exp is off by 2 + 1.2 |v|
// units of 2^-23.
__device__ __forceinline__ float dense_silu(float v) {
  const float e = __expf(-fabsf(v));
  return __fdividef(v < 0.f ? v * e : v, 1.f + e);
}
// v (1 + tanh z) / 2 = v sigmoid(2 z), the same way
__device__ __forceinline__ float dense_gelu_tanh(float v) {
  const float z2 = 1.5957691216057308f * v * fmaf(0.044715f * v, v, 1.f);
  const float e = __expf(-fabsf(z2));
  return __fdividef(z2 < 0.f ? v * e : v, 1.f + e);
}
// v (1 + erf(v / sqrt 2)) / 2 from erfc(z), z = |v| / sqrt 2: v erfc(z) / 2 below zero,
// where 1 + erf cancels (6 % of the result at -5, all of it from -5.5 on), v - v erfc(z) / 2
// above. e^(z^2) erfc(z) is a polynomial in t = 1 / (1 + 0.55 z) times t (the variable of
// Schonfelder's expansions, Math. Comp. 32, 1978; the coefficients are a relative
// least-squares fit of our own over z <= 10, off by 7e-9), in powers of t - 9/16: 4 units
// of 2^-24 with FP32's rounding. (1001 x 2080 x 2056 with a residual and 8192 x 2048 x
// 2048: 13.5 and 44.4 us, with erfcf 15.2 and 52.9, with the cancelling erff 13.0 and 44.0.)
__device__ __forceinline__ float dense_gelu(float v) {
  const float a = fminf(fabsf(v), 16.f);   // e^(-a^2 / 2) is 0 there
  const float t = __fdividef(1.f, fmaf(a, 0.388908744f, 1.f));
  const float s = t - 0.5625f;
  float r = 5.804775655e-02f;
  r = fmaf(r, s, -4.279274493e-02f);
  r = fmaf(r, s, -7.251586765e-02f);
  r = fmaf(r, s, 1.079753712e-01f);
  r = fmaf(r, s, 5.148212239e-02f);
  r = fmaf(r, s, -2.026180327e-01f);
  r = fmaf(r, s, -6.769769639e-02f);
  r = fmaf(r, s, 4.481518269e-01f);
  r = fmaf(r, s, 7.503036857e-01f);
  r = fmaf(r, s, 5.977187753e-01f);
  r *= t * exp2f(a * a * -0.72134751f);
  const float w = 0.5f * (v < 0.f ? v : a) * r;
  return v < 0.f ? w : v - w;   // (infinity and NaN stay what they are, -infinity is NaN)
}
// (NaN stays NaN)
__device__ __forceinline__ float dense_relu(float v) { return v < 0.f ? 0.f : v; }

// One switch for all of a thread's values.
template <int N>
__device__ __forceinline__ void dense_act(int act, float (&v)[N]) {
  if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = dense_relu(v[i]);
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = dense_silu(v[i]);
  } else if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = dense_gelu(v[i]);
  } else if (act == MOE_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = dense_gelu_tanh(v[i]);
  }
}

__device__ __forceinline__ float bf16_at(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

namespace tc {

// D (+)= A * B^T, both in shared memory, over both CTAs of a pair or in one.
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t" MOE_ELECT
        ".reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t" MOE_ELECT
        ".reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f16: FP32 D, bf16 A and B, both K-major.
__device__ __forceinline__ uint32_t f16_idesc(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void commit1(uint64_t* bar) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma1_load_2d(void* dst, const void* tmap, int x, int y,
                                             uint64_t* bar) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// A box from shared memory to a tensor, one of the issuing thread's bulk groups.
// Every lane may close and wait for groups: but for the elected one's they are empty.
__device__ __forceinline__ void tma_store_2d(const void* tmap, int x, int y, const void* src) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t}" ::"l"(tmap),
      "r"(x), "r"(y), "r"(smem_addr(src))
      : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ void tma2_load_4d(void* dst, const void* tmap, int c0, int c1, int c2,
                                             int c3, uint32_t bar) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// The inverse of stm4_trans.
__device__ __forceinline__ void ldm4_trans(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

}  // namespace tc

// The two halves of cluster_sync().
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// The first half without its release, which waits for this thread's stores to
// global memory too. What has to be seen goes ahead by a fence of its own.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
// Earlier writes to this CTA's shared memory, before a relaxed arrival.
__device__ __forceinline__ void release_shared() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}

// A whole warp's bounded wait on a phase of this CTA's mbarrier; a timeout
// marks the CTA dead, and with PAIR the other one of its pair (every role winds
// down).
template <bool PAIR>
__device__ __forceinline__ bool dense_wait(uint64_t* bar, uint32_t parity, const DenseParams& p,
                                           volatile int* dead) {
  constexpr Arrivals A = PAIR ? Arrivals::kPair : Arrivals::kOwn;
  if (__all_sync(kFull, prod_look<A>(bar, parity))) return true;
#pragma unroll 1
  for (uint32_t it = 0; it < p.polls; ++it) {
    if (__any_sync(kFull, *dead)) return false;
    if (__all_sync(kFull, prod_poll<A>(bar, parity))) return true;
  }
  atomicOr(p.err, kDeviceTimeout);
  *dead = 1;
  if constexpr (PAIR)
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(
                     tc::cluster_addr(const_cast<int*>(dead), (blockIdx.x & 1) ^ 1))
                 : "memory");
  return false;
}

// ---------------------------------------------------------------------------
// moe_dense_tiles. Roles:
//   warp 0      weights and rows by TMA
//   warp 1      (first CTA) the MMAs of both CTAs
//   warps 4-11  epilogue, one per lane quarter of tensor memory, two groups of
//               four that take chunks of 32 rows in turn
// Two accumulators in tensor memory let the epilogue of a tile overlap the next
// tile's MMAs. With SILU a tile is 128 neurons' gate and up rows, 16 and 16 in turn,
// so that each epilogue warp has a neuron's gate and up in one thread.
//
// The tensor cores cut a sum off at each step of 16 K instead of rounding it, which
// adds up along K (relative error of 8191 x 7168 x 256 by its 2-norm: 7.9e-6, of FP32
// FMAs 0.9e-6). bf16 outputs take all of a CTA's K in one accumulator all the same, as
// the library's products do: their error is 1.7e-3 and grows by less than 1e-4 of it, but
// at K = 7168 a sum lies on the other side of a rounding boundary in one output of 250,
// with SiLU(gate) * up of 140, which is then the neighbouring bf16 value (the 2-norm
// of these differences is 2e-4 and 3e-4; FP32 FMAs: 0.6e-4 and 0.8e-4). Where the
// outputs are FP32 (FLOAT), the sums of kDensePart stages in turn are added up in
// registers: 0.5e-6 with eight stages, 1.0e-6 with 16, in the same time.
// ---------------------------------------------------------------------------
constexpr int kDenseThreads = 384;
constexpr int kDensePart = 8;                  // stages
constexpr int kDenseFloatCols = 128;           // rows of x a tile with FLOAT, at most
constexpr int kDenseChunk = 32 * 256;   // epilogue staging: 32 rows of 128 bf16

constexpr int kDenseStages = 12;        // of the ring, at most
constexpr int kDenseSmemMax = 232448 - 1024;

// The ring takes what the epilogue's chunks leave: a slot's way from the MMA's
// release through a copy back to the MMA takes more than a microsecond, and narrow
// tiles' stages are small (router logits of 8191 x 7168 x 256 in tiles of 128 rows:
// 30.4 us with six stages, 27.5 with eight, 28.7 with the sums of FP32 outputs).
struct DenseSmem {
  static constexpr int out = 0;                     // [2 groups][2] chunks
  static constexpr int bars = out + 4 * kDenseChunk;
  static constexpr int ring = bars + 1024;
  __host__ __device__ static constexpr int stage(int nt) { return kDenseABytes + nt / 2 * kDenseK * 2; }
  __host__ __device__ static constexpr int stages(int nt) {
    return (kDenseSmemMax - ring) / stage(nt) < kDenseStages ? (kDenseSmemMax - ring) / stage(nt)
                                                             : kDenseStages;
  }
};
static_assert((2 * kDenseStages + 10) * 8 + 16 <= 1024, "barriers");
static_assert(DenseSmem::stages(kDenseCols) >= 6, "ring");

// Tile i of a call: bands of kDenseBand token tiles, within a band all token
// tiles of a weight tile in turn, so that pairs side by side share both
// operands in L2.
constexpr int kDenseBand = 8;
__device__ __forceinline__ void dense_tile(const DenseParams& p, int i, int& m, int& t) {
  const int band = i / (kDenseBand * p.mt), j = i - band * kDenseBand * p.mt;
  const int g = min(kDenseBand, p.tt - band * kDenseBand);
  m = j / g;
  t = band * kDenseBand + j - m * g;
}

template <bool SILU, bool FLOAT>
__global__ void __launch_bounds__(kDenseThreads, 1) moe_dense_tiles(
    const __grid_constant__ DenseParams p) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  using L = DenseSmem;
  constexpr int kOut = SILU ? kDenseRows / 2 : kDenseRows;   // outputs of a CTA's tile
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);   // used in the first CTA
  uint64_t* empty = full + kDenseStages;
  uint64_t* d_full = empty + kDenseStages;
  uint64_t* d_empty = d_full + 2;                                 // used in the first CTA
  uint64_t* drain = d_empty + 2;
  uint64_t* allocated = drain + 1;                                // used in the first CTA
  uint64_t* res_full = allocated + 1;                             // [2 groups][2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + 4);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;   // clusters are pairs of neighbours
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int tiles = p.mt * p.tt;
  const int stages = p.stages, stage_bytes = L::stage(p.nt);
  uint8_t* ring = smem + L::ring;

  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&p.tm_w);
    tc::prefetch_tmap(&p.tm_x);
    if (!FLOAT && p.vec) {
      tc::prefetch_tmap(&p.tm_out);
      if (p.residual) tc::prefetch_tmap(&p.tm_res);
    }
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1 + p.withheld);   // the announcement of both CTAs' bytes
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 16);   // both CTAs' epilogue warps
    }
    mbar_init(drain, 1);
    mbar_init(allocated, 2);
    for (int i = 0; i < 4; ++i) mbar_init(&res_full[i], 1);
    *dead = 0;
    mbar_init_fence();
    release_shared();
  }
  __syncwarp();
  // The copies wait for both CTAs' barriers, but not for tensor memory, nor, below,
  // the end for outputs on their way: with a barrier that does, 1001 x 2080 x 2056
  // took 12.5 us instead of 12.3, 256 x 2048 x 7168 13.6 instead of 13.1.
  cluster_arrive_relaxed();
  if (warp == 1) tc::tmem_alloc2(tmem_slot, 512);
  cluster_wait();   // the other CTA's barriers are ready too
  pdl_trigger();    // the next kernel's prologue may run beside this one
  // all of tensor memory is this CTA's, so its columns start at 0

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    RingPos rg(stages);
    const uint32_t full0 = tc::cluster_addr(full, 0);
    const int half = p.nt / 2;
    const uint32_t bytes = 2 * (kDenseABytes + half * kDenseK * 2);
    auto weights = [&](int s, int m, int kb) {
      uint8_t* dst = ring + s * stage_bytes;
      const int n = (2 * m + rank) * kOut;
      if (rank == 0) tc::expect(&full[s], bytes);
      if constexpr (!SILU) {
        tc::tma2_load_2d(dst, &p.tm_w, kb * kDenseK, n, full0 + 8 * s);
      } else if (p.groups) {
        tc::tma2_load_4d(dst, &p.tm_w, kb * kDenseK, 0, 0, n / 16, full0 + 8 * s);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tc::tma2_load_2d(dst + i * 16 * 128, &p.tm_w, kb * kDenseK,
                           n + 16 * (i >> 1) + (i & 1) * p.M, full0 + 8 * s);
      }
    };
    // the first stages' weights, which no earlier kernel writes, come before the
    // wait for the kernels before this one
    int ahead = 0, m, t;
    if (first < tiles) {
      dense_tile(p, first, m, t);
      for (; ahead < min(p.nk, stages); ++ahead) weights(ahead, m, ahead);
    }
    pdl_wait();
    int g = 0;
    bool ok = true;
    for (int i = first; ok && i < tiles; i += step) {
      dense_tile(p, i, m, t);
      const int r0 = t * p.nt + rank * half;
      for (int kb = 0; kb < p.nk; ++kb, ++g) {
        const int s = rg.slot;
        if (g >= stages && !dense_wait<true>(&empty[s], rg.phase ^ 1u, p, dead)) {
          ok = false;
          break;
        }
        if (g >= ahead) weights(s, m, kb);
        tc::tma2_load_2d(ring + s * stage_bytes + kDenseABytes, &p.tm_x, kb * kDenseK, r0, full0 + 8 * s);
        rg.next();
      }
    }
    // every arrival that the first CTA's MMAs make here, before this one may leave
    if (g < stages) rg.slot = 0, rg.phase = 1u;
    for (int j = 0; ok && j < min(g, stages); ++j) {
      ok = dense_wait<true>(&empty[rg.slot], rg.phase ^ 1u, p, dead);
      rg.next();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    tc::fence_before();
    tc::arrive_at(tc::cluster_addr(allocated, 0), rank != 0);
    if (rank == 0) {
      pdl_wait();   // no bounded wait begins before the kernels before this one end
      RingPos rg(stages);
      const uint32_t idesc = tc::f16_idesc(2 * kDenseRows, p.nt);
      int lt = 0;   // accumulators filled
      bool ok = dense_wait<true>(allocated, 0, p, dead);
      tc::fence_after();
      for (int i = first, k0 = 0; ok && i < tiles; ++lt) {
        const int buf = lt & 1;
        if (lt >= 2) ok = dense_wait<true>(&d_empty[buf], ((lt >> 1) - 1) & 1, p, dead);
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = buf * 256;
        const int k1 = FLOAT ? min(k0 + kDensePart, p.nk) : p.nk;
        for (int kb = k0; kb < k1; ++kb) {
          const int s = rg.slot;
          ok = dense_wait<true>(&full[s], rg.phase, p, dead);
          if (!ok) break;
          const uint32_t base = smem_addr(ring + s * stage_bytes);
          const uint64_t ad = tc::sdesc_sw128(base), bd = tc::sdesc_sw128(base + kDenseABytes);
#pragma unroll
          for (int q = 0; q < kDenseK / 16; ++q)   // 32 bytes further in the swizzled rows
            tc::mma_f16<true>(d, ad + 2 * q, bd + 2 * q, idesc, kb > k0 || q > 0 ? 1u : 0u);
          tc::commit2(&empty[s]);
          rg.next();
        }
        if (ok) tc::commit2(&d_full[buf]);
        k0 = k1;
        if (k0 == p.nk) k0 = 0, i += step;
      }
      tc::commit2(drain);
    }
  } else if (FLOAT && warp >= 4) {
    // ------------------------------------------------- epilogue, FP32 outputs
    const int q = warp & 3, et = threadIdx.x & 127, grp = (warp >> 2) - 1;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t d_empty0 = tc::cluster_addr(d_empty, 0);
    // a chunk of 32 rows of x by kOut outputs, turned in shared memory: column c of
    // row r lies at c ^ 8 ((r / 2) mod 4), so that the eight columns and four rows of
    // a warp's store lie in different banks
    float* turn = reinterpret_cast<float*>(smem + L::out + grp * 2 * kDenseChunk);
    constexpr int kPieces = kOut / 4, kRows = 128 / kPieces;
    const int pc = et & (kPieces - 1), pr = et / kPieces;
    const int sums_all =
        first < tiles ? ((tiles - 1 - first) / step + 1) * ((p.nk + kDensePart - 1) / kDensePart) : 0;
    int lt = 0;
    pdl_wait();
    for (int i = first; i < tiles; i += step) {
      int m, t;
      dense_tile(p, i, m, t);
      const int n0 = (2 * m + rank) * kOut, r0 = t * p.nt;
      const int n = min(p.nt, p.R - r0);
      // the tile's chunks 32 grp and 64 further; registers as in the epilogue below
      float sum[2][2][16];
#pragma unroll
      for (int x = 0; x < 64; ++x) sum[x >> 5][(x >> 4) & 1][x & 15] = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int k0 = 0; k0 < p.nk; k0 += kDensePart, ++lt) {
        const int buf = lt & 1;
        ok = dense_wait<true>(&d_full[buf], (lt >> 1) & 1, p, dead);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int c0 = 32 * grp + 64 * c;
          if (c0 >= n) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t raw[16];
            tc::ld_16x32(lanes + ((uint32_t)(16 * h) << 16) + buf * 256 + c0, raw);
            tc::wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) sum[c][h][x] += __uint_as_float(raw[x]);
          }
        }
        tc::fence_before();
        __syncwarp();
        // (to the last two nobody listens, nor would anyone wait for their way)
        if (lt + 2 < sums_all) tc::arrive_at(d_empty0 + 8 * buf, rank != 0);
      }
      // (a group's warps go on or leave together)
      if (!named_all(1 + grp, 128, ok)) break;
      float bias[4] = {};
      if (p.bias) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = SILU ? n0 + 16 * q + 8 * (k & 1) + (lane >> 2)
                               : n0 + 32 * q + 8 * k + (lane >> 2);
          if (row < p.M) bias[k] = bf16_at(p.bias + row + (SILU && k > 1 ? p.M : 0));
        }
      }
      float* out = static_cast<float*>(p.out);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int c0 = 32 * grp + 64 * c;
        if (c0 >= n) continue;
#pragma unroll
        for (int h = 0; h < (SILU ? 1 : 2); ++h) {
          float v[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            v[x] = sum[c][h][x] + bias[2 * h + ((x >> 1) & 1)];
            if constexpr (SILU) v[x] = dense_silu(v[x]) * (sum[c][1][x] + bias[2 + ((x >> 1) & 1)]);
          }
          if constexpr (!SILU) dense_act(p.act, v);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int row = 8 * (x >> 2) + 2 * (lane & 3) + (x & 1);
            const int col = kOut / 4 * q + 16 * h + 8 * ((x >> 1) & 1) + (lane >> 2);
            turn[row * kOut + (col ^ ((lane & 3) << 3))] = v[x];
          }
        }
        named_sync(1 + grp, 128);
        const int col = n0 + 4 * pc;
#pragma unroll
        for (int k = 0; k < 32 / kRows; ++k) {
          const int row = pr + kRows * k;
          if (c0 + row >= n || col >= p.M) continue;
          float4 w = *reinterpret_cast<const float4*>(
              turn + row * kOut + ((4 * pc) ^ (((row >> 1) & 3) << 3)));
          const size_t at = (size_t)(r0 + c0 + row) * p.M + col;
          if (p.vec) {
            if (p.residual) {
              const uint2 r = *reinterpret_cast<const uint2*>(p.residual + at);
              w.x += bf16_lo(r.x), w.y += bf16_hi(r.x), w.z += bf16_lo(r.y), w.w += bf16_hi(r.y);
            }
            *reinterpret_cast<float4*>(out + at) = w;
          } else {
            const float e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (col + j < p.M) out[at + j] = e[j] + (p.residual ? bf16_at(p.residual + at + j) : 0.f);
          }
        }
        named_sync(1 + grp, 128);   // the chunk's place is free again
      }
    }
  } else if (!FLOAT && warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, et = threadIdx.x & 127;
    const int grp = (warp >> 2) - 1;
    const int bar = 1 + grp;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t d_empty0 = tc::cluster_addr(d_empty, 0);
    // a chunk: 32 rows of x by kOut outputs, in blocks of 64 outputs: 16-byte piece i
    // of row r sits at i ^ (r & 7) of 128 bytes, as the copies' swizzle has it
    constexpr int kBlocks = kOut / 64, kBlockBytes = 32 * 128;
    // its row of the matrices that turn 32 columns of tensor memory into rows: piece
    // 4 q + i (with SILU 2 q + i) holds outputs 8 i.. of this warp's. Without SILU
    // matrix m of four is output group m, with SILU m & 1 of rows 8 (m >> 1) further
    const int mr = lane & 7, mm = lane >> 3;
    const uint32_t mat =
        SILU ? (8 * (mm >> 1) + mr) * 128 + (((2 * q + (mm & 1)) ^ mr) << 4)
             : (q >> 1) * kBlockBytes + mr * 128 + (((4 * (q & 1) + mm) ^ mr) << 4);
    // The group's first warp copies chunks in and out (vec): the residual's come a
    // chunk ahead, onto the place that the results leave from. (By registers and the
    // threads' own loads and stores 4096 x 768 x 2048 with a residual took 17.4 us
    // instead of 15.6, 1001 x 2080 x 2056 12.9 instead of 12.5, 8192 x 2048 x 7168
    // under load 152.4 instead of 151.3.)
    auto place = [&](int ch) { return smem + L::out + (2 * grp + (ch & 1)) * kDenseChunk; };
    auto ask = [&](int ch, int n0, int row) {
      uint64_t* landed = res_full + 2 * grp + (ch & 1);
      tc::expect(landed, kBlocks * kBlockBytes);
#pragma unroll
      for (int h = 0; h < kBlocks; ++h)
        tc::tma1_load_2d(place(ch) + h * kBlockBytes, &p.tm_res, n0 + 64 * h, row, landed);
    };
    // else a thread moves piece pc of rows pr + kRows k
    constexpr int kPieces = kOut / 8, kRows = 128 / kPieces, kMoves = 32 / kRows;
    const int pc = et & (kPieces - 1), pr = et / kPieces;
    const uint32_t moved = (pc >> 3) * kBlockBytes + pr * 128 + (((pc ^ pr) & 7) << 4);   // (kRows is a multiple of 8)
    int lt = 0, chunk = 0;
    bool ok = true;
    pdl_wait();
    for (int i = first; i < tiles; i += step, ++lt) {
      int m, t;
      dense_tile(p, i, m, t);
      const int n0 = (2 * m + rank) * kOut, r0 = t * p.nt;
      const int n = min(p.nt, p.R - r0), pn = n0 + 8 * pc;
      const int buf = lt & 1;
      // bias of this thread's weight rows 8 k + lane / 4 of the warp's 32 (with SILU the
      // last two are its neurons' up rows)
      float bias[4] = {};
      if (p.bias) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = SILU ? n0 + 16 * q + 8 * (k & 1) + (lane >> 2)
                               : n0 + 32 * q + 8 * k + (lane >> 2);
          if (row < p.M) bias[k] = bf16_at(p.bias + row + (SILU && k > 1 ? p.M : 0));
        }
      }
      if (p.residual && p.vec && q == 0 && ok) {
        tc::store_wait_read();   // both places are free
        if (32 * grp < n) ask(chunk, n0, r0 + 32 * grp);
        if (32 * grp + 64 < n) ask(chunk + 1, n0, r0 + 32 * grp + 64);
      }
      ok = dense_wait<true>(&d_full[buf], (lt >> 1) & 1, p, dead) && ok;
      // a group's warps go on or leave together: no named barrier below waits
      // for a warp that gave up
      ok = named_all(bar, 128, ok);
      if (!ok) break;
      tc::fence_after();
      for (int c0 = 32 * grp; c0 < n; c0 += 64, ++chunk) {
        uint8_t* stage = place(chunk);
        // register 4 b + 2 i + j of the two halves: weight row 8 i + lane / 4 (16
        // further in the second), row 8 b + 2 (lane % 4) + j of x
        constexpr int kVals = SILU ? 16 : 32;
        uint32_t raw[2][16];
        float v[kVals];
        tc::ld_16x32(lanes + buf * 256 + c0, raw[0]);
        tc::ld_16x32(lanes + (16u << 16) + buf * 256 + c0, raw[1]);
        tc::wait_ld();
        if constexpr (SILU) {
#pragma unroll
          for (int x = 0; x < 16; ++x)
            v[x] = dense_silu(__uint_as_float(raw[0][x]) + bias[(x >> 1) & 1]) *
                   (__uint_as_float(raw[1][x]) + bias[2 + ((x >> 1) & 1)]);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            v[x] = __uint_as_float(raw[x >> 4][x & 15]) + bias[2 * (x >> 4) + ((x >> 1) & 1)];
          dense_act(p.act, v);
        }
        // value of pair k (of two rows of x) of matrix set b: four matrices a set
        auto at = [](int b, int k) {
          return SILU ? 8 * b + 4 * (k >> 1) + 2 * (k & 1) : 16 * (k >> 1) + 4 * b + 2 * (k & 1);
        };
        constexpr int kSets = kVals / 8;
        constexpr uint32_t kSetBytes = (SILU ? 16 : 8) * 128;
        const uint32_t mats = smem_addr(stage) + mat;
        // the other place is free once its results have left
        if (p.vec && q == 0) {
          tc::store_wait_read();
          if (p.residual && ok && c0 >= 64 && c0 + 64 < n) ask(chunk + 1, n0, r0 + c0 + 64);
        }
        if (p.residual) {
          if (p.vec) {
            // (a timeout marks the pair dead; the group leaves together at its next tile)
            ok = dense_wait<true>(&res_full[2 * grp + (chunk & 1)], (chunk >> 1) & 1, p, dead) && ok;
          } else {
#pragma unroll
            for (int k = 0; k < kMoves; ++k) {
              const int row = c0 + pr + kRows * k;
              uint32_t w[4] = {};
              if (row < n) {
                const uint16_t* src = p.residual + (size_t)(r0 + row) * p.M + pn;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[j] = (pn + 2 * j < p.M ? src[2 * j] : 0u) |
                         (pn + 2 * j + 1 < p.M ? (uint32_t)src[2 * j + 1] << 16 : 0u);
              }
              *reinterpret_cast<uint4*>(stage + moved + k * kRows * 128) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            named_sync(bar, 128);
          }
#pragma unroll
          for (int b = 0; b < kSets; ++b) {
            uint32_t w[4];
            tc::ldm4_trans(mats + b * kSetBytes, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[at(b, k)] += bf16_lo(w[k]);
              v[at(b, k) + 1] += bf16_hi(w[k]);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < kSets; ++b) {
          auto pack = [&](int k) { return RowVec<8>::pack(v[at(b, k)], v[at(b, k) + 1]); };
          tc::stm4_trans(mats + b * kSetBytes, pack(0), pack(1), pack(2), pack(3));
        }
        if (p.vec) {
          tc::fence_proxy_async();
          named_sync(bar, 128);
          if (q == 0) {
#pragma unroll
            for (int h = 0; h < kBlocks; ++h)
              if (n0 + 64 * h < p.M)
                tc::tma_store_2d(&p.tm_out, n0 + 64 * h, r0 + c0, stage + h * kBlockBytes);
            tc::store_commit();
          }
        } else {
          named_sync(bar, 128);
          uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
          for (int k = 0; k < kMoves; ++k) {
            const int row = c0 + pr + kRows * k;
            if (row >= n) continue;
            const uint4 w = *reinterpret_cast<const uint4*>(stage + moved + k * kRows * 128);
            uint16_t* dst = out + (size_t)(r0 + row) * p.M + pn;
            const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (pn + j < p.M) dst[j] = (uint16_t)(e[j >> 1] >> (16 * (j & 1)));
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      // (as above)
      if (i + 2 * step < tiles) tc::arrive_at(d_empty0 + 8 * buf, rank != 0);
    }
    if (q == 0) tc::store_wait_read();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  // as in moe_product_tiles: before a CTA leaves and tensor memory is released,
  // every MMA is done, and with them every copy into a stage that they read,
  // which is all there are unless the pair is dead. Then copies may still be in
  // flight, and both CTAs stay for a time that is hundreds of times a copy's.
  if (warp == 1) prod_wait_end(drain, 0, p.err);
  if (warp == 0 && *dead)
    for (int i = 0; i < kProdSettleSleeps; ++i) __nanosleep(kWaitSuspendNs);
  __syncwarp();
  // No CTA leaves while the other may still reach into it: arrivals from there have
  // been waited for, MMAs are done (allocated, d_empty, empty, d_full, drain).
  cluster_arrive_relaxed();
  cluster_wait();
  tc::fence_after();
  if (warp == 1) tc::tmem_dealloc2(*tmem_slot, 512);
}

// ---------------------------------------------------------------------------
// moe_dense_split. One tile of 128 weight rows (with SILU 64 gate rows and their
// 64 up rows) by nt rows of x a cluster; CTA j of its S takes the j-th part of K.
// Warps 0-7 are the epilogue, two per lane quarter of tensor memory, warp 8
// copies, warp 9 issues the MMAs. Each part's sums go to the CTA that finishes the
// row of x they belong to (row r: CTA r mod S), which adds them in the order of the
// parts. (They go as stores to its shared memory: bulk copies from the CTA's own,
// 0.35 us more for 1 to 16 rows, gained nothing up to 1000.)
// ---------------------------------------------------------------------------
constexpr int kSplitEpilogue = 256;   // threads
constexpr int kSplitThreads = kSplitEpilogue + 64;
constexpr int kSplitMaxCols = 128;
constexpr int kSplitBars = 1024;   // bytes kept for barriers in front of the ring
constexpr int kSplitStages = 16;   // of the ring, at most

__host__ __device__ constexpr int split_stage_bytes(int nt) { return kDenseABytes + nt * kDenseK * 2; }
// Columns of an accumulator, and how many half of tensor memory holds.
__host__ __device__ constexpr int split_cols(int nt) { return nt <= 32 ? 32 : nt <= 64 ? 64 : 128; }
__host__ __device__ constexpr int split_accs(int nt) { return 256 / split_cols(nt); }
// What the parts of a tile's sums take in the CTAs that add them (a single part
// takes the ring's place, which is free then).
__host__ __device__ constexpr int split_sum_bytes(int nt, int S) {
  return S > 1 ? (nt + S - 1) / S * S * kDenseRows * 4 : 0;
}

// The results of outputs m.. m + 7 for row r of x from their sums v, with SILU the
// gates', and up; rows of out and residual in 16-byte accesses with p.vec.
template <bool SILU>
__device__ __forceinline__ void split_finish(const DenseParams& p, size_t r, int m, float (&v)[8],
                                             const float (&up)[8], const float (&bias)[8],
                                             const float (&up_bias)[8]) {
  const size_t at = r * p.M + m;
  float res[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) res[i] = 0.f;
  if (p.residual) {
    if (p.vec) {
      RowVec<8>::load(p.residual + at, res);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (m + i < p.M) res[i] = bf16_at(p.residual + at + i);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += bias[i];
  if constexpr (SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = dense_silu(v[i]) * (up[i] + up_bias[i]);
  } else {
    dense_act(p.act, v);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += res[i];
  if (p.out_float) {
    float* out = static_cast<float*>(p.out) + at;
    if (p.vec) {
      *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (m + i < p.M) out[i] = v[i];
    }
  } else {
    uint16_t* out = static_cast<uint16_t*>(p.out) + at;
    if (p.vec) {
      RowVec<8>::store(out, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (m + i < p.M) out[i] = f32_to_bf16_rn(v[i]);
    }
  }
}

template <bool SILU>
__global__ void __launch_bounds__(kSplitThreads) moe_dense_split(
    const __grid_constant__ DenseParams p, const int log_parts) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  constexpr int kTile = SILU ? kDenseRows / 2 : kDenseRows;   // outputs a tile
  const int S = 1 << log_parts;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kSplitStages;
  uint64_t* d_full = empty + kSplitStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(d_full + 1);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* ring = smem + kSplitBars;
  const int stage = split_stage_bytes(p.nt);
  // rows of x that a CTA finishes, and the parts of their sums [S][slots][128]
  const int slots = (p.nt + S - 1) >> log_parts;
  float* sums = reinterpret_cast<float*>(ring + (S > 1 ? p.stages * stage : 0));

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x & (S - 1), tile = blockIdx.x >> log_parts;
  const int m = tile % p.mt, t = tile / p.mt;
  const int n0 = m * kTile, r0 = t * p.nt;
  const int n = min(p.nt, p.R - r0);
  const int k0 = (int)((int64_t)p.nk * rank >> log_parts);
  const int k1 = (int)((int64_t)p.nk * (rank + 1) >> log_parts);
  const uint32_t tcols = split_cols(p.nt);
  // FP32 outputs: accumulators side by side take kDensePart stages each, at most as many
  // as half of tensor memory holds (two CTAs may share an SM's); a CTA's part of K is no
  // longer than that (plan_dense). 2 x 5816 x 316: error 1.1e-6 -> 0.5e-6, 3.9 -> 4.0 us.
  const int accs = p.out_float ? min((k1 - k0 + kDensePart - 1) / kDensePart, split_accs(p.nt)) : 1;
  const int acc_stages = (k1 - k0 + accs - 1) / accs;
  const uint32_t all_cols = tcols << (accs > 4 ? 3 : accs > 2 ? 2 : accs > 1 ? 1 : 0);

  if (warp == 8 && lane == 0) {
    tc::prefetch_tmap(&p.tm_w);
    tc::prefetch_tmap(&p.tm_x);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1 + p.withheld);
      mbar_init(&empty[i], 1);
    }
    mbar_init(d_full, 1);
    *dead = 0;
    mbar_init_fence();
  }
  if (warp == 9) tc::tmem_alloc(tmem_slot, all_cols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  if (S > 1) cluster_arrive();   // this CTA runs: others may write to it

  if (warp == 8) {
    RingPos rg(p.stages);
    const uint32_t bytes = stage;
    auto weights = [&](int s, int kb) {
      tc::expect(&full[s], bytes);
      tc::tma1_load_2d(ring + s * stage, &p.tm_w, kb * kDenseK, n0, &full[s]);
      if (SILU)
        tc::tma1_load_2d(ring + s * stage + kDenseABytes / 2, &p.tm_w, kb * kDenseK, p.M + n0,
                         &full[s]);
    };
    // weights, which no earlier kernel writes, before the wait for earlier kernels
    const int ahead = min(k1 - k0, p.stages);
    for (int g = 0; g < ahead; ++g) weights(g, k0 + g);
    pdl_wait();
    for (int g = 0; g < k1 - k0; ++g) {
      const int s = rg.slot;
      if (g >= p.stages && !dense_wait<false>(&empty[s], rg.phase ^ 1u, p, dead)) {
        ok = false;
        break;
      }
      if (g >= ahead) weights(s, k0 + g);
      tc::tma1_load_2d(ring + s * stage + kDenseABytes, &p.tm_x, (k0 + g) * kDenseK, r0, &full[s]);
      rg.next();
    }
  } else if (warp == 9) {
    pdl_wait();   // as in moe_dense_tiles
    RingPos rg(p.stages);
    const uint32_t idesc = tc::f16_idesc(kDenseRows, p.nt);
    uint32_t d = tmem;
    for (int kb = k0, in = 0; kb < k1; ++kb, ++in) {
      if (in == acc_stages) in = 0, d += tcols;
      const int s = rg.slot;
      ok = dense_wait<false>(&full[s], rg.phase, p, dead);
      if (!ok) break;
      const uint32_t base = smem_addr(ring + s * stage);
      const uint64_t ad = tc::sdesc_sw128(base), bd = tc::sdesc_sw128(base + kDenseABytes);
#pragma unroll
      for (int q = 0; q < kDenseK / 16; ++q)
        tc::mma_f16<false>(d, ad + 2 * q, bd + 2 * q, idesc, in > 0 || q > 0 ? 1u : 0u);
      tc::commit1(&empty[s]);
      rg.next();
    }
    tc::commit1(d_full);   // in any case: nothing leaves before the MMAs are done
    prod_wait_end(d_full, 0, p.err);
  }
  __syncwarp();
  // The sums go through shared memory, from a thread a weight row to a thread eight
  // outputs of one row of x (a thread a weight row to the end, with its 2-byte
  // accesses, took 84 ns a row of x).
  constexpr int kGroups = kTile / 8;
  const int grp = threadIdx.x & (kGroups - 1), out_m = n0 + 8 * grp;
  float bias[8], up_bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = up_bias[i] = 0.f;
  if (warp < 8) {
    pdl_wait();
    if (p.residual) {
      // on its way to L2 while the products are made, 128 bytes a request (64 x 2048 x
      // 7168: 9.4 us instead of 9.75)
      if ((grp & 7) == 0 && out_m < p.M)
#pragma unroll 1
        for (int slot = threadIdx.x / kGroups; (slot << log_parts) + rank < n;
             slot += kSplitEpilogue / kGroups)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(__cvta_generic_to_global(
              p.residual + (size_t)(r0 + (slot << log_parts) + rank) * p.M + out_m)));
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (out_m + i < p.M) {
          bias[i] = bf16_at(p.bias + out_m + i);
          if (SILU) up_bias[i] = bf16_at(p.bias + p.M + out_m + i);
        }
    }
    ok = dense_wait<false>(d_full, 0, p, dead);
    ok = named_all(1, kSplitEpilogue, ok && !*dead);
    tc::fence_after();
    if (S > 1) cluster_wait();   // every CTA runs
    if (ok) {
#pragma unroll 1
      for (int c0 = 16 * (warp >> 2); c0 < n; c0 += 32) {
        uint32_t raw[16];
        const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + c0;
        tc::ld16(from, raw);
        tc::wait_ld();
#pragma unroll 1
        for (int a = acc_stages, i = 1; a < k1 - k0; a += acc_stages, ++i) {
          uint32_t more[16];
          tc::ld16(from + i * tcols, more);
          tc::wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            raw[j] = __float_as_uint(__uint_as_float(raw[j]) + __uint_as_float(more[j]));
        }
        float* to = sums + rank * slots * kDenseRows + (threadIdx.x & 127);
        if (S == 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) to[(c0 + j) * kDenseRows] = __uint_as_float(raw[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int r = c0 + j;
            if (r >= n) break;
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(tc::cluster_addr(
                             to + (r >> log_parts) * kDenseRows, r & (S - 1))),
                         "r"(raw[j])
                         : "memory");
          }
        }
      }
      tc::fence_before();
    }
  } else if (S > 1) {
    cluster_wait();
  }
  __syncwarp();
  if (S > 1)
    cluster_sync();   // the parts have landed, and no CTA reaches into another after it
  else
    __syncthreads();
  if (warp < 8 && ok && out_m < p.M) {
#pragma unroll 2
    for (int slot = threadIdx.x / kGroups; (slot << log_parts) + rank < n;
         slot += kSplitEpilogue / kGroups) {
      float v[8], up[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = up[i] = 0.f;
#pragma unroll 2
      for (int j = 0; j < S; ++j) {
        const float4* from =
            reinterpret_cast<const float4*>(sums + (j * slots + slot) * kDenseRows + 8 * grp);
        const float4 a = from[0], b = from[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        if constexpr (SILU) {
          const float4 c = from[kTile / 4], d = from[kTile / 4 + 1];
          up[0] += c.x, up[1] += c.y, up[2] += c.z, up[3] += c.w;
          up[4] += d.x, up[5] += d.y, up[6] += d.z, up[7] += d.w;
        }
      }
      split_finish<SILU>(p, (size_t)(r0 + (slot << log_parts) + rank), out_m, v, up, bias, up_bias);
    }
  }
  __syncthreads();
  // copies of a dead CTA may still be in flight
  if (warp == 8 && *dead)
    for (int i = 0; i < kProdSettleSleeps; ++i) __nanosleep(kWaitSuspendNs);
  __syncthreads();
  tc::fence_after();
  if (warp == 9) tc::tmem_dealloc(tmem, all_cols);
}

}  // namespace moe
