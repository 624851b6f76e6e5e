// Ragged matrix products grouped by expert, on the tensor cores' block-scaled
// 8-bit MMA (tcgen05.mma kind::mxf8f6f4.block_scale): both operands enter as
// they are stored, E4M3 (or E2M1 weights) with one UE8M0 scale per 32 values
// along K, and the tensor cores apply the scales.
//
// Operands are swapped: an expert's weight rows are the MMA's M dimension
// (128 a tile, always full) and the rows of its group the N dimension (16 to
// kProdCols a tile, in steps of 16), so a ragged group wastes at most 15
// columns where the other way round it would waste up to 127 rows.
//
// One persistent CTA an SM walks the tiles (token tile of a group, 128 weight
// rows), found from the offsets on the device. Roles:
//   warp 0       weights, their scales and the group's rows by TMA (gathered
//                rows with the four-row gather form), per stage of 128 K
//   warp 1       scales to tensor memory (tcgen05.cp) and the MMAs
//   warps 4-7    epilogue, one per lane quarter of tensor memory
//   warps 8-11   the rows' scales: gathered words to shared memory in the
//                order tcgen05.cp takes
// Two FP32 accumulators in tensor memory let the epilogue of a tile overlap
// the next tile's MMAs.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "moe_device.cuh"
#include "moe_prompt_rows.cuh"
#include "moe_tcgen05.cuh"

namespace moe {

constexpr int kProdRows = 128;     // weight rows a tile (M)
// Rows of a group a tile (N). Two accumulators of 224 columns and four
// stages' scales (12 columns each) share the 512 columns of tensor memory.
constexpr int kProdCols = 224;
constexpr int kProdK = 128;        // K elements a stage: one 128-byte swizzle row
constexpr int kProdStages = 4;
constexpr int kProdBox = 32;       // rows of a TMA box when rows are contiguous
constexpr int kProdThreads = 384;
constexpr int kProdMaxE = 1024;
constexpr int kProdABytes = kProdRows * kProdK;
constexpr int kProdBBytes = kProdCols * kProdK;
constexpr int kProdSfaBytes = 512;
constexpr int kProdSfbBytes = 1024;
// tensor-memory columns
constexpr uint32_t kProdTmemCols = 512;
constexpr uint32_t kProdSfCol = 2 * kProdCols;
constexpr uint32_t kProdSfCols = 12;   // 4 of the weights' scales, 8 of the rows'
static_assert(2 * kProdCols + kProdStages * kProdSfCols <= kProdTmemCols, "tensor memory");
static_assert(kProdCols % kProdBox == 0 && kProdCols <= 256, "token tile");

struct ProductParams {
  CUtensorMap tm_w;
  CUtensorMap tm_a;        // boxes of kProdBox rows, or of one row to gather
  const uint8_t* sfa;      // weights' scales in tile order (moe_product_lay_scales)
  const uint8_t* a_scales; // [A, K/32]
  const int32_t* offsets;  // [E + 1]
  const int32_t* rows;     // [R] or null
  uint16_t* y;             // [R, N]
  uint8_t* codes;          // [R, N/2]
  uint8_t* scales;         // [R, N/64]
  uint32_t* err;
  int E, N, K, R, A;
  int mt;                  // weight tiles of an expert
  int sf_vec;              // scale bytes a load may take: 16, 4 or 1
  uint32_t w_bytes;        // bytes a weight tile's copy completes
  uint32_t a_format;       // the MMA's code for the weights' element type
};

struct ProductSmem {
  static constexpr int a = 0;
  static constexpr int b = a + kProdStages * kProdABytes;
  static constexpr int sfa = b + kProdStages * kProdBBytes;
  static constexpr int sfb = sfa + kProdStages * kProdSfaBytes;
  static constexpr int amax = sfb + kProdStages * kProdSfbBytes;   // [2][4][32] words
  static constexpr int off = amax + 2 * 4 * 32 * 4;                // [E + 1] group starts
  static constexpr int tiles = off + (kProdMaxE + 4) * 4;          // [E + 1] token tiles before
  static constexpr int bars = tiles + (kProdMaxE + 4) * 4;
  static constexpr int total = bars + (3 * kProdStages + 5) * 8 + 16;
};

namespace tc {

__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, int c0, int c1, int c2,
                                            int c3, int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar))
      : "memory");
}

// Four rows of a tensor map whose box is one row.
__device__ __forceinline__ void tma_gather4(void* dst, const void* tmap, int x, const int4& r,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(smem_addr(bar))
      : "memory");
}

// 512 bytes of scales (32 lanes of 16) -> 4 columns of tensor memory, repeated
// in its four lane quarters.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc =
      (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// D (+)= A * B^T with the operands' block scales.
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: A of format `fa` (0 E4M3, 5 E2M1),
// B E4M3, both K-major, M = 128, N = n, UE8M0 scales; the scale byte of the
// K = 32 step is added by mx_scale_id.
__device__ __forceinline__ uint32_t mx_idesc(uint32_t fa, int n) {
  return (fa << 7) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(kProdRows >> 4) << 24);
}
__device__ __forceinline__ uint32_t mx_scale_id(uint32_t j) { return (j << 4) | (j << 29); }

// 32 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

}  // namespace tc

// ---------------------------------------------------------------------------
// moe_product_lay_scales: the weights' scales in the order tcgen05.cp takes
// them, once per handle: for (expert, weight tile, stage) 512 bytes, lane l's
// 16 holding four scale bytes of each of the MMA rows l, l + 32, l + 64,
// l + 96. Places past N or K get 1 (their codes arrive as zeros).
// ---------------------------------------------------------------------------
// Weight row of an expert that MMA row `r` of tile m stands for. With SILU_MUL
// a tile is 64 gate rows and their 64 up rows in turns of 16, so that a gate
// and its up value meet in one warp of the epilogue; valid while the row's
// neuron is below I.
__host__ __device__ __forceinline__ bool product_row(bool silu, int N, int m, int r, int& row) {
  if (!silu) {
    row = m * kProdRows + r;
    return row < N;
  }
  const int I = N / 2, i = m * 64 + (r >> 5) * 16 + (r & 15);
  row = ((r >> 4) & 1) * I + i;
  return i < I;
}

__global__ void __launch_bounds__(128) moe_product_lay_scales(const uint8_t* s, uint8_t* out, int N,
                                                              int K, int mt, int silu) {
  const int ks = K / 32, nk = (K + kProdK - 1) / kProdK;
  const size_t block = blockIdx.x;            // ((e * mt) + m) * nk + kb
  const int kb = block % nk, m = (block / nk) % mt;
  const size_t e = block / nk / mt;
  const int l = threadIdx.x >> 2, g = threadIdx.x & 3;
  int row;
  const bool in = product_row(silu != 0, N, m, g * 32 + l, row);
  uint32_t v = 0;
  for (int j = 0; j < 4; ++j) {
    const int q = kb * 4 + j;
    v |= (in && q < ks ? (uint32_t)s[(e * N + row) * ks + q] : 127u) << (8 * j);
  }
  reinterpret_cast<uint32_t*>(out)[block * 128 + threadIdx.x] = v;
}

// ---------------------------------------------------------------------------
// moe_product_tiles
// ---------------------------------------------------------------------------

// Bounded wait; a timeout marks the CTA dead (every role winds down).
__device__ __forceinline__ bool prod_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                          volatile int* dead) {
  if (*dead) return false;
  if (mbar_wait(bar, parity, err)) return true;
  *dead = 1;
  return false;
}
__device__ __forceinline__ bool prod_wait_warp(uint64_t* bar, uint32_t parity, uint32_t* err,
                                               volatile int* dead) {
  const bool ok = prod_wait(bar, parity, err, dead);
  return __all_sync(kFull, ok);
}

// Barrier over `nthreads` threads on named barrier `id`: whether `ok` holds
// in all of them.
__device__ __forceinline__ bool named_all(int id, int nthreads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

struct ProductTile {
  int e, m;
  int r0, n;   // first row and rows (1..kProdCols) of the group's piece
};

// Tile `i` of the walk: weight tiles of one token tile in turn, so that CTAs
// working side by side share its rows in L2. A group of c rows is cut into
// the fewest pieces, of equal size but for rounding to 16.
__device__ __forceinline__ ProductTile product_tile(int i, int mt, int E, const int* off,
                                                    const int* tiles) {
  ProductTile t;
  const int q = i / mt;
  t.m = i - q * mt;
  int lo = 0, hi = E;   // tiles[lo] <= q < tiles[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tiles[mid] <= q) lo = mid; else hi = mid;
  }
  t.e = lo;
  const int pieces = tiles[lo + 1] - tiles[lo], j = q - tiles[lo];
  const int c = off[lo + 1] - off[lo];
  const int b = ((c + pieces - 1) / pieces + 15) & ~15;
  t.r0 = off[lo] + j * b;
  t.n = min(b, c - j * b);
  return t;
}

// Four stages' scale bytes (16) of one row from stage kb on; bytes past the
// row's end read as 127.
__device__ __forceinline__ uint4 load_row_scales(const uint8_t* row, int kb, int ks, int vec) {
  if (vec == 16) return *reinterpret_cast<const uint4*>(row + kb * 4);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int q = (kb + j) * 4;
    w[j] = 0x7f7f7f7fu;
    if (vec == 4) {
      if (q < ks) w[j] = *reinterpret_cast<const uint32_t*>(row + q);
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (q + b < ks) w[j] = (w[j] & ~(0xffu << (8 * b))) | ((uint32_t)row[q + b] << (8 * b));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool SILU>
__global__ void __launch_bounds__(kProdThreads, 1) moe_product_tiles(
    const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  using L = ProductSmem;
  int* off = reinterpret_cast<int*>(smem + L::off);
  int* tiles = reinterpret_cast<int*>(smem + L::tiles);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* sfb_full = full + kProdStages;
  uint64_t* empty = sfb_full + kProdStages;
  uint64_t* d_full = empty + kProdStages;
  uint64_t* d_empty = d_full + 2;
  uint64_t* drain = d_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nk = (p.K + kProdK - 1) / kProdK;

  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&p.tm_w);
    tc::prefetch_tmap(&p.tm_a);
    for (int i = 0; i < kProdStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&sfb_full[i], 4);   // the scale warps
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 4);    // the epilogue warps
    }
    mbar_init(drain, 1);
    *dead = 0;
    mbar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, kProdTmemCols);
  pdl_wait();
  if (warp == 2) {   // groups and the token tiles before each
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, nt = 0;
      if (e < p.E) {
        lo = min(max(p.offsets[e], 0), p.R);
        const int hi = min(max(p.offsets[e + 1], 0), p.R);
        nt = hi > lo ? (hi - lo + kProdCols - 1) / kProdCols : 0;
        off[e] = lo;
      }
      int incl = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += u;
      }
      if (e < p.E) tiles[e] = carry + incl - nt;
      carry += __shfl_sync(kFull, incl, 31);
    }
    if (lane == 0) {
      off[p.E] = min(max(p.offsets[p.E], 0), p.R);
      tiles[p.E] = carry;
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ntiles = tiles[p.E] * p.mt;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA copies
    RingPos rg(kProdStages);
    int g = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < ntiles; i += gridDim.x) {
      const ProductTile t = product_tile(i, p.mt, p.E, off, tiles);
      const int n16 = (t.n + 15) & ~15;
      int4 quad[2];   // gathered rows 4 lane .. + 3 and 4 (lane + 32) .. + 3
      if (p.rows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int q = min(4 * (lane + 32 * h) + j, t.n - 1);
            r[j] = min(max(p.rows[t.r0 + q], 0), p.A - 1);
          }
          quad[h] = make_int4(r[0], r[1], r[2], r[3]);
        }
      }
      const int boxes = (n16 + kProdBox - 1) / kProdBox;
      const uint32_t bytes =
          p.w_bytes + kProdSfaBytes + (p.rows ? n16 : boxes * kProdBox) * kProdK;
      const uint8_t* sfa = p.sfa + ((size_t)t.e * p.mt + t.m) * nk * kProdSfaBytes;
      for (int kb = 0; kb < nk; ++kb, ++g) {
        const int s = rg.slot;
        if (g >= kProdStages && !prod_wait_warp(&empty[s], rg.phase ^ 1u, p.err, dead)) {
          ok = false;
          break;
        }
        uint8_t* bdst = smem + L::b + s * kProdBBytes;
        if (lane == 0) {
          mbar_expect_tx(&full[s], bytes);
          uint8_t* adst = smem + L::a + s * kProdABytes;
          if (SILU)
            tc::tma_load_5d(adst, &p.tm_w, kb * kProdK, 0, 0, t.m * 4, t.e, &full[s]);
          else
            tma_load_3d(adst, &p.tm_w, kb * kProdK, t.m * kProdRows, t.e, &full[s]);
          bulk_copy_g2s(smem + L::sfa + s * kProdSfaBytes, sfa + (size_t)kb * kProdSfaBytes,
                        kProdSfaBytes, &full[s]);
        }
        __syncwarp();
        if (p.rows) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int q = lane + 32 * h;
            if (4 * q < n16) tc::tma_gather4(bdst + q * 4 * kProdK, &p.tm_a, kb * kProdK, quad[h], &full[s]);
          }
        } else if (lane < boxes) {
          tma_load_2d(bdst + lane * kProdBox * kProdK, &p.tm_a, kb * kProdK, t.r0 + lane * kProdBox,
                      &full[s]);
        }
        rg.next();
      }
    }
    // never leave with copies in flight
    if (lane == 0)
      for (int d = max(0, g - kProdStages); d < g; ++d)
        mbar_wait(&full[d % kProdStages], (d / kProdStages) & 1, p.err);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      RingPos rg(kProdStages);
      int lt = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < ntiles; i += gridDim.x, ++lt) {
        const ProductTile t = product_tile(i, p.mt, p.E, off, tiles);
        const int n16 = (t.n + 15) & ~15;
        const uint32_t idesc = tc::mx_idesc(p.a_format, n16);
        const int buf = lt & 1;
        if (lt >= 2) ok = prod_wait(&d_empty[buf], ((lt >> 1) - 1) & 1, p.err, dead);
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = tmem + buf * kProdCols;
        for (int kb = 0; kb < nk; ++kb) {
          const int s = rg.slot;
          ok = prod_wait(&full[s], rg.phase, p.err, dead) &&
               prod_wait(&sfb_full[s], rg.phase, p.err, dead);
          if (!ok) break;
          tc::fence_after();
          const uint32_t sfa = tmem + kProdSfCol + s * kProdSfCols, sfb = sfa + 4;
          const uint32_t sb = smem_addr(smem + L::sfb + s * kProdSfbBytes);
          tc::cp_scales(sfa, smem_addr(smem + L::sfa + s * kProdSfaBytes));
          tc::cp_scales(sfb, sb);
          if (n16 > 128) tc::cp_scales(sfb + 4, sb + 512);
          const uint32_t aa = smem_addr(smem + L::a + s * kProdABytes);
          const uint32_t ba = smem_addr(smem + L::b + s * kProdBBytes);
#pragma unroll
          for (int j = 0; j < kProdK / 32; ++j)
            tc::mma_mx(d, tc::sdesc_sw128(aa + 32 * j), tc::sdesc_sw128(ba + 32 * j),
                       idesc | tc::mx_scale_id(j), sfa, sfb, kb > 0 || j > 0 ? 1u : 0u);
          tc::commit(&empty[s]);
          rg.next();
        }
        if (ok) tc::commit(&d_full[buf]);
      }
      // every MMA done before tensor memory is released
      tc::commit(drain);
      mbar_wait(drain, 0, p.err);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------ the rows' scales
    const int r = threadIdx.x - 256;   // this thread's rows of a tile: r and r + 128
    const int ks = p.K / 32;
    uint32_t* dst0 = reinterpret_cast<uint32_t*>(smem + L::sfb) + (r & 31) * 4 + (r >> 5);
    RingPos rg(kProdStages);
    int g = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < ntiles; i += gridDim.x) {
      const ProductTile t = product_tile(i, p.mt, p.E, off, tiles);
      const uint8_t* src[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int q = t.r0 + min(r + 128 * h, t.n - 1);
        if (p.rows) q = min(max(p.rows[q], 0), p.A - 1);
        src[h] = p.a_scales + (size_t)q * ks;
      }
      const bool two = t.n > 128;
      uint4 w[2];
      w[0] = load_row_scales(src[0], 0, ks, p.sf_vec);
      w[1] = two ? load_row_scales(src[1], 0, ks, p.sf_vec) : w[0];
      for (int k0 = 0; ok && k0 < nk; k0 += 4) {
        const uint4 c[2] = {w[0], w[1]};
        if (k0 + 4 < nk) {   // the next four stages' words while these are handed over
          w[0] = load_row_scales(src[0], k0 + 4, ks, p.sf_vec);
          if (two) w[1] = load_row_scales(src[1], k0 + 4, ks, p.sf_vec);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k0 + j >= nk) break;
          const int s = rg.slot;
          if (g >= kProdStages && !prod_wait_warp(&empty[s], rg.phase ^ 1u, p.err, dead)) {
            ok = false;
            break;
          }
          uint32_t* dst = dst0 + s * (kProdSfbBytes / 4);
          dst[0] = j == 0 ? c[0].x : j == 1 ? c[0].y : j == 2 ? c[0].z : c[0].w;
          if (two) dst[128] = j == 0 ? c[1].x : j == 1 ? c[1].y : j == 2 ? c[1].z : c[1].w;
          tc::fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfb_full[s]);
          ++g;
          rg.next();
        }
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    uint32_t* amax = reinterpret_cast<uint32_t*>(smem + L::amax);
    int lt = 0, chunk = 0;
    for (int i = blockIdx.x; i < ntiles; i += gridDim.x, ++lt) {
      const ProductTile t = product_tile(i, p.mt, p.E, off, tiles);
      const int buf = lt & 1;
      bool ok = prod_wait_warp(&d_full[buf], (lt >> 1) & 1, p.err, dead);
      // the two warps of a block go on or leave together: the named barrier
      // below never waits for a warp that gave up
      if (SILU) ok = named_all(1 + (q >> 1), 64, ok);
      if (!ok) break;
      tc::fence_after();
      for (int c0 = 0; c0 < t.n; c0 += 32, ++chunk) {
        uint32_t v[32];
        tc::ld32(lanes + buf * kProdCols + c0, v);
        tc::wait_ld();
        if constexpr (!SILU) {
          // a lane holds one weight row of 32 columns (rows of the group):
          // neighbouring lanes swap, so that each stores two weight rows' bf16
          // values of every other column
          const int n = t.m * kProdRows + 32 * q + (lane & ~1);
          const int odd = lane & 1;
          uint16_t* y = p.y + (size_t)(t.r0 + c0) * p.N + n;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t give = odd ? v[j] : v[j + 1], keep = odd ? v[j + 1] : v[j];
            const uint32_t got = __shfl_xor_sync(kFull, give, 1);
            const float lo = __uint_as_float(odd ? got : keep);
            const float hi = __uint_as_float(odd ? keep : got);
            if (c0 + j + odd < t.n && n < p.N)
              *reinterpret_cast<uint32_t*>(y + (size_t)(j + odd) * p.N) = RowVec<8>::pack(lo, hi);
          }
        } else {
          // lanes 0-15 hold gate rows, lanes 16-31 the same neurons' up rows:
          // the halves swap, so that the low half finishes even columns and
          // the high half odd ones
          const int up = lane >> 4, I = p.N / 2;
          const int n = t.m * 64 + 16 * q + (lane & 15);
          float h[16];
          uint32_t mine = 0u;   // lane's column's largest magnitude among these 16 neurons
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t give = up ? v[2 * j] : v[2 * j + 1], keep = up ? v[2 * j + 1] : v[2 * j];
            const uint32_t got = __shfl_xor_sync(kFull, give, 16);
            const float gate = __uint_as_float(up ? got : keep);
            const float u = __uint_as_float(up ? keep : got);
            h[j] = gate / (1.0f + expf(-gate)) * u;
            uint32_t a = __float_as_uint(h[j]) & 0x7fffffffu;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(kFull, a, o));
            if ((lane & 15) == j) mine = a;
          }
          // lane l now holds column 2 (l & 15) + (l >> 4); the block's other 16
          // neurons are in the neighbouring warp
          const int col = 2 * (lane & 15) + up;
          uint32_t* mx = amax + (chunk & 1) * 128;
          mx[q * 32 + lane] = mine;
          named_sync(1 + (q >> 1), 64);
          mine = max(mine, mx[(q ^ 1) * 32 + lane]);
          const uint32_t sc = mx_scale_code(mine);
          if ((q & 1) == 0 && c0 + col < t.n && n < I)
            p.scales[(size_t)(t.r0 + c0 + col) * (I / 32) + t.m * 2 + (q >> 1)] = (uint8_t)sc;
          const float inv = mx_inverse(sc);
          uint8_t* out = p.codes + (size_t)(t.r0 + c0) * I + n;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x = h[j] * __shfl_sync(kFull, inv, j + (lane & 16));
            if (c0 + 2 * j + up < t.n && n < I)
              out[(size_t)(2 * j + up) * I] = (uint8_t)e4m3x2(x, x);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[buf]);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::tmem_dealloc(tmem, kProdTmemCols);
}

}  // namespace moe
