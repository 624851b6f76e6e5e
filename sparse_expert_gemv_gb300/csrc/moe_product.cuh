// Ragged matrix products grouped by expert, on the tensor cores' block-scaled
// 8-bit MMA (tcgen05.mma kind::mxf8f6f4.block_scale): both operands enter as
// they are stored, E4M3 (or E2M1 weights) with one UE8M0 scale per 32 values
// along K, and the tensor cores apply the scales.
//
// Operands are swapped: an expert's weight rows are the MMA's M dimension
// (256 a tile over the two SMs of a CTA pair) and the rows of its group the N
// dimension (32 to kProdCols a tile, in steps of 32), so a ragged group
// wastes at most 31 columns where the other way round it would waste up to
// 255 rows.
//
// One persistent pair of CTAs (a cluster of 2, cta_group::2) a pair of SMs
// walks the tiles (token tile of a group, 256 weight rows), found from the
// offsets on the device. Each CTA holds 128 of the weight rows and half of the
// group's rows in shared memory, per stage of 128 K, and its 128 rows of the
// accumulator in tensor memory; the first CTA issues the MMAs of both. Roles:
//   warp 0       weights by TMA
//   warp 1       (first CTA) scales to tensor memory (tcgen05.cp) and the MMAs
//   warp 2       the group's rows by TMA, where they are contiguous
//   warp 3       where they are gathered, word to the MMAs that they landed
//   warps 4-7    epilogue, one per lane quarter of tensor memory, and
//   warps 12-15  the same for every other chunk of 32 columns
//   warps 8-11   scales, 512 K at a time, into shared memory in the order
//                tcgen05.cp takes
//   warps 16-19  the group's rows where they are gathered
// Two FP32 accumulators in tensor memory let the epilogue of a tile overlap
// the next tile's MMAs.
//
// What bounds it, measured (us a call, E=128 k=8 H=2048 I=768 unless noted; the
// shorter figures are of runs too short to reach the board's power limit). Every
// call takes 5 until its first MMA: offsets, tiles, the first copies. Few rows an
// expert: HBM (gate/up of 8 tokens 30 to 33, 5.3 TB/s; of 256 tokens 68, 6.1).
// Hundreds of rows: 420 to 480 cycles a stage, of which its MMAs are 256 to 384,
// waits for rows and weights 120 to 140 and for scales 30 to 55, at a clock that the
// power limit takes from 2070 MHz to 1770 (gate/up of 2048 tokens, MXFP4, 54 to 59),
// 1560 (4096 tokens, 98 to 116) and 1300 (down of 32768 rows, E=32 H=7168 I=2048,
// 312 to 385, 2.5 to 3.1 PFLOP/s). Rows gathered or contiguous make no difference.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "moe_device.cuh"
#include "moe_prompt_rows.cuh"
#include "moe_tcgen05.cuh"

namespace moe {

constexpr int kProdRows = 128;     // weight rows a CTA (half of the MMA's M)
// Rows of a group a tile (N). Two accumulators of 192 columns and two batches
// of four stages' scales (12 columns a stage) share the 512 columns of tensor
// memory.
constexpr int kProdCols = 192;
constexpr int kProdK = 128;        // K elements a stage: one 128-byte swizzle row
// A slot's way from the MMA's release through a copy from L2 back to the MMA
// takes some 2000 cycles: six stages of one row each hide it better than three
// of two (down projection of 32768 rows, E32 H7168 I2048: 317 and 329 us).
constexpr int kProdStages = 6;
constexpr int kProdSfStages = 4;   // stages a batch of scales covers
constexpr int kProdThreads = 640;
constexpr int kProdMaxE = 1024;
constexpr int kProdSettleSleeps = 50;   // of kWaitSuspendNs: a dead pair's time for its copies
constexpr int kProdABytes = kProdRows * kProdK;
constexpr int kProdBBytes = kProdCols / 2 * kProdK;
constexpr int kProdSfaBytes = 512;    // a stage's weight scales of one CTA
constexpr int kProdSfbBytes = 1024;   // a stage's row scales (up to 256 rows)
constexpr int kProdSfBytes = kProdSfStages * (kProdSfaBytes + kProdSfbBytes);
// tensor-memory columns
constexpr uint32_t kProdTmemCols = 512;
constexpr uint32_t kProdSfCol = 2 * kProdCols;
constexpr uint32_t kProdSfCols = 12;   // a stage's: 4 of the weights, 8 of the rows
static_assert(2 * kProdCols + 2 * kProdSfStages * kProdSfCols <= kProdTmemCols, "tensor memory");
static_assert(kProdCols % 32 == 0 && kProdCols <= 256, "token tile");
// epilogue staging, two in turn for each of its two groups of four warps: a
// chunk of 32 columns as rows of 128 bf16 (16-byte pieces swizzled by the row),
// or of 64 codes padded to 80 bytes
constexpr int kProdStageOut = 32 * 256;
constexpr int kProdCodePitch = 80;

struct ProductParams {
  CUtensorMap tm_w;
  CUtensorMap tm_a[3];     // boxes of 16, 32 and 64 contiguous rows
  const uint8_t* a;        // [A, K]
  const uint8_t* sfa;      // weights' scales in tile order (moe_product_lay_scales)
  const uint8_t* a_scales; // [A, K/32]
  const int32_t* offsets;  // [E + 1]
  const int32_t* rows;     // [R] or null
  uint16_t* y;             // [R, N]
  uint8_t* codes;          // [R, N/2]
  uint8_t* scales;         // [R, N/64]
  uint32_t* err;
  int E, N, K, R, A;
  int mt;                  // tiles of kProdRows weight rows an expert has
  int sf_vec;              // scale bytes a load may take: 16, 4 or 1
  uint32_t w_bytes;        // bytes a CTA's weight copy completes
  uint32_t a_format;       // the MMA's code for the weights' element type
  uint32_t polls;          // of a bounded wait: kMbarPolls
  uint32_t withheld;       // 1: stages lack an arrival, so that waits run out (tests)
};

struct ProductSmem {
  static constexpr int a = 0;
  static constexpr int b = a + kProdStages * kProdABytes;
  static constexpr int sf = b + kProdStages * kProdBBytes;         // 2 batches
  static constexpr int out = sf + 2 * kProdSfBytes;                // [2][2] chunks
  static constexpr int amax = out + 4 * kProdStageOut;             // [2][2][4][32] words
  static constexpr int inv = amax + 2 * 2 * 4 * 32 * 4;            // [2][4][32] floats
  static constexpr int off = inv + 2 * 4 * 32 * 4;                 // [E + 1] group starts
  static constexpr int tiles = off + (kProdMaxE + 4) * 4;          // [E + 1] token tiles before
  static constexpr int piece = tiles + (kProdMaxE + 4) * 4;        // [E] rows of a group's pieces
  static constexpr int bars = piece + kProdMaxE * 2;
  static constexpr int total = bars + (3 * kProdStages + 9) * 8 + 16;
};

namespace tc {

// The wrappers below are called by whole, converged warps and act in one lane,
// always the same one, chosen inside the instruction sequence and by predicate.
// No branch on a lane appears in a role's loop: with a loop walked by lane 0
// alone a tensor-memory instruction cost 60 to 80 cycles and a wait on a
// barrier that had long completed over 200, and the MMA pipe idled for more
// than half of the time.
#define MOE_ELECT ".reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"

// The address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
// One arrival on an mbarrier of the first CTA, by this CTA or (`remote`) by the
// other one. What a remote one announces, scales and rows in this CTA's shared
// memory and columns of its tensor memory, is used by MMAs that the first CTA
// issues, so it is a release at cluster scope, of shared memory alone: that fence
// waits for no global load or store (gate/up of 4096 tokens 97 us, 264 with a
// release of all memory; down projection of 32768 rows 312 and 454).
__device__ __forceinline__ void arrive_at(uint32_t bar, bool remote) {
  if (remote)
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t{\n\t" MOE_ELECT
                 "@e mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar)
                 : "memory");
  else
    asm volatile("{\n\t" MOE_ELECT
                 "@e mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar)
                 : "memory");
}
// One arrival on this CTA's mbarrier that announces `bytes` of copies.
__device__ __forceinline__ void expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("{\n\t" MOE_ELECT
               "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Tensor-map tiles into this CTA's shared memory, completing on an mbarrier of
// either CTA of the pair.
__device__ __forceinline__ void tma2_load_2d(void* dst, const void* tmap, int x, int y,
                                             uint32_t bar) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma2_load_3d(void* dst, const void* tmap, int x, int y, int z,
                                             uint32_t bar) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma2_load_5d(void* dst, const void* tmap, int c0, int c1, int c2,
                                             int c3, int c4, uint32_t bar) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n\t}" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

// 16 bytes global -> shared, asynchronously; `bytes` 0 fills with zeros and
// reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// This thread's arrival on an mbarrier, once its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void copy_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// 512 bytes of scales (32 lanes of 16) at the same place of both CTAs' shared
// memory -> 4 columns of their tensor memory, repeated in its four quarters.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc =
      (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
  asm volatile("{\n\t" MOE_ELECT "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(
                   taddr),
               "l"(desc)
               : "memory");
}

// D (+)= A * B^T with the operands' block scales, over both CTAs.
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t" MOE_ELECT
      ".reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: A of format `fa` (0 E4M3, 5 E2M1),
// B E4M3, both K-major, M = 256 over the pair, N = n, UE8M0 scales; the scale
// byte of the K = 32 step is added by mx_scale_id.
__device__ __forceinline__ uint32_t mx_idesc(uint32_t fa, int n) {
  return (fa << 7) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(2 * kProdRows >> 4) << 24);
}
__device__ __forceinline__ uint32_t mx_scale_id(uint32_t j) { return (j << 4) | (j << 29); }

// Arrive once on the mbarrier at `bar` of both CTAs when every MMA and copy
// issued so far is done.
__device__ __forceinline__ void commit2(uint64_t* bar) {
  asm volatile(
      "{\n\t" MOE_ELECT
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;\n\t}" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// 32 columns of lanes 0-15 of this warp's quarter (16-31 from taddr + 16
// lanes): register 4b + 2i + j of thread t holds lane 8i + t / 4, column
// 8b + 2 (t % 4) + j.
__device__ __forceinline__ void ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Four transposed 8x8 matrices of 16-bit values: thread t's register m holds
// rows 2 (t % 4) + {0, 1}, column t / 4 of matrix m, whose row r goes to the
// 16 bytes at the address of lane 8m + r.
__device__ __forceinline__ void stm4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                           uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

}  // namespace tc

// ---------------------------------------------------------------------------
// moe_product_lay_scales: the weights' scales in the order tcgen05.cp takes
// them, once per handle: for (expert, 128-row tile, stage) 512 bytes, lane l's
// 16 holding four scale bytes of each of the MMA rows l, l + 32, l + 64,
// l + 96. Places past N or K get 1 (their codes arrive as zeros).
// ---------------------------------------------------------------------------
// Weight row of an expert that MMA row `r` of 128-row tile m stands for. With
// SILU_MUL a tile is 64 neurons in four groups of 16: a group's 16 gate rows,
// then its 16 up rows, even neurons before odd ones, so that one thread of the
// epilogue holds the gates and ups of two neighbouring neurons. False past the
// last row.
__host__ __device__ __forceinline__ bool product_row(bool silu, int N, int m, int r, int& row) {
  if (!silu) {
    row = m * kProdRows + r;
    return row < N;
  }
  const int I = N / 2, i = m * 64 + (r >> 5) * 16 + 2 * (r & 7) + ((r >> 3) & 1);
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

// err[1] = the error word err[0], which is cleared.
__global__ void moe_product_take_error(uint32_t* err) { err[1] = atomicExch(err, 0u); }

// ---------------------------------------------------------------------------
// moe_product_tiles
// ---------------------------------------------------------------------------

// Whose arrivals a wait is for: kPair, an mbarrier on which the other CTA or the
// MMAs of both arrive, acquired at cluster scope (1% of the gathered gate/up's
// time), or kOwn, one of this CTA alone.
enum class Arrivals { kOwn, kPair };

// One look at a barrier's phase: without a time the instruction returns after
// the hardware's own short wait, with one it may sleep that long.
template <Arrivals A>
__device__ __forceinline__ bool prod_look(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  if constexpr (A == Arrivals::kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], "
        "%2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], "
        "%2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
  return done != 0;
}
template <Arrivals A>
__device__ __forceinline__ bool prod_poll(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  if constexpr (A == Arrivals::kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], "
        "%2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kWaitSuspendNs)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], "
        "%2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kWaitSuspendNs)
        : "memory");
  return done != 0;
}
// A whole warp's bounded wait on a phase of this CTA's mbarrier; a timeout
// marks both CTAs of the pair dead (every role winds down).
template <Arrivals A = Arrivals::kPair>
__device__ __forceinline__ bool prod_wait(uint64_t* bar, uint32_t parity, const ProductParams& p,
                                          volatile int* dead) {
  if (__all_sync(kFull, prod_look<A>(bar, parity))) return true;
#pragma unroll 1
  for (uint32_t it = 0; it < p.polls; ++it) {
    if (__any_sync(kFull, *dead)) return false;
    if (__all_sync(kFull, prod_poll<A>(bar, parity))) return true;
  }
  atomicOr(p.err, kDeviceTimeout);
  *dead = 1;
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(
                   tc::cluster_addr(const_cast<int*>(dead), (blockIdx.x & 1) ^ 1))
               : "memory");
  return false;
}
// The wait for what must have ended before a CTA may leave: neither a dead pair
// nor p.polls shortens it.
__device__ __forceinline__ void prod_wait_end(uint64_t* bar, uint32_t parity, uint32_t* err) {
#pragma unroll 1
  for (uint32_t it = 0; it < kMbarPolls; ++it)
    if (__all_sync(kFull, prod_poll<Arrivals::kPair>(bar, parity))) return;
  atomicOr(err, kDeviceTimeout);
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

// The value of lane 0, which all lanes hold already: tells the compiler that
// it is the same in the whole warp, so that what follows from it (loop bounds,
// descriptors, tensor-memory addresses) is computed once a warp and reaches
// the tensor-memory instructions without a move per operand.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kFull, v, 0); }

struct ProductTile {
  int e, m;
  int r0, n;   // first row and rows (1..kProdCols) of the group's piece
  // the MMA's N and each CTA's half of it
  __device__ __forceinline__ int cols() const { return (n + 31) & ~31; }
  __device__ __forceinline__ int half() const { return cols() >> 1; }
};

// A CTA pair's walk over the tiles first, first + step, ...: the pairs of
// weight tiles of one token tile in turn, so that pairs of CTAs working side
// by side share its rows in L2. A group of c rows is cut into the fewest
// pieces, of equal size but for rounding to 32. Every lane of the warp takes
// part: the next token tile's expert is found 32 experts at a time (a search
// and divisions cost each role a thousand cycles a tile).
struct ProductWalk {
  const int *off, *tiles;           // [E + 1]
  const uint16_t* piece;            // [E]
  int rank, pairs, E, ntok;
  int q, m, dq, dm;                 // token tile and pair of weight tiles, and a step's
  int e;                            // expert of q, once found
  __device__ __forceinline__ ProductWalk(const int* off_, const int* tiles_,
                                         const uint16_t* piece_, int rank_, int pairs_, int E_,
                                         int first, int step)
      : off(off_), tiles(tiles_), piece(piece_), rank(rank_), pairs(pairs_), E(E_),
        ntok(uniform(tiles_[E_])), q(first / pairs_), m(first % pairs_), dq(step / pairs_),
        dm(step % pairs_), e(0) {}
  __device__ __forceinline__ bool valid() const { return q < ntok; }
  __device__ __forceinline__ void next() {
    q += dq;
    m += dm;
    if (m >= pairs) m -= pairs, ++q;
  }
  __device__ __forceinline__ ProductTile tile() {
    const int lane = threadIdx.x & 31;
    for (;;) {   // tiles[e] <= q < tiles[e + 1]; the last entry is above q
      const int i = e + 1 + lane;
      const unsigned past = __ballot_sync(kFull, i <= E && tiles[i] <= q);
      e += __popc(past);
      if (past != kFull) break;
    }
    ProductTile t;
    const int b = piece[e], r0 = off[e] + (q - tiles[e]) * b;
    t.e = uniform(e);
    t.m = 2 * m + rank;
    t.r0 = uniform(r0);
    t.n = uniform(min(b, off[e + 1] - r0));
    return t;
  }
};

// A batch's scale bytes (16, four stages) of one row from stage kb on; bytes
// past the row's end read as 127.
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

// What a thread of the scale warps holds of a tile: the two rows (r and
// r + 128 of the tile) whose scales it brings. load() only issues the loads of
// gathered rows; settle() uses them, a tile later.
struct ScaleRows {
  int row[2];
  ProductTile t;
  __device__ __forceinline__ void load(const ProductParams& p, const ProductTile& tile, int r) {
    t = tile;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row[h] = t.r0 + min(r + 128 * h, t.n - 1);
      if (p.rows) row[h] = p.rows[row[h]];
    }
  }
  __device__ __forceinline__ void settle(const ProductParams& p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) row[h] = min(max(row[h], 0), p.A - 1);
  }
};

// What a thread of the copying warps holds of a tile: the gathered rows
// (r / 8 + 16 c of this CTA's half) of which it copies 16 bytes a stage.
struct CopyRows {
  int row[kProdCols / 32];
  int half;
  __device__ __forceinline__ void load(const ProductParams& p, const ProductTile& t, int rank,
                                       int r) {
    half = t.half();
#pragma unroll
    for (int c = 0; c < kProdCols / 32; ++c) {
      row[c] = 0;
      if (16 * c < half) row[c] = p.rows[t.r0 + min(rank * half + (r >> 3) + 16 * c, t.n - 1)];
    }
  }
};

template <bool SILU>
__global__ void __launch_bounds__(kProdThreads, 1) moe_product_tiles(
    const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  using L = ProductSmem;
  int* off = reinterpret_cast<int*>(smem + L::off);
  int* tiles = reinterpret_cast<int*>(smem + L::tiles);
  uint16_t* piece = reinterpret_cast<uint16_t*>(smem + L::piece);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);   // used in the first CTA
  uint64_t* empty = full + kProdStages;
  uint64_t* copied = empty + kProdStages;                         // gathered rows
  uint64_t* sf_full = copied + kProdStages;                       // used in the first CTA
  uint64_t* sf_empty = sf_full + 2;
  uint64_t* d_full = sf_empty + 2;
  uint64_t* d_empty = d_full + 2;                                 // used in the first CTA
  uint64_t* drain = d_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;   // clusters are pairs of neighbours
  const int nk = (p.K + kProdK - 1) / kProdK;
  const int pairs = (p.mt + 1) / 2;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&p.tm_w);
    for (int i = 0; i < kProdStages; ++i) {
      // the announcement of both CTAs' TMA bytes, and with gathered rows both
      // CTAs' word that their copies have landed
      mbar_init(&full[i], (p.rows ? 3 : 1) + p.withheld);
      mbar_init(&empty[i], 1);
      mbar_init(&copied[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sf_full[i], 8);    // both CTAs' scale warps
      mbar_init(&sf_empty[i], 1);
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 16);   // both CTAs' epilogue warps
    }
    mbar_init(drain, 1);
    *dead = 0;
    mbar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc2(tmem_slot, kProdTmemCols);
  pdl_wait();
  pdl_trigger();   // the next kernel's prologue may run beside this one
  for (int e = threadIdx.x; e <= p.E; e += kProdThreads)
    off[e] = min(max(p.offsets[e], 0), p.R);
  __syncthreads();
  if (warp == 2) {   // the token tiles before each group
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int nt = 0;
      if (e < p.E) {
        const int c = off[e + 1] - off[e];
        nt = c > 0 ? (c + kProdCols - 1) / kProdCols : 0;
        piece[e] = (uint16_t)(nt ? ((c + nt - 1) / nt + 31) & ~31 : 0);
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
    if (lane == 0) tiles[p.E] = carry;
  }
  tc::fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's barriers are ready too
  tc::fence_after();
  // all of tensor memory is this CTA's, so its columns start at 0
  constexpr uint32_t tmem = 0;
  ProductWalk walk(off, tiles, piece, rank, pairs, p.E, first, step);

  if (warp == 0) {
    // --------------------------------------------------------------- weights
    RingPos rg(kProdStages);
    const uint32_t full0 = tc::cluster_addr(full, 0);
    int g = 0;
    bool ok = true;
    for (; ok && walk.valid(); walk.next()) {
      const ProductTile t = walk.tile();
      const uint32_t bytes = 2 * p.w_bytes + (p.rows ? 0 : t.cols() * kProdK);
      // the groups of 16 neurons of all experts' gate and up rows in one row
      const int grp = SILU ? t.e * (p.N / 16) + t.m * 4 : 0;
      for (int kb = 0; kb < nk; ++kb, ++g) {
        const int s = rg.slot;
        if (g >= kProdStages && !prod_wait(&empty[s], rg.phase ^ 1u, p, dead)) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + L::a + s * kProdABytes;
        if (rank == 0) tc::expect(&full[s], bytes);
        if (SILU)
          tc::tma2_load_5d(dst, &p.tm_w, kb * kProdK, 0, 0, 0, grp, full0 + 8 * s);
        else
          tc::tma2_load_3d(dst, &p.tm_w, kb * kProdK, t.m * kProdRows, t.e, full0 + 8 * s);
        rg.next();
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (rank == 0) {
      RingPos rg(kProdStages), rs(2);
      int lt = 0;
      bool ok = true;
      ProductTile t, after;
      bool more = walk.valid();
      if (more) after = walk.tile();
      for (; more; ++lt) {
        t = after;
        const int n = t.cols();
        const uint32_t idesc = tc::mx_idesc(p.a_format, n);
        const int buf = lt & 1;
        if (lt >= 2) ok = prod_wait(&d_empty[buf], ((lt >> 1) - 1) & 1, p, dead);
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = tmem + buf * kProdCols;
        for (int k0 = 0; ok && k0 < nk; k0 += kProdSfStages) {
          const int ns = min(kProdSfStages, nk - k0);
          ok = prod_wait(&sf_full[rs.slot], rs.phase, p, dead);
          if (!ok) break;
          const uint32_t sfc = tmem + kProdSfCol + rs.slot * kProdSfStages * kProdSfCols;
          const uint32_t sfs = smem_addr(smem + L::sf + rs.slot * kProdSfBytes);
          for (int j = 0; j < ns; ++j) {
            const uint32_t c = sfc + j * kProdSfCols;
            const uint32_t sb = sfs + kProdSfStages * kProdSfaBytes + j * kProdSfbBytes;
            tc::cp_scales(c, sfs + j * kProdSfaBytes);
            tc::cp_scales(c + 4, sb);
            if (n > 128) tc::cp_scales(c + 8, sb + 512);
          }
          for (int j = 0; j < ns; ++j) {
            const int s = rg.slot;
            ok = prod_wait(&full[s], rg.phase, p, dead);
            if (!ok) break;
            const uint64_t ad = tc::sdesc_sw128(smem_addr(smem + L::a + s * kProdABytes));
            const uint64_t bd = tc::sdesc_sw128(smem_addr(smem + L::b + s * kProdBBytes));
            const uint32_t c = sfc + j * kProdSfCols;
#pragma unroll
            for (int q = 0; q < kProdK / 32; ++q)   // 32 bytes further in the swizzled rows
              tc::mma_mx(d, ad + 2 * q, bd + 2 * q, idesc | tc::mx_scale_id(q), c, c + 4,
                         k0 + j + q > 0 ? 1u : 0u);
            tc::commit2(&empty[s]);
            rg.next();
          }
          // the batch's places in shared and tensor memory are free when its
          // MMAs are done
          if (!ok) break;
          tc::commit2(&sf_empty[rs.slot]);
          rs.next();
          if (k0 == 0) {   // find the next tile while MMAs are under way
            walk.next();
            more = walk.valid();
            if (more) after = walk.tile();
          }
        }
        if (!ok) break;
        tc::commit2(&d_full[buf]);
      }
      tc::commit2(drain);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------- contiguous rows
    if (!p.rows) {
      RingPos rg(kProdStages);
      const uint32_t full0 = tc::cluster_addr(full, 0);
      int g = 0;
      bool ok = true;
      for (; ok && walk.valid(); walk.next()) {
        const ProductTile t = walk.tile();
        const int half = t.half(), r0 = t.r0 + rank * half;
        for (int kb = 0; kb < nk; ++kb, ++g) {
          const int s = rg.slot;
          if (g >= kProdStages && !prod_wait(&empty[s], rg.phase ^ 1u, p, dead)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + L::b + s * kProdBBytes;
          int r = 0;   // half = 64 + 32 + 16 where those bits are set (at most two boxes)
#pragma unroll
          for (int b = 2; b >= 0; --b)
            if (half & (16 << b)) {
              tc::tma2_load_2d(dst + r * kProdK, &p.tm_a[b], kb * kProdK, r0 + r, full0 + 8 * s);
              r += 16 << b;
            }
          rg.next();
        }
      }
    }
  } else if (warp == 3) {
    // ------------------------------------ word of gathered rows to the MMAs
    // One warp waits for a stage's copies, makes them visible to the tensor
    // cores and tells the first CTA, so that the copying warps never wait for
    // what they issued.
    if (p.rows) {
      RingPos rg(kProdStages);
      const uint32_t full0 = tc::cluster_addr(full, 0);
      bool ok = true;
      for (; ok && walk.valid(); walk.next())
        for (int kb = 0; kb < nk; ++kb) {
          if (!prod_wait<Arrivals::kOwn>(&copied[rg.slot], rg.phase, p, dead)) {
            ok = false;
            break;
          }
          tc::fence_proxy_async();
          __syncwarp();
          tc::arrive_at(full0 + 8 * rg.slot, rank != 0);
          rg.next();
        }
    }
  } else if (warp >= 16) {
    // --------------------------------------------------------- gathered rows
    if (p.rows) {
      const int r = threadIdx.x - 512;
      // this thread's 16 bytes of each row: piece r % 8, where the 128-byte
      // swizzle puts it
      const int within = (r & 7) * 16;
      const uint32_t dst =
          smem_addr(smem + L::b) + (r >> 3) * kProdK + (((r & 7) ^ ((r >> 3) & 7)) << 4);
      RingPos rg(kProdStages);
      int g = 0;
      CopyRows cur, nxt;
      bool ok = true, more = walk.valid();
      if (more) nxt.load(p, walk.tile(), rank, r);
      while (ok && more) {
        cur = nxt;
        const uint8_t* src[kProdCols / 32];
#pragma unroll
        for (int c = 0; c < kProdCols / 32; ++c)
          src[c] = p.a + (size_t)min(max(cur.row[c], 0), p.A - 1) * p.K;
        walk.next();
        more = walk.valid();
        if (more) nxt.load(p, walk.tile(), rank, r);   // used a tile later
        for (int kb = 0; kb < nk; ++kb, ++g) {
          const int s = rg.slot, at = kb * kProdK + within;
          if (g >= kProdStages && !prod_wait(&empty[s], rg.phase ^ 1u, p, dead)) {
            ok = false;
            break;
          }
          const uint32_t bytes = at < p.K ? 16u : 0u;
          const int from = bytes ? at : 0;
#pragma unroll
          for (int c = 0; c < kProdCols / 32; ++c)
            if (16 * c < cur.half)
              tc::copy16(dst + s * kProdBBytes + c * 16 * kProdK, src[c] + from, bytes);
          tc::copy_arrive(&copied[s]);
          rg.next();
        }
      }
      tc::copy_wait_all();
    }
  } else if ((warp >> 2) == 2) {
    // ---------------------------------------------------------------- scales
    const int r = threadIdx.x - 256;
    const int ks = p.K / 32;
    const uint32_t sf_full0 = tc::cluster_addr(sf_full, 0);
    RingPos rs(2);
    int gb = 0;
    ScaleRows cur, nxt;
    bool ok = true, more = walk.valid();
    uint4 wsf = make_uint4(0, 0, 0, 0), rsf[2] = {wsf, wsf};
    auto load_batch = [&](const ScaleRows& sr, int k0) {
      if (r < 32 * min(kProdSfStages, nk - k0))
        wsf = *reinterpret_cast<const uint4*>(
            p.sfa + (((size_t)sr.t.e * 2 * pairs + sr.t.m) * nk + k0) * kProdSfaBytes + r * 16);
      rsf[0] = load_row_scales(p.a_scales + (size_t)sr.row[0] * ks, k0, ks, p.sf_vec);
      if (sr.t.n > 128)
        rsf[1] = load_row_scales(p.a_scales + (size_t)sr.row[1] * ks, k0, ks, p.sf_vec);
    };
    if (more) {
      cur.load(p, walk.tile(), r);
      cur.settle(p);
      load_batch(cur, 0);
    }
    while (ok && more) {
      walk.next();
      more = walk.valid();
      if (more) nxt.load(p, walk.tile(), r);
      for (int k0 = 0; k0 < nk; k0 += kProdSfStages, ++gb) {
        if (gb >= 2 && !prod_wait(&sf_empty[rs.slot], rs.phase ^ 1u, p, dead)) {
          ok = false;
          break;
        }
        uint8_t* sf = smem + L::sf + rs.slot * kProdSfBytes;
        *reinterpret_cast<uint4*>(sf + r * 16) = wsf;
        uint32_t* dst = reinterpret_cast<uint32_t*>(sf + kProdSfStages * kProdSfaBytes) +
                        (r & 31) * 4 + (r >> 5);
        dst[0] = rsf[0].x, dst[256] = rsf[0].y, dst[512] = rsf[0].z, dst[768] = rsf[0].w;
        if (cur.t.n > 128)
          dst[128] = rsf[1].x, dst[384] = rsf[1].y, dst[640] = rsf[1].z, dst[896] = rsf[1].w;
        tc::fence_proxy_async();
        __syncwarp();
        tc::arrive_at(sf_full0 + 8 * rs.slot, rank != 0);
        rs.next();
        // the next batch's loads run while this one is used
        if (k0 + kProdSfStages < nk) {
          load_batch(cur, k0 + kProdSfStages);
        } else if (more) {
          nxt.settle(p);
          load_batch(nxt, 0);
        }
      }
      cur = nxt;
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, et = threadIdx.x & 127;
    const int grp = warp >> 3;   // chunks of 32 columns go to the two groups in turn
    const int bar = 1 + 3 * grp;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t d_empty0 = tc::cluster_addr(d_empty, 0);
    uint32_t* amax = reinterpret_cast<uint32_t*>(smem + L::amax) + grp * 256;
    float* inv = reinterpret_cast<float*>(smem + L::inv) + (grp * 4 + q) * 32;
    int lt = 0, chunk = 0;
    for (; walk.valid(); walk.next(), ++lt) {
      const ProductTile t = walk.tile();
      const int buf = lt & 1;
      bool ok = prod_wait(&d_full[buf], (lt >> 1) & 1, p, dead);
      // a group's warps go on or leave together: no named barrier below waits
      // for a warp that gave up
      ok = named_all(bar, 128, ok);
      if (!ok) break;
      tc::fence_after();
      for (int c0 = 32 * grp; c0 < t.n; c0 += 64, ++chunk) {
        uint8_t* stage = smem + L::out + (2 * grp + (chunk & 1)) * kProdStageOut;
        uint32_t lo[16], hi[16];
        tc::ld_16x32(lanes + buf * kProdCols + c0, lo);
        tc::ld_16x32(lanes + (16u << 16) + buf * kProdCols + c0, hi);
        tc::wait_ld();
        if constexpr (!SILU) {
          // 32 rows of the group x this warp's 32 weight rows, transposed on
          // the way to shared memory: 16-byte piece 4q + m of row r holds
          // weight rows 8m.. and sits at piece ^ (r & 7)
          const int m = lane >> 3, r = lane & 7;
          const uint32_t dst = smem_addr(stage) + r * 256 + (((4 * q + m) ^ r) << 4);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            auto pack = [](uint32_t x, uint32_t y) {
              return RowVec<8>::pack(__uint_as_float(x), __uint_as_float(y));
            };
            tc::stm4_trans(dst + b * 8 * 256, pack(lo[4 * b], lo[4 * b + 1]),
                           pack(lo[4 * b + 2], lo[4 * b + 3]), pack(hi[4 * b], hi[4 * b + 1]),
                           pack(hi[4 * b + 2], hi[4 * b + 3]));
          }
          named_sync(bar, 128);
          const int pc = et & 15, n = t.m * kProdRows + 8 * pc;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = (et >> 4) + 8 * k;
            if (c0 + row < t.n && n < p.N)
              *reinterpret_cast<uint4*>(p.y + (size_t)(t.r0 + c0 + row) * p.N + n) =
                  *reinterpret_cast<const uint4*>(stage + row * 256 + ((pc ^ (row & 7)) << 4));
          }
        } else {
          // this thread's gates (lo) and ups (hi) of neurons 2 (lane / 4) + {0, 1}
          // of the warp's 16, columns 8 b + 2 (lane % 4) + {0, 1}
          float h[16];
          uint32_t mx[8];   // magnitudes of columns 2 b + j, over those two neurons
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float gate = __uint_as_float(lo[x]), up = __uint_as_float(hi[x]);
            // SiLU with e = exp(-|gate|) <= 1: nothing overflows, and the divisor
            // stays where the short division is good to two units. The short
            // exp is off by 2 + 1.2 |gate| units, far below the 2^-4 that E4M3
            // keeps. Over eight inputs of 4096 tokens the codes' error against 64
            // bits is 1.16e-4 so, 1.15e-4 with expf and 1.19e-4 with exact division
            // as well (the FP32 sum's order decides); at 2048 tokens of 4-bit
            // weights 8.4e-5, 7.9e-5 and 8.2e-5. Those take 98.3, 100.6, 107.5 us
            // and 53.8, 55.1, 61.6.
            const float e = __expf(-fabsf(gate));
            h[x] = __fdividef(gate < 0.f ? gate * e : gate, 1.0f + e) * up;
          }
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const int x = (b >> 1) * 4 + (b & 1);
            mx[b] = max(__float_as_uint(h[x]) & 0x7fffffffu, __float_as_uint(h[x + 2]) & 0x7fffffffu);
          }
          // over the warp's 16 neurons (lane bits 4, 3, 2), each lane keeping
          // half of its columns a step and one in the end
#pragma unroll
          for (int w = 4; w > 0; w >>= 1) {
            const bool high = (lane & (4 * w)) != 0;
#pragma unroll
            for (int b = 0; b < w; ++b) {
              const uint32_t give = high ? mx[b] : mx[b + w], keep = high ? mx[b + w] : mx[b];
              mx[b] = max(keep, __shfl_xor_sync(kFull, give, 4 * w));
            }
          }
          const int v = lane >> 2, col = 8 * (v >> 1) + 2 * (lane & 3) + (v & 1);
          // the block's other 16 neurons are in the neighbouring warp
          uint32_t* am = amax + (chunk & 1) * 128;
          am[q * 32 + col] = mx[0];
          named_sync(bar + 1 + (q >> 1), 64);
          const uint32_t sc = mx_scale_code(max(mx[0], am[(q ^ 1) * 32 + col]));
          const int I = p.N / 2, nb = t.m * 2 + (q >> 1);   // block of 32 neurons
          if ((q & 1) == 0 && c0 + col < t.n && nb * 32 < I)
            p.scales[(size_t)(t.r0 + c0 + col) * (I / 32) + nb] = (uint8_t)sc;
          inv[col] = mx_inverse(sc);
          __syncwarp();
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int cb = 8 * b + 2 * (lane & 3);
            const float2 f = *reinterpret_cast<const float2*>(inv + cb);
            uint16_t* dst = reinterpret_cast<uint16_t*>(stage + cb * kProdCodePitch + 16 * q) + v;
            dst[0] = (uint16_t)e4m3x2(h[4 * b] * f.x, h[4 * b + 2] * f.x);
            dst[kProdCodePitch / 2] = (uint16_t)e4m3x2(h[4 * b + 1] * f.y, h[4 * b + 3] * f.y);
          }
          named_sync(bar, 128);
          const int row = et >> 2, n = t.m * 64 + 16 * (et & 3);
          if (c0 + row < t.n && n < I)
            *reinterpret_cast<uint4*>(p.codes + (size_t)(t.r0 + c0 + row) * I + n) =
                *reinterpret_cast<const uint4*>(stage + row * kProdCodePitch + 16 * (et & 3));
        }
      }
      tc::fence_before();
      __syncwarp();
      tc::arrive_at(d_empty0 + 8 * buf, rank != 0);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  // Before a CTA leaves and tensor memory is released, every MMA is done (they
  // read both CTAs' shared memory and arrive on both CTAs' barriers), and with
  // them every copy into a stage that they read, which is all there are unless
  // the pair is dead. Then copies of this CTA may still be in flight, and those
  // of the second CTA complete on the first one's barriers: both stay for a time
  // that is hundreds of times a copy's.
  if (warp == 1) prod_wait_end(drain, 0, p.err);
  if (warp == 0 && *dead)
    for (int i = 0; i < kProdSettleSleeps; ++i) __nanosleep(kWaitSuspendNs);
  __syncwarp();
  cluster_sync();   // no CTA leaves while the other may still reach into it
  tc::fence_after();
  if (warp == 1) tc::tmem_dealloc2(*tmem_slot, kProdTmemCols);
}

}  // namespace moe
