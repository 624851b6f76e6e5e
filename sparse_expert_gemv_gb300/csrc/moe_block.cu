// Host side of the C ABI declared in include/moe_block.h: argument checks,
// launch shapes and the dense product's handle.
#include "moe_block.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <new>

#include "moe_block_rows.cuh"
#include "moe_dense.cuh"
#include "moe_host.cuh"

struct moe_dense : moe::Handle {
  moe_dense_config_t cfg;
  int num_sms;
  CUtensorMap tm_tiles, tm_split;   // the weight as the two kernels take it
  int groups;                       // tm_tiles has groups of 16 rows
  const uint16_t* weight;
  const uint16_t* bias;
  std::atomic<bool> armed;   // the next run's waits run out (moe_dense_arm_timeout)
};

namespace {

// Rows of a call and outputs of a product: what rounding up to a tile does not take
// past 32 bits.
constexpr int32_t kMaxRows = 0x7fffff00;

using moe::aligned;
using moe::launch;
using moe::overlap;
using moe::Span;

// ---- routing -----------------------------------------------------------------

// What route_row with R experts a lane needs of p.
template <int R>
void route_prepare(moe::RouteParams& p) {
  p.vec = p.E % R == 0 && aligned(p.logits, std::min(16, R * (p.bf16 ? 2 : 4)));
  p.lane_shift = -1;
  if (p.per % R == 0)
    for (int s = 0; s <= 5; ++s)
      if (p.per / R == 1 << s) p.lane_shift = s;
  p.bias_vec = p.E % R == 0 && aligned(p.bias, 16);
  p.smem = std::max(p.E * (int)sizeof(double), 128 * (R + 1));   // route_slow's, sorted keys
}

template <int R>
moe_status_t route_launch(moe::RouteParams p, void* stream) {
  route_prepare<R>(p);
  const size_t smem = (size_t)moe::kRouteWarps * p.smem;
  const unsigned grid = (p.T + moe::kRouteWarps - 1) / moe::kRouteWarps;
  return p.bf16 && !p.bias ? launch(moe::moe_route_experts_rows<R, true>, grid,
                                    moe::kRouteWarps * 32, smem, stream, 1, p)
                           : launch(moe::moe_route_experts_rows<R, false>, grid,
                                    moe::kRouteWarps * 32, smem, stream, 1, p);
}

// W lanes a token; rows that need it are decided by a whole warp.
template <int W>
moe_status_t route_packed_launch(moe::RouteParams p, void* stream) {
  route_prepare<W>(p);
  p.packed_shift = 0;
  while (32 << p.packed_shift < p.per) ++p.packed_shift;
  const int tokens = moe::kRouteWarps * (32 / W);
  const size_t smem = (size_t)moe::kRouteWarps * p.smem;
  const unsigned grid = (p.T + tokens - 1) / tokens;
  return p.bf16 && !p.bias ? launch(moe::moe_route_experts_packed<W, true>, grid,
                                    moe::kRouteWarps * 32, smem, stream, 1, p)
                           : launch(moe::moe_route_experts_packed<W, false>, grid,
                                    moe::kRouteWarps * 32, smem, stream, 1, p);
}

// Whether moe_route_experts_packed takes a call: many tokens, where it is the faster
// one (figures at the kernel), lanes of 32 experts read in aligned vectors, groups of
// whole lanes (and 2^n of them).
bool route_packed(const moe::RouteParams& p) {
  return p.T >= 4096 && (p.E == 64 || p.E == 128 || (p.E == 256 && !p.bias)) && p.k <= 8 &&
         aligned(p.logits, 16) && aligned(p.bias, 16) &&
         (p.groups == 1 || (p.per % 32 == 0 && (p.per / 32 & (p.per / 32 - 1)) == 0));
}

// ---- norms -------------------------------------------------------------------

// NV vectors a thread; rows of at most 32 threads several a CTA.
template <int V, int NV>
moe_status_t norm_pair_rows(const moe::NormPairParams& p, void* stream) {
  const int threads = ((p.H / V + NV - 1) / NV + 31) / 32 * 32;
  const int rows = threads == 32 ? 8 : 1;
  const unsigned grid = (p.T + rows - 1) / rows;
  const dim3 block(threads, rows);
  return p.gate && !p.gate_row
             ? launch(moe::moe_norm_add_norm_rows<V, NV, true>, grid, block, 0, stream, 1, p)
             : launch(moe::moe_norm_add_norm_rows<V, NV, false>, grid, block, 0, stream, 1, p);
}

moe_status_t norm_pair_launch(const moe::NormPairParams& p, bool vec, void* stream) {
  if (!vec) {
    if (p.H <= 1024) return norm_pair_rows<1, 1>(p, stream);
    if (p.H <= 4096) return norm_pair_rows<1, 4>(p, stream);
    return norm_pair_rows<1, 16>(p, stream);
  }
  const int nv = p.H / 8;
  // Few values: as many threads as a row takes, for the latency (us of 300 rows of
  // 1024 with one, two and four vectors a thread 2.1, 2.4, 3.4). Many: more values a
  // thread spread the two reductions' instructions further (16384 rows of 2048
  // 50 / 47 / 48, 8191 of 7168 90 / 87 / 71, with eight 72; 2000 of 16384 with two 57,
  // with eight 46).
  if ((int64_t)p.T * nv < 65536)
    return nv <= 1024 ? norm_pair_rows<8, 1>(p, stream) : norm_pair_rows<8, 2>(p, stream);
  if (nv <= 32) return norm_pair_rows<8, 1>(p, stream);
  if (nv <= 256) return norm_pair_rows<8, 2>(p, stream);
  if (nv <= 1024) return norm_pair_rows<8, 4>(p, stream);
  return norm_pair_rows<8, 8>(p, stream);
}

// ---- dense products ------------------------------------------------------------

bool is_silu(const moe_dense_config_t& c) { return c.activation == MOE_ACT_SILU_MUL; }

// bf16 [rows, K] in boxes of `box` rows by one stage of K (64 values)
bool encode_rows(CUtensorMap* tm, const void* base, int rows, int K, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
  const cuuint32_t b[2] = {moe::kDenseK, (cuuint32_t)box};
  return moe::encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, b);
}

// The gate and up rows of neurons 16 g.. as [g][gate, up][16][K], four groups a box.
bool encode_groups(CUtensorMap* tm, const void* w, int I, int K) {
  const cuuint64_t row = (cuuint64_t)K * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)K, 16, 2, (cuuint64_t)I / 16};
  const cuuint64_t strides[3] = {row, I * row, 16 * row};
  const cuuint32_t box[4] = {moe::kDenseK, 16, 2, 4};
  return moe::encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, w, dims, strides, box);
}

bool encode_weight(moe_dense* m, const uint16_t* w) {
  const moe_dense_config_t& c = m->cfg;
  if (!is_silu(c))
    return encode_rows(&m->tm_tiles, w, c.N, c.K, moe::kDenseRows) &&
           encode_rows(&m->tm_split, w, c.N, c.K, moe::kDenseRows);
  m->groups = c.N / 2 % 16 == 0;
  return (m->groups ? encode_groups(&m->tm_tiles, w, c.N / 2, c.K)
                    : encode_rows(&m->tm_tiles, w, c.N, c.K, 16)) &&
         encode_rows(&m->tm_split, w, c.N, c.K, moe::kDenseRows / 2);
}

// How a call is cut.
struct DensePlan {
  bool split;
  int nt;       // rows of x a tile
  int S;        // parts of K (split)
  int stages;   // of the ring
  double us;    // by the model below
};

// Shared memory of a CTA of moe_dense_split: half an SM's or all of it. A third CTA
// never fits on an SM, so that the tensor memory of those that do is never more
// than there is: none waits for it while it holds up its cluster.
constexpr int kSplitHalf = 113 * 1024, kSplitFull = 226 * 1024, kSplitSmemMin = 78 * 1024;

int split_stages(int nt, int S, int room) {
  room -= 1024 + moe::kSplitBars + moe::split_sum_bytes(nt, S);
  return std::min(moe::kSplitStages, room / moe::split_stage_bytes(nt));
}

size_t split_smem(const DensePlan& p) {
  const int need = 1024 + moe::kSplitBars + p.stages * moe::split_stage_bytes(p.nt) +
                   moe::split_sum_bytes(p.nt, p.S);
  return std::max(need, kSplitSmemMin);
}

// The cheapest cut by a model of its time, in us. Its constants were fitted to some
// 500 timings (30 shapes from 1 to 8192 rows, every cut of each, inputs beyond L2);
// its choices are on average 1.1 % slower than the best of them, 12 % at worst. All
// but a few of them had bf16 outputs of 16-byte rows: the model does not know what the
// element-wise epilogue (p.vec = 0) or that of FP32 outputs takes.
//   split   a start, then the stages of a CTA at what an SM, shared by the CTAs on
//           it, or all of L2 delivers, or its ring's latency allows where it turns;
//           the parts' exchange; clusters that find no room wait for a round more
//   tiles   rounds of tiles over the pairs, whose stages take their MMAs or their
//           bytes' way into an SM
DensePlan plan_dense(const moe_dense_config_t& c, int R, bool out_float, int num_sms) {
  const bool silu = is_silu(c);
  const int M = silu ? c.N / 2 : c.N;
  const int nk = (c.K + moe::kDenseK - 1) / moe::kDenseK;
  constexpr double kStart = 0.16, kL2 = 14.7e6;   // us, bytes a us
  DensePlan best{false, 0, 1, 0, 0.0};
  auto take = [&](const DensePlan& p) {
    if (!best.nt || p.us < best.us) best = p;
  };
  const int pairs = std::max(1, num_sms / 2);
  for (int nt = out_float ? moe::kDenseFloatCols : moe::kDenseCols; nt >= 32; nt -= 32) {
    if (nt - 32 >= R) continue;
    const double tiles = std::ceil(M / (silu ? 128.0 : 256.0)) * std::ceil((double)R / nt);
    const double bytes = moe::DenseSmem::stage(nt);   // a stage's, of one CTA
    const double stage = std::max({0.0012 * nt, bytes / 108.8e3,
                                   std::min<double>(tiles, pairs) * 2 * bytes / kL2});
    take({false, nt, 1, moe::DenseSmem::stages(nt), kStart + 1.2 + std::ceil(tiles / pairs) * nk * stage +
                               0.0082 * std::min(nt, R)});
  }
  const double hbm = 2.0 * c.K * ((double)c.N + R) / 6.8e6;
  for (int nt = moe::kSplitMaxCols; nt >= 16; nt -= 16) {
    if (nt - 16 >= R) continue;
    const int n = std::min(nt, R), bytes = moe::split_stage_bytes(nt);
    for (int S = 1; S <= 8 && S <= nk; S *= 2) {
      // FP32 outputs: an accumulator takes kDensePart stages at most (and fewer than
      // eight parts no more than two accumulators)
      if (out_float && (nk + S - 1) / S > moe::kDensePart * (S < 8 ? 2 : moe::split_accs(nt))) continue;
      for (const int room : {kSplitFull, kSplitHalf}) {
        const int stages = split_stages(nt, S, room);
        if (stages < 2) continue;
        const bool half = room == kSplitHalf;
        const double ctas = std::ceil(M / (silu ? 64.0 : 128.0)) * std::ceil((double)R / nt) * S;
        // CTAs that run at once: clusters of 4 and 8 leave SMs of a GPC over
        const double most = num_sms * (half ? (S == 8 ? 288 : S == 4 ? 296 : 304)
                                            : (S == 8 ? 120 : S == 4 ? 144 : 152)) / 152.0;
        const double run = std::min(ctas, most), shared = half ? std::min(2.0, std::ceil(run / num_sms)) : 1;
        const double g = std::ceil((double)nk / S);
        const double rate = std::min(153e3 / shared, g > stages ? stages * bytes / 1.83 : 153e3);
        const double stream = std::max(g * bytes / rate, run * g * bytes / kL2);
        const double per = 1.65 + stream + n * (0.005 / S + (S > 1 ? 0.0112 : 0)) + 0.118 * (S - 1);
        take({true, nt, S, stages, kStart + std::max(std::ceil(ctas / most) * per, hbm + 1.65)});
      }
    }
  }
  return best;
}

int log2_of(int v) {
  int l = 0;
  while (1 << (l + 1) <= v) ++l;
  return l;
}

constexpr size_t kDenseSmem = moe::kDenseSmemMax + 1024;
static_assert(kDenseSmem <= 232448, "shared memory of a CTA");

template <bool SILU>
bool set_dense_attributes() {
  return cudaFuncSetAttribute(moe::moe_dense_tiles<SILU, false>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)kDenseSmem) == cudaSuccess &&
         cudaFuncSetAttribute(moe::moe_dense_tiles<SILU, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)kDenseSmem) == cudaSuccess &&
         cudaFuncSetAttribute(moe::moe_dense_split<SILU>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSplitFull) == cudaSuccess;
}

moe_status_t check_dense(const moe_dense_config_t& c) {
  if (c.N < 1 || c.K < 1 || c.activation < MOE_ACT_NONE || c.activation > MOE_ACT_SILU_MUL)
    return MOE_ERR_INVALID_ARG;
  return c.K % 8 || c.K > kMaxRows || c.N > kMaxRows || (is_silu(c) && c.N % 2)
             ? MOE_ERR_UNSUPPORTED_SHAPE
             : MOE_OK;
}

// Tiles along M and R and the CTAs of a launch; false when there are too many.
bool dense_grid(const moe_dense_config_t& c, const DensePlan& p, int R, int num_sms, int& mt, int& tt,
                int& ctas) {
  const int64_t M = is_silu(c) ? c.N / 2 : c.N, rows = (p.split ? 128 : 256) / (is_silu(c) ? 2 : 1);
  if (R > kMaxRows) return false;
  const int64_t m = (M + rows - 1) / rows, t = ((int64_t)R + p.nt - 1) / p.nt;
  if (m * t * p.S > 0x3fffffff) return false;
  mt = (int)m;
  tt = (int)t;
  ctas = (int)(p.split ? m * t * p.S : 2 * std::min<int64_t>(std::max(1, num_sms / 2), m * t));
  return true;
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
  if (c.E > moe::kRouteMaxE || c.k > 32 || c.groups > 32 || T > kMaxRows)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c.E % c.groups || c.k > c.top_groups * (c.E / c.groups)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !w) return MOE_ERR_INVALID_ARG;
  const bool bf16 = (c.flags & MOE_ROUTE_BF16) != 0;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(w, 4))
    return MOE_ERR_MISALIGNED;
  const size_t rows = T, size = bf16 ? 2 : 4;
  const Span in{logits, rows * c.E * size}, add{bias, (size_t)c.E * 4};
  const Span out{ids, rows * c.k * 4}, weights{w, rows * c.k * 4};
  if (overlap(out, in) || overlap(out, add) || overlap(weights, in) || overlap(weights, add) ||
      overlap(out, weights))
    return MOE_ERR_INVALID_ARG;
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
  if (route_packed(p)) {
    if (c.E == 64) return route_packed_launch<2>(p, stream);
    if (c.E == 128) return route_packed_launch<4>(p, stream);
    return route_packed_launch<8>(p, stream);
  }
  if (c.E <= 32) return route_launch<1>(p, stream);
  if (c.E <= 64) return route_launch<2>(p, stream);
  if (c.E <= 128) return route_launch<4>(p, stream);
  if (c.E <= 256) return route_launch<8>(p, stream);
  if (c.E <= 512) return route_launch<16>(p, stream);
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
  if (H > moe::kNormMaxH || (codes && H % 32) || T > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!x || !residual || !sum || (pre_weight == nullptr) != (!y && !codes) ||
      (codes == nullptr) != (scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  for (const uint16_t* a : {x, residual, post_weight, pre_weight, gate,
                            const_cast<const uint16_t*>(sum), const_cast<const uint16_t*>(y)})
    if (!aligned(a, 2)) return MOE_ERR_MISALIGNED;
  // A thread reads its elements of x and residual before it writes the same ones of
  // sum or y, so that those may lie there; nothing else may.
  const size_t all = (size_t)T * H * 2, row = (size_t)H * 2;
  const Span outs[] = {{sum, all}, {y, all}, {codes, all / 2}, {scales, all / 64}};
  const Span ins[] = {{x, all}, {residual, all}, {post_weight, row}, {pre_weight, row},
                      {gate, flags & MOE_NORM_GATE_FULL  ? all
                             : flags & MOE_NORM_GATE_ROW ? (size_t)T * 2
                                                         : row}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < 5; ++j)
      if (overlap(outs[i], ins[j]) && !(i < 2 && j < 2 && outs[i].at == ins[j].at))
        return MOE_ERR_INVALID_ARG;
  }
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
  p.T = T;
  p.H = H;
  p.inv_h = 1.f / (float)H;
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
  return norm_pair_launch(p, vec, stream);
}

moe_status_t moe_dense_create(const moe_dense_config_t* cfg, const uint16_t* weight,
                              const uint16_t* bias, moe_dense_t* out) {
  if (out) *out = nullptr;
  if (!cfg || !out || !weight) return MOE_ERR_INVALID_ARG;
  const moe_dense_config_t c = *cfg;
  const moe_status_t st = check_dense(c);
  if (st != MOE_OK) return st;
  if (!aligned(weight, 16) || !aligned(bias, 2)) return MOE_ERR_MISALIGNED;
  moe_dense* m = new (std::nothrow) moe_dense();
  if (!m) return MOE_ERR_CUDA;
  m->cfg = c;
  m->weight = weight;
  m->bias = bias;
  const bool ok =
      cudaGetDevice(&m->device) == cudaSuccess &&
      cudaDeviceGetAttribute(&m->num_sms, cudaDevAttrMultiProcessorCount, m->device) ==
          cudaSuccess &&
      encode_weight(m, weight) &&
      (is_silu(c) ? set_dense_attributes<true>() : set_dense_attributes<false>()) &&
      m->acquire(nullptr) && cudaStreamSynchronize(nullptr) == cudaSuccess;
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
  const bool silu = is_silu(c);
  const size_t outputs = (size_t)R * (silu ? c.N / 2 : c.N);
  const Span result{out, outputs * (out_float ? 4 : 2)};
  if (overlap(result, {x, (size_t)R * c.K * 2}) ||
      overlap(result, {m->weight, (size_t)c.N * c.K * 2}) ||
      overlap(result, {m->bias, (size_t)c.N * 2}) ||
      (overlap(result, {residual, outputs * 2}) && (out_float || out != residual)))
    return MOE_ERR_INVALID_ARG;
  const DensePlan plan = plan_dense(c, R, out_float != 0, m->num_sms);
  moe::DenseParams p;
  p.M = silu ? c.N / 2 : c.N;
  p.nt = plan.nt;
  p.nk = (c.K + moe::kDenseK - 1) / moe::kDenseK;
  int ctas;
  if (!dense_grid(c, plan, R, m->num_sms, p.mt, p.tt, ctas)) return MOE_ERR_UNSUPPORTED_SHAPE;
  p.tm_w = plan.split ? m->tm_split : m->tm_tiles;
  p.groups = m->groups;
  if (!encode_rows(&p.tm_x, x, R, c.K, plan.split ? plan.nt : plan.nt / 2)) return MOE_ERR_CUDA;
  p.vec = p.M % 8 == 0 && aligned(out, 16) && aligned(residual, 16);
  if (!plan.split && !out_float && p.vec &&
      !(encode_rows(&p.tm_out, out, R, p.M, 32) &&
        (!residual || encode_rows(&p.tm_res, residual, R, p.M, 32))))
    return MOE_ERR_CUDA;
  p.bias = m->bias;
  p.residual = residual;
  p.out = out;
  p.err = m->d_err;
  p.R = R;
  p.act = c.activation;
  p.out_float = out_float != 0;
  p.stages = plan.stages;
  const bool armed = m->armed.exchange(false, std::memory_order_relaxed);
  p.polls = armed ? 50 : moe::kMbarPolls;   // a millisecond
  p.withheld = armed;
  moe_status_t st;
  if (plan.split)
    st = launch(silu ? moe::moe_dense_split<true> : moe::moe_dense_split<false>, ctas,
                moe::kSplitThreads, split_smem(plan), stream, plan.S, p, log2_of(plan.S));
  else
    st = launch(silu ? (out_float ? moe::moe_dense_tiles<true, true> : moe::moe_dense_tiles<true, false>)
                     : (out_float ? moe::moe_dense_tiles<false, true> : moe::moe_dense_tiles<false, false>),
                ctas,
                moe::kDenseThreads, kDenseSmem, stream, 2, p);
  if (st == MOE_OK) m->mark_done(static_cast<cudaStream_t>(stream));
  return st;
}

moe_status_t moe_dense_plan(const moe_dense_config_t* cfg, int32_t R, int32_t out_float,
                            int32_t num_sms, moe_dense_plan_t* out) {
  if (!cfg || !out || R < 1 || num_sms < 1) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_dense(*cfg);
  if (st != MOE_OK) return st;
  const bool silu = is_silu(*cfg);
  const DensePlan p = plan_dense(*cfg, R, out_float != 0, num_sms);
  int mt, tt, ctas;
  if (!dense_grid(*cfg, p, R, num_sms, mt, tt, ctas)) return MOE_ERR_UNSUPPORTED_SHAPE;
  out->split = p.split;
  out->nt = p.nt;
  out->parts = p.S;
  out->stages = p.stages;
  out->smem = (int)(p.split ? split_smem(p) : kDenseSmem);
  out->ctas = ctas;
  return MOE_OK;
}

moe_status_t moe_dense_arm_timeout(moe_dense_t m) {
  if (!m) return MOE_ERR_INVALID_ARG;
  m->armed.store(true, std::memory_order_relaxed);
  return MOE_OK;
}

moe_status_t moe_dense_get_error(moe_dense_t m, void* stream, uint32_t* device_flags) {
  if (device_flags) *device_flags = 0;
  if (!m || !device_flags) return MOE_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return MOE_ERR_CUDA;
  return m->read_error(device_flags);
}

}  // extern "C"
