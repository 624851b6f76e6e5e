/*
 * moe_prompt.h -- the operators around the routed experts for calls of many
 * tokens (prompts, large batches), in libmoe_decode.so beside the decode
 * layer of moe_decode.h. Together they are the mixture-of-experts half of a
 * transformer block with the activations between them in MXFP8, the format
 * the GC-MoE summary (onedev.kr/papers/1690, "How it is used") names for
 * routed activations (E4M3 codes, one UE8M0 scale per 32 values along the
 * reduction axis):
 *
 *   moe_add_rms_norm    s = bf16(x + residual);  n = s / rms(s) * weight
 *   moe_group           counting sort of the routed (token, slot) pairs by expert
 *   moe_product_run     per expert, its group's rows times its MXFP8 or MXFP4
 *                       weights: plain (the down projection), or gate and up
 *                       finished to SiLU(g) * u and requantised to MXFP8
 *   moe_combine         out[t] = residual[t] + sum_j w[t, j] * y[slot of (t, j)]
 *
 * Conventions are moe_decode.h's: contiguous row-major tensors, device
 * pointers, work enqueued on `stream` without waiting, argument errors found
 * on the host (nothing is enqueued then), results bitwise reproducible.
 * T = 0 or R = 0 is a successful no-op. Calls keep no state between them
 * except a product handle's error word.
 *
 * MXFP8 quantisation, wherever it is an output: per block of 32 values along
 * a row, E = floor(log2 amax) - 8 clamped to [-127, 127] (0 for a block of
 * zeros), scale code E + 127, codes E4M3(v * 2^-E) rounded to nearest even
 * and saturated to 448. A block that holds an infinity or a NaN becomes NaN
 * as a whole (scale code 255, every code 0x7F).
 */
#ifndef MOE_PROMPT_H
#define MOE_PROMPT_H

#include <stdint.h>

#include "moe_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition and root-mean-square norm of T rows of H values, one
 * pass over the data:
 *   s[t]  = bf16(x[t] + residual[t])           (x[t] when residual is NULL)
 *   n[t]  = s[t] * rsqrt(mean(s[t]^2) + eps) * weight    in FP32
 * Outputs, each optional but at least one of y and codes:
 *   sum     bf16 [T, H]   s; NULL to skip; may be `x` or `residual` itself
 *   y       bf16 [T, H]   bf16(n)
 *   codes   uint8 [T, H], scales uint8 [T, H/32]   MXFP8(n), both or neither
 * x, residual bf16 [T, H], weight bf16 [H]. H in 1..16384, a multiple of 32
 * for MXFP8. bf16 tensors 2-byte aligned; 16-byte aligned ones with H a
 * multiple of 8 take the vector form.
 */
moe_status_t moe_add_rms_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual,
                              const uint16_t* weight, float eps, uint16_t* sum, uint16_t* y,
                              uint8_t* codes, uint8_t* scales, void* stream);

/*
 * Groups the routed slots p = t * k + j by expert, keeping their order:
 *   topk_ids  int32 [T, k]
 *   offsets   int32 [E + 1]  group e is rows offsets[e] .. offsets[e + 1] - 1
 *   rows      int32 [T * k]  token of every grouped row; -1 from offsets[E] on
 *   slots     int32 [T, k]   grouped row of every slot; -1 where its id lies
 *                            outside [0, E) (an unused slot: it joins no
 *                            group, and offsets[E] < T * k tells that some did)
 * E in 1..1024, T * k <= 2^30.
 */
moe_status_t moe_group(int32_t T, int32_t k, int32_t E, const int32_t* topk_ids, int32_t* offsets,
                       int32_t* rows, int32_t* slots, void* stream);

/*
 * Routing-weighted sum of a token's expert rows, in slot order, in FP32:
 *   out[t] = bf16(residual[t] + sum_j w[t, j] * y[slots[t, j]])
 *   y         bf16 [R, H]
 *   slots     int32 [T, k]; a slot outside [0, R) contributes nothing
 *   w         float [T, k]
 *   residual  bf16 [T, H], or NULL for none
 *   out       bf16 [T, H]; may be `residual` itself
 */
moe_status_t moe_combine(int32_t T, int32_t k, int32_t H, int32_t R, const uint16_t* y,
                         const int32_t* slots, const float* w, const uint16_t* residual,
                         uint16_t* out, void* stream);

/* ---- ragged products grouped by expert ---------------------------------- */

/* Flags of moe_product_config_t (MOE_FLAG_MXFP4 as for the decode layer). */
#define MOE_PRODUCT_SILU_MUL 0x10u /* the N = 2I rows of an expert are I gate
                                      rows, then I up rows; the output is
                                      MXFP8(SiLU(gate) * up) of I values */

typedef struct {
  int32_t E;      /* experts, 1..1024 */
  int32_t N;      /* weight rows of an expert: a multiple of 8; with
                     MOE_PRODUCT_SILU_MUL a multiple of 64 */
  int32_t K;      /* reduction length: a multiple of 32; of 128 with MOE_FLAG_MXFP4 */
  uint32_t flags; /* MOE_FLAG_MXFP4, MOE_PRODUCT_SILU_MUL */
} moe_product_config_t;

typedef struct moe_product* moe_product_t;

/*
 * A handle over one stack of expert weights on the current device.
 *   w         uint8 [E, N, K] E4M3 codes, or [E, N, K/2] packed E2M1 codes;
 *             32-byte aligned, borrowed until moe_product_destroy
 *   w_scales  uint8 [E, N, K/32] UE8M0; read here only: the handle keeps a
 *             copy in the order in which the tensor cores take them (padded to
 *             128 rows and 128 K elements), laid out by a kernel on `stream`,
 *             for which this call waits (so not while a graph is captured)
 * Allocates that copy and the error word, one CUDA event and one non-blocking
 * stream (for reading the error word).
 */
moe_status_t moe_product_create(const moe_product_config_t* cfg, const uint8_t* w,
                                const uint8_t* w_scales, moe_product_t* out, void* stream);
moe_status_t moe_product_destroy(moe_product_t handle);

/*
 * For every expert e and row q in [offsets[e], offsets[e + 1]), with
 * a[q] = the MXFP8 row rows[q] of codes (row q itself when rows is NULL):
 *   plain     y[q, n] = bf16(sum_K W[e, n, K] * a[q, K])
 *   SILU_MUL  h[q, i] = SiLU(sum W[e, i] a[q]) * (sum W[e, I + i] a[q]),
 *             codes[q], scales[q] = MXFP8(h[q])
 * with FP32 accumulation on the tensor cores' block-scaled 8-bit MMA. The
 * current device has to be the handle's.
 *   R         rows of the output; offsets are read as clamped to [0, R], rows
 *             outside every group are left as they are
 *   A         rows of a
 *   a         uint8 [A, K] E4M3, 16-byte aligned;  a_scales uint8 [A, K/32]
 *   offsets   int32 [E + 1], on the device, ascending
 *   rows      int32 [R] or NULL (then A = R); entries of a group's rows lie in
 *             [0, A) (others are read as the nearest bound)
 *   y         bf16 [R, N], 16-byte aligned (plain);  codes uint8 [R, N/2] and
 *             scales uint8 [R, N/64] (SILU_MUL); the other outputs NULL
 */
moe_status_t moe_product_run(moe_product_t handle, int32_t R, int32_t A, const uint8_t* a,
                             const uint8_t* a_scales, const int32_t* offsets, const int32_t* rows,
                             uint16_t* y, uint8_t* codes, uint8_t* scales, void* stream);

/* Read and clear, in one step, the handle's device error word
 * (MOE_DEVICE_TIMEOUT: a bounded device wait gave up and outputs are undefined)
 * after waiting for the handle's latest run that was not being captured into a
 * graph, and moe_product_get_error for `stream` too (which covers graphs
 * replayed there). The return value is MOE_ERR_DEVICE_FAULT when a bit was set. */
moe_status_t moe_product_get_error(moe_product_t handle, void* stream, uint32_t* device_flags);
moe_status_t moe_product_get_error_latest(moe_product_t handle, uint32_t* device_flags);

/* Test support: in the next run that launches something, the MMAs wait for an
 * arrival that nothing makes, with a limit of some milliseconds instead of a
 * second. Every role gives up, the launch completes with unspecified outputs,
 * the handle reports MOE_DEVICE_TIMEOUT and its later runs are unaffected. */
moe_status_t moe_product_arm_timeout(moe_product_t handle);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PROMPT_H */
