/*
 * moe_block.h -- what a transformer block with routed experts needs between
 * them, in libmoe_decode.so beside the decode layer of moe_decode.h and the
 * prompt operators of moe_prompt.h:
 *
 *   moe_route_experts   the router's choice: softmax or sigmoid scores, a bias
 *                       that balances the choice, groups of experts, top-k,
 *                       renormalised and scaled weights
 *   moe_norm_add_norm   the norm after a block, its gate and scale, the residual
 *                       addition and the norm before the next block
 *   moe_dense_run       a matrix product of bf16 rows with bias, activation and
 *                       residual in its epilogue: router logits, shared experts,
 *                       projections
 *
 * Conventions are moe_decode.h's: contiguous row-major tensors, device
 * pointers, work enqueued on `stream` without waiting, argument errors found
 * on the host (nothing is enqueued then), results bitwise reproducible.
 * T = 0 or R = 0 is a successful no-op. Calls keep no state between them
 * except a dense product's error word. An output shares no memory with another
 * tensor of its call, but for those that are named as the same below; other calls
 * are refused (MOE_ERR_INVALID_ARG).
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include <stdint.h>

#include "moe_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- routing --------------------------------------------------------------- */

/* Flags of moe_route_config_t. */
#define MOE_ROUTE_BF16 0x1u        /* logits are bf16, not float */
#define MOE_ROUTE_SIGMOID 0x2u     /* scores are sigmoids, not a softmax */
#define MOE_ROUTE_GROUP_TOP2 0x4u  /* a group's score is the sum of its two largest
                                      choice scores (its one, where it has but one),
                                      not its largest */
#define MOE_ROUTE_RENORMALIZE 0x8u /* weights are divided by their sum */

typedef struct {
  int32_t E;          /* experts, 1..1024 */
  int32_t k;          /* experts a token takes, 1..32 */
  int32_t groups;     /* 1..32, a divisor of E; experts of a group are neighbours */
  int32_t top_groups; /* groups a token's experts come from, 1..groups;
                         k <= top_groups * E / groups */
  float scale;        /* of the weights, finite */
  uint32_t flags;     /* MOE_ROUTE_* */
} moe_route_config_t;

/*
 * For every token t:
 *   s[e]    = softmax or sigmoid of logits[t]
 *   c[e]    = s[e] + bias[e]       (the choice scores; s[e] when bias is NULL)
 *   the top_groups groups of the best group scores are kept, and of their
 *   experts the k of the best choice scores chosen
 *   ids[t]  = the chosen experts, best choice score first
 *   w[t]    = scale * s[ids] (/ sum of s[ids], with MOE_ROUTE_RENORMALIZE)
 * Of equal scores the lower index is the better one. The choice is that of
 * FP64 arithmetic on the given inputs, whatever lies how close: scores too close
 * for FP32 are compared in FP64. (Without a bias experts compare by their logits,
 * which is exact; beside a bias a score below 2^-53 of it is none.)
 * An expert whose logit is NaN or -inf is switched off: it counts in no sum and
 * is never chosen; one whose bias is NaN or -inf is never chosen. Slots for
 * which no expert is left get the id -1 and the weight 0. moe_group takes -1 as an
 * unused slot. To the decode layer it is an id outside [0, E) like any other: it
 * adds nothing and sets MOE_DEVICE_BAD_ID, which then tells of no fault. Softmax
 * over infinite logits is shared by those alone; chosen scores that are all 0 give
 * weights of 0.
 *   logits  float or bf16 [T, E]
 *   bias    float [E] or NULL
 *   ids     int32 [T, k];  w float [T, k]
 */
moe_status_t moe_route_experts(const moe_route_config_t* cfg, int32_t T, const void* logits,
                               const float* bias, int32_t* ids, float* w, void* stream);

/* ---- norms around a block's end --------------------------------------------- */

/* Flags of moe_norm_add_norm; at most one of the gate's shape and one of its
 * function. */
#define MOE_NORM_GATE_ROW 0x1u      /* gate is [T], one value a row */
#define MOE_NORM_GATE_FULL 0x2u     /* gate is [T, H] */
#define MOE_NORM_GATE_SIGMOID 0x4u  /* the branch is multiplied by sigmoid(gate) */
#define MOE_NORM_GATE_TANH 0x8u     /* or by tanh(gate) */
#define MOE_NORM_UNIT_OFFSET 0x10u  /* norm weights are stored less one */

/*
 * The end of one block and the start of the next, per row of H values:
 *   p    = x * rsqrt(mean(x^2) + eps) * post_weight    (x when post_weight is NULL)
 *   s    = bf16(residual_scale * residual + scale * g(gate) * p)
 *   n    = s * rsqrt(mean(s^2) + eps) * pre_weight
 * with g the identity, sigmoid or tanh (1 without a gate), in FP32. Outputs:
 *   sum     bf16 [T, H]   s, the new residual stream; may be `x` or `residual`
 *   y       bf16 [T, H]   bf16(n), or NULL; may be the one of them that `sum` is not
 *   codes   uint8 [T, H], scales uint8 [T, H/32]   MXFP8(n) as moe_prompt.h
 *           defines it, both or neither
 * Without pre_weight there is no n: y, codes and scales are NULL.
 *   x, residual bf16 [T, H];  post_weight, pre_weight bf16 [H] or NULL
 *   gate    bf16 [H] (a scale per channel), or of the shape that flags tell; or NULL
 * H in 1..16384, a multiple of 32 for MXFP8. bf16 tensors 2-byte aligned;
 * 16-byte aligned ones with H a multiple of 8 take the vector form.
 */
moe_status_t moe_norm_add_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual,
                               const uint16_t* post_weight, const uint16_t* pre_weight,
                               const uint16_t* gate, float scale, float residual_scale, float eps,
                               uint32_t flags, uint16_t* sum, uint16_t* y, uint8_t* codes,
                               uint8_t* scales, void* stream);

/* ---- dense products ----------------------------------------------------------- */

/* Activations of moe_dense_config_t. */
#define MOE_ACT_NONE 0
#define MOE_ACT_RELU 1
#define MOE_ACT_SILU 2
#define MOE_ACT_GELU 3      /* v (1 + erf(v / sqrt 2)) / 2 */
#define MOE_ACT_GELU_TANH 4 /* v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2 */
#define MOE_ACT_SILU_MUL 5  /* the N = 2I weight rows are I gate rows, then I up
                               rows; the result is the I values SiLU(gate) * up */

typedef struct {
  int32_t N;          /* weight rows; even for MOE_ACT_SILU_MUL */
  int32_t K;          /* reduction length, a multiple of 8 */
  int32_t activation; /* MOE_ACT_* */
} moe_dense_config_t;

typedef struct moe_dense* moe_dense_t;

/*
 * A handle over one weight matrix on the current device.
 *   weight  bf16 [N, K], 16-byte aligned;  bias bf16 [N] or NULL
 * Both are borrowed until moe_dense_destroy. They hold their values when this is
 * called, their writers' work being over (that of the default stream is waited for
 * here), and keep them until then: a run reads them before it waits for earlier
 * work on its stream. Allocates
 * an error word, one CUDA event and one non-blocking stream (for reading the error
 * word), so it is made outside graph captures; runs may be captured, and runs on
 * several streams may overlap. N and K up to 2^31 - 256.
 */
moe_status_t moe_dense_create(const moe_dense_config_t* cfg, const uint16_t* weight,
                              const uint16_t* bias, moe_dense_t* out);
moe_status_t moe_dense_destroy(moe_dense_t handle);

/*
 *   out[r] = act(x[r] weight^T + bias) + residual[r]
 * with FP32 accumulation and epilogue, rounded once. M = N, or N / 2 with
 * MOE_ACT_SILU_MUL. The current device has to be the handle's.
 * The tensor cores cut their sums off at each 16 of K. FP32 outputs add them up
 * every 512 K (relative 2-norm of the error 0.5e-6 on random values); bf16 outputs
 * take longer ones, which their rounding hides but for a neighbouring value now and
 * then. SiLU and the GELUs are off by at most 2^-23 (6 + 5 a) of their value, a the
 * magnitude of their exponential's argument (values below 2^-126 may be 0).
 *   x         bf16 [R, K], 16-byte aligned
 *   residual  bf16 [R, M] or NULL; may be `out` where that is bf16
 *   out       bf16 [R, M], or float [R, M] with out_float != 0
 */
moe_status_t moe_dense_run(moe_dense_t handle, int32_t R, const uint16_t* x,
                           const uint16_t* residual, void* out, int32_t out_float, void* stream);

/* Read and clear, in one step, the handle's device error word
 * (MOE_DEVICE_TIMEOUT: a bounded device wait gave up and outputs are undefined)
 * after waiting for the handle's latest run that was not being captured into a
 * graph and for `stream` (which covers graphs replayed there). The return
 * value is MOE_ERR_DEVICE_FAULT when a bit was set. */
moe_status_t moe_dense_get_error(moe_dense_t handle, void* stream, uint32_t* device_flags);

/* Test support: how a run of R rows, with FP32 outputs or bf16 ones, is cut on a GPU
 * of num_sms SMs, computed on the host (no device needed). */
typedef struct {
  int32_t split;  /* 1: moe_dense_split, 0: moe_dense_tiles */
  int32_t nt;     /* rows of x a tile */
  int32_t parts;  /* of K, one CTA of a cluster each (split) */
  int32_t stages; /* of the operands' ring */
  int32_t smem;   /* dynamic shared memory of a CTA, bytes */
  int32_t ctas;   /* of the launch */
} moe_dense_plan_t;
moe_status_t moe_dense_plan(const moe_dense_config_t* cfg, int32_t R, int32_t out_float,
                            int32_t num_sms, moe_dense_plan_t* out);

/* Test support: in the next run that launches something, the MMAs wait for an
 * arrival that nothing makes, with a limit of some milliseconds instead of a
 * second. Every role gives up, the launch completes with unspecified outputs,
 * the handle reports MOE_DEVICE_TIMEOUT and its later runs are unaffected. */
moe_status_t moe_dense_arm_timeout(moe_dense_t handle);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
