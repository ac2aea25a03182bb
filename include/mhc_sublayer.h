/*
 * mhc_sublayer.h -- C ABI of the operators between two mHC boundaries.
 *
 * A boundary (mhc_boundary.h) gives the next sublayer its BF16 layer input
 * and takes the sublayer's output back as a partial.  These operators are
 * what a sublayer computes between the two:
 *
 *   add_rms_norm  r = x + residual;  y = r * rsqrt(mean(r^2) + eps) * weight
 *   quantize      x in 8 bits
 *   swiglu        silu(gate) * up in 8 bits
 *   matmul        (a * a_scales) (w * w_scales)^T of 8-bit tensors
 *   moe           a whole mixture-of-experts layer for up to 32 tokens
 *
 * The 8-bit format: E4M3 values with FP32 scales.  An activation [m][k] has
 * one scale for each 128 consecutive values of a row (the last block of a
 * row may be shorter), [m][ceil(k/128)]; a weight [n][k] has one scale for
 * each 128 x 128 block, [ceil(n/128)][ceil(k/128)].  A value stands for
 * value * scale.  The quantisers take scale = amax / 448 with the block's
 * largest magnitude, floored at 2^-100, as amax, and round x * (448 / amax)
 * to nearest-even.  The quotients are taken as amax * (1 / 448) and (1 / amax) *
 * 448, every step rounded to nearest in FP32 (but 1 / amax may be the neighbour
 * below where amax has 24 significant bits, all ones).  A block that holds an
 * infinity or a NaN has a non-finite scale.
 *
 * Conventions: as in mhc_boundary.h (device pointers, caller-owned buffers,
 * every argument checked before the first launch, nothing aborts or traps).
 * Matrices are row-major with contiguous rows; a *_stride is the distance of
 * two rows in elements.  BF16 and 8-bit rows start on 16-byte boundaries.
 * Outputs overlap neither inputs nor one another, but where a call allows it.
 * Calls with m = 0 succeed and launch nothing (but for moe, whose m is in
 * [1, max_moe_tokens]).  A handle owns scratch that its moe calls use: its
 * calls run one after another, on one stream or on streams that the caller
 * orders.
 */
#ifndef MHC_SUBLAYER_H
#define MHC_SUBLAYER_H

#include "mhc_boundary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Router score of mhc_sublayer_moe. */
enum {
  MHC_SCORE_SOFTMAX = 0, /* softmax over all experts */
  MHC_SCORE_SIGMOID = 1  /* sigmoid of each logit */
};

/* Config flags. */
enum {
  /* The expert weights are 8-bit with block scales (else BF16). */
  MHC_SUBLAYER_FP8 = 1u << 0,
  /* Divide the chosen experts' scores by their sum. */
  MHC_SUBLAYER_RENORMALIZE = 1u << 1,
  /* The router weight is FP32 (else BF16). */
  MHC_SUBLAYER_ROUTER_F32 = 1u << 2
};

/* Construction arguments.  num_experts = 0: a handle without moe (the other
 * MoE fields are then ignored).  Else hidden and intermediate are positive
 * multiples of 8 (16 with MHC_SUBLAYER_FP8), hidden <= 16384, intermediate
 * <= 16384, num_experts <= 512, 1 <= top_k <= min(16, num_experts),
 * 0 <= shared_experts <= 8, 1 <= max_moe_tokens <= 32. */
typedef struct {
  int32_t hidden;
  int32_t intermediate;   /* an expert's width between its two products */
  int32_t num_experts;    /* routed experts */
  int32_t shared_experts; /* experts that every token takes with weight 1 */
  int32_t top_k;
  int32_t max_moe_tokens;
  int32_t score;          /* MHC_SCORE_* */
  float routed_scale;     /* factor of the routed experts' weights */
  uint32_t flags;         /* MHC_SUBLAYER_* */
} mhc_sublayer_config_t;

typedef struct mhc_sublayer mhc_sublayer_t; /* opaque, library-owned */

/* h: a positive multiple of 8, at most 16384; strides multiples of 8.
 * r = x + residual (x where residual is NULL) in FP32, not rounded before the
 * norm.  Outputs, each optional but at least one given: residual_out [m][h]
 * bf16 (needs residual), output [m][h] bf16, values and scales (both or
 * neither).  residual_out and output may each be x or residual itself where
 * that is dense (its stride h, or m = 1); no output may overlap an input in
 * another way. */
typedef struct {
  int32_t m, h;
  const void *x;           /* [m][h] bf16 */
  int64_t x_stride;
  const void *residual;    /* [m][h] bf16 or NULL */
  int64_t residual_stride;
  const void *norm_weight; /* [h] bf16 */
  float eps;
  void *residual_out;
  void *output;
  uint8_t *values;         /* [m][h] e4m3 */
  float *scales;           /* [m][ceil(h/128)] */
} mhc_sublayer_norm_args_t;

/* h: a positive multiple of 8.  quantize reads x [m][h]; swiglu reads [m][2h]
 * rows, gate then up, and quantises gate / (1 + exp(-gate)) * up.  output is
 * swiglu's optional BF16 copy (NULL for quantize). */
typedef struct {
  int32_t m, h;
  const void *x;           /* bf16 */
  int64_t x_stride;
  void *output;            /* [m][h] bf16 or NULL */
  uint8_t *values;         /* [m][h] e4m3 */
  float *scales;           /* [m][ceil(h/128)] */
} mhc_sublayer_quantize_args_t;

/* output [m][n] = (values * scales) (weight * weight_scales)^T, summed in
 * FP32.  k: a positive multiple of 16; values_stride and weight_stride
 * multiples of 16; n any positive size. */
typedef struct {
  int32_t m, n, k;
  const uint8_t *values;      /* [m][k] e4m3 */
  int64_t values_stride;
  const float *scales;        /* [m][ceil(k/128)] */
  int64_t scales_stride;
  const uint8_t *weight;      /* [n][k] e4m3 */
  int64_t weight_stride;
  const float *weight_scales; /* [ceil(n/128)][ceil(k/128)], dense */
  void *output;               /* [m][n] bf16, or f32 with output_f32 */
  int64_t output_stride;
  int32_t output_f32;
} mhc_sublayer_matmul_args_t;

/* One MoE layer over m tokens.  With E = num_experts, S = shared_experts,
 * H = hidden, I = intermediate, all dense:
 *   logits = x router^T; score = softmax or sigmoid; the top_k experts of the
 *   largest score (+ bias, where given) are chosen, ties to the lowest index,
 *   a NaN below every number; weight = score (divided by the chosen scores'
 *   sum with MHC_SUBLAYER_RENORMALIZE) * routed_scale;
 *   expert(x) = (silu(x gate^T) * (x up^T)) down^T;
 *   output = sum of weight * expert over the chosen, plus the S shared
 *   experts (the last S of the weight tensors) with weight 1.
 * The products sum in FP32 and take the BF16 x exactly with BF16 weights; with
 * 8-bit weights exactly down to 2^-17 of its row's largest magnitude, or of
 * 2^-100 where that is larger, and off by at most 2^-25 of it below.  The
 * activation between them is held to 16 significant bits with BF16 weights; with
 * 8-bit weights it is off by at most 2^-12 of itself or 2^-25 of the largest of
 * its block of 128.  A row of x with an infinity or a NaN has no finite
 * output. */
typedef struct {
  int32_t m;
  const void *x;               /* [m][H] bf16 */
  const void *router;          /* [E][H] bf16, or f32 with MHC_SUBLAYER_ROUTER_F32 */
  const float *bias;           /* [E] selection bias or NULL */
  const void *gate_up;         /* [E+S][2I][H]: I gate rows, then I up rows */
  const float *gate_up_scales; /* [E+S][2][ceil(I/128)][ceil(H/128)], MHC_SUBLAYER_FP8 only */
  const void *down;            /* [E+S][H][I] */
  const float *down_scales;    /* [E+S][ceil(H/128)][ceil(I/128)], MHC_SUBLAYER_FP8 only */
  void *output;                /* [m][H] bf16 */
  int32_t *idx;                /* [m][top_k] chosen experts, largest first, or NULL */
  float *weights;              /* [m][top_k] their weights, or NULL */
} mhc_sublayer_moe_args_t;

mhc_status_t mhc_sublayer_create(const mhc_sublayer_config_t *config, int device, mhc_sublayer_t **out);
mhc_status_t mhc_sublayer_add_rms_norm(mhc_sublayer_t *s, const mhc_sublayer_norm_args_t *args,
                                       mhc_stream_t stream);
mhc_status_t mhc_sublayer_quantize(mhc_sublayer_t *s, const mhc_sublayer_quantize_args_t *args,
                                   mhc_stream_t stream);
mhc_status_t mhc_sublayer_swiglu(mhc_sublayer_t *s, const mhc_sublayer_quantize_args_t *args,
                                 mhc_stream_t stream);
mhc_status_t mhc_sublayer_matmul(mhc_sublayer_t *s, const mhc_sublayer_matmul_args_t *args, mhc_stream_t stream);
mhc_status_t mhc_sublayer_moe(mhc_sublayer_t *s, const mhc_sublayer_moe_args_t *args, mhc_stream_t stream);
/* Synchronises the device and reports MHC_ERR_TIMEOUT if a kernel of an
 * earlier call gave up a bounded wait (its outputs are not valid); the report
 * is then cleared and the scratch made ready for the next call. */
mhc_status_t mhc_sublayer_check_errors(mhc_sublayer_t *s);
mhc_status_t mhc_sublayer_destroy(mhc_sublayer_t *s);
/* Message of the last failing call on `s` (NULL: of the last failing create). */
const char *mhc_sublayer_last_error(const mhc_sublayer_t *s);

#ifdef __cplusplus
}
#endif

#endif
