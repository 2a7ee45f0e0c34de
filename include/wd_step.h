/*
 * wd_step.h - the small operators of a decode step around the attention of
 * wd_kv.h and the MoE layer of wd_moe.h: the norm before each of them, the
 * routing to experts, and what is done to the logits before a token is chosen.
 * (The rotation of queries and keys is wd_kv_append_rotated in wd_kv.h.)
 *
 * As in wd_moe.h every call is asynchronous on `stream`, allocates nothing and
 * checks its arguments on the host before any launch.  None of these needs a
 * workspace, so calls on different streams share nothing; every result is the same
 * from run to run.  Strides are in elements; the last dimension is contiguous.
 * Outputs must not overlap inputs except where a call says so.
 */
#ifndef WD_STEP_H_
#define WD_STEP_H_

#include <stddef.h>
#include <stdint.h>

#include "wd_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum wd_dtype { WD_BF16 = 0, WD_FP16 = 1, WD_FP32 = 2 } wd_dtype;

/* Largest row of wd_rms_norm, most experts of wd_route, most experts of a token,
 * largest vocabulary and longest history of wd_adjust_logits. */
#define WD_NORM_MAX_H 16384
#define WD_ROUTE_MAX_EXPERTS 1024
#define WD_ROUTE_MAX_K 64
#define WD_LOGITS_MAX_V (1 << 24)
#define WD_LOGITS_MAX_HISTORY (1 << 20)

/* Root-mean-square norm of each row, after the residual's addition:
 *
 *   r = x + residual,   y = r / sqrt(mean(r^2) + eps) * weight
 *
 * x: `tokens` times `heads` rows of H elements of `dtype`, row (t, h) at
 * x + t * x_stride_token + h * x_stride_head (the heads of a fused projection; 1
 * head for ordinary rows).  weight [H], of `weight_dtype` (`dtype` or WD_FP32), or
 * NULL for ones.  residual (or NULL): rows like x with strides of its own.  Outputs
 * are contiguous, [tokens, heads, H]: residual_out (needs residual; may be NULL)
 * receives r in `dtype`, y (may be NULL) the norm in `dtype`, codes and scales (both
 * or neither) the norm in MXFP8 as the expert weights have it: of each 32 elements
 * E4M3 codes and one E8M0 byte s = floor(log2 of the largest magnitude) - 8 + 127,
 * at least 0 (127 for a block of zeros; 255 and codes of 0 if one is not finite).  Codes
 * are rounded to nearest even and saturate at 448.  y or codes is wanted; MXFP8
 * wants H a multiple of 32.  residual_out may be residual, and y may be x, where that
 * is contiguous.
 *
 * Numbers: r, its squares' sum and the norm are FP32 and each output is rounded once
 * from them (y is made of r, not of what residual_out keeps of it); rows whose squares
 * leave FP32 are summed again smaller, so any finite r has its norm.  eps: at least 1e-37,
 * finite.  A row that is not finite gives NaN.  1 <= H <= WD_NORM_MAX_H, tokens * heads < 2^31. */
WD_API wd_status wd_rms_norm(const void* x, wd_dtype dtype, int64_t x_stride_token,
                             int64_t x_stride_head, int64_t tokens, int heads, int H,
                             const void* weight, wd_dtype weight_dtype, const void* residual,
                             int64_t residual_stride_token, int64_t residual_stride_head,
                             void* residual_out, float eps, void* y, uint8_t* codes,
                             uint8_t* scales, wd_stream_t stream);

typedef enum wd_scores { WD_SOFTMAX = 0, WD_SIGMOID = 1 } wd_scores;

/* Routing of `tokens` tokens to K of E experts, as wd_moe_decode takes it.
 *
 *   score = softmax(logits) or sigmoid(logits),   key = score + bias
 *
 * The experts stand in `groups` equal groups; a group's value is the sum of its
 * `group_best` (1 or 2) largest keys, and the top_groups groups of the largest values are chosen.
 * Of their experts the K with the largest keys are, largest first; of equal keys (or
 * values) the lowest index.  Weights are the scores, without the bias, divided by
 * their sum over the K if `renormalise`, times `scale`.
 *
 * logits [tokens, E] of `dtype`; bias FP32 [E] or NULL; ids int32 and weights FP32
 * [tokens, K], contiguous.  A logit of -inf or NaN masks its expert: score 0, chosen
 * after all that are not masked whatever its bias, and without part in its group's
 * value.  Logits of +inf share the softmax among them.  Where the scores of
 * the chosen are all 0, the weights are 0.  Weights are made of FP32 scores: one below 2^-126
 * loses bits or counts as 0 (but sigmoids that are renormalised keep theirs if all of the K are below e^-40).
 *
 * Without a bias keys are compared by their logits, which order as they do.  Where keys or
 * groups' sums have to be compared, the FP32 ones decide unless two are nearer to each other than their
 * error; that token's are then compared in 64 bits, so that ids are those of the definition.
 * Groups of one expert and no bias go by the logits, too.
 *
 * E <= WD_ROUTE_MAX_EXPERTS, groups <= 32 divides E, a group has at most 1024 / groups
 * experts with groups rounded up to a power of two; K <= min(WD_ROUTE_MAX_K, top_groups * E / groups);
 * scale finite. */
WD_API wd_status wd_route(const void* logits, wd_dtype dtype, int64_t stride_token, int64_t tokens,
                          int E, int K, wd_scores scores, const float* bias, int groups,
                          int top_groups, int group_best, int renormalise, float scale,
                          int32_t* ids, float* weights, wd_stream_t stream);

/* The tokens so far of a batch's requests, for wd_adjust_logits. */
typedef struct wd_history {
  const int32_t* tokens;         /* [slots][columns], rows `stride` apart; NULL: no history */
  const int32_t* lengths;        /* [slots]: how many of a row count, prompt and answer */
  const int32_t* prompt_lengths; /* [slots]: how many of them are the prompt; NULL: none */
  const int32_t* seqs;           /* [B]: the slot of each row of logits; NULL: slot b */
  int64_t stride;
  int32_t slots, columns;        /* columns <= WD_LOGITS_MAX_HISTORY */
} wd_history;

/* What is done to logits before a token is chosen.  For each row b and token v:
 *
 *   1. v in the prompt or the answer:  l = l > 0 ? l * (1 / repetition[b]) : l * repetition[b]
 *   2. v n > 0 times in the answer:    l = l - (n * frequency[b] + presence[b])
 *   3. v named by the row's biases:    l = l + its value (the sum of them in their order, if it is named several times)
 *   4. temperature[b] > 0:             l = l * (1 / temperature[b])
 *   5. bit v of the row's mask is 0:   l = -inf
 *
 * logits [B, V] of `dtype`, rows `stride` apart; out [B, V] of `out_dtype` (`dtype` or
 * WD_FP32), rows `out_stride` >= V apart; out may be logits where type and stride are the same.
 * repetition, presence, frequency, temperature: FP32 [B], each NULL to leave its step out.
 * Biases: row b's are entries bias_start[b] .. bias_start[b + 1] - 1 of bias_ids and
 * bias_values (all NULL for none; `biases` entries in all).  mask: int32 words, rows mask_stride words
 * apart, bit v % 32 of word v / 32 (NULL: all allowed).  Steps and reciprocals are FP32
 * (1 / x of x below 2^-128 is infinite), and the result is rounded once to out_dtype.  What is out of range counts
 * for nothing: tokens and biases outside the vocabulary, slots, a row's biases if its entries of bias_start are no
 * range 0 <= from <= to <= biases; lengths are cut to 0 .. columns. */
WD_API wd_status wd_adjust_logits(const void* logits, wd_dtype dtype, int64_t stride, int B, int V,
                                  const wd_history* history, const float* repetition,
                                  const float* presence, const float* frequency,
                                  const int32_t* bias_start, const int32_t* bias_ids,
                                  const float* bias_values, int biases, const float* temperature,
                                  const int32_t* mask, int64_t mask_stride, void* out,
                                  wd_dtype out_dtype, int64_t out_stride, wd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WD_STEP_H_ */
