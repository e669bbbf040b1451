/*
 * moonep_ops.h -- C ABI of the operators around the layer path of moonep.h:
 *
 *   moonep_router_forward            top-K experts and gates of every token, per-expert
 *                                    counts and the balance loss
 *   moonep_router_backward           gradient of the gates and of the balance loss with
 *                                    respect to the router's logits
 *   moonep_mxfp4_quantize            rows of bf16 values to MXFP4
 *   moonep_mxfp4_quantize_weights    expert weights [H][Hp] to MXFP4, transposed
 *   moonep_mxfp4_dequantize          MXFP4 rows back to bf16 (exact)
 *   moonep_mxfp4_dispatch            moonep_dispatch that quantises each token on the way
 *   moonep_mxfp4_prefetch_weights    moonep_prefetch_weights on MXFP4 weights
 *   moonep_mxfp4_grouped_gemm        moonep_grouped_gemm on MXFP4 operands
 *
 * The router makes what moonep_plan and moonep_combine take (topk_idx, gates)
 * and takes what moonep_combine_backward makes (d_gates); the MXFP4 calls take
 * the place of their bf16 namesakes between moonep_plan and moonep_combine.
 * The conventions of moonep.h hold: the caller owns every buffer, pointers are
 * 16-byte aligned device pointers unless stated, arrays are dense and
 * row-major, nothing allocates or synchronises, host-detected errors come back
 * before anything is enqueued, and calls that take a plan workspace write
 * nothing if the plan failed.  Buffers of one call do not overlap.
 */
#ifndef MOONEP_OPS_H
#define MOONEP_OPS_H

#include "moonep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- router ---------------------------------------------------------------
 * l [T][E] logits.  Per token: s = softmax(l) or sigmoid(l); the K experts with
 * the largest logits, largest first, equal logits in ascending expert id (-0 and
 * +0 are equal; a NaN ranks below -inf); gate k = scale * s[id_k], divided by
 * the sum of the K chosen s when `normalise` is set.  A token whose token_mask is 0 still gets K distinct ids, as the plan
 * needs them, but its gates are 0, it is not counted and its gradient is 0.
 *
 * Balance loss over segments of `segment` consecutive tokens (the last may be
 * shorter; G = ceil(T / segment) of them), n_g unmasked tokens in segment g:
 *   counts[g][e]   = unmasked tokens of g with e among their K experts
 *   prob_sum[g][e] = sum over the unmasked tokens of g of q_e, where q = s for
 *                    softmax and q = s / sum_e s for sigmoid
 *   loss = 1/G sum_g E / (K n_g^2) sum_e counts[g][e] prob_sum[g][e]
 * (1 when counts and probabilities are even; a segment with n_g = 0 adds 0).
 *
 * A row that holds only -inf has q = 0 and gates 0.  Other rows with NaN (softmax:
 * or +inf) give NaN where the formulas do.  Gates, sums and the loss are computed
 * in fp32 or wider; the result is the same in every run (sums across blocks are
 * integer sums of fixed-point values).  Smallest values: scores below 2^-126
 * read 0, and where several blocks share a segment each rounds its part of
 * prob_sum to a multiple of 2^-46 (of 2^(b - 62) for segments of more than 2^16
 * tokens, 2^b the power of two at or above their length). */
typedef struct moonep_router_dims {
  int32_t T, E, K;
  int32_t segment;    /* tokens per segment of the balance loss, 1 .. T (0: T) */
  int32_t score;      /* 0 = softmax, 1 = sigmoid                              */
  int32_t normalise;  /* 1 = gates divided by their sum                        */
  int32_t dtype;      /* logits and their gradient: 0 = fp32, 1 = bf16         */
  float scale;        /* factor on every gate                                  */
} moonep_router_dims;

/* Bytes of scratch for moonep_router_forward's loss (host only). */
int moonep_router_workspace_bytes(const moonep_router_dims* dims, size_t* bytes);

/* logits [T][E], token_mask uint8 [T] or NULL, topk_idx int32 [T][K] and gates
 * fp32 [T][K] (written).  The balance outputs are all given or all NULL: ws
 * (overwritten), counts int32 [G][E], prob_sum fp32 [G][E], seg_tokens int32
 * [G] (n_g), loss fp32 [1] (4-byte aligned).
 * MOONEP_ERR_SHAPE: K > E, K > 128, E > 4096, T*K reaches 2^31 - 4096, G*E
 * reaches 2^31, or segment > T.  Two calls that overlap on the GPU need two workspaces. */
int moonep_router_forward(const moonep_router_dims* dims, const void* logits,
                          const uint8_t* token_mask, int32_t* topk_idx, float* gates, void* ws,
                          int32_t* counts, float* prob_sum, int32_t* seg_tokens, float* loss,
                          void* stream);

/* d_logits [T][E] (written) = gradient of sum d_gates * gates + d_loss * loss
 * with the choice of experts, and so counts and n_g, held fixed.  topk_idx,
 * counts and seg_tokens as the forward pass wrote them (an id outside [0, E)
 * contributes nothing).  d_gates fp32 [T][K] or NULL; counts, seg_tokens and
 * d_loss (fp32 [1] on the device, 4-byte aligned) all given or all NULL; at
 * least one of the two gradients is given.  Sigmoid without d_loss: a token's
 * gradient depends on its chosen logits alone, whatever the others hold. */
int moonep_router_backward(const moonep_router_dims* dims, const void* logits,
                           const uint8_t* token_mask, const int32_t* topk_idx,
                           const float* d_gates, const int32_t* counts,
                           const int32_t* seg_tokens, const float* d_loss, void* d_logits,
                           void* stream);

/* ---- MXFP4 ----------------------------------------------------------------
 * Blocks of 32 consecutive values of a row share the scale 2^(b - 127), b one
 * byte (the OCP microscaling format's E8M0); a value is a 4-bit E2M1 code: sign
 * and magnitude 0, 0.5, 1, 1.5, 2, 3, 4 or 6, codes 0..7 in that order.  A row
 * of `cols` values is cols/2 bytes of codes (the even column in the low half)
 * and a row of MOONEP_MXFP4_SCALE_PITCH(cols) scale bytes, of which the first
 * cols/32 are used and the rest are 0.
 * Quantisation: b = max(exponent of the block's largest magnitude - 2, -127) +
 * 127, values rounded to the nearest code, ties to the even code, at most 6;
 * a block that holds an infinity or a NaN gets b = 255 and codes 0, and stands
 * for NaN throughout. */
#define MOONEP_MXFP4_SCALE_PITCH(cols) ((((cols) / 32 + 15) / 16) * 16)

/* src bf16 [rows][cols] -> codes uint8 [rows][cols/2], scales uint8
 * [rows][pitch].  cols a multiple of 32 (MOONEP_ERR_SHAPE), rows >= 0. */
int moonep_mxfp4_quantize(int64_t rows, int32_t cols, const uint16_t* src, uint8_t* codes,
                          uint8_t* scales, void* stream);

/* The inverse: dst bf16 [rows][cols].  Every MXFP4 value that quantisation
 * makes is a bf16 value, so nothing is rounded; scale bytes of 253 and more can
 * pass bf16's range and give infinities. */
int moonep_mxfp4_dequantize(int64_t rows, int32_t cols, const uint8_t* codes,
                            const uint8_t* scales, uint16_t* dst, void* stream);

/* n matrices bf16 [H][Hp] -> codes uint8 [n][Hp][H/2], scales uint8
 * [n][Hp][pitch of H]: the rows of W^T, quantised along H, the contraction of
 * the grouped product.  H and Hp multiples of 64 (MOONEP_ERR_SHAPE). */
int moonep_mxfp4_quantize_weights(int32_t n, int32_t H, int32_t Hp, const uint16_t* w,
                                  uint8_t* codes, uint8_t* scales, void* stream);

/* moonep_prefetch_weights on quantised weights.  home: [E][Hp][..], slots:
 * [R][B][Hp][..], codes of H/2 and scales of pitch(H) bytes a row.  An expert's
 * codes stay below 16 GiB (MOONEP_ERR_SHAPE). */
int moonep_mxfp4_prefetch_weights(const moonep_dims* dims, void* plan_ws, const uint8_t* home_codes,
                                  const uint8_t* home_scales, uint8_t* slot_codes,
                                  uint8_t* slot_scales, void* stream);

/* moonep_dispatch that writes MXFP4 rows: each token is quantised once and
 * scattered to its K rows.  x bf16 [R][S][H]; recv_codes uint8 [R][C][H/2],
 * recv_scales uint8 [R][C][pitch(H)] (every row written). */
int moonep_mxfp4_dispatch(const moonep_dims* dims, void* plan_ws, const uint16_t* x,
                          uint8_t* recv_codes, uint8_t* recv_scales, void* stream);

/* moonep_grouped_gemm on MXFP4 operands: y = recv x W with both as quantised
 * above, products and sums in the block-scaled tensor-core instruction with
 * fp32 accumulation, y bf16 [R][C][Hp] (round to nearest even).  Slot pointers
 * may be NULL when B == 0.  N, R*B*Hp and E*Hp must stay below 2^31 - 512
 * (MOONEP_ERR_SHAPE).  Uses the plan's work tiles.
 * The gradients stay in bf16, on the same plan: moonep_grouped_gemm_dx takes
 * bf16 weights [E][H][Hp] with their slots (moonep_prefetch_weights), and
 * moonep_grouped_gemm_dw bf16 rows (H a multiple of 128).  These are the
 * caller's weights and moonep_dispatch's rows; or, for the gradients of the
 * product as it was computed, what moonep_mxfp4_dequantize makes of the codes:
 * recv as it stands, the weights turned by the caller from [E][Hp][H] to
 * [E][H][Hp] first. */
int moonep_mxfp4_grouped_gemm(const moonep_dims* dims, void* plan_ws, const uint8_t* recv_codes,
                              const uint8_t* recv_scales, const uint8_t* home_codes,
                              const uint8_t* home_scales, const uint8_t* slot_codes,
                              const uint8_t* slot_scales, uint16_t* y, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOONEP_OPS_H */
