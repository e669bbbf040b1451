/*
 * moonep_ffn.h -- C ABI of the feed-forward network and the end of the layer:
 *
 *   moonep_linear                    out = residual + act(x w + bias): shared experts, the
 *                                    router's logits
 *   moonep_linear_dx, _dw            its gradients with respect to x and w
 *   moonep_act_backward              gradient of an activation, with that of the bias
 *   moonep_grouped_gemm_act          moonep_grouped_gemm with bias and activation
 *   moonep_grouped_act_backward      moonep_act_backward on the plan's rows, a bias an expert
 *   moonep_combine_dropout           moonep_combine with dropout, added to the residual
 *   moonep_combine_dropout_backward  its gradient
 *
 * An expert of two projections runs on one plan: moonep_grouped_gemm_act with the
 * first weights, then moonep_grouped_gemm with the second ones and dims that differ
 * from the plan's in H and Hp alone (a plan depends on neither), then
 * moonep_combine_dropout.  A shared expert is moonep_linear twice, the second time
 * with the layer's input as residual and its output the combine's residual.
 * The gradients go back through moonep_combine_dropout_backward,
 * moonep_grouped_gemm_dw and _dx, moonep_grouped_act_backward and _dw and _dx again.
 * The conventions of moonep.h hold: the caller owns every buffer, pointers are
 * 16-byte aligned device pointers unless stated, arrays are dense and row-major,
 * nothing allocates or synchronises, host-detected errors come back before anything
 * is enqueued, and calls that take a plan workspace write nothing if the plan
 * failed.  Buffers of one call do not overlap.  moonep_grouped_gemm_act is one of the
 * grouped products that must not run at the same time on one plan.
 */
#ifndef MOONEP_FFN_H
#define MOONEP_FFN_H

#include "moonep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- products ---------------------------------------------------------------
 * bf16 operands, fp32 accumulation and epilogue, one rounding at the end (to nearest
 * even).  Activations of z: */
enum moonep_activation {
  MOONEP_ACT_NONE = 0,
  MOONEP_ACT_RELU = 1,
  MOONEP_ACT_GELU = 2,   /* z P(N(0,1) <= z)                                        */
  MOONEP_ACT_SILU = 3,   /* z / (1 + e^-z); 0 below z = -87.33, where it is under
                            1.1e-36 (swiglu and the gradients likewise)             */
  MOONEP_ACT_SWIGLU = 4  /* silu(z_j) z_(F+j), j < F: the first half of a row's
                            columns are gates, 2F columns of z give F of the output */
};

typedef struct moonep_linear_dims {
  int32_t T, K, N;  /* rows (0: nothing to do), depth, columns of w and z           */
  int32_t act;      /* moonep_activation                                            */
  int32_t out_f32;  /* moonep_linear's out: 0 = bf16, 1 = fp32                      */
} moonep_linear_dims;

/* z = x w + bias, out = residual + act(z).  x bf16 [T][K], w bf16 [K][N], bias fp32
 * [N] or NULL, residual bf16 [T][C] or NULL, out [T][C] (written), with C = N or, for
 * swiglu, N / 2; z bf16 [T][N] (written) or NULL: what the activation's gradient
 * needs (out is computed from z before it is rounded).
 * status: int32 on the device (4-byte aligned), zeroed by the caller before its first
 * use; a device wait that runs out ORs MOONEP_ERR_TIMEOUT into it, and a call that
 * finds it other than 0 writes nothing.
 * K and N multiples of 8 (N of 16 for swiglu), sizes below 2^31 - 512 and tiles of
 * 128 x 128 below 2^31 - 512 in number (MOONEP_ERR_SHAPE). */
int moonep_linear(const moonep_linear_dims* dims, const uint16_t* x, const uint16_t* w,
                  const float* bias, const uint16_t* residual, void* out, uint16_t* z,
                  int32_t* status, void* stream);

/* d_x bf16 [T][K] = d_z w^T, with d_z bf16 [T][N] (of moonep_act_backward, or the
 * output's gradient itself where there is no activation).  dims->act and out_f32 play
 * no part here and in moonep_linear_dw. */
int moonep_linear_dx(const moonep_linear_dims* dims, const uint16_t* d_z, const uint16_t* w,
                     uint16_t* d_x, int32_t* status, void* stream);

/* d_w fp32 [K][N] = x^T d_z, or with accumulate = 1 d_w += x^T d_z.  (T = 0 and
 * accumulate = 0: d_w is zeroed and status neither read nor needed.) */
int moonep_linear_dw(const moonep_linear_dims* dims, const uint16_t* x, const uint16_t* d_z,
                     float* d_w, int32_t accumulate, int32_t* status, void* stream);

/* Scratch of moonep_act_backward with d_bias (host only). */
int moonep_act_backward_workspace_bytes(int64_t rows, int32_t cols, size_t* bytes);

/* d_z = act'(z) d_out (bf16; relu'(0) = 0) and d_bias = the column sums of d_z before
 * it is rounded (fp32, always in the same order; written, or added to with
 * accumulate = 1).  z bf16 [rows][cols], d_out bf16 [rows][cols, or cols / 2 for
 * swiglu], d_z bf16 [rows][cols]; d_bias fp32 [cols] or NULL, and scratch (overwritten)
 * with it.  With MOONEP_ACT_NONE z is not read and may be NULL, and so may d_z if
 * d_bias is not.  cols a multiple of 8 (16 for swiglu) below 2^31 - 512, 0 <= rows <
 * 2^40 (MOONEP_ERR_SHAPE). */
int moonep_act_backward(int64_t rows, int32_t cols, int32_t act, const uint16_t* z,
                        const uint16_t* d_out, uint16_t* d_z, float* d_bias, int32_t accumulate,
                        void* scratch, void* stream);

/* moonep_grouped_gemm with an epilogue: for each rank u and group g, of expert e,
 * z = recv W(u,g) + bias[e], y = act(z).  recv, w_home, w_slot as there; bias fp32
 * [E][Hp] or NULL (a slot takes the bias of the expert it holds); y bf16 [R][C][Hp, or
 * Hp / 2 for swiglu] (written); z bf16 [R][C][Hp] (written) or NULL.  E*H, R*B*H and N
 * below 2^31 - 512 (MOONEP_ERR_SHAPE). */
int moonep_grouped_gemm_act(const moonep_dims* dims, void* plan_ws, int32_t act, const uint16_t* recv,
                            const uint16_t* w_home, const uint16_t* w_slot, const float* bias,
                            uint16_t* y, uint16_t* z, void* stream);

/* Scratch of moonep_grouped_act_backward with d_bias (host only). */
int moonep_grouped_act_backward_workspace_bytes(const moonep_dims* dims, size_t* bytes);

/* moonep_act_backward on rows as moonep_grouped_gemm_act makes them: z, d_z bf16
 * [R][C][Hp], d_y bf16 [R][C][Hp, or Hp / 2]; d_bias fp32 [E][Hp] or NULL: every
 * expert's sum over all its rows, home or slot (0 for an expert without rows).  d_z
 * then goes to moonep_grouped_gemm_dx and _dw.  Hp up to 65535 x 1024
 * (MOONEP_ERR_SHAPE). */
int moonep_grouped_act_backward(const moonep_dims* dims, void* plan_ws, int32_t act,
                                const uint16_t* z, const uint16_t* d_y, uint16_t* d_z, float* d_bias,
                                int32_t accumulate, void* scratch, void* stream);

/* ---- combine with dropout and residual --------------------------------------
 * out[r][s] = bf16( residual[r][s] + m sum over k ascending of gates[r][s][k]
 * y[dst[r][s][k]] ), fp32 sums; residual bf16 [R][S][Hp] or NULL.
 * m of the output's element i (counted from 0, row by row) is 0 for a dropped element
 * (whose product is 0 whatever the sum) and 65536 / (65536 - c) for one that stays,
 * c = floor(65536 p + 1/2).  Element i is dropped if the (i % 8)-th of eight 16-bit
 * numbers is below c: the halves, low first, of the four words of Philox4x32-10 with
 * the seed as its key and (i / 8, offset), 64 bits each, low words first, as its
 * counter.  rng: int64 [2] on the device, {seed, offset}, read when the kernel runs (a
 * replayed graph can be given new ones); may be NULL if c = 0.  0 <= p < 1, c < 65536
 * (MOONEP_ERR_ARG).  Nothing of the mask is stored: the gradient draws it again from
 * the same rng. */
int moonep_combine_dropout(const moonep_dims* dims, void* plan_ws, const uint16_t* y,
                           const float* gates, const uint16_t* residual, uint16_t* out, double p,
                           const int64_t* rng, void* stream);

/* moonep_combine_backward behind it: with d = m d_out, d_y[dst[r][s][k]] =
 * bf16(gates[r][s][k] d[r][s]) and d_gates[r][s][k] = <y[dst[r][s][k]], d[r][s]>, where
 * a dropped element counts as 0 whatever y, the gate and d_out are.  (The residual's
 * gradient is d_out itself.)  K <= 128, Hp <= 8192 (MOONEP_ERR_SHAPE). */
int moonep_combine_dropout_backward(const moonep_dims* dims, void* plan_ws, const uint16_t* y,
                                    const float* gates, const uint16_t* d_out, uint16_t* d_y,
                                    float* d_gates, double p, const int64_t* rng, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOONEP_FFN_H */
