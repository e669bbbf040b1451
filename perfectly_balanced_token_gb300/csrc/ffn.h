// Host-side launchers of the operators declared in include/moonep_ffn.h.
#pragma once

#include "../../include/moonep_ffn.h"
#include "common.cuh"

namespace moonep {

struct LinearDims {
  int T, K, N, act, f32;
  int half;  // swiglu: N / 2, otherwise 0
};

cudaError_t launch_linear(const LinearDims&, const void* x, const void* w, const float* bias,
                          const void* residual, void* out, void* z, int32_t* status, cudaStream_t,
                          int*);
cudaError_t launch_linear_dx(const LinearDims&, const void* d_z, const void* w, void* d_x,
                             int32_t* status, cudaStream_t, int*);
cudaError_t launch_linear_dw(const LinearDims&, const void* x, const void* d_z, float* d_w, int add,
                             int32_t* status, cudaStream_t, int*);
cudaError_t launch_grouped_gemm_act(const Dims&, const PlanPtrs&, int act, const void* recv,
                                    const void* w_home, const void* w_slot, const float* bias, void* y,
                                    void* z, cudaStream_t, int*);

int64_t act_chunks(int64_t rows);  // rows of sums that the dense gradient leaves in scratch
cudaError_t launch_act_backward(int64_t rows, int cols, int act, const void* z, const void* d_out,
                                void* d_z, float* d_bias, int add, float* scratch, cudaStream_t, int*);
cudaError_t launch_grouped_act_backward(const Dims&, const PlanPtrs&, int act, const void* z,
                                        const void* d_y, void* d_z, float* d_bias, int add,
                                        float* scratch, cudaStream_t, int*);

struct Dropout {
  uint32_t cut;  // 16-bit numbers below it are dropped; 0: nothing is, and rng is not read
  float scale;   // of what stays
  const int64_t* rng;
};
cudaError_t launch_combine_dropout(const Dims&, const PlanPtrs&, const void* y, const float* gates,
                                   const void* residual, void* out, const Dropout&, cudaStream_t, int*);
cudaError_t launch_combine_dropout_backward(const Dims&, const PlanPtrs&, const void* y,
                                            const float* gates, const void* d_out, void* d_y,
                                            float* d_gates, const Dropout&, cudaStream_t, int*);

}  // namespace moonep
