// Host-side launchers of the operators declared in include/moonep_ops.h.
#pragma once

#include "../../include/moonep_ops.h"
#include "common.cuh"

namespace moonep {

struct RouterDims {
  int T, E, K, segment, score, normalise, bf16;
  float scale;
  int G;                  // segments
  int shift;              // fixed-point bits below one of the probability sums
  int per_block, blocks;  // launch shape: tokens a block, set by the launcher
};

// The router's scratch: what is zeroed before a launch comes first.
struct RouterScratch {
  unsigned long long* done;    // [1] segments finished
  unsigned long long* joined;  // [G] blocks finished, above unmasked tokens (32 bits)
  int32_t* bad;           // [G] set where a sum met a value that is not finite
  int32_t* counts;        // [G][E]
  unsigned long long* q;  // [G][E] fixed-point probability sums
  float* seg_loss;        // [G], written before it is read
  size_t zero_bytes, total_bytes;
};
RouterScratch router_scratch(const RouterDims& d, void* ws);

struct RouterOut {
  int32_t* topk_idx;
  float* gates;
  int32_t* counts;
  float* prob_sum;
  int32_t* seg_tokens;
  float* loss;  // NULL: no balance outputs
};

cudaError_t launch_router_forward(const RouterDims&, const void* logits, const uint8_t* mask,
                                  const RouterOut&, const RouterScratch&, cudaStream_t, int*);
cudaError_t launch_router_backward(const RouterDims&, const void* logits, const uint8_t* mask,
                                   const int32_t* topk_idx, const float* d_gates,
                                   const int32_t* counts, const int32_t* seg_tokens,
                                   const float* d_loss, void* d_logits, cudaStream_t, int*);

cudaError_t launch_mxfp4_quantize(int64_t rows, int cols, const void* src, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t, int*);
cudaError_t launch_mxfp4_dequantize(int64_t rows, int cols, const uint8_t* codes,
                                    const uint8_t* scales, void* dst, cudaStream_t, int*);
cudaError_t launch_mxfp4_quantize_weights(int n, int H, int Hp, const void* w, uint8_t* codes,
                                          uint8_t* scales, cudaStream_t, int*);
cudaError_t launch_mxfp4_dispatch(const Dims&, const PlanPtrs&, const void* x, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t, int*);
cudaError_t launch_mxfp4_prefetch(const Dims&, const PlanPtrs&, const uint8_t* home_codes,
                                  const uint8_t* home_scales, uint8_t* slot_codes,
                                  uint8_t* slot_scales, cudaStream_t, int*);
cudaError_t launch_mxfp4_grouped_gemm(const Dims&, const PlanPtrs&, const uint8_t* a,
                                      const uint8_t* a_scales, const uint8_t* home,
                                      const uint8_t* home_scales, const uint8_t* slot,
                                      const uint8_t* slot_scales, void* y, cudaStream_t, int*);

}  // namespace moonep
