// Host side of the C ABI declared in include/moonep_ops.h: argument checks and
// launches.
#include <cmath>

#include "host.h"
#include "ops.h"

namespace moonep {

static int check_router(const moonep_router_dims* in, RouterDims* d) {
  if (in == nullptr) return MOONEP_ERR_ARG;
  const moonep_router_dims& x = *in;
  if (x.T <= 0 || x.E <= 0 || x.K <= 0 || x.segment < 0) return MOONEP_ERR_ARG;
  if (x.score != 0 && x.score != 1) return MOONEP_ERR_ARG;
  if (x.normalise != 0 && x.normalise != 1) return MOONEP_ERR_ARG;
  if (x.dtype != 0 && x.dtype != 1) return MOONEP_ERR_ARG;
  if (!std::isfinite(x.scale)) return MOONEP_ERR_ARG;
  if (x.K > x.E || x.K > 128 || x.E > kMaxExperts || x.segment > x.T) return MOONEP_ERR_SHAPE;
  // (token counters run a block past the last token)
  if ((int64_t)x.T * x.K >= (int64_t(1) << 31) - 4096) return MOONEP_ERR_SHAPE;
  d->T = x.T;
  d->E = x.E;
  d->K = x.K;
  d->segment = x.segment ? x.segment : x.T;
  d->score = x.score;
  d->normalise = x.normalise;
  d->bf16 = x.dtype;
  d->scale = x.scale;
  d->G = (int)(((int64_t)x.T + d->segment - 1) / d->segment);
  d->per_block = d->blocks = 0;
  if ((int64_t)d->G * d->E >= (int64_t(1) << 31)) return MOONEP_ERR_SHAPE;
  int bits = 0;  // a sum of `segment` probabilities fits 62 bits
  while ((int64_t(1) << bits) < d->segment) ++bits;
  d->shift = std::min(46, 62 - bits);
  return MOONEP_OK;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace moonep

using namespace moonep;

extern "C" {

int moonep_router_workspace_bytes(const moonep_router_dims* dims, size_t* bytes) {
  RouterDims d;
  const int rc = check_router(dims, &d);
  if (rc != MOONEP_OK) return rc;
  if (bytes == nullptr) return MOONEP_ERR_ARG;
  *bytes = router_scratch(d, nullptr).total_bytes;
  return MOONEP_OK;
}

int moonep_router_forward(const moonep_router_dims* dims, const void* logits,
                          const uint8_t* token_mask, int32_t* topk_idx, float* gates, void* ws,
                          int32_t* counts, float* prob_sum, int32_t* seg_tokens, float* loss,
                          void* stream) {
  RouterDims d;
  const int rc = check_router(dims, &d);
  if (rc != MOONEP_OK) return rc;
  MOONEP_NEED(logits);
  MOONEP_NEED(topk_idx);
  MOONEP_NEED(gates);
  if (!aligned16(token_mask)) return MOONEP_ERR_ALIGN;
  if (ws || counts || prob_sum || seg_tokens || loss) {
    MOONEP_NEED(ws);
    MOONEP_NEED(counts);
    MOONEP_NEED(prob_sum);
    MOONEP_NEED(seg_tokens);
    if (loss == nullptr) return MOONEP_ERR_ARG;
    if (!aligned4(loss)) return MOONEP_ERR_ALIGN;
  }
  const RouterOut out{topk_idx, gates, counts, prob_sum, seg_tokens, loss};
  int n = 0;
  const cudaError_t e = launch_router_forward(d, logits, token_mask, out, router_scratch(d, ws),
                                              (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_router_backward(const moonep_router_dims* dims, const void* logits,
                           const uint8_t* token_mask, const int32_t* topk_idx,
                           const float* d_gates, const int32_t* counts,
                           const int32_t* seg_tokens, const float* d_loss, void* d_logits,
                           void* stream) {
  RouterDims d;
  const int rc = check_router(dims, &d);
  if (rc != MOONEP_OK) return rc;
  MOONEP_NEED(logits);
  MOONEP_NEED(topk_idx);
  MOONEP_NEED(d_logits);
  if (!aligned16(token_mask) || !aligned16(d_gates)) return MOONEP_ERR_ALIGN;
  if (counts || seg_tokens || d_loss) {
    MOONEP_NEED(counts);
    MOONEP_NEED(seg_tokens);
    if (d_loss == nullptr) return MOONEP_ERR_ARG;
    if (!aligned4(d_loss)) return MOONEP_ERR_ALIGN;
  } else if (d_gates == nullptr) {
    return MOONEP_ERR_ARG;
  }
  int n = 0;
  const cudaError_t e =
      launch_router_backward(d, logits, token_mask, topk_idx, d_gates, counts, seg_tokens, d_loss,
                             d_logits, (cudaStream_t)stream, &n);
  return finish(e, n);
}

static int check_rows(int64_t rows, int32_t cols) {
  if (rows < 0 || cols <= 0) return MOONEP_ERR_ARG;
  if (cols % 32 != 0 || rows >= (int64_t(1) << 40)) return MOONEP_ERR_SHAPE;
  return MOONEP_OK;
}

int moonep_mxfp4_quantize(int64_t rows, int32_t cols, const uint16_t* src, uint8_t* codes,
                          uint8_t* scales, void* stream) {
  const int rc = check_rows(rows, cols);
  if (rc != MOONEP_OK) return rc;
  if (rows == 0) return MOONEP_OK;
  MOONEP_NEED(src);
  MOONEP_NEED(codes);
  MOONEP_NEED(scales);
  int n = 0;
  const cudaError_t e =
      launch_mxfp4_quantize(rows, cols, src, codes, scales, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_mxfp4_dequantize(int64_t rows, int32_t cols, const uint8_t* codes,
                            const uint8_t* scales, uint16_t* dst, void* stream) {
  const int rc = check_rows(rows, cols);
  if (rc != MOONEP_OK) return rc;
  if (rows == 0) return MOONEP_OK;
  MOONEP_NEED(codes);
  MOONEP_NEED(scales);
  MOONEP_NEED(dst);
  int n = 0;
  const cudaError_t e =
      launch_mxfp4_dequantize(rows, cols, codes, scales, dst, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_mxfp4_quantize_weights(int32_t n, int32_t H, int32_t Hp, const uint16_t* w,
                                  uint8_t* codes, uint8_t* scales, void* stream) {
  if (n < 0 || H <= 0 || Hp <= 0) return MOONEP_ERR_ARG;
  if (H % 64 != 0 || Hp % 64 != 0 || Hp / 64 > 65535) return MOONEP_ERR_SHAPE;
  if ((int64_t)n * (MOONEP_MXFP4_SCALE_PITCH(H) / 8) >= (int64_t(1) << 31)) return MOONEP_ERR_SHAPE;
  if (n == 0) return MOONEP_OK;
  MOONEP_NEED(w);
  MOONEP_NEED(codes);
  MOONEP_NEED(scales);
  int k = 0;
  const cudaError_t e =
      launch_mxfp4_quantize_weights(n, H, Hp, w, codes, scales, (cudaStream_t)stream, &k);
  return finish(e, k);
}

int moonep_mxfp4_prefetch_weights(const moonep_dims* dims, void* plan_ws, const uint8_t* home_codes,
                                  const uint8_t* home_scales, uint8_t* slot_codes,
                                  uint8_t* slot_scales, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(home_codes);
  MOONEP_NEED(home_scales);
  if (d.B > 0) {
    MOONEP_NEED(slot_codes);
    MOONEP_NEED(slot_scales);
  }
  int n = 0;
  if ((int64_t)d.Hp * (d.H / 2) / 16 >= (int64_t(1) << 30)) return MOONEP_ERR_SHAPE;
  const cudaError_t e = launch_mxfp4_prefetch(d, P, home_codes, home_scales, slot_codes,
                                              slot_scales, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_mxfp4_dispatch(const moonep_dims* dims, void* plan_ws, const uint16_t* x,
                          uint8_t* recv_codes, uint8_t* recv_scales, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(x);
  MOONEP_NEED(recv_codes);
  MOONEP_NEED(recv_scales);
  int n = 0;
  const cudaError_t e =
      launch_mxfp4_dispatch(d, P, x, recv_codes, recv_scales, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_mxfp4_grouped_gemm(const moonep_dims* dims, void* plan_ws, const uint8_t* recv_codes,
                              const uint8_t* recv_scales, const uint8_t* home_codes,
                              const uint8_t* home_scales, const uint8_t* slot_codes,
                              const uint8_t* slot_scales, uint16_t* y, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(recv_codes);
  MOONEP_NEED(recv_scales);
  MOONEP_NEED(home_codes);
  MOONEP_NEED(home_scales);
  MOONEP_NEED(y);
  if (d.B > 0) {
    MOONEP_NEED(slot_codes);
    MOONEP_NEED(slot_scales);
  }
  // rows are addressed by 32-bit coordinates, up to a tile past the last one
  const int64_t most = (int64_t(1) << 31) - 512;
  if (d.N >= most || (int64_t)d.E * d.Hp >= most || (int64_t)d.R * d.B * d.Hp >= most)
    return MOONEP_ERR_SHAPE;
  int n = 0;
  const cudaError_t e =
      launch_mxfp4_grouped_gemm(d, P, recv_codes, recv_scales, home_codes, home_scales, slot_codes,
                                slot_scales, y, (cudaStream_t)stream, &n);
  return finish(e, n);
}

}  // extern "C"
