// Host side of the C ABI declared in include/moonep_ffn.h: argument checks and
// launches.
#include <cmath>

#include "ffn.h"
#include "host.h"

namespace moonep {

// coordinates run a tile past the last row and column; tiles are counted in 32 bits
constexpr int64_t kMostRows = (int64_t(1) << 31) - 512;

static int check_linear(const moonep_linear_dims* in, LinearDims* d) {
  if (in == nullptr) return MOONEP_ERR_ARG;
  const moonep_linear_dims& x = *in;
  if (x.T < 0 || x.K <= 0 || x.N <= 0) return MOONEP_ERR_ARG;
  if (x.act < MOONEP_ACT_NONE || x.act > MOONEP_ACT_SWIGLU) return MOONEP_ERR_ARG;
  if (x.out_f32 != 0 && x.out_f32 != 1) return MOONEP_ERR_ARG;
  const int step = x.act == MOONEP_ACT_SWIGLU ? 16 : 8;
  if (x.K % 8 != 0 || x.N % step != 0) return MOONEP_ERR_SHAPE;
  if (x.T >= kMostRows || x.K >= kMostRows || x.N >= kMostRows) return MOONEP_ERR_SHAPE;
  const int64_t t = x.T / 128 + 1, k = x.K / 128 + 1, n = x.N / 128 + 1;
  if (t * n >= kMostRows || t * k >= kMostRows || k * n >= kMostRows) return MOONEP_ERR_SHAPE;
  d->T = x.T;
  d->K = x.K;
  d->N = x.N;
  d->act = x.act;
  d->f32 = x.out_f32;
  d->half = x.act == MOONEP_ACT_SWIGLU ? x.N / 2 : 0;
  return MOONEP_OK;
}

static int check_status(const int32_t* status) {
  if (status == nullptr) return MOONEP_ERR_ARG;
  return (reinterpret_cast<uintptr_t>(status) & 3u) ? MOONEP_ERR_ALIGN : MOONEP_OK;
}

static int check_act(int act, int cols) {
  if (act < MOONEP_ACT_NONE || act > MOONEP_ACT_SWIGLU) return MOONEP_ERR_ARG;
  return cols % (act == MOONEP_ACT_SWIGLU ? 16 : 8) ? MOONEP_ERR_SHAPE : MOONEP_OK;
}

static int check_act_rows(int64_t rows, int32_t cols, int act) {
  if (rows < 0 || cols <= 0) return MOONEP_ERR_ARG;
  const int rc = check_act(act, cols);
  if (rc != MOONEP_OK) return rc;
  return rows >= (int64_t(1) << 40) || cols >= kMostRows ? MOONEP_ERR_SHAPE : MOONEP_OK;
}

// the arguments that the activation's two gradients share
static int check_act_buffers(int act, const void* z, const void* d_out, const void* d_z,
                             const void* d_bias, const void* scratch) {
  MOONEP_NEED(d_out);
  if (act != MOONEP_ACT_NONE) {
    MOONEP_NEED(z);
    MOONEP_NEED(d_z);
  }
  if (!aligned16(z) || !aligned16(d_z) || !aligned16(d_bias)) return MOONEP_ERR_ALIGN;
  if (d_bias != nullptr) {
    MOONEP_NEED(scratch);
  } else if (d_z == nullptr) {
    return MOONEP_ERR_ARG;
  }
  return MOONEP_OK;
}

static int check_dropout(double p, const int64_t* rng, Dropout* out) {
  if (!(p >= 0.0 && p < 1.0)) return MOONEP_ERR_ARG;
  const double cut = std::floor(p * 65536.0 + 0.5);
  if (cut > 65535.0) return MOONEP_ERR_ARG;
  out->cut = (uint32_t)cut;
  out->scale = (float)(65536.0 / (65536.0 - cut));
  out->rng = rng;
  if (out->cut) MOONEP_NEED(rng);
  return MOONEP_OK;
}

}  // namespace moonep

using namespace moonep;

#define MOONEP_CHECK(call)                  \
  do {                                      \
    const int rc_ = (call);                 \
    if (rc_ != MOONEP_OK) return rc_;       \
  } while (0)

extern "C" {

int moonep_linear(const moonep_linear_dims* dims, const uint16_t* x, const uint16_t* w,
                  const float* bias, const uint16_t* residual, void* out, uint16_t* z,
                  int32_t* status, void* stream) {
  LinearDims d;
  MOONEP_CHECK(check_linear(dims, &d));
  if (d.T == 0) return MOONEP_OK;
  MOONEP_NEED(x);
  MOONEP_NEED(w);
  MOONEP_NEED(out);
  if (!aligned16(bias) || !aligned16(residual) || !aligned16(z)) return MOONEP_ERR_ALIGN;
  MOONEP_CHECK(check_status(status));
  int n = 0;
  const cudaError_t e =
      launch_linear(d, x, w, bias, residual, out, z, status, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_linear_dx(const moonep_linear_dims* dims, const uint16_t* d_z, const uint16_t* w,
                     uint16_t* d_x, int32_t* status, void* stream) {
  LinearDims d;
  MOONEP_CHECK(check_linear(dims, &d));
  if (d.T == 0) return MOONEP_OK;
  MOONEP_NEED(d_z);
  MOONEP_NEED(w);
  MOONEP_NEED(d_x);
  MOONEP_CHECK(check_status(status));
  int n = 0;
  const cudaError_t e = launch_linear_dx(d, d_z, w, d_x, status, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_linear_dw(const moonep_linear_dims* dims, const uint16_t* x, const uint16_t* d_z,
                     float* d_w, int32_t accumulate, int32_t* status, void* stream) {
  LinearDims d;
  MOONEP_CHECK(check_linear(dims, &d));
  if (accumulate != 0 && accumulate != 1) return MOONEP_ERR_ARG;
  MOONEP_NEED(d_w);
  if (d.T == 0) {  // a sum of nothing
    if (accumulate) return MOONEP_OK;
    return finish(cudaMemsetAsync(d_w, 0, (size_t)d.K * d.N * 4, (cudaStream_t)stream), 0);
  }
  MOONEP_NEED(x);
  MOONEP_NEED(d_z);
  MOONEP_CHECK(check_status(status));
  int n = 0;
  const cudaError_t e =
      launch_linear_dw(d, x, d_z, d_w, accumulate, status, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_act_backward_workspace_bytes(int64_t rows, int32_t cols, size_t* bytes) {
  MOONEP_CHECK(check_act_rows(rows, cols, MOONEP_ACT_NONE));
  if (bytes == nullptr) return MOONEP_ERR_ARG;
  *bytes = std::max<size_t>(1, (size_t)act_chunks(rows)) * cols * sizeof(float);
  return MOONEP_OK;
}

int moonep_act_backward(int64_t rows, int32_t cols, int32_t act, const uint16_t* z,
                        const uint16_t* d_out, uint16_t* d_z, float* d_bias, int32_t accumulate,
                        void* scratch, void* stream) {
  MOONEP_CHECK(check_act_rows(rows, cols, act));
  if (accumulate != 0 && accumulate != 1) return MOONEP_ERR_ARG;
  if (rows == 0) {
    if (d_bias == nullptr || accumulate) return MOONEP_OK;
    MOONEP_NEED(d_bias);
    return finish(cudaMemsetAsync(d_bias, 0, (size_t)cols * 4, (cudaStream_t)stream), 0);
  }
  MOONEP_CHECK(check_act_buffers(act, z, d_out, d_z, d_bias, scratch));
  int n = 0;
  const cudaError_t e = launch_act_backward(rows, cols, act, z, d_out, d_z, d_bias, accumulate,
                                            (float*)scratch, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_grouped_gemm_act(const moonep_dims* dims, void* plan_ws, int32_t act, const uint16_t* recv,
                            const uint16_t* w_home, const uint16_t* w_slot, const float* bias,
                            uint16_t* y, uint16_t* z, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_CHECK(check_act(act, d.Hp));
  MOONEP_NEED(recv);
  MOONEP_NEED(w_home);
  MOONEP_NEED(y);
  if (d.B > 0) MOONEP_NEED(w_slot);
  if (!aligned16(bias) || !aligned16(z)) return MOONEP_ERR_ALIGN;
  if (d.N >= kMostRows || (int64_t)d.E * d.H >= kMostRows || (int64_t)d.R * d.B * d.H >= kMostRows ||
      (int64_t)d.max_mtiles * (d.Hp / 128 + 1) >= kMostRows)
    return MOONEP_ERR_SHAPE;
  int n = 0;
  const cudaError_t e = launch_grouped_gemm_act(d, P, act, recv, w_home, w_slot, bias, y, z,
                                                (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_grouped_act_backward_workspace_bytes(const moonep_dims* dims, size_t* bytes) {
  Dims d;
  MOONEP_CHECK(check_dims(dims, &d));
  if (bytes == nullptr) return MOONEP_ERR_ARG;
  *bytes = (size_t)d.max_mtiles * d.Hp * sizeof(float);
  return MOONEP_OK;
}

int moonep_grouped_act_backward(const moonep_dims* dims, void* plan_ws, int32_t act,
                                const uint16_t* z, const uint16_t* d_y, uint16_t* d_z, float* d_bias,
                                int32_t accumulate, void* scratch, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_CHECK(check_act(act, d.Hp));
  if (accumulate != 0 && accumulate != 1) return MOONEP_ERR_ARG;
  MOONEP_CHECK(check_act_buffers(act, z, d_y, d_z, d_bias, scratch));
  if (d.Hp > 65535 * 1024) return MOONEP_ERR_SHAPE;  // 1024 columns of d_bias a block, blocks in y
  int n = 0;
  const cudaError_t e = launch_grouped_act_backward(d, P, act, z, d_y, d_z, d_bias, accumulate,
                                                    (float*)scratch, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_combine_dropout(const moonep_dims* dims, void* plan_ws, const uint16_t* y,
                           const float* gates, const uint16_t* residual, uint16_t* out, double p,
                           const int64_t* rng, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  Dropout drop;
  MOONEP_CHECK(check_dropout(p, rng, &drop));
  MOONEP_NEED(y);
  MOONEP_NEED(gates);
  MOONEP_NEED(out);
  if (!aligned16(residual)) return MOONEP_ERR_ALIGN;
  int n = 0;
  const cudaError_t e =
      launch_combine_dropout(d, P, y, gates, residual, out, drop, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_combine_dropout_backward(const moonep_dims* dims, void* plan_ws, const uint16_t* y,
                                    const float* gates, const uint16_t* d_out, uint16_t* d_y,
                                    float* d_gates, double p, const int64_t* rng, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  Dropout drop;
  MOONEP_CHECK(check_dropout(p, rng, &drop));
  MOONEP_NEED(y);
  MOONEP_NEED(gates);
  MOONEP_NEED(d_out);
  MOONEP_NEED(d_y);
  MOONEP_NEED(d_gates);
  if (d.K > 128 || d.Hp > 8192) return MOONEP_ERR_SHAPE;
  int n = 0;
  const cudaError_t e = launch_combine_dropout_backward(d, P, y, gates, d_out, d_y, d_gates, drop,
                                                        (cudaStream_t)stream, &n);
  return finish(e, n);
}

}  // extern "C"
