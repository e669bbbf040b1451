// Host side of the C ABI declared in include/moonep.h: argument checks, the
// plan-workspace layout and the launches.  Nothing here allocates device
// memory; only moonep_read_status and moonep_plan_export synchronise.
#include <algorithm>
#include <mutex>

#include "host.h"

namespace moonep {
cudaError_t launch_plan(const Dims&, const int32_t*, const PlanPtrs&, cudaStream_t, int*);
cudaError_t launch_prefetch(const Dims&, const PlanPtrs&, const void*, void*, cudaStream_t, int*);
cudaError_t launch_dispatch(const Dims&, const PlanPtrs&, const void*, void*, cudaStream_t, int*);
cudaError_t launch_dispatch_send_once(const Dims&, const PlanPtrs&, const void*, const float*, void*,
                                      float*, cudaStream_t, int*);
cudaError_t launch_grouped_gemm(const Dims&, const PlanPtrs&, const void*, const void*, const void*,
                                void*, cudaStream_t, int*);
cudaError_t launch_combine(const Dims&, const PlanPtrs&, const void*, const float*, void*,
                           cudaStream_t, int*);
cudaError_t launch_reduce(const Dims&, const PlanPtrs&, float*, float*, cudaStream_t, int*);
cudaError_t launch_grouped_gemm_dx(const Dims&, const PlanPtrs&, const void*, const void*, const void*,
                                   void*, cudaStream_t, int*);
cudaError_t launch_grouped_gemm_dw(const Dims&, const PlanPtrs&, const void*, const void*, float*,
                                   float*, cudaStream_t, int*);
cudaError_t launch_combine_backward(const Dims&, const PlanPtrs&, const void*, const float*,
                                    const void*, void*, float*, cudaStream_t, int*);
cudaError_t launch_dispatch_backward(const Dims&, const PlanPtrs&, const void*, void*, cudaStream_t,
                                     int*);
cudaError_t launch_wait_selftest(int32_t*, uint32_t, int32_t*, cudaStream_t, int*);

}  // namespace moonep

using namespace moonep;

extern "C" {

int moonep_plan_workspace_bytes(const moonep_dims* dims, size_t* bytes) {
  Dims d;
  const int rc = check_dims(dims, &d);
  if (rc != MOONEP_OK) return rc;
  if (bytes == nullptr) return MOONEP_ERR_ARG;
  *bytes = make_layout(d).pub.total_bytes;
  return MOONEP_OK;
}

int moonep_get_plan_layout(const moonep_dims* dims, moonep_plan_layout* out) {
  Dims d;
  const int rc = check_dims(dims, &d);
  if (rc != MOONEP_OK) return rc;
  if (out == nullptr) return MOONEP_ERR_ARG;
  *out = make_layout(d).pub;
  return MOONEP_OK;
}

int moonep_plan_views(const moonep_dims* dims, const void* plan_ws, moonep_plan_view* out) {
  Dims d;
  const int rc = check_dims(dims, &d);
  if (rc != MOONEP_OK) return rc;
  if (plan_ws == nullptr || out == nullptr) return MOONEP_ERR_ARG;
  if (!aligned16(plan_ws)) return MOONEP_ERR_ALIGN;
  const moonep_plan_layout L = make_layout(d).pub;
  const uint8_t* b = static_cast<const uint8_t*>(plan_ws);
  out->cu_seqlens = reinterpret_cast<const int32_t*>(b + L.cu_seqlens);
  out->dst = reinterpret_cast<const int32_t*>(b + L.dst);
  out->inverse = reinterpret_cast<const int32_t*>(b + L.inverse);
  out->slot_expert = reinterpret_cast<const int32_t*>(b + L.slot_expert);
  out->status = reinterpret_cast<const int32_t*>(b + L.status);
  return MOONEP_OK;
}

int moonep_plan(const moonep_dims* dims, const int32_t* topk_idx, void* plan_ws, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(topk_idx);
  int n = 0;
  const cudaError_t e = launch_plan(d, topk_idx, P, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_prefetch_weights(const moonep_dims* dims, void* plan_ws, const uint16_t* w_home,
                            uint16_t* w_slot, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(w_home);
  if (d.B > 0) MOONEP_NEED(w_slot);
  int n = 0;
  const cudaError_t e = launch_prefetch(d, P, w_home, w_slot, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_dispatch(const moonep_dims* dims, void* plan_ws, const uint16_t* x, uint16_t* recv,
                    void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(x);
  MOONEP_NEED(recv);
  int n = 0;
  const cudaError_t e = launch_dispatch(d, P, x, recv, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_dispatch_send_once(const moonep_dims* dims, void* plan_ws, const uint16_t* x,
                              const float* gates, uint16_t* recv, float* recv_weight,
                              void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(x);
  MOONEP_NEED(gates);
  MOONEP_NEED(recv);
  MOONEP_NEED(recv_weight);
  if (d.K > 128) return MOONEP_ERR_SHAPE;  // one thread per route entry in the send pass
  int n = 0;
  const cudaError_t e = launch_dispatch_send_once(d, P, x, gates, recv, recv_weight,
                                                  (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_grouped_gemm(const moonep_dims* dims, void* plan_ws, const uint16_t* recv,
                        const uint16_t* w_home, const uint16_t* w_slot, uint16_t* y,
                        void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(recv);
  MOONEP_NEED(w_home);
  MOONEP_NEED(y);
  if (d.B > 0) MOONEP_NEED(w_slot);
  int n = 0;
  const cudaError_t e = launch_grouped_gemm(d, P, recv, w_home, w_slot, y, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_combine(const moonep_dims* dims, void* plan_ws, const uint16_t* y, const float* gates,
                   uint16_t* out, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(y);
  MOONEP_NEED(gates);
  MOONEP_NEED(out);
  int n = 0;
  const cudaError_t e = launch_combine(d, P, y, gates, out, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_reduce_grad(const moonep_dims* dims, void* plan_ws, float* g_home, float* g_slot,
                       void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(g_home);
  if (d.B > 0) MOONEP_NEED(g_slot);
  int n = 0;
  const cudaError_t e = launch_reduce(d, P, g_home, g_slot, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_combine_backward(const moonep_dims* dims, void* plan_ws, const uint16_t* y,
                            const float* gates, const uint16_t* d_out, uint16_t* d_y,
                            float* d_gates, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(y);
  MOONEP_NEED(gates);
  MOONEP_NEED(d_out);
  MOONEP_NEED(d_y);
  MOONEP_NEED(d_gates);
  if (d.K > 128 || d.Hp > 8192) return MOONEP_ERR_SHAPE;
  int n = 0;
  const cudaError_t e = launch_combine_backward(d, P, y, gates, d_out, d_y, d_gates,
                                                (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_grouped_gemm_dx(const moonep_dims* dims, void* plan_ws, const uint16_t* d_y,
                           const uint16_t* w_home, const uint16_t* w_slot, uint16_t* d_recv,
                           void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(d_y);
  MOONEP_NEED(w_home);
  MOONEP_NEED(d_recv);
  if (d.B > 0) MOONEP_NEED(w_slot);
  int n = 0;
  const cudaError_t e = launch_grouped_gemm_dx(d, P, d_y, w_home, w_slot, d_recv,
                                               (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_grouped_gemm_dw(const moonep_dims* dims, void* plan_ws, const uint16_t* recv,
                           const uint16_t* d_y, float* g_home, float* g_slot, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(recv);
  MOONEP_NEED(d_y);
  MOONEP_NEED(g_home);
  if (d.B > 0) MOONEP_NEED(g_slot);
  if (d.mode != 0) return MOONEP_ERR_ARG;       // gradients exist in training only
  if (d.H % 128 != 0) return MOONEP_ERR_SHAPE;  // 128-row tiles of H
  int n = 0;
  const cudaError_t e = launch_grouped_gemm_dw(d, P, recv, d_y, g_home, g_slot,
                                               (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_dispatch_backward(const moonep_dims* dims, void* plan_ws, const uint16_t* d_recv,
                             uint16_t* d_x, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(d_recv);
  MOONEP_NEED(d_x);
  int n = 0;
  const cudaError_t e = launch_dispatch_backward(d, P, d_recv, d_x, (cudaStream_t)stream, &n);
  return finish(e, n);
}

int moonep_read_status(const moonep_dims* dims, const void* plan_ws, int32_t* host_status,
                       void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  if (host_status == nullptr) return MOONEP_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (cudaMemcpyAsync(host_status, P.status, sizeof(int32_t), cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return MOONEP_ERR_CUDA;
  return cudaStreamSynchronize(st) == cudaSuccess ? MOONEP_OK : MOONEP_ERR_CUDA;
}

int moonep_plan_export(const moonep_dims* dims, const void* plan_ws, void* host_dst, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  (void)P;
  if (host_dst == nullptr) return MOONEP_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (cudaMemcpyAsync(host_dst, plan_ws, lay.pub.total_bytes, cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return MOONEP_ERR_CUDA;
  return cudaStreamSynchronize(st) == cudaSuccess ? MOONEP_OK : MOONEP_ERR_CUDA;
}

const char* moonep_status_string(int s) {
  switch (s) {
    case MOONEP_OK: return "ok";
    case MOONEP_ERR_ARG: return "invalid argument (null pointer, non-positive dimension, bad mode, policy or gemm_rows)";
    case MOONEP_ERR_ALIGN: return "pointer not 16-byte aligned";
    case MOONEP_ERR_SLOTS: return "training mode needs B >= E/R prefetch slots";
    case MOONEP_ERR_SHAPE: return "unsupported shape (E%R, K>E, E>4096, B>E, H or Hp not a multiple of 64, or a size >= 2^31)";
    case MOONEP_ERR_CUDA: return "CUDA runtime error or launch failure";
    case MOONEP_ERR_SCRATCH: return "dims need more planner scratch than the fixed no-allocation capacity (4 MiB)";
    default: break;
  }
  if (s & MOONEP_ERR_ROUTING) return "device: expert id out of range or repeated within a token";
  if (s & MOONEP_ERR_INTERNAL) return "device: planner invariant failed";
  if (s & MOONEP_ERR_TIMEOUT) return "device: a bounded wait in the GEMM pipeline expired";
  return "unknown status";
}

uint64_t moonep_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int moonep_selftest_bounded_wait(int32_t* dev_status, uint32_t limit_us, int32_t* dev_elapsed_us,
                                 void* stream) {
  if (dev_status == nullptr || dev_elapsed_us == nullptr) return MOONEP_ERR_ARG;
  if (limit_us == 0 || limit_us > 1000000u) return MOONEP_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(dev_status) & 3u) || (reinterpret_cast<uintptr_t>(dev_elapsed_us) & 3u))
    return MOONEP_ERR_ALIGN;
  int n = 0;
  const cudaError_t e = launch_wait_selftest(dev_status, limit_us, dev_elapsed_us,
                                             (cudaStream_t)stream, &n);
  return finish(e, n);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// moonep_plan_noalloc: the planner with its internal scratch in a static
// device array, for callers that cannot allocate device memory.
// ---------------------------------------------------------------------------
namespace moonep {

constexpr size_t kNoAllocBytes = MOONEP_NOALLOC_SCRATCH_BYTES;
constexpr int kNoAllocMaxDevices = 64;

// Lives in the library's device image on every GPU that loads it; host code
// must not use this name as an address (it is a host-side stand-in).
static __device__ __align__(256) int32_t g_noalloc_scratch[kNoAllocBytes / sizeof(int32_t)];

static std::mutex g_noalloc_mutex;
static void* g_noalloc_base[kNoAllocMaxDevices] = {};

// Device address of g_noalloc_scratch on the current device, looked up once
// per device with that device current.
static int noalloc_base(void** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kNoAllocMaxDevices)
    return MOONEP_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  if (g_noalloc_base[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr)
      return MOONEP_ERR_CUDA;
    g_noalloc_base[dev] = p;
  }
  *out = g_noalloc_base[dev];
  return MOONEP_OK;
}

// Offsets of the planner's internal tables inside the static array.
struct NoAllocLayout {
  size_t counts, pieces, piece_n, piece_base, home_base, rank_tiles, rank_groups, total;
};

static NoAllocLayout noalloc_layout(const Dims& d) {
  NoAllocLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + std::max<size_t>(bytes, 4));
    return at;
  };
  const size_t R = d.R, E = d.E;
  L.counts = take(4 * R * d.nchunk * E);
  L.pieces = take(sizeof(Piece) * E * R);
  L.piece_n = take(4 * E);
  L.piece_base = take(4 * E * R);
  L.home_base = take(4 * E);
  L.rank_tiles = take(4 * (R + 1));
  L.rank_groups = take(4 * (R + 1));
  L.total = off;
  return L;
}

}  // namespace moonep

extern "C" int moonep_plan_noalloc(const moonep_dims* dims, const int32_t* topk_idx,
                                   void* plan_ws, void* stream) {
  MOONEP_PROLOGUE(dims, plan_ws);
  MOONEP_NEED(topk_idx);
  const NoAllocLayout S = noalloc_layout(d);
  if (S.total > kNoAllocBytes) return MOONEP_ERR_SCRATCH;
  void* base = nullptr;
  const int rc = noalloc_base(&base);
  if (rc != MOONEP_OK) return rc;
  char* b = static_cast<char*>(base);
  PlanPtrs Q = P;
  Q.counts = (int32_t*)(b + S.counts);
  Q.pieces = (Piece*)(b + S.pieces);
  Q.piece_n = (int32_t*)(b + S.piece_n);
  Q.piece_base = (int32_t*)(b + S.piece_base);
  Q.home_base = (int32_t*)(b + S.home_base);
  Q.rank_tiles = (int32_t*)(b + S.rank_tiles);
  Q.rank_groups = (int32_t*)(b + S.rank_groups);
  int n = 0;
  const cudaError_t e = launch_plan(d, topk_idx, Q, (cudaStream_t)stream, &n);
  return finish(e, n);
}
