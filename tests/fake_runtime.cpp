// A CUDA runtime of two devices that launches nothing, for host-side tests of the library's
// launchers: linked with the library's objects in place of the real one.  It keeps what is
// a device's own there (the shared-memory opt-in of a kernel, the number of multiprocessors),
// refuses a launch that asks for more shared memory than the current device was told of,
// and prints each launch.
//
//   fake_runtime CALL DEVICE [DEVICE ...]   CALL on each device in turn
//   fake_runtime offset CALL BYTES          CALL with a workspace BYTES past a 256-byte boundary
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

static int atomicOr(int*, int) { return 0; }  // (named by a device function of the header)
#include "../perfectly_balanced_token_gb300/csrc/common.cuh"
#include "../include/moonep_ops.h"

namespace {
int device = 0;
const int kSms[2] = {152, 76};
std::map<const void*, std::string> names;
std::map<const void*, int> opted_in[2];

cudaError_t launch(const void* f, dim3 grid, size_t smem, void** args) {
  const std::string& name = names[f];
  const int most = opted_in[device].count(f) ? opted_in[device][f] : 48 << 10;
  const bool ok = smem <= (size_t)most;
  std::printf("device %d %s grid %u %s", device, name.c_str(), grid.x, ok ? "ok" : "refused");
  // the kernels that edit tensor maps: where their copies lie (argument of type PlanPtrs)
  const int at = name.find("k_mxfp4_gemm") != std::string::npos     ? 10
                 : name.find("k_ggemm_2sm") != std::string::npos    ? 6
                 : name.find("k_ggemm_dw_2sm") != std::string::npos ? 5
                                                                    : -1;
  if (at >= 0 && args) {
    const auto* p = static_cast<const moonep::PlanPtrs*>(args[at]);
    std::printf(" maps %zu", (size_t)p->tmaps);
  }
  std::printf("\n");
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}
CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) { return *v = kSms[d], cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int v) {
  opted_in[device][f] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  return *n = kSms[device] / 2, cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t,
                                                                   unsigned) {
  return *n = 1, cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void** p, const void*) { return *p = nullptr, cudaErrorNotSupported; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = (void*)encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  return launch(f, c->gridDim, c->dynamicSmemBytes, args);
}

// what the compiler's host code for <<< >>> and for registering kernels calls
struct Pushed {
  dim3 grid, block;
  size_t smem;
  cudaStream_t stream;
};
static std::vector<Pushed> pushed;
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t s, cudaStream_t st) {
  pushed.push_back({g, b, s, st});
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* s, void* st) {
  *g = pushed.back().grid, *b = pushed.back().block, *s = pushed.back().smem;
  *(cudaStream_t*)st = pushed.back().stream;
  pushed.pop_back();
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) { return *k = (cudaKernel_t)f, cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 g, dim3, void** args, size_t smem, cudaStream_t) {
  return launch((const void*)k, g, smem, args);
}
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*,
                            dim3*, dim3*, int*) {
  names[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
}

// Addresses that nothing reads or writes
static uint8_t* at(size_t a) { return reinterpret_cast<uint8_t*>(a); }

static int call(const std::string& what, void* ws) {
  moonep_dims d;
  std::memset(&d, 0, sizeof d);
  d.R = 2, d.E = 8, d.B = 4, d.K = 2, d.S = 4096, d.H = 512, d.Hp = 512;
  auto* a = (uint16_t*)at(0x100000);
  auto* b = (uint8_t*)at(0x200000);
  auto* f = (float*)at(0x300000);
  if (what == "mxfp4_grouped_gemm") return moonep_mxfp4_grouped_gemm(&d, ws, b, b, b, b, b, b, a, nullptr);
  if (what == "grouped_gemm") return moonep_grouped_gemm(&d, ws, a, a, a, a, nullptr);
  if (what == "grouped_gemm_dx") return moonep_grouped_gemm_dx(&d, ws, a, a, a, a, nullptr);
  if (what == "grouped_gemm_dw") return moonep_grouped_gemm_dw(&d, ws, a, a, f, f, nullptr);
  std::exit(2);
}

int main(int argc, char** argv) {
  if (argc == 4 && !std::strcmp(argv[1], "offset")) {
    std::printf("returned %d\n", call(argv[2], at(0x10000000 + std::strtoul(argv[3], nullptr, 0))));
    return 0;
  }
  for (int i = 2; i < argc; ++i) {
    device = std::atoi(argv[i]);
    std::printf("returned %d\n", call(argv[1], at(0x10000000)));
  }
  return 0;
}
