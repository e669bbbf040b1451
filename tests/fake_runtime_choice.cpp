// The runtime of fake_runtime.cpp with as many clusters at once as the GPU has (of 2, 4 and 8 CTAs: 76, 36
// and 15 on the first device, half of it on the second), for what the launchers choose by size.
//
//   fake_runtime_choice DEVICE CALL SIZES...   linear T K N ACT F32, dx T K N, dw T K N:
//                                              the kernel, its grid and the columns of its tiles
//                                              experts R E B K S H Hp ACT: the same of the plan's product
//                                              act_bias E Hp: the gradient with the experts' bias sums
#include <cuda_runtime.h>

#define main fake_runtime_main
#define cudaLaunchKernelExC fake_launch
#define cudaOccupancyMaxActiveClusters fake_clusters
#include "fake_runtime.cpp"
#undef main
#undef cudaLaunchKernelExC
#undef cudaOccupancyMaxActiveClusters

#include "../include/moonep_ffn.h"

static int refused = 0;

extern "C" {
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  const unsigned x = c->attrs[0].val.clusterDim.x;
  *n = (x == 2 ? 76 : (x == 4 ? 36 : 15)) / (device + 1);
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  if (c->gridDim.y > 65535 || c->gridDim.z > 65535) {
    ++refused;
    std::printf("refused grid %u %u %u\n", c->gridDim.x, c->gridDim.y, c->gridDim.z);
    return cudaErrorInvalidConfiguration;
  }
  const std::string& name = names[f];
  int columns = 0;  // (the tiles' columns: an argument of k_product, where product.cu says)
  if (name.find("k_product_split") == std::string::npos && name.find("k_product") != std::string::npos)
    columns = static_cast<const int*>(args[1])[7];
  std::printf("%s %u %u %d\n", name.c_str(), c->gridDim.x, c->gridDim.y, columns);
  return cudaSuccess;
}
}

int main(int argc, char** argv) {
  if (argc < 4) return 2;
  device = std::atoi(argv[1]);
  const std::string what = argv[2];
  int v[8] = {};
  for (int i = 3; i < argc && i < 11; ++i) v[i - 3] = std::atoi(argv[i]);
  auto* a = (uint16_t*)at(0x100000);
  auto* f = (float*)at(0x300000);
  auto* s = (int32_t*)at(0x400000);
  moonep_linear_dims d = {v[0], v[1], v[2], 0, 0};
  moonep_dims m;
  std::memset(&m, 0, sizeof m);
  int rc = -1;
  if (what == "linear") {
    d.act = v[3], d.out_f32 = v[4];
    rc = moonep_linear(&d, a, a, f, nullptr, a, a, s, nullptr);
  } else if (what == "dx") {
    rc = moonep_linear_dx(&d, a, a, a, s, nullptr);
  } else if (what == "dw") {
    rc = moonep_linear_dw(&d, a, a, f, 0, s, nullptr);
  } else if (what == "experts") {
    m.R = v[0], m.E = v[1], m.B = v[2], m.K = v[3], m.S = v[4], m.H = v[5], m.Hp = v[6], m.mode = m.B == 0;
    rc = moonep_grouped_gemm_act(&m, at(0x10000000), v[7], a, a, a, f, a, a, nullptr);
  } else if (what == "act_bias") {
    m.R = 1, m.E = v[0], m.K = 1, m.S = 1, m.H = 64, m.Hp = v[1], m.mode = 1;
    rc = moonep_grouped_act_backward(&m, at(0x10000000), MOONEP_ACT_RELU, a, a, a, f, 0, f, nullptr);
  }
  std::printf("returned %d refused %d\n", rc, refused);
  return 0;
}
