// The runtime of fake_runtime.cpp, with calls of the feed-forward operators.
//
//   fake_runtime_ffn CALL DEVICE [DEVICE ...]   CALL on each device in turn
#define main fake_runtime_main
#include "fake_runtime.cpp"
#undef main

#include "../include/moonep_ffn.h"

static int ffn_call(const std::string& what) {
  moonep_dims d;
  std::memset(&d, 0, sizeof d);
  d.R = 2, d.E = 8, d.B = 4, d.K = 2, d.S = 4096, d.H = 512, d.Hp = 512;
  void* ws = at(0x10000000);
  auto* a = (uint16_t*)at(0x100000);
  auto* f = (float*)at(0x300000);
  auto* s = (int32_t*)at(0x400000);
  moonep_linear_dims few = {1, 4096, 512, MOONEP_ACT_NONE, 0};
  moonep_linear_dims many = {65536, 4096, 4096, MOONEP_ACT_SWIGLU, 0};
  if (what == "linear") return moonep_linear(&many, a, a, f, nullptr, a, a, s, nullptr);
  if (what == "linear_few") return moonep_linear(&few, a, a, f, nullptr, a, a, s, nullptr);
  if (what == "linear_dx") return moonep_linear_dx(&many, a, a, a, s, nullptr);
  if (what == "linear_dw") return moonep_linear_dw(&many, a, a, f, 0, s, nullptr);
  if (what == "act_backward")
    return moonep_act_backward(65536, 4096, MOONEP_ACT_GELU, a, a, a, f, 0, f, nullptr);
  if (what == "grouped_gemm_act")
    return moonep_grouped_gemm_act(&d, ws, MOONEP_ACT_SILU, a, a, a, f, a, a, nullptr);
  std::exit(2);
}

int main(int argc, char** argv) {
  for (int i = 2; i < argc; ++i) {
    device = std::atoi(argv[i]);
    std::printf("returned %d\n", ffn_call(argv[1]));
  }
  return 0;
}
