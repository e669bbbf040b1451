// Eight bf16 values, one 16-byte access, as fp32 and back.
#pragma once

#include "tcgen05.cuh"

namespace moonep {

__device__ __forceinline__ void unpack8(float (&f)[8], const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16x2(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace moonep
