// The combine with dropout and residual, forward and backward.  Bound by memory: 16-byte accesses,
// each value read and written once, eight copies' loads in flight in every thread.
#include <algorithm>

#include "ffn.h"
#include "pdl.cuh"
#include "vec.cuh"

namespace moonep {

// ---------------------------------------------------------------------------
// dropout: Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
// as 1, 2, 3", 2011), its counter (element / 8, offset) and its key the seed: the four words are the
// 16-bit numbers of eight elements, one 16-byte access.  No mask is stored: the backward pass draws
// the same numbers again, about 80 instructions for 16 (K + 2) bytes of traffic.
// ---------------------------------------------------------------------------
struct Philox {
  uint32_t k0, k1, o0, o1;
  __device__ __forceinline__ explicit Philox(const int64_t* rng) {
    const uint64_t seed = (uint64_t)__ldg(reinterpret_cast<const long long*>(rng));
    const uint64_t offset = (uint64_t)__ldg(reinterpret_cast<const long long*>(rng) + 1);
    k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
  }
  __device__ __forceinline__ void numbers(uint64_t group, uint32_t (&w)[4]) const {
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = o0, c3 = o1, a = k0, b = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t m0 = (uint64_t)c0 * 0xD2511F53u, m1 = (uint64_t)c2 * 0xCD9E8D57u;
      c0 = (uint32_t)(m1 >> 32) ^ c1 ^ a;
      c2 = (uint32_t)(m0 >> 32) ^ c3 ^ b;
      c1 = (uint32_t)m1;
      c3 = (uint32_t)m0;
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
  }
  // f[i] scaled or dropped, for the eight elements of a group
  __device__ __forceinline__ void apply(uint64_t group, uint32_t cut, float scale, float (&f)[8]) const {
    uint32_t w[4];
    numbers(group, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = (w[i] & 0xffffu) >= cut ? f[2 * i] * scale : 0.f;
      f[2 * i + 1] = (w[i] >> 16) >= cut ? f[2 * i + 1] * scale : 0.f;
    }
  }
};

constexpr int kRowThreads = 128;

// out[t] = bf16( residual[t] + dropout( sum over k ascending of gates[t][k] y[dst[t][k]] ) )
template <int KC, bool DROP, bool RES>
__global__ void __launch_bounds__(kRowThreads)
k_combine_dropout(Dims d, PlanPtrs p, const uint4* __restrict__ y, const float* __restrict__ gates,
                  const uint4* __restrict__ residual, uint4* __restrict__ out, Dropout drop) {
  grid_wait();
  grid_trigger();
  if (plan_failed(p.status)) return;
  const int hv = d.Hp / 8;
  const int ntok = d.R * d.S;
  for (int t = blockIdx.x; t < ntok; t += gridDim.x) {
    const int32_t* dt = p.dst + (size_t)t * d.K;
    const float* gt = gates + (size_t)t * d.K;
    for (int a = threadIdx.x; a < hv; a += kRowThreads) {
      uint4 res;
      if (RES) res = __ldcs(residual + (size_t)t * hv + a);
      float acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      for (int k0 = 0; k0 < d.K; k0 += KC) {
        uint4 v[KC];
        float g[KC];
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          if (k0 + k < d.K) {
            v[k] = __ldcs(y + (size_t)__ldg(dt + k0 + k) * hv + a);
            g[k] = __ldg(gt + k0 + k);
          }
        }
#pragma unroll
        for (int k = 0; k < KC; ++k)
          if (k0 + k < d.K) {
            float f[8];
            unpack8(f, v[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[k], f[i], acc[i]);
          }
      }
      if (DROP) Philox(drop.rng).apply((uint64_t)t * hv + a, drop.cut, drop.scale, acc);
      if (RES) {
        float f[8];
        unpack8(f, res);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
      }
      __stcs(out + (size_t)t * hv + a, pack8(acc));
    }
  }
}

// With d = dropout(d_out[t]) (the forward pass's mask and scale):
//   d_y[dst(t,k)] = bf16(gates[t][k] d)   and   d_gates[t][k] = <y[dst(t,k)], d>
// A block a token; its slice of d stays in registers, the copies come KC at a time.
constexpr int kDropMaxK = 128;

template <int VPT, int KC, bool DROP>
__global__ void __launch_bounds__(kRowThreads)
k_combine_dropout_bwd(Dims d, PlanPtrs p, const uint4* __restrict__ y,
                      const float* __restrict__ gates, const uint4* __restrict__ dout,
                      uint4* __restrict__ dy, float* __restrict__ dgates, Dropout drop) {
  __shared__ float part[kRowThreads / 32][kDropMaxK];
  grid_wait();
  grid_trigger();
  if (plan_failed(p.status)) return;
  const int hv = d.Hp / 8;
  const int ntok = d.R * d.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = blockIdx.x; t < ntok; t += gridDim.x) {
    float o[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int a = threadIdx.x + i * kRowThreads;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[i][j] = 0.f;
      if (a < hv) {
        unpack8(o[i], __ldcs(dout + (size_t)t * hv + a));
        if (DROP) Philox(drop.rng).apply((uint64_t)t * hv + a, drop.cut, drop.scale, o[i]);
      }
    }
    const int32_t* dt = p.dst + (size_t)t * d.K;
    const float* gt = gates + (size_t)t * d.K;
    for (int k0 = 0; k0 < d.K; k0 += KC) {
      size_t row[KC];
      float g[KC];
      uint4 v[KC][VPT];
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        row[k] = k0 + k < d.K ? (size_t)__ldg(dt + k0 + k) : 0;
        g[k] = k0 + k < d.K ? __ldg(gt + k0 + k) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < KC; ++k)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int a = threadIdx.x + i * kRowThreads;
          if (k0 + k < d.K && a < hv) v[k][i] = __ldcs(y + row[k] * hv + a);
        }
      float dot[KC];
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        dot[k] = 0.f;
        if (k0 + k < d.K) {
#pragma unroll
          for (int i = 0; i < VPT; ++i) {
            const int a = threadIdx.x + i * kRowThreads;
            if (a < hv) {
              float f[8], w[8];
              unpack8(f, v[k][i]);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                dot[k] = fmaf(f[j], o[i][j], dot[k]);
                w[j] = g[k] * o[i][j];
              }
              __stcs(dy + row[k] * hv + a, pack8(w));
            }
          }
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < KC; ++k) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], off);
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < KC; ++k)
          if (k0 + k < d.K) part[warp][k0 + k] = dot[k];
      }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < d.K; k += kRowThreads) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kRowThreads / 32; ++w) sum += part[w][k];
      dgates[(size_t)t * d.K + k] = sum;
    }
    __syncthreads();
  }
}

// -- host side ------------------------------------------------------------------
cudaError_t launch_combine_dropout(const Dims& d, const PlanPtrs& p, const void* y, const float* gates,
                                   const void* residual, void* out, const Dropout& drop,
                                   cudaStream_t st, int* launches) {
  const int grid = std::min(d.R * d.S, sm_count_gemm() * 16);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    e = launch_after(kernel, grid, kRowThreads, 0, st, 1, d, p, (const uint4*)y, gates,
                     (const uint4*)residual, (uint4*)out, drop);
  };
  const bool r = residual != nullptr;
  if (drop.cut) {
    if (d.K >= 8) r ? go(k_combine_dropout<8, true, true>) : go(k_combine_dropout<8, true, false>);
    else r ? go(k_combine_dropout<4, true, true>) : go(k_combine_dropout<4, true, false>);
  } else {
    if (d.K >= 8) r ? go(k_combine_dropout<8, false, true>) : go(k_combine_dropout<8, false, false>);
    else r ? go(k_combine_dropout<4, false, true>) : go(k_combine_dropout<4, false, false>);
  }
  *launches += 1;
  return e;
}

cudaError_t launch_combine_dropout_backward(const Dims& d, const PlanPtrs& p, const void* y,
                                            const float* gates, const void* d_out, void* d_y,
                                            float* d_gates, const Dropout& drop, cudaStream_t st,
                                            int* launches) {
  const int grid = std::min(d.R * d.S, sm_count_gemm() * 16);
  const int vpt = (d.Hp / 8 + kRowThreads - 1) / kRowThreads;
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    e = launch_after(kernel, grid, kRowThreads, 0, st, 1, d, p, (const uint4*)y, gates,
                     (const uint4*)d_out, (uint4*)d_y, d_gates, drop);
  };
  const bool m = drop.cut != 0;
  // KC x VPT row vectors in flight in a thread: 8 for every row width
  if (vpt <= 1) m ? go(k_combine_dropout_bwd<1, 8, true>) : go(k_combine_dropout_bwd<1, 8, false>);
  else if (vpt <= 2) m ? go(k_combine_dropout_bwd<2, 4, true>) : go(k_combine_dropout_bwd<2, 4, false>);
  else if (vpt <= 4) m ? go(k_combine_dropout_bwd<4, 2, true>) : go(k_combine_dropout_bwd<4, 2, false>);
  else if (vpt <= 8) m ? go(k_combine_dropout_bwd<8, 1, true>) : go(k_combine_dropout_bwd<8, 1, false>);
  else return cudaErrorInvalidValue;
  *launches += 1;
  return e;
}

}  // namespace moonep
