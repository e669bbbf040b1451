// The combine with dropout and residual, forward and backward.  Bound by memory: 16-byte accesses, each
// value read and written once, several copies' loads in flight in every thread.  Measured at 32768
// tokens x 8 x 7168 with dropout and residual: 699 us forward (6.7 TB/s), 1168 us backward (6.8).
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
    const uint64_t seed = (uint64_t)rng[0];
    const uint64_t offset = (uint64_t)rng[1];
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
  // f[i] scaled or dropped, for the eight elements of a group of numbers
  static __device__ __forceinline__ void apply(const uint32_t (&w)[4], uint32_t cut, float scale,
                                               float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = (w[i] & 0xffffu) >= cut ? f[2 * i] * scale : 0.f;
      f[2 * i + 1] = (w[i] >> 16) >= cut ? f[2 * i + 1] * scale : 0.f;
    }
  }
};

constexpr int kRowThreads = 128;

// out[t] = bf16( residual[t] + dropout( sum over k ascending of gates[t][k] y[dst[t][k]] ) )
// `lanes` threads (a power of two) take a token, so that short rows leave none of a block without work.
// Four copies are in flight in a thread, eight blocks a multiprocessor: with eight copies fewer blocks fit
// (32768 x 8 x 7168 with residual: 732 us and 700 with four, without dropout 715 and 693).
constexpr int kCopies = 4;

template <bool DROP, bool RES>
__global__ void __launch_bounds__(kRowThreads, 8)
k_combine_dropout(Dims d, PlanPtrs p, const uint4* y, const float* gates,
                  const uint4* residual, uint4* __restrict__ out, Dropout drop, int lanes) {
  grid_wait();
  grid_trigger();
  if (plan_failed(p.status)) return;
  const int hv = d.Hp / 8;
  const uint32_t ntok = (uint32_t)d.R * d.S;  // (below 2^31: a step past the last one fits)
  const uint32_t tokens = kRowThreads / lanes;  // of a block at a time
  for (uint32_t t = blockIdx.x * tokens + threadIdx.x / lanes; t < ntok; t += gridDim.x * tokens) {
    const int32_t* dt = p.dst + (size_t)t * d.K;
    const float* gt = gates + (size_t)t * d.K;
    for (int a = threadIdx.x & (lanes - 1); a < hv; a += lanes) {
      uint4 res;
      if (RES) res = __ldcs(residual + (size_t)t * hv + a);
      float acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      uint32_t random[4];
      for (int k0 = 0; k0 < d.K; k0 += kCopies) {
        uint4 v[kCopies];
        float g[kCopies];
#pragma unroll
        for (int k = 0; k < kCopies; ++k) {
          if (k0 + k < d.K) {
            v[k] = __ldcs(y + (size_t)dt[k0 + k] * hv + a);
            g[k] = gt[k0 + k];
          }
        }
        // (drawn while the first copies are on their way)
        if (DROP && k0 == 0) Philox(drop.rng).numbers((uint64_t)t * hv + a, random);
#pragma unroll
        for (int k = 0; k < kCopies; ++k)
          if (k0 + k < d.K) {
            float f[8];
            unpack8(f, v[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[k], f[i], acc[i]);
          }
      }
      if (DROP) Philox::apply(random, drop.cut, drop.scale, acc);
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
// A token is a warp's or, with long rows, a block's; a thread's slice of d stays in registers, the copies
// come KC at a time, the first of them on their way while the random numbers are drawn.
constexpr int kDropMaxK = 128;

// A thread's part of a copy's dot product and of its d_y, where an element that was dropped counts as 0
// whatever y and the gate are.
template <int TEAM>
__device__ __forceinline__ float drop_alone(const uint4* y, const uint4* dout, uint4* dy, float g, int hv,
                                            uint64_t group0, const Dropout& drop) {
  float dot = 0.f;
#pragma unroll 1
  for (int a = threadIdx.x % TEAM; a < hv; a += TEAM) {
    float f[8], o[8], w[8], kept[8];
    unpack8(f, __ldcs(y + a));
    unpack8(o, __ldcs(dout + a));
#pragma unroll
    for (int j = 0; j < 8; ++j) kept[j] = 1.f;
    uint32_t random[4];
    Philox(drop.rng).numbers(group0 + a, random);
    Philox::apply(random, drop.cut, 1.f, kept);
    Philox::apply(random, drop.cut, drop.scale, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dot = fmaf(kept[j] != 0.f ? f[j] : 0.f, o[j], dot);
      w[j] = kept[j] != 0.f ? g * o[j] : 0.f;
    }
    __stcs(dy + a, pack8(w));
  }
  return dot;
}

// Blocks a multiprocessor: as many as the vectors in flight leave registers for.  (Left to itself the
// compiler takes 96 registers and spills where 128 threads share a token of four vectors each: 32768 x 8 x
// 4096 718 us and 667 with four blocks; and 128 without dropout where a warp does: 8192 x 2 x 1024 10.5 and 9.5.)
constexpr int back_blocks(int team, int vpt, int kc, bool drop) {
  if (vpt * kc == 4) return 8;
  if (vpt == 4) return team == 32 && !drop ? 5 : 4;
  return vpt == 2 ? 5 : 4;
}

template <int TEAM, int VPT, int KC, bool DROP>
__global__ void __launch_bounds__(kRowThreads, back_blocks(TEAM, VPT, KC, DROP))
k_combine_dropout_bwd(Dims d, PlanPtrs p, const uint4* y,
                      const float* gates, const uint4* dout,
                      uint4* __restrict__ dy, float* __restrict__ dgates, Dropout drop) {
  static_assert(TEAM == 32 || TEAM == kRowThreads, "threads of a token");
  __shared__ float part[TEAM / 32][TEAM == 32 ? 1 : kDropMaxK];
  grid_wait();
  grid_trigger();
  if (plan_failed(p.status)) return;
  const int hv = d.Hp / 8;
  const uint32_t ntok = (uint32_t)d.R * d.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, member = threadIdx.x % TEAM;
  constexpr uint32_t TEAMS = kRowThreads / TEAM;
  for (uint32_t t = blockIdx.x * TEAMS + threadIdx.x / TEAM; t < ntok; t += gridDim.x * TEAMS) {
    const int32_t* dt = p.dst + (size_t)t * d.K;
    const float* gt = gates + (size_t)t * d.K;
    size_t row[KC];
    float g[KC];
    uint4 v[KC][VPT];
    auto load = [&](int k0) {  // copies k0 .. of the token
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        row[k] = k0 + k < d.K ? (size_t)dt[k0 + k] : 0;
        g[k] = k0 + k < d.K ? gt[k0 + k] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < KC; ++k)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int a = member + i * TEAM;
          if (k0 + k < d.K && a < hv) v[k][i] = __ldcs(y + row[k] * hv + a);
        }
    };
    uint4 dv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int a = member + i * TEAM;
      dv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (a < hv) dv[i] = __ldcs(dout + (size_t)t * hv + a);
    }
    load(0);
    float o[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack8(o[i], dv[i]);
      const int a = member + i * TEAM;
      if (DROP && a < hv) {
        uint32_t random[4];
        Philox(drop.rng).numbers((uint64_t)t * hv + a, random);
        Philox::apply(random, drop.cut, drop.scale, o[i]);
      }
    }
    float probe = 0.f;  // 0, or a NaN: a gate or a dot product is not finite (alike in all lanes of a warp)
    for (int k0 = 0; k0 < d.K; k0 += KC) {
      if (k0 > 0) load(k0);
      float dot[KC];
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        dot[k] = 0.f;
        if (k0 + k < d.K) {
#pragma unroll
          for (int i = 0; i < VPT; ++i) {
            const int a = member + i * TEAM;
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
      if (DROP) {
#pragma unroll
        for (int k = 0; k < KC; ++k) probe = fmaf(g[k], 0.f, fmaf(dot[k], 0.f, probe));
      }
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < KC; ++k)
          if (k0 + k < d.K) (TEAM == 32 ? dgates[(size_t)t * d.K + k0 + k] : part[warp][k0 + k]) = dot[k];
      }
    }
    if (DROP && probe != 0.f) {
      // 0 times what is not finite is a NaN, where the element was dropped as well: the token once more,
      // element by element (finite ones pay two instructions a copy for it)
#pragma unroll 1
      for (int k = 0; k < d.K; ++k) {
        const size_t at = (size_t)dt[k] * hv;
        float sum = drop_alone<TEAM>(y + at, dout + (size_t)t * hv, dy + at, gt[k], hv, (uint64_t)t * hv,
                                     drop);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) (TEAM == 32 ? dgates[(size_t)t * d.K + k] : part[warp][k]) = sum;
      }
    }
    if (TEAM == 32) continue;
    __syncthreads();
    for (int k = threadIdx.x; k < d.K; k += TEAM) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < TEAM / 32; ++w) sum += part[w][k];
      dgates[(size_t)t * d.K + k] = sum;
    }
    __syncthreads();
  }
}

// -- host side ------------------------------------------------------------------
cudaError_t launch_combine_dropout(const Dims& d, const PlanPtrs& p, const void* y, const float* gates,
                                   const void* residual, void* out, const Dropout& drop,
                                   cudaStream_t st, int* launches) {
  // as many lanes a token as a block has threads, or fewer where that leaves fewer of them idle
  const int hv = d.Hp / 8;
  int lanes = kRowThreads;
  for (int n = lanes / 2; n >= 8; n /= 2)
    if ((hv + n - 1) / n * n * 8 <= (hv + lanes - 1) / lanes * lanes * 7) lanes = n;
  const int tokens = kRowThreads / lanes;
  const int grid = std::min((int)(((int64_t)d.R * d.S + tokens - 1) / tokens), sm_count_gemm() * 16);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    e = launch_after(kernel, grid, kRowThreads, 0, st, 1, d, p, (const uint4*)y, gates,
                     (const uint4*)residual, (uint4*)out, drop, lanes);
  };
  const bool r = residual != nullptr;
  if (drop.cut) r ? go(k_combine_dropout<true, true>) : go(k_combine_dropout<true, false>);
  else r ? go(k_combine_dropout<false, true>) : go(k_combine_dropout<false, false>);
  *launches += 1;
  return e;
}

cudaError_t launch_combine_dropout_backward(const Dims& d, const PlanPtrs& p, const void* y,
                                            const float* gates, const void* d_out, void* d_y,
                                            float* d_gates, const Dropout& drop, cudaStream_t st,
                                            int* launches) {
  const int hv = d.Hp / 8;
  cudaError_t e = cudaSuccess;
  auto launch = [&](auto kernel, int team) {
    const int teams = kRowThreads / team;
    const int64_t blocks = ((int64_t)d.R * d.S + teams - 1) / teams;
    e = launch_after(kernel, (unsigned)std::min<int64_t>(blocks, sm_count_gemm() * 16), kRowThreads, 0, st,
                     1, d, p, (const uint4*)y, gates, (const uint4*)d_out, (uint4*)d_y, d_gates, drop);
  };
#define MOONEP_GO(team, vpt, kc)                                                                  \
  (drop.cut ? launch(k_combine_dropout_bwd<team, vpt, kc, true>, team)                            \
            : launch(k_combine_dropout_bwd<team, vpt, kc, false>, team))
  // Rows of up to 128 vectors are a warp's, longer ones a block's (65536 x 4 x 512: 233 -> 98 us with
  // warps); KC x VPT vectors of y in flight in a thread, 8 of them, 4 where there are few copies
  if (hv <= 32) d.K <= 4 ? MOONEP_GO(32, 1, 4) : MOONEP_GO(32, 1, 8);
  else if (hv <= 64) d.K <= 2 ? MOONEP_GO(32, 2, 2) : MOONEP_GO(32, 2, 4);
  else if (hv <= 128) MOONEP_GO(32, 4, 2);
  else if (hv <= 256) d.K <= 2 ? MOONEP_GO(128, 2, 2) : MOONEP_GO(128, 2, 4);
  else if (hv <= 512) MOONEP_GO(128, 4, 2);
  else if (hv <= 1024) MOONEP_GO(128, 8, 1);
#undef MOONEP_GO
  else return cudaErrorInvalidValue;
  *launches += 1;
  return e;
}

}  // namespace moonep
