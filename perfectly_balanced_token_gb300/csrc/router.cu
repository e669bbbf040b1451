// The router: top-K experts and gates of every token, per-expert counts and the
// balance loss in one pass over the logits, and the gradient in one more.
//
// A warp takes one token; its lanes hold the row in registers, so a logit is
// read once.  The blocks' probability sums are joined as integers (fixed
// point), so the order of the atomics changes nothing.
#include <cuda_bf16.h>

#include <algorithm>

#include "ops.h"

namespace moonep {

constexpr unsigned kAll = 0xffffffffu;

// How a lane's N values lie in the row: four neighbours at a time in steps of
// 128 (rows whose length 4 divides: vector loads), or every 32nd value.
template <int N, bool VEC>
__device__ __forceinline__ int place(int j, int lane) {
  return VEC ? (j >> 2) * 128 + lane * 4 + (j & 3) : j * 32 + lane;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}

// A row's values of this lane; -inf past the row's end, where a value adds
// nothing to any sum of exponentials.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int lane,
                                         float (&l)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const int at = c * 128 + lane * 4;
      float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (at < E) {
        if constexpr (sizeof(T) == 4) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(row + at));
          v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + at));
          v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
          v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) l[4 * c + i] = v[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int at = j * 32 + lane;
      l[j] = at < E ? to_f32(row[at]) : -INFINITY;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {  // NaN is passed over
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// The lanes' values sorted downwards over the warp (bitonic network).
__device__ __forceinline__ float warp_sort_down(float v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1) {
      const float o = __shfl_xor_sync(kAll, v, j);
      v = (((lane & k) == 0) == ((lane & j) == 0)) ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
}

// Rank of a logit as an integer: larger logits first, equal ones (-0 and +0
// too) by ascending expert; a NaN below -inf.
__device__ __forceinline__ unsigned long long rank_key(float v, int e) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t k = v != v ? 1u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return ((unsigned long long)k << 32) | (uint32_t)~e;
}
__device__ __forceinline__ int key_expert(unsigned long long k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_logit(unsigned long long key) {
  const uint32_t k = (uint32_t)(key >> 32);
  if (k == 1u) return __uint_as_float(0x7fffffffu);
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// The K best keys of a token, by rank, into top[0..K): at most 128.
//
// With K <= 32 the K-th largest of the 32 lanes' maxima is a bound that at least
// K values reach, and few more (K = 8 of 384 normal logits: 11 on average), so
// the values that reach it are gathered and each finds its rank by counting the
// larger ones.  More than 32 of them (ties), a bound of -inf and K > 32 take the K
// largest one after the other.
template <int N, bool VEC>
__device__ __forceinline__ void select_top(const float (&l)[N], int E, int K, int lane,
                                           float sorted, unsigned long long* cand,
                                           unsigned long long* top) {
  const float bound = __shfl_sync(kAll, sorted, min(K, 32) - 1);
  // a bound of -inf would let in the places past the row's end
  if (K <= 32 && bound > -INFINITY) {
    int mine = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) mine += l[j] >= bound;
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, before, o);
      if (lane >= o) before += v;
    }
    const int total = __shfl_sync(kAll, before, 31);
    if (total <= 32) {
      int at = before - mine;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (l[j] >= bound) cand[at++] = rank_key(l[j], place<N, VEC>(j, lane));
      __syncwarp();
      const unsigned long long key = lane < total ? cand[lane] : 0;
      int rank = 0;
      for (int i = 0; i < total; ++i) rank += cand[i] > key;
      if (lane < total && rank < K) top[rank] = key;
      __syncwarp();
      return;
    }
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < K; ++k) {
    unsigned long long best = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = place<N, VEC>(j, lane);
      const unsigned long long key = e < E ? rank_key(l[j], e) : 0;
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long v = __shfl_xor_sync(kAll, best, o);
      best = v > best ? v : best;
    }
    if (lane == 0) top[k] = best;
    last = best;
  }
  __syncwarp();
}

constexpr int kRouterMaxK = 128;

template <int N>
constexpr int router_warps() {
  return N > 32 ? 4 : 8;
}

// Sum over the block in a fixed order (every thread gets it).
__device__ __forceinline__ double block_sum(double v, double* s) {
  s[threadIdx.x] = v;
  __syncthreads();
  for (int o = blockDim.x >> 1; o; o >>= 1) {
    if ((int)threadIdx.x < o) s[threadIdx.x] += s[threadIdx.x + o];
    __syncthreads();
  }
  const double r = s[0];
  __syncthreads();
  return r;
}

template <typename T, int N, bool VEC, bool LOSS>
__global__ void __launch_bounds__(router_warps<N>() * 32)
k_router(RouterDims d, const T* __restrict__ logits, const uint8_t* __restrict__ mask,
         RouterOut out, RouterScratch ws) {
  constexpr int W = router_warps<N>();
  __shared__ unsigned long long s_cand[W][32];
  __shared__ unsigned long long s_top[W][kRouterMaxK];
  extern __shared__ unsigned long long s_dyn[];  // LOSS: q sums [E], then counts [E]
  __shared__ int s_tokens, s_bad, s_last;
  unsigned long long* s_q = s_dyn;
  int32_t* s_cnt = reinterpret_cast<int32_t*>(s_dyn + d.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int g = LOSS ? blockIdx.x / d.cps : 0;
  const int base = LOSS ? g * d.segment : 0;  // first token of the segment
  const int t0 = base + (LOSS ? blockIdx.x % d.cps : blockIdx.x) * d.chunk;
  const int t1 = min(min(t0 + d.chunk, LOSS ? base + d.segment : d.T), d.T);
  if (LOSS) {
    for (int e = threadIdx.x; e < d.E; e += blockDim.x) {
      s_q[e] = 0;
      s_cnt[e] = 0;
    }
    if (threadIdx.x == 0) s_tokens = s_bad = 0;
    __syncthreads();
  }

  float acc[LOSS ? N : 1];
#pragma unroll
  for (int j = 0; j < (LOSS ? N : 1); ++j) acc[j] = 0.f;
  int live_tokens = 0;

  for (int t = t0 + warp; t < t1; t += W) {
    float l[N];
    load_row<T, N, VEC>(logits + (size_t)t * d.E, d.E, lane, l);
    const bool live = mask == nullptr || mask[t] != 0;
    float most = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      most = fmaxf(most, l[j]);  // passes NaN over
      nan |= l[j] != l[j];
    }
    const float sorted = warp_sort_down(most, lane);
    float m = __shfl_sync(kAll, sorted, 0);
    if (m == -INFINITY) m = 0.f;  // nothing but -inf (and NaN): exponentials of 0
    select_top<N, VEC>(l, d.E, d.K, lane, sorted, s_cand[warp], s_top[warp]);

    // 1 / sum of the row's s (softmax: of the exponentials before they are divided)
    float inv = 1.f;
    if (LOSS || (d.score == 0 && !d.normalise)) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        l[j] = d.score == 0 ? __expf(l[j] - m) : sigmoid(l[j]);
        sum += l[j];
      }
      sum = warp_sum(sum);
      inv = sum == 0.f ? 0.f : 1.f / sum;
    }
    if (LOSS && live) {
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = fmaf(l[j], inv, acc[j]);
      ++live_tokens;
    }

    float gate[kRouterMaxK / 32], total = 0.f;
#pragma unroll
    for (int i = 0; i < kRouterMaxK / 32; ++i) {
      const int k = i * 32 + lane;
      gate[i] = 0.f;
      if (k < d.K) {
        const float v = key_logit(s_top[warp][k]);
        gate[i] = d.score == 0 ? __expf(v - m) : sigmoid(v);
        total += gate[i];
      }
    }
    float factor = d.score == 0 ? inv : 1.f;
    if (d.normalise) {
      total = warp_sum(total);
      factor = total == 0.f ? 0.f : 1.f / total;
    }
    factor *= d.scale;
    // a NaN anywhere in the row is in every softmax score, so in every gate
    if (d.score == 0 && __any_sync(kAll, nan)) factor = NAN;
#pragma unroll
    for (int i = 0; i < kRouterMaxK / 32; ++i) {
      const int k = i * 32 + lane;
      if (k < d.K) {
        const int e = key_expert(s_top[warp][k]);
        out.topk_idx[(size_t)t * d.K + k] = e;
        out.gates[(size_t)t * d.K + k] = live ? gate[i] * factor : 0.f;
        if (LOSS && live) atomicAdd(&s_cnt[e], 1);
      }
    }
    __syncwarp();  // the next token reuses the lists
  }
  if (!LOSS) return;

  // The warps' sums as integers: a step of 2^-shift, so the order of the
  // additions changes nothing; what is not finite is only noted (q of such a
  // token is NaN for every expert).
  const float one = ldexpf(1.f, d.shift);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = place<N, VEC>(j, lane);
    if (e < d.E) {
      if (!isfinite(acc[j])) s_bad = 1;
      else if (acc[j] != 0.f) atomicAdd(&s_q[e], __float2ull_rn(acc[j] * one));
    }
  }
  if (lane == 0) atomicAdd(&s_tokens, live_tokens);
  __syncthreads();

  const bool alone = d.cps == 1;  // the segment's only block
  if (!alone) {
    for (int e = threadIdx.x; e < d.E; e += blockDim.x) {
      if (s_q[e]) atomicAdd(&ws.q[(size_t)g * d.E + e], s_q[e]);
      if (s_cnt[e]) atomicAdd(&ws.counts[(size_t)g * d.E + e], s_cnt[e]);
    }
    if (threadIdx.x == 0) {
      atomicAdd(&ws.tokens[g], s_tokens);
      if (s_bad) atomicOr(&ws.bad[g], 1);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = atomicAdd(&ws.seg_done[g], 1) == d.cps - 1;
      __threadfence();
      if (s_last) {
        s_tokens = __ldcg(&ws.tokens[g]);
        s_bad = __ldcg(&ws.bad[g]);
      }
    }
    __syncthreads();
    if (!s_last) return;
  }

  // the segment's outputs and its part of the loss
  __shared__ double s_red[W * 32];
  const double step = ldexp(1.0, -d.shift);
  double part = 0.0;
  for (int e = threadIdx.x; e < d.E; e += blockDim.x) {
    const size_t at = (size_t)g * d.E + e;
    const int32_t c = alone ? s_cnt[e] : __ldcg(&ws.counts[at]);
    const double q = s_bad ? (double)NAN : (double)(alone ? s_q[e] : __ldcg(&ws.q[at])) * step;
    out.counts[at] = c;
    out.prob_sum[at] = (float)q;
    part += (double)c * q;
  }
  const double sum = block_sum(part, s_red);
  const double n = s_tokens;
  const double seg = s_tokens ? (double)d.E * sum / ((double)d.K * n * n) : 0.0;
  if (threadIdx.x == 0) {
    out.seg_tokens[g] = s_tokens;
    if (d.G > 1) {
      ws.seg_loss[g] = seg;
      __threadfence();
      s_last = atomicAdd(ws.done, 1) == d.G - 1;
      __threadfence();
    } else {
      *out.loss = (float)seg;
    }
  }
  if (d.G == 1) return;
  __syncthreads();
  if (!s_last) return;
  double mean = 0.0;
  for (int i = threadIdx.x; i < d.G; i += blockDim.x) mean += __ldcg(&ws.seg_loss[i]);
  mean = block_sum(mean, s_red);
  if (threadIdx.x == 0) *out.loss = (float)(mean / d.G);
}

// The gradient.  With w_e = d_loss E counts_e / (G K n^2), a_k what the gate k
// gives its expert's s times s, and dot = sum_e q_e w_e:
//   softmax:  dl_e = q_e (w_e - dot) + a_e,           a sums to 0 when normalised;
//             else dot takes in sum a
//   sigmoid:  dl_e = (1 - s_e) (q_e (w_e - dot) + a_e)
//   a_k = scale n_k (d_gate_k - sum_j n_j d_gate_j), n = chosen s / their sum, when
//   normalised; else scale s_k d_gate_k
// The chosen experts' a lie in a row of shared memory that is zero elsewhere.
template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(router_warps<N>() * 32)
k_router_backward(RouterDims d, const T* __restrict__ logits, const uint8_t* __restrict__ mask,
                  const int32_t* __restrict__ topk_idx, const float* __restrict__ d_gates,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ seg_tokens,
                  const float* __restrict__ d_loss, T* __restrict__ d_logits) {
  constexpr int W = router_warps<N>();
  extern __shared__ float s_a[];  // [W][E rounded up to 4]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E4 = (d.E + 3) & ~3;
  float* a = s_a + (size_t)warp * E4;
  for (int e = lane; e < E4; e += 32) a[e] = 0.f;
  __syncwarp();

  const int g = blockIdx.x / d.cps;
  const int base = g * d.segment;
  const int t0 = base + (blockIdx.x % d.cps) * d.chunk;
  const int t1 = min(min(t0 + d.chunk, base + d.segment), d.T);

  float w[N];
  float coef = 0.f;
  if (d_loss != nullptr) {
    const float n = (float)seg_tokens[g];
    if (n > 0.f) coef = *d_loss * ((float)d.E / ((float)d.G * (float)d.K * n)) / n;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = place<N, VEC>(j, lane);
    w[j] = d_loss != nullptr && e < d.E ? coef * (float)counts[(size_t)g * d.E + e] : 0.f;
  }

  for (int t = t0 + warp; t < t1; t += W) {
    const T* row = logits + (size_t)t * d.E;
    T* drow = d_logits + (size_t)t * d.E;
    const bool live = mask == nullptr || mask[t] != 0;
    float l[N];
    float dl[N];
    if (live) {
      load_row<T, N, VEC>(row, d.E, lane, l);
      int id[kRouterMaxK / 32];
      float s[kRouterMaxK / 32], dg[kRouterMaxK / 32];
      if (d_gates != nullptr) {
#pragma unroll
        for (int i = 0; i < kRouterMaxK / 32; ++i) {
          const int k = i * 32 + lane;
          id[i] = -1;
          if (k < d.K) {
            const int e = topk_idx[(size_t)t * d.K + k];
            dg[i] = d_gates[(size_t)t * d.K + k];
            if (e >= 0 && e < d.E) {
              id[i] = e;
              s[i] = to_f32(row[e]);
            }
          }
        }
      }
      float m = 0.f;
      if (d.score == 0) {
        m = -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, l[j]);
        m = warp_max(m);
        if (m == -INFINITY) m = 0.f;
      }
      // s, the sum of s and of s w
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (d.score == 0) {
          l[j] = __expf(l[j] - m);
          dl[j] = 1.f;
        } else {
          const float x = __expf(-l[j]);
          const float v = __fdividef(1.f, 1.f + x);
          dl[j] = l[j] > 0.f ? x * v : 1.f - v;  // 1 - s, near s = 1 without cancellation
          l[j] = v;
        }
        sum += l[j];
        dot = fmaf(l[j], w[j], dot);
      }
      sum = warp_sum(sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      dot = warp_sum(dot) * inv;

      if (d_gates != nullptr) {
        float total = 0.f, with = 0.f;
#pragma unroll
        for (int i = 0; i < kRouterMaxK / 32; ++i)
          if (id[i] >= 0) {
            s[i] = d.score == 0 ? __expf(s[i] - m) : sigmoid(s[i]);
            total += s[i];
            with = fmaf(s[i], dg[i], with);
          }
        float factor = d.score == 0 ? inv : 1.f, mean = 0.f;
        if (d.normalise) {
          total = warp_sum(total);
          factor = total == 0.f ? 0.f : 1.f / total;
          mean = warp_sum(with) * factor;
        } else if (d.score == 0) {
          dot = fmaf(warp_sum(with), d.scale * inv, dot);
        }
#pragma unroll
        for (int i = 0; i < kRouterMaxK / 32; ++i)
          if (id[i] >= 0) a[id[i]] = d.scale * (s[i] * factor) * (dg[i] - mean);
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = place<N, VEC>(j, lane);
        const float own = d_gates != nullptr && e < d.E ? a[e] : 0.f;
        dl[j] *= fmaf(l[j] * inv, w[j] - dot, own);
      }
      if (d_gates != nullptr) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kRouterMaxK / 32; ++i)
          if (id[i] >= 0) a[id[i]] = 0.f;
        __syncwarp();
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) dl[j] = 0.f;
    }
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < N / 4; ++c) {
        const int at = c * 128 + lane * 4;
        if (at < d.E) {
          if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(drow + at) =
                make_float4(dl[4 * c], dl[4 * c + 1], dl[4 * c + 2], dl[4 * c + 3]);
          } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(dl[4 * c], dl[4 * c + 1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(dl[4 * c + 2], dl[4 * c + 3]);
            uint2 u;
            u.x = *reinterpret_cast<const uint32_t*>(&lo);
            u.y = *reinterpret_cast<const uint32_t*>(&hi);
            *reinterpret_cast<uint2*>(drow + at) = u;
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int at = j * 32 + lane;
        if (at < d.E) drow[at] = (T)dl[j];
      }
    }
  }
}

RouterScratch router_scratch(const RouterDims& d, void* ws) {
  char* b = static_cast<char*>(ws);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* at = b + off;
    off = align256(off + bytes);
    return at;
  };
  RouterScratch r{};
  const size_t G = d.G, GE = (size_t)d.G * d.E;
  r.done = (int32_t*)take(4);
  r.seg_done = (int32_t*)take(4 * G);
  r.tokens = (int32_t*)take(4 * G);
  r.bad = (int32_t*)take(4 * G);
  r.counts = (int32_t*)take(4 * GE);
  r.q = (unsigned long long*)take(8 * GE);
  // one block a segment: only the count of finished segments is kept here
  r.zero_bytes = d.cps > 1 ? off : (d.G > 1 ? 4 : 0);
  r.seg_loss = (double*)take(8 * G);
  r.total_bytes = off;
  return r;
}

template <typename Kernel>
static cudaError_t with_smem(Kernel* k, size_t bytes) {
  return bytes > (32u << 10)
             ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
             : cudaSuccess;
}

template <typename T, int N, bool VEC>
static cudaError_t forward(RouterDims d, const void* logits, const uint8_t* mask,
                           const RouterOut& out, const RouterScratch& ws, cudaStream_t st) {
  constexpr int W = router_warps<N>();
  if (out.loss == nullptr) {
    d.chunk = W;
    k_router<T, N, VEC, false>
        <<<(d.T + W - 1) / W, W * 32, 0, st>>>(d, (const T*)logits, mask, out, ws);
    return cudaGetLastError();
  }
  if (ws.zero_bytes) {
    const cudaError_t e = cudaMemsetAsync(ws.done, 0, ws.zero_bytes, st);
    if (e != cudaSuccess) return e;
  }
  const size_t smem = (size_t)d.E * 12;
  const cudaError_t e = with_smem(k_router<T, N, VEC, true>, smem);
  if (e != cudaSuccess) return e;
  k_router<T, N, VEC, true>
      <<<d.G * d.cps, W * 32, smem, st>>>(d, (const T*)logits, mask, out, ws);
  return cudaGetLastError();
}

template <typename T, int N, bool VEC>
static cudaError_t backward(const RouterDims& d, const void* logits, const uint8_t* mask,
                            const int32_t* topk_idx, const float* d_gates, const int32_t* counts,
                            const int32_t* seg_tokens, const float* d_loss, void* d_logits,
                            cudaStream_t st) {
  constexpr int W = router_warps<N>();
  const size_t smem = (size_t)W * ((d.E + 3) & ~3) * 4;
  const cudaError_t e = with_smem(k_router_backward<T, N, VEC>, smem);
  if (e != cudaSuccess) return e;
  k_router_backward<T, N, VEC><<<d.G * d.cps, W * 32, smem, st>>>(
      d, (const T*)logits, mask, topk_idx, d_gates, counts, seg_tokens, d_loss, (T*)d_logits);
  return cudaGetLastError();
}

// Calls f with the kernel's row shape: values per lane, and whether they lie in
// vectors of four.  Rows of up to 128 experts are spread over all lanes one
// value at a time (vectors would leave lanes empty); so are rows that 4 does not
// divide and rows of more than 1024.
template <typename T, typename F>
static cudaError_t by_row(int E, F&& f) {
#define ROW(n, vec) return f.template operator()<T, n, vec>()
  if (E % 4 == 0 && E > 128 && E <= 1024) {
    switch ((E + 127) / 128) {
      case 2: ROW(8, true);
      case 3: ROW(12, true);
      case 4: ROW(16, true);
      case 5: ROW(20, true);
      case 6: ROW(24, true);
      case 7: ROW(28, true);
      default: ROW(32, true);
    }
  }
  if (E <= 32) ROW(1, false);
  if (E <= 64) ROW(2, false);
  if (E <= 128) ROW(4, false);
  if (E <= 256) ROW(8, false);
  if (E <= 512) ROW(16, false);
  if (E <= 1024) ROW(32, false);
  if (E <= 2048) ROW(64, false);
  ROW(128, false);
#undef ROW
}

struct ForwardCall {
  const RouterDims& d;
  const void* logits;
  const uint8_t* mask;
  const RouterOut& out;
  const RouterScratch& ws;
  cudaStream_t st;
  template <typename T, int N, bool VEC>
  cudaError_t operator()() const {
    return forward<T, N, VEC>(d, logits, mask, out, ws, st);
  }
};

struct BackwardCall {
  const RouterDims& d;
  const void* logits;
  const uint8_t* mask;
  const int32_t* topk_idx;
  const float* d_gates;
  const int32_t* counts;
  const int32_t* seg_tokens;
  const float* d_loss;
  void* d_logits;
  cudaStream_t st;
  template <typename T, int N, bool VEC>
  cudaError_t operator()() const {
    return backward<T, N, VEC>(d, logits, mask, topk_idx, d_gates, counts, seg_tokens, d_loss,
                               d_logits, st);
  }
};

cudaError_t launch_router_forward(const RouterDims& d, const void* logits, const uint8_t* mask,
                                  const RouterOut& out, const RouterScratch& ws, cudaStream_t st,
                                  int* launches) {
  const ForwardCall call{d, logits, mask, out, ws, st};
  const cudaError_t e = d.bf16 ? by_row<__nv_bfloat16>(d.E, call) : by_row<float>(d.E, call);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

cudaError_t launch_router_backward(const RouterDims& d, const void* logits, const uint8_t* mask,
                                   const int32_t* topk_idx, const float* d_gates,
                                   const int32_t* counts, const int32_t* seg_tokens,
                                   const float* d_loss, void* d_logits, cudaStream_t st,
                                   int* launches) {
  const BackwardCall call{d,      logits,     mask,   topk_idx, d_gates,
                          counts, seg_tokens, d_loss, d_logits, st};
  const cudaError_t e = d.bf16 ? by_row<__nv_bfloat16>(d.E, call) : by_row<float>(d.E, call);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace moonep
