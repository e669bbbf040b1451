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

// Rank of a logit (not NaN) as an integer: larger logits first, equal ones (-0 and
// +0 too) by ascending expert.
__device__ __forceinline__ unsigned long long rank_key(float v, int e) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return ((unsigned long long)k << 32) | (uint32_t)~e;
}

// e^x in one multiplication and the hardware's power of two (off by 2 ulp and by
// what rounding x log2(e) leaves: |x| 2^-24); results below 2^-126 are 0.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {  // 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A row's scores up to a common factor, from its largest logit m:
//   softmax: e^(l - m);  the factor is 1 / their sum
//   sigmoid: 1 / (e^(b - l) + e^b) with b = min(m, 0), which is sigmoid(l) e^-b: at
//   least 1/2 for l = m, so a sum of them never vanishes, however low the row's logits
// (a row of nothing but -inf takes m = 0, and all its scores are 0).
struct Scores {
  int kind;
  float shift, one;  // m; or b and e^b
  __device__ __forceinline__ Scores(int kind_, float m) : kind(kind_) {
    if (m == -INFINITY) m = 0.f;
    shift = kind == 0 ? m : fminf(m, 0.f);
    one = fast_exp(shift);
  }
  __device__ __forceinline__ float operator()(float l) const {
    return kind == 0 ? fast_exp(l - shift) : fast_rcp(fast_exp(shift - l) + one);
  }
};

// The K largest of a token, one after the other; f(k, logit, expert) for each.
// (Compared as logits and experts, not as keys: keys of a whole row would be kept
// in registers through the kernel.)
template <int N, bool VEC, typename F>
__device__ __forceinline__ void select_in_turn(const float (&l)[N], int E, int K, int lane, F&& f) {
  float last = INFINITY;
  int last_e = -1;
  bool nans = false;  // all that is left is NaN
#pragma unroll 1
  for (int k = 0; k < K;) {
    float best = -INFINITY;
    int best_e = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = place<N, VEC>(j, lane);
      const bool later = e > last_e;
      const bool left = nans ? (l[j] != l[j] && later) : (l[j] < last || (l[j] == last && later));
      if (left && e < E && (best_e == 0x7fffffff || l[j] > best)) best = l[j], best_e = e;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float v = __shfl_xor_sync(kAll, best, o);
      const int e = __shfl_xor_sync(kAll, best_e, o);
      if (e != 0x7fffffff && (best_e == 0x7fffffff || v > best || (!(v < best) && e < best_e)))
        best = v, best_e = e;
    }
    if (best_e == 0x7fffffff) {  // (only once, as K <= E)
      nans = true;
      last_e = -1;
      continue;
    }
    f(k++, best, best_e);
    last = best, last_e = best_e;
  }
}

// The K <= 32 largest of a token: lanes with 0 <= rank < K hold one each.
//
// The K-th largest of the 32 lanes' maxima is a bound that at least K values reach,
// and few more (K = 8 of 384 normal logits: 9 on average), so the values that reach
// it are gathered, and each finds its rank by counting the larger ones.  More than
// 32 of them (ties) and a bound of -inf (which the places past the row's end reach
// too) take the K largest one after the other.
template <int N, bool VEC>
__device__ __forceinline__ void select_top(const float (&l)[N], int E, int K, int lane,
                                           float bound, unsigned long long* cand, int& rank,
                                           float& value, int& expert) {
  rank = 32;
  value = 0.f, expert = 0;
  if (bound > -INFINITY) {
    int total = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const unsigned who = __ballot_sync(kAll, l[j] >= bound);
      if (who) {
        const int at = total + __popc(who & ((1u << lane) - 1u));
        if ((who >> lane & 1u) && at < 32)
          cand[at] = ((unsigned long long)__float_as_uint(l[j]) << 32) | (uint32_t)place<N, VEC>(j, lane);
        total += __popc(who);
      }
    }
    if (total <= 32) {
      __syncwarp();
      unsigned long long key = 0;
      if (lane < total) {
        const unsigned long long c = cand[lane];
        value = __uint_as_float((uint32_t)(c >> 32)), expert = (int)(uint32_t)c;
        key = rank_key(value, expert);
      }
      __syncwarp();
      cand[lane] = key;  // 0 past the last: counts for nobody
      __syncwarp();
      int r = 0;
#pragma unroll 1
      for (int i = 0; i < total; i += 4) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(cand + i);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(cand + i + 2);
        r += (a.x > key) + (a.y > key) + (b.x > key) + (b.y > key);
      }
      __syncwarp();
      if (lane < total) rank = r;
      return;
    }
  }
  __syncwarp();
  select_in_turn<N, VEC>(l, E, K, lane, [&](int k, float v, int e) {
    if (lane == k) value = v, expert = e, rank = k;
  });
}

constexpr int kRouterMaxK = 128;

template <int N>
constexpr int router_warps() {
  return N > 32 ? 4 : 8;
}
// Blocks a multiprocessor has to hold, which caps the registers
template <int N>
constexpr int router_blocks() {
  return N <= 8 ? 5 : N <= 16 ? 4 : N <= 32 ? 2 : 1;
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

// The end of a block with the loss: its warps' probability sums s_q [W][E], counts
// s_cnt [E] and tokens go to its segment's, and the last block of a segment writes
// the segment's outputs, the last segment the loss.
template <int W>
__device__ __forceinline__ void join_blocks(const RouterDims& d, const RouterOut& out,
                                            const RouterScratch& ws, int g, const float* s_q,
                                            const int32_t* s_cnt, int& s_tokens, int& s_bad) {
  __shared__ int s_last;
  const bool alone = d.cps == 1;  // the segment's only block
  if (!alone) {
    // Joined across blocks as integers (steps of 2^-shift), so the order of the
    // atomics changes nothing; what is not finite is only noted (q of such a token is
    // NaN for every expert).
    const float one = ldexpf(1.f, d.shift);
    for (int e = threadIdx.x; e < d.E; e += blockDim.x) {
      float q = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) q += s_q[(size_t)w * d.E + e];
      if (!isfinite(q)) s_bad = 1;
      else if (q != 0.f) atomicAdd(&ws.q[(size_t)g * d.E + e], __float2ull_rn(q * one));
      if (s_cnt[e]) atomicAdd(&ws.counts[(size_t)g * d.E + e], s_cnt[e]);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      atomicAdd(&ws.tokens[g], s_tokens);
      if (s_bad) atomicOr(&ws.bad[g], 1);
      __threadfence();
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
    int32_t c;
    double q;
    if (alone) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += s_q[(size_t)w * d.E + e];
      c = s_cnt[e], q = v;
    } else {
      c = __ldcg(&ws.counts[at]);
      q = s_bad ? (double)NAN : (double)__ldcg(&ws.q[at]) * step;
    }
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

// A block takes `chunk` tokens of one segment, a warp every W-th of them.
// SHORT: K <= 32.
template <typename T, int N, bool VEC, bool LOSS, bool SHORT>
__global__ void __launch_bounds__(router_warps<N>() * 32, router_blocks<N>())
k_router(RouterDims d, const T* __restrict__ logits, const uint8_t* __restrict__ mask,
         RouterOut out, RouterScratch ws) {
  constexpr int W = router_warps<N>();
  constexpr int KI = SHORT ? 1 : kRouterMaxK / 32;
  __shared__ __align__(16) unsigned long long s_list[W][SHORT ? 32 : kRouterMaxK];  // candidates
  extern __shared__ float s_dyn[];  // LOSS: the warps' sums [W][E], then counts [E]
  __shared__ int s_tokens, s_bad;
  int32_t* s_cnt = reinterpret_cast<int32_t*>(s_dyn + (size_t)W * d.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int g = LOSS ? blockIdx.x / d.cps : 0;
  const int base = LOSS ? g * d.segment : 0;  // first token of the segment
  const int t0 = base + (LOSS ? blockIdx.x % d.cps : blockIdx.x) * d.chunk;
  const int t1 = min(min(t0 + d.chunk, LOSS ? base + d.segment : d.T), d.T);
  if (LOSS) {
    for (int e = threadIdx.x; e < d.E; e += blockDim.x) s_cnt[e] = 0;
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
    float most = l[0];
#pragma unroll
    for (int j = 1; j < N; ++j) most = fmaxf(most, l[j]);  // passes NaN over
    if (N == 1) most = fmaxf(most, -INFINITY);
    const float sorted = warp_sort_down(most, lane);
    const Scores score(d.score, __shfl_sync(kAll, sorted, 0));

    // the chosen ones of this lane: SHORT, the one with rank `rank`; else those with
    // rank i * 32 + lane
    float value[KI];
    int expert[KI], rank = 0;
    if constexpr (SHORT) {
      select_top<N, VEC>(l, d.E, d.K, lane, __shfl_sync(kAll, sorted, d.K - 1), s_list[warp], rank,
                         value[0], expert[0]);
    } else {
      select_in_turn<N, VEC>(l, d.E, d.K, lane, [&](int k, float v, int e) {
        if (lane == 0)
          s_list[warp][k] = ((unsigned long long)__float_as_uint(v) << 32) | (uint32_t)e;
      });
      __syncwarp();
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const unsigned long long c = i * 32 + lane < d.K ? s_list[warp][i * 32 + lane] : 0;
        value[i] = __uint_as_float((uint32_t)(c >> 32)), expert[i] = (int)(uint32_t)c;
      }
      __syncwarp();
    }

    // 1 / sum of the row's scores, where it is needed; a NaN in the row, which is in
    // every softmax score, shows in it
    float inv = 1.f;
    bool nan = false;
    if (LOSS || (d.score == 0 && !d.normalise)) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        l[j] = score(l[j]);
        sum += l[j];
      }
      sum = warp_sum(sum);
      inv = sum == 0.f ? 0.f : fast_rcp(sum);
      nan = sum != sum;
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) nan |= l[j] != l[j];
      nan = __any_sync(kAll, nan);
    }
    if (LOSS && live) {
#pragma unroll
      for (int j = 0; j < (LOSS ? N : 1); ++j) acc[j] = fmaf(l[j], inv, acc[j]);
      ++live_tokens;
    }

    float gate[KI], total = 0.f;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const bool mine = SHORT ? rank < d.K : i * 32 + lane < d.K;
      gate[i] = mine ? score(value[i]) : 0.f;
      total += gate[i];
    }
    float factor = d.score == 0 ? inv : score.one;
    if (d.normalise) {
      total = warp_sum(total);
      factor = total == 0.f ? 0.f : fast_rcp(total);
    }
    factor *= d.scale;
    if (d.score == 0 && nan) factor = NAN;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int k = SHORT ? rank : i * 32 + lane;
      if (k < d.K) {
        out.topk_idx[(size_t)t * d.K + k] = expert[i];
        out.gates[(size_t)t * d.K + k] = live ? gate[i] * factor : 0.f;
        if (LOSS && live) atomicAdd(&s_cnt[expert[i]], 1);
      }
    }
  }
  if constexpr (LOSS) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = place<N, VEC>(j, lane);
      if (e < d.E) s_dyn[(size_t)warp * d.E + e] = acc[j];
    }
    if (lane == 0) atomicAdd(&s_tokens, live_tokens);
    __syncthreads();
    join_blocks<W>(d, out, ws, g, s_dyn, s_cnt, s_tokens, s_bad);
  }
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
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, l[j]);
      const Scores score(d.score, warp_max(m));
      // the scores (up to their common factor), their sum and that with w
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (d.score == 0) {
          l[j] = score(l[j]);
          dl[j] = 1.f;
        } else {
          const float x = fast_exp(score.shift - l[j]);
          const float v = fast_rcp(x + score.one);
          // 1 - s; near s = 1 (then the shift is 0) without cancellation
          dl[j] = l[j] > 0.f ? x * v : fmaf(-v, score.one, 1.f);
          l[j] = v;
        }
        sum += l[j];
        dot = fmaf(l[j], w[j], dot);
      }
      sum = warp_sum(sum);
      const float inv = sum == 0.f ? 0.f : fast_rcp(sum);
      dot = warp_sum(dot) * inv;

      if (d_gates != nullptr) {
        float total = 0.f, with = 0.f;
#pragma unroll
        for (int i = 0; i < kRouterMaxK / 32; ++i)
          if (id[i] >= 0) {
            s[i] = score(s[i]);
            total += s[i];
            with = fmaf(s[i], dg[i], with);
          }
        float factor = d.score == 0 ? inv : score.one, mean = 0.f;
        if (d.normalise) {
          total = warp_sum(total);
          factor = total == 0.f ? 0.f : fast_rcp(total);
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
  r.zero_bytes = off;
  r.seg_loss = (double*)take(8 * G);
  r.total_bytes = off;
  return r;
}

// Launch shape of a router kernel: blocks for one round of what fits the GPU at
// once, so that all warps take equally many tokens; whole rounds of the block's
// warps, and at most 64 tokens a warp, so that a warp's fp32 sums stay short.
template <typename Kernel>
static cudaError_t plan_blocks(Kernel* k, int warps, size_t smem, RouterDims& d) {
  if (smem > (32u << 10)) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, warps * 32, smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = std::max(1, sms * per_sm);
  // blocks a segment in that round, or one where there are more segments than blocks
  const int64_t each = std::max<int64_t>(1, blocks / d.G);
  int64_t chunk = (d.segment + each - 1) / each;
  chunk = (chunk + warps - 1) / warps * warps;
  d.chunk = (int)std::min<int64_t>(chunk, 64 * warps);
  d.cps = (d.segment + d.chunk - 1) / d.chunk;
  return cudaSuccess;
}

template <typename T, int N, bool VEC, bool LOSS, bool SHORT>
static cudaError_t forward(RouterDims d, const void* logits, const uint8_t* mask,
                           const RouterOut& out, const RouterScratch& ws, cudaStream_t st) {
  constexpr int W = router_warps<N>();
  auto* kernel = k_router<T, N, VEC, LOSS, SHORT>;
  const size_t smem = LOSS ? (size_t)d.E * 4 * (W + 1) : 0;
  if (!LOSS) d.G = 1, d.segment = d.T;
  cudaError_t e = plan_blocks(kernel, W, smem, d);
  if (e != cudaSuccess) return e;
  if (LOSS) {  // one block a segment: only the count of finished segments is used
    const size_t zero = d.cps > 1 ? ws.zero_bytes : (d.G > 1 ? 4 : 0);
    if (zero) e = cudaMemsetAsync(ws.done, 0, zero, st);
    if (e != cudaSuccess) return e;
  }
  kernel<<<d.G * d.cps, W * 32, smem, st>>>(d, (const T*)logits, mask, out, ws);
  return cudaGetLastError();
}

template <typename T, int N, bool VEC>
static cudaError_t backward(RouterDims d, const void* logits, const uint8_t* mask,
                            const int32_t* topk_idx, const float* d_gates, const int32_t* counts,
                            const int32_t* seg_tokens, const float* d_loss, void* d_logits,
                            cudaStream_t st) {
  constexpr int W = router_warps<N>();
  const size_t smem = (size_t)W * ((d.E + 3) & ~3) * 4;
  const cudaError_t e = plan_blocks(k_router_backward<T, N, VEC>, W, smem, d);
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
    if (out.loss == nullptr)
      return d.K <= 32 ? forward<T, N, VEC, false, true>(d, logits, mask, out, ws, st)
                       : forward<T, N, VEC, false, false>(d, logits, mask, out, ws, st);
    return d.K <= 32 ? forward<T, N, VEC, true, true>(d, logits, mask, out, ws, st)
                     : forward<T, N, VEC, true, false>(d, logits, mask, out, ws, st);
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
