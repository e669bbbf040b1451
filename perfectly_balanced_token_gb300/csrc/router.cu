// The router: top-K experts and gates of every token, per-expert counts and the
// balance loss in one pass over the logits, and the gradient in one more.
//
// A warp takes one token; its lanes hold the row in registers, so a logit is
// read once.  The blocks' probability sums are joined as integers (fixed
// point), so the order of the atomics changes nothing.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "ops.h"

namespace moonep {

constexpr unsigned kAll = 0xffffffffu;

// How a lane's N values lie in the row: four neighbours at a time in steps of
// 128 (rows whose length 4 divides: vector loads), or every 32nd value.
template <int N, bool VEC>
__device__ __forceinline__ int place(int j, int lane) {
  return VEC ? (j >> 2) * 128 + lane * 4 + (j & 3) : j * 32 + lane;
}

// Whether step c (of four neighbours, or of one value) of a lane lies in the row of E.
// Vector rows have as many steps as E needs: only the last one can lie outside.
template <int N, bool VEC>
__device__ __forceinline__ bool inside(int c, int lane, int E) {
  return VEC ? c < N / 4 - 1 || c * 128 + lane * 4 < E : c * 32 + lane < E;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}

// Starts the copy of a row (VEC) into the warp's row of shared memory, every lane the
// values that are its own.
template <typename T, int N>
__device__ __forceinline__ void fetch_row(T* s_row, const T* __restrict__ row, int E, int lane) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(s_row + lane * 4);
  const T* from = row + lane * 4;
#pragma unroll
  for (int c = 0; c < N / 4; ++c) {
    if (inside<N, true>(c, lane, E))
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + c * 128 * (int)sizeof(T)),
                   "l"(from + c * 128), "n"(4 * sizeof(T))
                   : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void await_row() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}

// A row's values of this lane; -inf past the row's end, where a value adds
// nothing to any sum of exponentials.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, float (&l)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const int at = c * 128 + lane * 4;
      float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (inside<N, true>(c, lane, E)) {
        if constexpr (sizeof(T) == 4) {
          const float4 f = *reinterpret_cast<const float4*>(row + at);
          v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(row + at);
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

// A row as choosing sees it: its values, the largest of this lane's (NaN passed over),
// a bit for each that reaches a bound, and the expert that a bit stands for.
template <typename T, int N, bool VEC>
struct Row {
  static constexpr int kWords = (N + 31) / 32;
  float l[N];
  __device__ __forceinline__ void load(const T* row, int E, int lane) {
    load_row<T, N, VEC>(row, E, lane, l);
  }
  __device__ __forceinline__ float operator()(int j) const { return l[j]; }
  __device__ __forceinline__ float most() const {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, l[j]);
    return m;
  }
  __device__ __forceinline__ bool nan() const {
    bool n = false;
#pragma unroll
    for (int j = 0; j < N; ++j) n |= l[j] != l[j];
    return n;
  }
  __device__ __forceinline__ void reach(float bound, uint32_t (&bits)[kWords]) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (l[j] >= bound) bits[j / 32] |= 1u << (j & 31);
  }
  __device__ __forceinline__ static int expert(int word, int bit, int lane) {
    return place<N, VEC>(word * 32 + bit, lane);
  }
};
// bf16 vectors stay as they are, two values a register: an instruction takes both
// (bits p and p + 16 for pair p).
template <int N>
struct Row<__nv_bfloat16, N, true> {
  static constexpr int kWords = 1;
  static_assert(N % 4 == 0 && N <= 32);
  uint32_t pair[N / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int E, int lane) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      uint2 u = make_uint2(0xff80ff80u, 0xff80ff80u);  // -inf
      if (inside<N, true>(c, lane, E)) u = *reinterpret_cast<const uint2*>(row + c * 128 + lane * 4);
      pair[2 * c] = u.x, pair[2 * c + 1] = u.y;
    }
  }
  __device__ __forceinline__ static __nv_bfloat162 both(uint32_t u) {
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  }
  __device__ __forceinline__ float operator()(int j) const {
    const uint32_t u = pair[j >> 1];
    return __uint_as_float(j & 1 ? u & 0xffff0000u : u << 16);
  }
  __device__ __forceinline__ float most() const {
    __nv_bfloat162 m = both(pair[0]);
#pragma unroll
    for (int p = 1; p < N / 2; ++p) m = __hmax2(m, both(pair[p]));
    const float a = __low2float(m), b = __high2float(m);
    return fmaxf(fmaxf(a, b), -INFINITY);
  }
  __device__ __forceinline__ bool nan() const {
    unsigned n = 0;
#pragma unroll
    for (int p = 0; p < N / 2; ++p) n |= __hneu2_mask(both(pair[p]), both(pair[p]));
    return n != 0;
  }
  __device__ __forceinline__ void reach(float bound, uint32_t (&bits)[1]) const {
    const __nv_bfloat162 b = __bfloat162bfloat162(__float2bfloat16_ru(bound));
#pragma unroll
    for (int p = 0; p < N / 2; ++p) bits[0] |= __hge2_mask(both(pair[p]), b) & (0x00010001u << p);
  }
  __device__ __forceinline__ static int expert(int, int bit, int lane) {
    const int p = bit & 15;
    return (p >> 1) * 128 + lane * 4 + (p & 1) * 2 + (bit >> 4);
  }
};

template <typename T, int N, bool VEC>
__device__ __forceinline__ void store_row(T* __restrict__ row, int E, int lane,
                                          const float (&l)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const int at = c * 128 + lane * 4;
      if (!inside<N, true>(c, lane, E)) continue;
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(row + at) =
            make_float4(l[4 * c], l[4 * c + 1], l[4 * c + 2], l[4 * c + 3]);
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(l[4 * c], l[4 * c + 1]);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(l[4 * c + 2], l[4 * c + 3]);
        *reinterpret_cast<uint2*>(row + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                         *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int at = j * 32 + lane;
      if (at < E) row[at] = (T)l[j];
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {  // NaN is passed over
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The lanes' values sorted downwards over the warp (bitonic network).  `keep` has a
// bit for each step where the lane keeps the larger value: see sort_directions.
__device__ __forceinline__ uint32_t sort_directions(int lane) {
  uint32_t keep = 0, bit = 1;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1, bit <<= 1)
      if (((lane & k) == 0) == ((lane & j) == 0)) keep |= bit;
  return keep;
}
__device__ __forceinline__ float warp_sort_down(float v, uint32_t keep) {
  uint32_t bit = 1;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1, bit <<= 1) {
      const float o = __shfl_xor_sync(kAll, v, j);
      v = (keep & bit) ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
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
// KIND: 0 softmax, 1 sigmoid, -1 as the call says.
template <int KIND>
struct Scores {
  int called;
  float shift, one;  // m; or b and e^b
  __device__ __forceinline__ Scores(int called_, float m) : called(called_) {
    if (m == -INFINITY) m = 0.f;
    shift = softmax() ? m : fminf(m, 0.f);
    one = fast_exp(shift);
  }
  __device__ __forceinline__ bool softmax() const { return KIND < 0 ? called == 0 : KIND == 0; }
  __device__ __forceinline__ float operator()(float l) const {
    return softmax() ? fast_exp(l - shift) : fast_rcp(fast_exp(shift - l) + one);
  }
};

// The K largest of a token, one after the other; f(k, logit, expert) for each.
// (Compared as logits and experts, not as keys: keys of a whole row would be kept
// in registers through the kernel.)
template <typename T, int N, bool VEC, typename F>
__device__ __forceinline__ void select_in_turn(const Row<T, N, VEC>& l, int E, int K, int lane,
                                               F&& f) {
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
      const float v = l(j);
      const bool left = nans ? (v != v && later) : (v < last || (v == last && later));
      if (left && e < E && (best_e == 0x7fffffff || v > best)) best = v, best_e = e;
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

// A bf16 logit (not NaN) and its expert as one integer: larger logits first, equal
// ones (-0 and +0 too) by ascending expert.
__device__ __forceinline__ uint32_t bf16_key(float v, int e) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return ((u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) & 0xffff0000u) | (0xffffu - (uint32_t)e);
}

// Candidates of a warp: all logits that reach a bound, at most 32.
struct __align__(16) Candidates {
  uint32_t value[32];  // bf16 rows: the key above; fp32 rows: the logit
  int32_t expert[32];
};

// The K <= 32 largest of a token: a lane with rank < K holds the one of that rank.
//
// The logits that reach a bound are gathered, one a lane, and each finds its rank by
// counting the larger ones; any bound that K to 32 logits reach gives the same
// result.  The bound of the token before is tried first, moved each time so that
// about `target` logits reach it (on the model that their number falls off
// exponentially up to the row's largest, m; on normal logits 84 to 90 tokens of a
// hundred succeed at once).  Where too few reach it, the K-th largest of the lanes'
// maxima is a bound that at least K do; where too many do, it is raised, then halved
// in on.  What no bound tells apart (ties) and a bound of -inf (which the places past
// the row's end reach too) take the K largest one after the other.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void select_top(const Row<T, N, VEC>& l, const T* row, int E, int K,
                                           int lane, float most, float m, uint32_t keep,
                                           float& guess, Candidates& list, int& rank, float& value,
                                           int& expert) {
  constexpr int NW = Row<T, N, VEC>::kWords;
  rank = 32;
  value = 0.f, expert = 0;
  const float target = (float)min(K + 8, (K + 30) / 2);
  const float pull = fast_rcp(target * __logf(target));
  float bound = guess, low = -INFINITY, high = INFINITY;  // too many reach low, too few high
  bool fresh = !(bound > -INFINITY);
  if (fresh) bound = __shfl_sync(kAll, warp_sort_down(most, keep), K - 1);
#pragma unroll 1
  for (int tries = 0; tries < 8 && bound > -INFINITY; ++tries) {
    uint32_t reach[NW] = {};
    l.reach(bound, reach);
    int mine = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) mine += __popc(reach[w]);
    const int total = __reduce_add_sync(kAll, mine);
    if (total < K) {
      high = bound;
      bound = low;
      if (!(low > -INFINITY)) {
        bound = __shfl_sync(kAll, warp_sort_down(most, keep), K - 1);
        fresh = true;
        continue;
      }
    }
    if (total < K || total > 32) {
      low = bound;
      bound = high < INFINITY
                  ? low + 0.5f * (high - low)
                  : low + (m - low) * (1.f - __log2f(target) * fast_rcp(__log2f((float)total)));
      if (!(bound > low && bound < high)) break;
      continue;
    }
    // the next token's bound: a number off by a part x of the target asks for a step of
    // x / log(target) of the way to m; a quarter of it, but all after a fresh start
    guess = fmaf((m - bound) * pull, (fresh ? 1.f : 0.25f) * ((float)total - target), bound);
    if (!(fabsf(guess) < INFINITY)) guess = -INFINITY;

    int base = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w)
      while (const unsigned who = __ballot_sync(kAll, reach[w] != 0)) {
        if (reach[w])
          list.expert[base + __popc(who & ((1u << lane) - 1u))] =
              Row<T, N, VEC>::expert(w, __ffs(reach[w]) - 1, lane);
        reach[w] &= reach[w] - 1;
        base += __popc(who);
      }
    __syncwarp();
    uint32_t own = sizeof(T) == 2 ? 0u : 0xff800000u;  // larger than none
    if (lane < total) {
      expert = list.expert[lane];
      value = to_f32(row[expert]);
      own = sizeof(T) == 2 ? bf16_key(value, expert) : __float_as_uint(value);
    }
    list.value[lane] = own;
    __syncwarp();
    int r = 0;
#pragma unroll 1
    for (int i = 0; i < total; i += 4) {
      const uint4 c = *reinterpret_cast<const uint4*>(&list.value[i]);
      if constexpr (sizeof(T) == 2)
        r += (c.x > own) + (c.y > own) + (c.z > own) + (c.w > own);
      else
        r += (__uint_as_float(c.x) > value) + (__uint_as_float(c.y) > value) +
             (__uint_as_float(c.z) > value) + (__uint_as_float(c.w) > value);
    }
    if constexpr (sizeof(T) == 4) {
      // equal logits share a rank: then the lower expert goes first
      if (__reduce_add_sync(kAll, lane < total ? r : 0) != total * (total - 1) / 2) {
        for (int i = 0; i < total; ++i)
          r += __uint_as_float(list.value[i]) == value && list.expert[i] < expert;
      }
    }
    __syncwarp();
    if (lane < total) rank = r;
    return;
  }
  select_in_turn<T, N, VEC>(l, E, K, lane, [&](int k, float v, int e) {
    if (lane == k) value = v, expert = e, rank = k;
  });
}

constexpr int kRouterMaxK = 128;

// Warps of a block
template <int N>
constexpr int router_warps() {
  return N > 32 ? 4 : 8;
}
// Blocks a multiprocessor has to hold, which caps the registers
template <int N>
constexpr int router_blocks() {
  return N <= 8 ? 5 : N <= 16 ? 4 : N <= 32 ? 3 : 1;
}
// The same for the router with balance outputs.  A block ends with up to two atomics an
// expert: for rows of more than 512 all warps of a multiprocessor are one block (65536 x
// 896: 77 us, in blocks of 8 warps 79.5); for shorter ones that gains 0.6 us at 65536 x
// 384 (51.8, 52.4) and costs as much on eight tokens.
template <int N, bool LOSS>
constexpr int forward_warps() {
  return LOSS && N > 16 && N <= 32 ? 24 : router_warps<N>();
}
template <int N, bool LOSS>
constexpr int forward_blocks() {
  return LOSS && N > 16 && N <= 32 ? 1 : router_blocks<N>();
}
// Rows of more than 512 keep the warp's probability sums in shared memory: in
// registers, next to the row, they cost a third of the warps that fit.
template <int N>
constexpr bool sums_in_smem() {
  return N > 16;
}

// Rows of more than 512 come by way of shared memory, one row ahead: with 24 warps on a
// multiprocessor, loads waited for at once cost a quarter of the time between two
// instructions (65536 x 896 bf16: 86 us so, 80 ahead).  With the 32 warps of shorter rows
// the copy costs as much as it saves (65536 x 384 fp32: 52.5 us at once, 53.6 ahead).
template <int N, bool VEC>
constexpr bool rows_ahead() {
  return VEC && N > 16;
}

// Sum over the block in a fixed order, to thread 0.  (fp32: each of these sums has
// terms of one sign, so its error is a few 2^-24 of it; this GPU's 64-bit units would
// take longer than the whole call on eight tokens.)
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  v = (int)threadIdx.x < warps ? s[threadIdx.x] : 0.f;
  return threadIdx.x < 32 ? warp_sum(v) : 0.f;
}

// An expert's sum over the warps that had a token.
__device__ __forceinline__ float sum_of_warps(const float* s_q, int E, int e, int warps) {
  float q = 0.f;
#pragma unroll 8
  for (int w = 0; w < warps; ++w) q += s_q[(size_t)w * E + e];
  return q;
}

// A block's part of a segment that several blocks share: its warps' probability sums
// s_q [warps][E] and counts s_cnt [E] are added to the segment's as integers (steps of
// 2^-shift), so the order of the atomics changes nothing; what is not finite is only
// noted (q of such a token is NaN for every expert).
__device__ __forceinline__ void add_to_segment(const RouterDims& d, const RouterScratch& ws, int g,
                                               const float* s_q, const int32_t* s_cnt, int warps) {
  const float one = ldexpf(1.f, d.shift);
  for (int e = threadIdx.x; e < d.E; e += blockDim.x) {
    const float q = sum_of_warps(s_q, d.E, e, warps);
    if (!isfinite(q)) atomicOr(&ws.bad[g], 1);
    else if (q != 0.f) atomicAdd(&ws.q[(size_t)g * d.E + e], __float2ull_rn(q * one));
    if (s_cnt[e]) atomicAdd(&ws.counts[(size_t)g * d.E + e], s_cnt[e]);
  }
}

// The outputs of a segment of `tokens` tokens and its part of the loss, from the block's
// own sums (ALONE) or the joined ones.  All threads.
template <bool ALONE>
__device__ __forceinline__ void finish_segment(const RouterDims& d, const RouterOut& out,
                                               const RouterScratch& ws, int g, int tokens,
                                               const float* s_q = nullptr,
                                               const int32_t* s_cnt = nullptr, int warps = 0) {
  __shared__ float s_red[32];
  const float step = ldexpf(1.f, -d.shift);
  const bool bad = !ALONE && __ldcg(&ws.bad[g]);
  float part = 0.f;
  for (int e = threadIdx.x; e < d.E; e += blockDim.x) {
    const size_t at = (size_t)g * d.E + e;
    int32_t c;
    float q;
    if constexpr (ALONE) {
      q = sum_of_warps(s_q, d.E, e, warps);
      c = s_cnt[e];
    } else {
      c = __ldcg(&ws.counts[at]);
      q = bad ? NAN : __ull2float_rn(__ldcg(&ws.q[at])) * step;
    }
    out.counts[at] = c;
    out.prob_sum[at] = q;
    part = fmaf((float)c, q, part);
  }
  part = block_sum(part, s_red);
  if (threadIdx.x == 0) {
    const float n = (float)tokens;
    const float seg = tokens ? part / n * ((float)d.E / ((float)d.K * n)) : 0.f;
    out.seg_tokens[g] = tokens;
    *(d.G > 1 ? &ws.seg_loss[g] : out.loss) = seg;
  }
  __syncthreads();
}

// Adds to a counter of the GPU, after all that this thread has written or, over a
// barrier, has seen written; what other threads wrote before theirs is seen after it.
__device__ __forceinline__ unsigned long long add_in_order(unsigned long long* at,
                                                           unsigned long long v) {
  unsigned long long before;
  asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;" : "=l"(before) : "l"(at), "l"(v) : "memory");
  return before;
}

// A block's end.  Its `joined` (0 to 2) segments shared with other blocks are told off;
// the last block of a segment writes its outputs, and the block that finishes the last
// segment the loss.  `finished`: segments that this block has had to itself.
__device__ __forceinline__ void join_blocks(const RouterDims& d, const RouterOut& out,
                                            const RouterScratch& ws, int first_seg, int last_seg,
                                            int joined, int* s_tokens, int finished) {
  // (s_all is a word of its own: a warp may still be reading s_last when thread 0 writes it)
  __shared__ int s_last[2], s_all;
  if (joined) {
    // (the barrier before this orders the block's additions before these)
    if ((int)threadIdx.x < joined) {
      const int g = threadIdx.x ? last_seg : first_seg;
      const int from = (int)((int64_t)g * d.segment / d.per_block);
      const int to = (int)((min((int64_t)(g + 1) * d.segment, (int64_t)d.T) - 1) / d.per_block);
      // the blocks so far above the tokens so far
      const unsigned long long before =
          add_in_order(&ws.joined[g], 1ull << 32 | (uint32_t)s_tokens[threadIdx.x]);
      s_last[threadIdx.x] = (int)(before >> 32) == to - from;
      s_tokens[threadIdx.x] += (int)(uint32_t)before;
    }
    __syncthreads();
    for (int i = 0; i < joined; ++i)
      if (s_last[i]) {
        finish_segment<false>(d, out, ws, i ? last_seg : first_seg, s_tokens[i]);
        ++finished;
      }
  }
  if (d.G == 1 || finished == 0) return;
  if (threadIdx.x == 0) {
    s_all = (int)add_in_order(ws.done, finished) + finished == d.G;
  }
  __syncthreads();
  if (!s_all) return;
  __shared__ float s_red[32];
  float mean = 0.f;
  for (int i = threadIdx.x; i < d.G; i += blockDim.x) mean += __ldcg(&ws.seg_loss[i]);
  mean = block_sum(mean, s_red);
  if (threadIdx.x == 0) *out.loss = mean / (float)d.G;
}

// A block takes per_block consecutive tokens, a warp every W-th of them; with the
// loss, segment by segment.  SHORT: K <= 32.
//
// Bound by instructions and by the latency of a token's own chain (test the bound, gather,
// rank, score): about 290 instructions a token to choose the experts and place them, and
// per logit 1 to 4 more there and 7 in scores and sums.  While blocks run, 66 % (384
// experts) and 74 % (896) of the issue slots are used, 55 and 61 % of the launch with its
// start and end; of the 10.5 clocks between two instructions of a warp at 384, 2.6 are
// waits for the row, 1.4 for shared memory and shuffles, 1.9 for results of fixed latency,
// 0.75 for the block.  Measured with the loss: 65536 x 384 fp32, K 8: 49.2 us (without
// 35.3; its bytes 15.6); 65536 x 896 bf16, K 16, sigmoid: 69.7 us (without 45; its bytes
// 18.8, its 2 special functions a score 25).
template <typename T, int N, bool VEC, bool LOSS, bool SHORT, int KIND>
__global__ void __launch_bounds__(forward_warps<N, LOSS>() * 32, forward_blocks<N, LOSS>())
k_router(RouterDims d, const T* __restrict__ logits, const uint8_t* __restrict__ mask,
         RouterOut out, RouterScratch ws) {
  constexpr int W = forward_warps<N, LOSS>();
  constexpr bool kSmemSums = LOSS && sums_in_smem<N>(), kRegSums = LOSS && !kSmemSums;
  constexpr bool kAhead = rows_ahead<N, VEC>();
  constexpr int KI = SHORT ? 1 : kRouterMaxK / 32;
  __shared__ Candidates s_cand[SHORT ? W : 1];
  __shared__ unsigned long long s_list[SHORT ? 1 : W][kRouterMaxK];
  // LOSS: the warps' sums [W][E], then counts [E]; rows ahead: the warps' [W][E]
  extern __shared__ __align__(16) float s_dyn[];
  __shared__ int s_tokens[2];  // of the shared segments, and of the one at work
  int32_t* s_cnt = reinterpret_cast<int32_t*>(s_dyn + (size_t)W * d.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T* s_row = reinterpret_cast<T*>(s_dyn + (LOSS ? (size_t)(W + 1) * d.E : 0)) + (size_t)warp * d.E;
  const uint32_t keep = sort_directions(lane);
  float guess = -INFINITY;
  int joined = 0, finished = 0, first_seg = 0, last_seg = 0;

  const int first = blockIdx.x * d.per_block;
  const int last = min(first + d.per_block, d.T);
  for (int begin = first; begin < last;) {
    const int g = LOSS ? begin / d.segment : 0;
    const int end = LOSS ? (int)min((int64_t)last, (int64_t)(g + 1) * d.segment) : last;
    float acc[kRegSums ? N : 1];
    float* sums = s_dyn + (size_t)warp * d.E;  // this warp's, in its lanes' own places
    int live_tokens = 0;
    if constexpr (LOSS) {
#pragma unroll
      for (int j = 0; j < (kRegSums ? N : 1); ++j) acc[j] = 0.f;
      if constexpr (kSmemSums) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (place<N, VEC>(j, lane) < d.E) sums[place<N, VEC>(j, lane)] = 0.f;
      }
      for (int e = threadIdx.x; e < d.E; e += blockDim.x) s_cnt[e] = 0;
      if (threadIdx.x == 0) s_tokens[joined] = 0;
      __syncthreads();
    }

    if (kAhead && begin + warp < end)
      fetch_row<T, N>(s_row, logits + (size_t)(begin + warp) * d.E, d.E, lane);
    for (int t = begin + warp; t < end; t += W) {
      Row<T, N, VEC> logit;
      const T* row = kAhead ? s_row : logits + (size_t)t * d.E;
      if constexpr (kAhead) await_row();
      logit.load(row, d.E, lane);
      const bool live = mask == nullptr || mask[t] != 0;
      const float most = logit.most();
      const float m = warp_max(most);
      const Scores<KIND> score(d.score, m);

      // the chosen ones of this lane, with their ranks (K and more: none)
      float value[KI];
      int expert[KI], rank[KI];
      if constexpr (SHORT) {
        select_top<T, N, VEC>(logit, row, d.E, d.K, lane, most, m, keep, guess, s_cand[warp],
                              rank[0], value[0], expert[0]);
      } else {
        select_in_turn<T, N, VEC>(logit, d.E, d.K, lane, [&](int k, float v, int e) {
          if (lane == 0)
            s_list[warp][k] = ((unsigned long long)__float_as_uint(v) << 32) | (uint32_t)e;
        });
        __syncwarp();
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          rank[i] = i * 32 + lane;
          const unsigned long long c = rank[i] < d.K ? s_list[warp][rank[i]] : 0;
          value[i] = __uint_as_float((uint32_t)(c >> 32)), expert[i] = (int)(uint32_t)c;
        }
        __syncwarp();
      }

      // all that was read of this row has been used (and the warp is together): the next
      // one's way from memory is behind the scores, sums and gates of this one
      if (kAhead && t + W < end) fetch_row<T, N>(s_row, logits + (size_t)(t + W) * d.E, d.E, lane);

      // 1 / sum of the row's scores, where it is needed; a NaN in the row, which is in
      // every softmax score, shows in it
      float inv = 1.f;
      bool nan = score.softmax() && m == INFINITY;
      float l[N];
      if (LOSS || (score.softmax() && !d.normalise)) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          l[j] = score(logit(j));
          sum += l[j];
        }
        sum = warp_sum(sum);
        inv = sum == 0.f ? 0.f : fast_rcp(sum);
        nan |= score.softmax() && sum != sum;
      } else if (score.softmax()) {
        nan |= logit.nan();
      }
      if (LOSS && live) {
        ++live_tokens;
        if constexpr (kRegSums) {
#pragma unroll
          for (int j = 0; j < N; ++j) acc[j] = fmaf(l[j], inv, acc[j]);
        } else if constexpr (kSmemSums && VEC) {
#pragma unroll
          for (int c = 0; c < N / 4; ++c)
            if (inside<N, true>(c, lane, d.E)) {
              float4& q = *reinterpret_cast<float4*>(sums + c * 128 + lane * 4);
              q = make_float4(fmaf(l[4 * c], inv, q.x), fmaf(l[4 * c + 1], inv, q.y),
                              fmaf(l[4 * c + 2], inv, q.z), fmaf(l[4 * c + 3], inv, q.w));
            }
        } else if constexpr (kSmemSums) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (j * 32 + lane < d.E) sums[j * 32 + lane] = fmaf(l[j], inv, sums[j * 32 + lane]);
        }
      }

      // The chosen scores are at most 1 and the largest of them at least 1/2: summed as
      // integers, in steps of 2^-24, the sum does not depend on which lane holds which.
      float gate[KI];
      uint32_t part = 0;
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        gate[i] = rank[i] < d.K ? score(value[i]) : 0.f;
        nan |= gate[i] != gate[i];
        part += __float2uint_rn(gate[i] * 16777216.f);
      }
      float factor = score.softmax() ? inv : score.one;
      if (d.normalise) {
        const float total = (float)__reduce_add_sync(kAll, part);
        factor = total == 0.f ? 0.f : 16777216.f * fast_rcp(total);
      }
      factor *= d.scale;
      if (__any_sync(kAll, nan) && (score.softmax() || d.normalise)) factor = NAN;
#pragma unroll
      for (int i = 0; i < KI; ++i)
        if (rank[i] < d.K) {
          const size_t at = (size_t)t * d.K + rank[i];
          out.topk_idx[at] = expert[i];
          out.gates[at] = live ? gate[i] * factor : 0.f;
          if (LOSS && live) atomicAdd(&s_cnt[expert[i]], 1);
        }
    }
    if constexpr (LOSS) {
      if constexpr (kRegSums) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (place<N, VEC>(j, lane) < d.E) sums[place<N, VEC>(j, lane)] = acc[j];
      }
      if (lane == 0) atomicAdd(&s_tokens[joined], live_tokens);
      __syncthreads();
      // A segment with a token in another block: at most the block's first one and its
      // last.  Only the additions are made here, and waited for at the block's end
      // (waiting for them twice in a block: 1.1 us more at 65536 x 896).
      const bool alone = first <= (int64_t)g * d.segment &&
                         min((int64_t)(g + 1) * d.segment, (int64_t)d.T) <= (int64_t)first + d.per_block;
      if (alone) {
        finish_segment<true>(d, out, ws, g, s_tokens[joined], s_dyn, s_cnt, min(W, end - begin));
        ++finished;
      } else {
        cudaGridDependencySynchronize();  // the scratch is zero
        add_to_segment(d, ws, g, s_dyn, s_cnt, min(W, end - begin));
        *(joined ? &last_seg : &first_seg) = g;
        ++joined;
      }
      __syncthreads();  // the next segment uses the sums' memory
    }
    begin = end;
  }
  if constexpr (LOSS) {
    cudaGridDependencySynchronize();
    join_blocks(d, out, ws, first_seg, last_seg, joined, s_tokens, finished);
  }
}

// The gradient.  With w_e = d_loss E counts_e / (G K n^2), a_k what the gate k
// gives its expert's s times s, and dot = sum_e q_e w_e:
//   softmax:  dl_e = q_e (w_e - dot) + a_e,           a sums to 0 when normalised;
//             else dot takes in sum a
//   sigmoid:  dl_e = (1 - s_e) (q_e (w_e - dot) + a_e)
//   a_k = scale n_k (d_gate_k - sum_j n_j d_gate_j), n = chosen s / their sum, when
//   normalised; else scale s_k d_gate_k
// (sigmoid without the loss, w = 0: dl_e = (1 - s_e) a_e, and 0 where e is not chosen)
// The chosen experts' a lie in a row of shared memory that is zero elsewhere; w, one for
// a segment, lies there too, as three rows in registers left a third of the warps.
//
// Bound by bytes at 65536 x 384 fp32 (37.9 us, 5.4 TB/s; its bytes 30.5), by instructions
// and their latency at 65536 x 896 bf16 (58 us, 68 % of the issue slots while blocks run;
// with w in registers 79 us; its bytes 35).
template <typename T, int N, bool VEC, bool SHORT, int KIND>
__global__ void __launch_bounds__(router_warps<N>() * 32, router_blocks<N>())
k_router_backward(RouterDims d, const T* __restrict__ logits, const uint8_t* __restrict__ mask,
                  const int32_t* __restrict__ topk_idx, const float* __restrict__ d_gates,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ seg_tokens,
                  const float* __restrict__ d_loss, T* __restrict__ d_logits) {
  constexpr int W = router_warps<N>();
  constexpr int KI = SHORT ? 1 : kRouterMaxK / 32;
  constexpr int V = VEC ? 4 : 1;  // neighbours in a lane
  // w [E rounded up to 4], the warps' a [W][same], VEC: the warps' rows [W][E]
  extern __shared__ __align__(16) float s_dyn[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E4 = (d.E + 3) & ~3;
  float* w = s_dyn;
  float* a = s_dyn + (size_t)(1 + warp) * E4;
  T* s_row = reinterpret_cast<T*>(s_dyn + (size_t)(1 + W) * E4) + (size_t)warp * d.E;
  for (int e = lane; e < E4; e += 32) a[e] = 0.f;
  __syncwarp();
  // V values of a row of shared memory
  auto values = [](const float* at, float (&v)[V]) {
    if constexpr (VEC) {
      const float4 f = *reinterpret_cast<const float4*>(at);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      v[0] = *at;
    }
  };

  const int first = blockIdx.x * d.per_block;
  const int last = min(first + d.per_block, d.T);
  for (int begin = first; begin < last;) {
    const int g = d_loss != nullptr ? begin / d.segment : 0;
    const int end = d_loss != nullptr ? (int)min((int64_t)last, (int64_t)(g + 1) * d.segment) : last;
    float coef = 0.f;
    if (d_loss != nullptr) {
      const float n = (float)seg_tokens[g];
      coef = n > 0.f ? *d_loss * ((float)d.E / ((float)d.G * (float)d.K * n)) / n : 0.f;
    }
    __syncthreads();  // the last segment's w has been read
    for (int e = threadIdx.x; e < E4; e += blockDim.x)
      w[e] = d_loss != nullptr && e < d.E ? coef * (float)__ldg(counts + (size_t)g * d.E + e) : 0.f;
    __syncthreads();

    // a token's chosen experts and their gradients, loaded one token ahead
    int id[KI], next_id[KI];
    float dg[KI], next_dg[KI];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const int k = i * 32 + lane;
        const bool there = d_gates != nullptr && t < end && k < d.K;
        next_id[i] = there ? topk_idx[(size_t)t * d.K + k] : -1;
        next_dg[i] = there ? d_gates[(size_t)t * d.K + k] : 0.f;
      }
    };
    auto is_live = [&](int t) { return t < end && (mask == nullptr || mask[t] != 0); };
    fetch(begin + warp);
    bool live = is_live(begin + warp);
    if (VEC && live) fetch_row<T, N>(s_row, logits + (size_t)(begin + warp) * d.E, d.E, lane);
    for (int t = begin + warp; t < end; t += W) {
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        id[i] = next_id[i] < d.E ? next_id[i] : -1;
        dg[i] = next_dg[i];
      }
      fetch(t + W);
      const bool next_live = is_live(t + W);
      const T* next_row = logits + (size_t)(t + W) * d.E;
      T* drow = d_logits + (size_t)t * d.E;
      float l[N];
      if (live) {
        const T* row = VEC ? s_row : logits + (size_t)t * d.E;
        if constexpr (VEC) await_row();
        load_row<T, N, VEC>(row, d.E, lane, l);
        float s[KI];
#pragma unroll
        for (int i = 0; i < KI; ++i) s[i] = id[i] >= 0 ? to_f32(row[id[i]]) : 0.f;
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, l[j]);
        const Scores<KIND> score(d.score, warp_max(m));
        // the scores (up to their common factor), their sum and that with w.  A
        // sigmoid's place keeps the smaller of s and 1 - s without cancellation (where
        // that is 1 - s, l > 0, the factor is 1): the other follows, and their product
        // is all that the gradient needs.
        // A sigmoid's gates without the loss depend on the chosen logits alone: the row's
        // sums are left out, with what a NaN at another expert would make of them
        const bool row_sums = score.softmax() || d_loss != nullptr;
        float sum = 0.f, dot = 0.f;
#pragma unroll
        for (int c = 0; c < N / V; ++c) {
          if (!row_sums) break;
          const int at = place<N, VEC>(c * V, lane);
          float wv[V] = {};
          if (inside<N, VEC>(c, lane, d.E)) values(w + at, wv);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float& v = l[c * V + i];
            float q;
            if (score.softmax()) {
              v = q = score(v);
            } else {
              const float x = fast_exp(score.shift - v);
              q = fast_rcp(x + score.one);
              v = v > 0.f ? x * q : q;
            }
            sum += q;
            dot = fmaf(q, wv[i], dot);
          }
        }
        sum = warp_sum(sum);
        const float inv = sum == 0.f ? 0.f : fast_rcp(sum);
        dot = warp_sum(dot) * inv;

        if (d_gates != nullptr) {
          float total = 0.f, with = 0.f;
          float rest[KI];  // sigmoid: 1 - s
#pragma unroll
          for (int i = 0; i < KI; ++i) {
            rest[i] = 1.f;
            if (!score.softmax()) {
              const float x = fast_exp(score.shift - s[i]), q = fast_rcp(x + score.one);
              rest[i] = s[i] > 0.f ? x * q : fmaf(-q, score.one, 1.f);
            }
            s[i] = id[i] >= 0 ? score(s[i]) : 0.f;
            total += s[i];
            with = fmaf(s[i], dg[i], with);
          }
          float factor = score.softmax() ? inv : score.one, mean = 0.f;
          if (d.normalise) {
            total = warp_sum(total);
            factor = total == 0.f ? 0.f : fast_rcp(total);
            mean = warp_sum(with) * factor;
          } else if (score.softmax()) {
            dot = fmaf(warp_sum(with), d.scale * inv, dot);
          }
#pragma unroll
          for (int i = 0; i < KI; ++i)
            if (id[i] >= 0) a[id[i]] = d.scale * (s[i] * factor) * (dg[i] - mean) * rest[i];
        }
        __syncwarp();
        // all that was read of this row has been used: the next one's way from memory
        // is behind what is left of this one
        if (VEC && next_live) fetch_row<T, N>(s_row, next_row, d.E, lane);
        const float dot_inv = dot * inv;
        // (two loops: a choice for each element costs 1 us at 65536 x 896)
        if (row_sums) {
#pragma unroll
          for (int c = 0; c < N / V; ++c) {
            const int at = place<N, VEC>(c * V, lane);
            float wv[V] = {}, av[V] = {};
            if (inside<N, VEC>(c, lane, d.E)) values(w + at, wv), values(a + at, av);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              float& v = l[c * V + i];
              if (!score.softmax()) v *= fmaf(-v, score.one, 1.f);
              v = fmaf(v, fmaf(wv[i], inv, -dot_inv), av[i]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < N / V; ++c) {
            float av[V] = {};
            if (inside<N, VEC>(c, lane, d.E)) values(a + place<N, VEC>(c * V, lane), av);
#pragma unroll
            for (int i = 0; i < V; ++i) l[c * V + i] = av[i];
          }
        }
        if (d_gates != nullptr) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < KI; ++i)
            if (id[i] >= 0) a[id[i]] = 0.f;
          __syncwarp();
        }
      } else {
        if (VEC && next_live) fetch_row<T, N>(s_row, next_row, d.E, lane);
#pragma unroll
        for (int j = 0; j < N; ++j) l[j] = 0.f;
      }
      store_row<T, N, VEC>(drow, d.E, lane, l);
      live = next_live;
    }
    begin = end;
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
  r.done = (unsigned long long*)take(8);
  r.joined = (unsigned long long*)take(8 * G);
  r.bad = (int32_t*)take(4 * G);
  r.counts = (int32_t*)take(4 * GE);
  r.q = (unsigned long long*)take(8 * GE);
  r.zero_bytes = off;
  r.seg_loss = (float*)take(4 * G);
  r.total_bytes = off;
  return r;
}

// Blocks of `kernel` that fit the current device at once.  What the runtime answers
// is kept for each device and size of shared memory (the last one asked for): the
// three questions take longer than a small launch.
template <auto kernel, int N, int W>
static cudaError_t blocks_at_once(size_t smem, size_t most, int64_t* blocks) {
  constexpr int kDevices = 64;
  static std::atomic<uint64_t> known[kDevices];  // shared memory, blocks
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  const uint64_t k = known[dev].load(std::memory_order_relaxed);
  if (k != 0 && (uint32_t)(k >> 32) == (uint32_t)smem) {
    *blocks = (uint32_t)k;
    return cudaSuccess;
  }
  if (most > (32 << 10)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
  }
  int sms = 0, per_sm = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, W * 32, smem);
  if (e != cudaSuccess) return e;
  *blocks = std::max(1, sms * per_sm);
  known[dev].store((uint64_t)smem << 32 | (uint64_t)*blocks, std::memory_order_relaxed);
  return cudaSuccess;
}

// Launch shape: one round of blocks with equally many tokens: whole rounds of the
// block's warps, and at most 64 tokens a warp, so that a warp's fp32 sums stay short.
template <auto kernel, int N, int W>
static cudaError_t plan_blocks(size_t smem, size_t most, RouterDims& d) {
  int64_t blocks = 0;
  const cudaError_t e = blocks_at_once<kernel, N, W>(smem, most, &blocks);
  if (e != cudaSuccess) return e;
  const int64_t each = ((int64_t)d.T + blocks * W - 1) / (blocks * W);  // tokens a warp
  d.per_block = (int)std::min<int64_t>(each, 64) * W;
  d.blocks = (int)(((int64_t)d.T + d.per_block - 1) / d.per_block);
  return cudaSuccess;
}

// Zeroes the scratch; the router's kernel is launched while it runs and waits for it
// before it joins its sums (programmatic dependent launch).
__global__ void k_router_zero(uint4* at, size_t n) {
  cudaTriggerProgrammaticLaunchCompletion();
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
    at[i] = make_uint4(0, 0, 0, 0);
}

template <typename T, int N, bool VEC, bool LOSS, bool SHORT, int KIND>
static cudaError_t forward(RouterDims d, const void* logits, const uint8_t* mask,
                           const RouterOut& out, const RouterScratch& ws, cudaStream_t st,
                           int* launches) {
  constexpr int W = forward_warps<N, LOSS>();
  constexpr auto kernel = k_router<T, N, VEC, LOSS, SHORT, KIND>;
  const size_t per_expert = (LOSS ? 4 * (W + 1) : 0) + (rows_ahead<N, VEC>() ? sizeof(T) * W : 0);
  const size_t smem = d.E * per_expert;
  cudaError_t e = plan_blocks<kernel, N, W>(smem, 32 * N * per_expert, d);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d.blocks);
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  if (LOSS && (d.blocks > 1 || d.G > 1)) {
    // (one block joins nothing and only counts the segments)
    const size_t n = (d.blocks > 1 ? ws.zero_bytes : 16) / 16;
    k_router_zero<<<(unsigned)std::min<size_t>((n + 255) / 256, 1024), 256, 0, st>>>((uint4*)ws.done, n);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *launches += 1;
  }
  *launches += 1;
  return cudaLaunchKernelEx(&cfg, kernel, d, (const T*)logits, mask, out, ws);
}

// Calls f with the kernel's row shape: values per lane, whether they lie in vectors
// of four, K <= 32, and the score.  Rows of up to 128 experts are spread over all
// lanes one value at a time (vectors would leave lanes empty); so are rows that 4
// does not divide, rows of more than 1024, and K > 32.
template <typename T, typename F>
static cudaError_t by_row(const RouterDims& d, F&& f) {
#define ROW(n)                                                   \
  return d.score == 0 ? f.template operator()<T, n, true, true, 0>() \
                      : f.template operator()<T, n, true, true, 1>()
#define LONG_ROW(n)                                                   \
  return d.K <= 32 ? f.template operator()<T, n, false, true, -1>() \
                   : f.template operator()<T, n, false, false, -1>()
  const int E = d.E;
  if (E % 4 == 0 && E > 128 && E <= 1024 && d.K <= 32) {
    switch ((E + 127) / 128) {
      case 2: ROW(8);
      case 3: ROW(12);
      case 4: ROW(16);
      case 5: ROW(20);
      case 6: ROW(24);
      case 7: ROW(28);
      default: ROW(32);
    }
  }
  if (E <= 32) LONG_ROW(1);
  if (E <= 128) LONG_ROW(4);
  if (E <= 512) LONG_ROW(16);
  if (E <= 1024) LONG_ROW(32);
  LONG_ROW(128);
#undef ROW
#undef LONG_ROW
}

struct ForwardCall {
  const RouterDims& d;
  const void* logits;
  const uint8_t* mask;
  const RouterOut& out;
  const RouterScratch& ws;
  cudaStream_t st;
  int* launches;
  template <typename T, int N, bool VEC, bool SHORT, int KIND>
  cudaError_t operator()() const {
    return out.loss == nullptr
               ? forward<T, N, VEC, false, SHORT, KIND>(d, logits, mask, out, ws, st, launches)
               : forward<T, N, VEC, true, SHORT, KIND>(d, logits, mask, out, ws, st, launches);
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
  template <typename T, int N, bool VEC, bool SHORT, int KIND>
  cudaError_t operator()() const {
    constexpr int W = router_warps<N>();
    constexpr auto kernel = k_router_backward<T, N, VEC, SHORT, KIND>;
    const size_t per_expert = 4 * (W + 1) + (VEC ? sizeof(T) * W : 0);
    const size_t smem = ((d.E + 3) & ~3) * per_expert;
    RouterDims r = d;
    const cudaError_t e = plan_blocks<kernel, N, W>(smem, 32 * N * per_expert, r);
    if (e != cudaSuccess) return e;
    kernel<<<r.blocks, W * 32, smem, st>>>(r, (const T*)logits, mask, topk_idx, d_gates, counts,
                                           seg_tokens, d_loss, (T*)d_logits);
    return cudaGetLastError();
  }
};

cudaError_t launch_router_forward(const RouterDims& d, const void* logits, const uint8_t* mask,
                                  const RouterOut& out, const RouterScratch& ws, cudaStream_t st,
                                  int* launches) {
  const ForwardCall call{d, logits, mask, out, ws, st, launches};
  return d.bf16 ? by_row<__nv_bfloat16>(d, call) : by_row<float>(d, call);
}

cudaError_t launch_router_backward(const RouterDims& d, const void* logits, const uint8_t* mask,
                                   const int32_t* topk_idx, const float* d_gates,
                                   const int32_t* counts, const int32_t* seg_tokens,
                                   const float* d_loss, void* d_logits, cudaStream_t st,
                                   int* launches) {
  const BackwardCall call{d,      logits,     mask,   topk_idx, d_gates,
                          counts, seg_tokens, d_loss, d_logits, st};
  const cudaError_t e = d.bf16 ? by_row<__nv_bfloat16>(d, call) : by_row<float>(d, call);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace moonep
