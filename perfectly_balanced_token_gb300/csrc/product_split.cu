// The dense product of few rows, or of few tiles: every multiprocessor gets a share of the depth.
//
// The operands change sides: 128 columns of w are the M of the instruction and up to 256 rows of x,
// any multiple of 16, its N, so that one token costs a 16-wide instruction and not a 128-row tile.
// A cluster of 1, 2, 4 or 8 CTAs shares the depth of one tile: each runs its part through a ring of
// TMA-fed stages into TMEM, then sends its partial sums of a token to the CTA that owns the token
// (stores to the shared memory of the cluster, into the stages that are done), which adds them in
// rank order in fp32, applies bias, activation and residual and stores the rows.  No scratch memory,
// no atomics, one launch.
// What bounds it: at few rows reading w once (all of it is in flight over the multiprocessors'
// rings at any time), towards 256 rows a tile the rate at which L2 feeds the rings.
#include <algorithm>

#include "product.cuh"

namespace moonep {

constexpr int kSplitThreads = 256;
constexpr int kSplitWarps = kSplitThreads / 32;
constexpr int kSplitStages = 12;          // at most
constexpr int kSplitRing = 204 * 1024;    // bytes of stages, at most
constexpr int kSplitSmem = kSplitRing + 1024 + (2 * kSplitStages + 2) * 8 + 16;
static_assert(kSplitSmem <= 232448, "shared memory of a CTA");

struct SplitArgs {
  int T, columns, depth;  // rows of x, columns of w (or rows, input gradient), depth
  int half, act, f32;
  int tokens, splits, stages;
  const float* bias;
  const uint16_t* residual;
  void* out;
  uint16_t* z;
  int32_t* status;
};

// four columns' partial sums, added in rank order
__device__ __forceinline__ void add_parts(float (&v)[4], const float* at, int stride, int splits) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 f = *reinterpret_cast<const float4*>(at + (size_t)s * stride);
    v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
  }
}
__device__ __forceinline__ void add_bias4(float (&v)[4], const float* bias) {
  if (bias == nullptr) return;
  const float4 f = __ldg(reinterpret_cast<const float4*>(bias));
  v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
}
__device__ __forceinline__ void store4(uint16_t* at, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(__float_as_uint(v[0]), __float_as_uint(v[1])),
                                             pack_bf16x2(__float_as_uint(v[2]), __float_as_uint(v[3])));
}

template <int KIND>
__global__ void __launch_bounds__(kSplitThreads, 1)
k_product_split(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                const __grid_constant__ SplitArgs a) {
  constexpr bool AMN = KIND == kForward;  // w runs along its columns, w^T along the depth
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(smem + kSplitRing);
  uint32_t* tmem_slot = (uint32_t*)(bars + 2 * kSplitStages + 2);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kSplitStages + s); };
  const uint32_t done = bar0 + 8u * (2 * kSplitStages);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.splits, rank = S > 1 ? (int)pair_rank() : 0;
  const int step = a.half ? 64 : 128;  // output columns of a tile
  const int ncols = a.half ? a.half : a.columns;
  const int CT = (ncols + step - 1) / step;
  const int tile = (int)blockIdx.x / S;
  const int c0 = (tile % CT) * step, t0 = (tile / CT) * a.tokens;
  const int KB = (a.depth + kDepth - 1) / kDepth;
  const int kb0 = (int)((int64_t)KB * rank / S), kb1 = (int)((int64_t)KB * (rank + 1) / S);
  const uint32_t stage_bytes = 2 * kPanelBytes + a.tokens * 128;
  const int stages = a.stages;
  const uint32_t tmem_cols = a.tokens <= 32 ? 32 : (a.tokens <= 64 ? 64 : (a.tokens <= 128 ? 128 : 256));

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    // (a CTA that finds the status set does nothing but take part in its cluster's barriers: one that
    // started earlier may not have seen it, and stores to this one's shared memory)
    *abort_flag = plan_failed(a.status) ? 1 : 0;
    fence_barrier_init();
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const bool live = *abort_flag == 0;
  __syncthreads();  // read by all before a role may raise it

  if (warp == 0) {
    if (live && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int kb = kb0;
      for (; kb < kb1; ++kb) {
        if (!mbar_wait(empty(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
        mbar_expect_tx(full(stage), stage_bytes);
        const uint32_t sa = smem_u32(smem) + stage * stage_bytes;
        const int k0 = kb * kDepth;
        if (AMN) {
          tma_load_2d(sa, &tm_w, full(stage), c0, k0);
          tma_load_2d(sa + kPanelBytes, &tm_w, full(stage), a.half ? a.half + c0 : c0 + 64, k0);
        } else {
          tma_load_2d(sa, &tm_w, full(stage), k0, c0);
        }
        tma_load_2d(sa + 2 * kPanelBytes, &tm_x, full(stage), k0, t0);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) {
        *abort_flag = 1;
        set_error(a.status, MOONEP_ERR_TIMEOUT);
        for (int i = 0; i < min(kb - kb0, stages); ++i) {  // the copies in flight, time-bounded
          if (stage == 0) { stage = stages - 1; phase ^= 1u; } else { --stage; }
          mbar_wait(full(stage), phase, nullptr, 200000000ull);
        }
      }
    }
  } else if (warp == 1) {
    if (live && elect_one()) {
      const uint32_t idesc = product_idesc(128, a.tokens, AMN, false);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(full(stage), phase, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem) + stage * stage_bytes;
        const uint32_t sb = sa + 2 * kPanelBytes;
#pragma unroll
        for (int k = 0; k < kDepth / 16; ++k)
          umma_bf16(tmem_base, stage_desc(sa, k, AMN), stage_desc(sb, k, false), idesc,
                    kb != kb0 || k != 0);
        umma_commit(empty(stage));
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) {
        *abort_flag = 1;
        set_error(a.status, MOONEP_ERR_TIMEOUT);
      }
      umma_commit(done);  // once every MMA issued so far is done
    }
  }
  __syncwarp();
  // every thread waits for the sums: the stages are then free, here and, past the cluster's barrier,
  // in its other CTAs.  A CTA that gave up still takes part in the barriers.
  const bool here = !live || mbar_wait(done, 0, nullptr, 3 * kWaitNs);
  const bool ok = __syncthreads_and(here) && !*abort_flag;
  if (live && !ok && threadIdx.x == 0) set_error(a.status, MOONEP_ERR_TIMEOUT);
  __syncwarp();
  tc_fence_after();
  if (S > 1) pair_sync();

  const int valid = min(a.tokens, a.T - t0);  // rows of this tile
  const int per = (valid + S - 1) / S;        // that a CTA owns
  const uint32_t red = smem_u32(smem);        // [splits][per][128] partial sums
  if (ok) {
    const int qw = warp & 3;  // TMEM lanes 32 qw .. : columns of w
#pragma unroll 1
    for (int t = 16 * (warp >> 2); t < valid; t += 16 * (kSplitWarps / 4)) {
      uint32_t r[16];
      tmem_ld_x16(tmem_base + ((uint32_t)(qw * 32) << 16) + (uint32_t)t, r);
      tmem_ld_wait();
      int owner = t / per, local = t - owner * per;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (t + j < valid) {
          const uint32_t at = red + (((rank * per + local) * 128) + qw * 32 + lane) * 4;
          if (S > 1)
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(pair_map(at, owner)), "r"(r[j]) : "memory");
          else
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(r[j]) : "memory");
        }
        if (++local == per) { local = 0; ++owner; }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) pair_sync();

  if (ok) {
    const float* sums = reinterpret_cast<const float*>(smem);
    const int mine = min(per, valid - rank * per);
    const int width = a.half ? 16 : 32;  // lanes a row, four columns each
    const int col = 4 * (lane & (width - 1)), x = c0 + col;
    for (int l = (threadIdx.x / width); l < mine; l += kSplitThreads / width) {
      if (x >= ncols) break;
      const size_t row = (size_t)(t0 + rank * per + l);
      float v[4];
      add_parts(v, sums + l * 128 + col, per * 128, S);
      if (KIND == kForward) {
        add_bias4(v, a.bias ? a.bias + x : nullptr);
        if (a.z != nullptr) store4(a.z + row * a.columns + x, v);
        if (a.half) {
          float u[4];
          add_parts(u, sums + l * 128 + 64 + col, per * 128, S);
          add_bias4(u, a.bias ? a.bias + a.half + x : nullptr);
          if (a.z != nullptr) store4(a.z + row * a.columns + a.half + x, u);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = v[i] * sigmoid_f(v[i]) * u[i];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = act_value(a.act, v[i]);
        }
        if (a.residual != nullptr) {
          const uint2 r = __ldg(reinterpret_cast<const uint2*>(a.residual + row * ncols + x));
          v[0] += __uint_as_float(r.x << 16), v[1] += __uint_as_float(r.x & 0xffff0000u);
          v[2] += __uint_as_float(r.y << 16), v[3] += __uint_as_float(r.y & 0xffff0000u);
        }
      }
      if (a.f32)
        *reinterpret_cast<float4*>((float*)a.out + row * ncols + x) = make_float4(v[0], v[1], v[2], v[3]);
      else
        store4((uint16_t*)a.out + row * ncols + x, v);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
}

// -- host side ------------------------------------------------------------------
// How the rows are cut and the depth is split, or splits = 0 where the pair kernel's tiles are the
// better choice.  Times in microseconds of the two kernels on one box: a block of 64 of the depth
// costs the larger of its loads and its instructions.
SplitPlan plan_split(int T, int columns, int half, int depth) {
  static PerDevice kept;
  int sms = 0;
  if (kept(&sms, [](int* n) { return *n = sm_count_gemm(), cudaSuccess; }) != cudaSuccess) sms = 152;
  const int64_t CT = half ? (half + 63) / 64 : (columns + 127) / 128;
  const int KB = (depth + kDepth - 1) / kDepth;
  const int64_t pairs = std::max(1, sms / 2);
  const int64_t pair_tiles =
      ((T + 255) / 256) * (int64_t)(half ? (half + 127) / 128 : (columns + 255) / 256);
  SplitPlan best{0, 0};
  double cost = (double)((pair_tiles + pairs - 1) / pairs) * (KB * 0.36 + 1.0) + 6.0;
  for (int S = 1; S <= 8 && (S == 1 || KB >= 2 * S); S *= 2)
    for (int waves = 0; waves <= 3; ++waves) {  // 0: as few cuts as there can be
      const int64_t fewest = (T + 255) / 256;
      const int64_t cuts = waves ? waves * sms / (CT * S) : fewest;
      if (cuts < fewest) continue;
      const int tokens = (int)(((T + cuts - 1) / cuts + 15) / 16 * 16);
      const int64_t ctas = (T + tokens - 1) / tokens * CT * S;
      const double block = std::max(0.10, 0.06 + tokens * 0.0014);
      const double c = (double)((ctas + sms - 1) / sms) *
                           ((KB + S - 1) / S * block + 1.5 + tokens * 0.01) + 5.0 + 0.3 * (S > 1);
      if (c < cost) cost = c, best = {tokens, S};
    }
  return best;
}

template <int KIND>
static cudaError_t launch_kind(const CUtensorMap& w, const CUtensorMap& x, const SplitArgs& a,
                               int64_t ctas, cudaStream_t st) {
  auto* kernel = k_product_split<KIND>;
  static PerDevice kept;
  int set = 0;
  const cudaError_t e = kept(&set, [&](int* done) {
    *done = 1;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = a.splits;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = kSplitSmem;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = a.splits > 1 ? 1 : 0;
  void* args[] = {const_cast<CUtensorMap*>(&w), const_cast<CUtensorMap*>(&x),
                  const_cast<SplitArgs*>(&a)};
  return cudaLaunchKernelExC(&cfg, (const void*)kernel, args);
}

cudaError_t launch_split(Kind kind, const LinearDims& d, SplitPlan plan, const void* x, const void* w,
                         const float* bias, const void* residual, void* out, void* z, int32_t* status,
                         cudaStream_t st) {
  SplitArgs a = {};
  a.T = d.T;
  a.tokens = plan.tokens;
  a.splits = plan.splits;
  a.stages = std::min(kSplitStages, kSplitRing / (2 * kPanelBytes + plan.tokens * 128));
  a.out = out;
  a.status = status;
  CUtensorMap tw, tx;
  if (kind == kForward) {
    a.columns = d.N, a.depth = d.K;
    a.half = d.half, a.act = d.act, a.f32 = d.f32;
    a.bias = bias;
    a.residual = (const uint16_t*)residual;
    a.z = (uint16_t*)z;
    if (!encode_matrix(&tw, w, d.N, d.K, d.N, 64)) return cudaErrorInvalidValue;
  } else {
    a.columns = d.K, a.depth = d.N;
    if (!encode_matrix(&tw, w, d.N, d.K, d.N, 128)) return cudaErrorInvalidValue;
  }
  if (!encode_matrix(&tx, x, a.depth, d.T, a.depth, plan.tokens)) return cudaErrorInvalidValue;
  const int64_t CT = a.half ? (a.half + 63) / 64 : (a.columns + 127) / 128;
  const int64_t ctas = ((d.T + plan.tokens - 1) / plan.tokens) * CT * plan.splits;
  return kind == kForward ? launch_kind<kForward>(tw, tx, a, ctas, st)
                          : launch_kind<kInputGrad>(tw, tx, a, ctas, st);
}

}  // namespace moonep
