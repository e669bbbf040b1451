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

// (the reduction is short chains of dependent instructions: eight warps took 2.2 times as long)
constexpr int kSplitThreads = 512;
constexpr int kSplitWarps = kSplitThreads / 32;
constexpr int kSplitStages = 12;          // at most
constexpr int kSplitRing = 204 * 1024;    // bytes of stages, at most
constexpr int kSplitSmem = kSplitRing + 1024 + (2 * kSplitStages + 2) * 8 + 16;
static_assert(kSplitSmem <= 232448, "shared memory of a CTA");

struct SplitArgs {
  int T, columns, depth;  // rows of x, columns of w (or rows, input gradient), depth
  int half, act, f32;
  int tokens, splits, stages, parts;
  const float* bias;
  const uint16_t* residual;
  void* out;
  uint16_t* z;
  int32_t* status;
};

// Four tokens' partial sums of a column, added in rank order.
__device__ __forceinline__ float4 add_parts(const float4* at, int stride, int splits) {
  float4 v = *at;
#pragma unroll 2
  for (int s = 1; s < splits; ++s) {
    at += stride;
    const float4 f = *at;
    v.x += f.x, v.y += f.y, v.z += f.z, v.w += f.w;
  }
  return v;
}

// act of the two columns' four tokens
__device__ __forceinline__ void act_pairs(int act, float (&v)[2][4]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = f(v[i >> 2][i & 3]);
  };
  if (act == kActRelu) each([](float z) { return act_value(kActRelu, z); });
  else if (act == kActGelu) each([](float z) { return act_value(kActGelu, z); });
  else if (act == kActSilu) each([](float z) { return act_value(kActSilu, z); });
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
  const uint32_t span = a.tokens <= 32 ? 32 : (a.tokens <= 64 ? 64 : (a.tokens <= 128 ? 128 : 256));
  const uint32_t tmem_cols = span * a.parts;  // a.parts is a power of two

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
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
  grid_wait();  // (what is above runs while the kernel before this one ends)

  if (warp == 0) {
    if (elect_one()) {
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
    if (elect_one()) {
      const uint32_t idesc = product_idesc(128, a.tokens, AMN, false);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      // the depth's parts, one after the other, have an accumulator each
      const int blocks = kb1 - kb0, of_part = (blocks + a.parts - 1) / a.parts;
      uint32_t acc = tmem_base;
      for (int kb = 0, left = 0; kb < blocks; ++kb) {
        if (!mbar_wait(full(stage), phase, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (left == 0 && kb != 0) acc += span;
        const uint32_t sa = smem_u32(smem) + stage * stage_bytes;
        const uint32_t sb = sa + 2 * kPanelBytes;
#pragma unroll
        for (int k = 0; k < kDepth / 16; ++k)
          umma_bf16(acc, stage_desc(sa, k, AMN), stage_desc(sb, k, false), idesc, left != 0 || k != 0);
        if (++left == of_part) left = 0;
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
  grid_trigger();
  // every thread waits for the sums: the stages are then free, here and, past the cluster's barrier,
  // in its other CTAs.  A CTA that gave up still takes part in the barriers; so does one that finds
  // the status set, which stops the stores alone (the rest harms nobody).
  const bool live = !plan_failed(a.status);
  const bool here = mbar_wait(done, 0, nullptr, 3 * kWaitNs);
  const bool ok = __syncthreads_and(here) && !*abort_flag;
  if (!ok && threadIdx.x == 0) set_error(a.status, MOONEP_ERR_TIMEOUT);
  __syncwarp();
  tc_fence_after();
  if (S > 1) pair_sync();

  const int valid = min(a.tokens, a.T - t0);   // rows of this tile
  const int fours = (valid + 3) / 4;           // in groups of four
  const int per = (fours + S - 1) / S;         // groups that a CTA owns
  const uint32_t red = smem_u32(smem);         // [splits][per][128 columns][4 tokens] partial sums
  if (ok) {
    const int qw = warp & 3;  // TMEM lanes 32 qw .. : columns of w
    const int of_part = (kb1 - kb0 + a.parts - 1) / a.parts;
    const int filled = (kb1 - kb0 + of_part - 1) / of_part;  // parts that hold a sum
    const uint32_t own = red + (rank * per * 128 + qw * 32 + lane) * 16;
    for (int g = 4 * (warp >> 2); g < fours; g += 4 * (kSplitWarps / 4)) {
      const uint32_t at = tmem_base + ((uint32_t)(qw * 32) << 16) + (uint32_t)(4 * g);
      uint32_t r[16];
      tmem_ld_x16(at, r);
      tmem_ld_wait();
      for (int k = 1; k < filled; ++k) {
        uint32_t more[16];
        tmem_ld_x16(at + k * span, more);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(more[j]));
      }
      int owner = S > 1 ? g / per : 0, local = g - owner * per;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (g + j < fours) {
          uint32_t to = own + local * (128 * 16);
          if (S > 1) to = pair_map(to, owner);
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(r[4 * j]),
                       "r"(r[4 * j + 1]), "r"(r[4 * j + 2]), "r"(r[4 * j + 3])
                       : "memory");
        }
        if (++local == per) { local = 0; ++owner; }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) pair_sync();

  if (ok && live) {
    // a lane has two columns (and, for swiglu, the two of the same numbers in the up half), a warp
    // 64 columns of every 8th (16th) group
    const int mine = min(per, fours - rank * per);
    const int c = 2 * lane + (a.half ? 0 : 64 * (warp & 1)), x = c0 + c;
    const int step = a.half ? kSplitWarps : kSplitWarps / 2;
    const int g0 = a.half ? warp : warp >> 1;
    if (x < ncols && g0 < mine) {
      const float4* sums = reinterpret_cast<const float4*>(smem) + g0 * 128 + c;
      const int stride = per * 128;
      const bool biased = KIND == kForward && a.bias != nullptr;
      float2 bias = make_float2(0.f, 0.f), bias_up = bias;
      if (biased) {
        bias = __ldg(reinterpret_cast<const float2*>(a.bias + x));
        if (a.half) bias_up = __ldg(reinterpret_cast<const float2*>(a.bias + a.half + x));
      }
      auto get = [&](float (&to)[2][4], int at, float2 b) {
        const float4 p = add_parts(sums + at, stride, S), q = add_parts(sums + at + 1, stride, S);
        to[0][0] = p.x, to[0][1] = p.y, to[0][2] = p.z, to[0][3] = p.w;
        to[1][0] = q.x, to[1][1] = q.y, to[1][2] = q.z, to[1][3] = q.w;
        if (biased) {
#pragma unroll
          for (int j = 0; j < 4; ++j) to[0][j] += b.x, to[1][j] += b.y;
        }
      };
      const int first = 4 * (rank * per + g0);  // token of the tile
      size_t at = (size_t)(t0 + first) * ncols + x, at_z = (size_t)(t0 + first) * a.columns + x;
#pragma unroll 1
      for (int left = valid - first, g = g0; g < mine; g += step, left -= 4 * step) {
        auto put = [&](uint16_t* to, int pitch, const float (&f)[2][4]) {
#pragma unroll
          for (int j = 0; j < 4; ++j, to += pitch)
            if (j < left)
              *reinterpret_cast<uint32_t*>(to) =
                  pack_bf16x2(__float_as_uint(f[0][j]), __float_as_uint(f[1][j]));
        };
        float v[2][4];
        get(v, 0, bias);
        if (KIND == kForward) {
          uint32_t res[4] = {};
          if (a.residual != nullptr) {
            const uint16_t* r = a.residual + at;
#pragma unroll
            for (int j = 0; j < 4; ++j, r += ncols)
              if (j < left) res[j] = __ldg(reinterpret_cast<const uint32_t*>(r));
          }
          if (a.z != nullptr) put(a.z + at_z, a.columns, v);
          if (a.half) {
            float u[2][4];
            get(u, 64, bias_up);
            if (a.z != nullptr) put(a.z + at_z + a.half, a.columns, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float& z = v[i >> 2][i & 3];
              z = z * sigmoid_f(z) * u[i >> 2][i & 3];
            }
          } else if (a.act != kActNone) {
            act_pairs(a.act, v);
          }
          if (a.residual != nullptr) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[0][j] += __uint_as_float(res[j] << 16);
              v[1][j] += __uint_as_float(res[j] & 0xffff0000u);
            }
          }
        }
        if (a.f32) {
          float* o = (float*)a.out + at;
#pragma unroll
          for (int j = 0; j < 4; ++j, o += ncols)
            if (j < left) *reinterpret_cast<float2*>(o) = make_float2(v[0][j], v[1][j]);
        } else {
          put((uint16_t*)a.out + at, ncols, v);
        }
        sums += step * 128;
        at += (size_t)(4 * step) * ncols;
        at_z += (size_t)(4 * step) * a.columns;
      }
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
  return launch_after(kernel, (unsigned)ctas, kSplitThreads, kSplitSmem, st, a.splits, w, x, a);
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
  a.parts = 1;
  if (a.f32) {
    const int blocks = ((a.depth + kDepth - 1) / kDepth + plan.splits - 1) / plan.splits;
    const int span = plan.tokens <= 32 ? 32 : (plan.tokens <= 64 ? 64 : (plan.tokens <= 128 ? 128 : 256));
    while (a.parts * kPartBlocks < blocks && a.parts * span < 512) a.parts *= 2;
  }
  return kind == kForward ? launch_kind<kForward>(tw, tx, a, ctas, st)
                          : launch_kind<kInputGrad>(tw, tx, a, ctas, st);
}

}  // namespace moonep
