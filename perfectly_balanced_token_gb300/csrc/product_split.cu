// The dense product of few rows, or of few tiles: every multiprocessor gets a share of the depth.
//
// The operands change sides: 128 columns of w are the M of the instruction and up to 256 rows of x,
// any multiple of 16, its N, so that one token costs a 16-wide instruction and not a 128-row tile.
// (Weight gradient: d_z takes the place of w and x^T that of x, the depth is the number of tokens.)
// A cluster of 1, 2, 4 or 8 CTAs shares the depth of one tile: each runs its part through a ring of
// TMA-fed stages into TMEM, then sends its partial sums of a token to the CTA that owns the token
// (stores to the shared memory of the cluster, into the stages that are done), which adds them in
// rank order in fp32, applies bias, activation and residual and stores the rows.  No scratch memory,
// no atomics, one launch.  The plan's tiles run the same way where they are few (1 token x 2 of 14 experts,
// 4864 x 1664 of swiglu: 33 us with tiles of one CTA, 9.7 so).
// What bounds it: at few rows reading w once (all of it is in flight over the multiprocessors'
// rings at any time), towards 256 rows a tile the rate at which L2 feeds the rings.  Measured: 1 x 7168
// x 4096 of swiglu 13.4 us (58.7 MB: 8.8 us at the copy's rate), 256 rows 18.9, 1024 x 7168 x 2048 27
// (pair tiles: 37), 100 x 512 x 4096 4.9; and between the smallest kernels of a chain 2.9 us.
#include <algorithm>
#include <cmath>

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
  int T, columns, depth;  // rows and columns of the result, depth
  int half, act, f32, add;
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

// GROUPED: a tile is one of the plan's work tiles (all of them within `tokens` rows) instead of rows of x;
// the grid has room for as many as there can be, and clusters without one end at once.
template <int KIND, bool GROUPED>
__global__ void __launch_bounds__(kSplitThreads, 1)
k_product_split(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_slots,
                const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ SplitArgs a,
                const __grid_constant__ PlanPtrs p) {
  constexpr bool AMN = KIND != kInputGrad;  // w runs along its columns, w^T along the depth
  constexpr bool BMN = KIND == kWeightGrad;  // x runs along the depth, x^T does not
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
  const int c0 = (tile % CT) * step;
  int t0 = (tile / CT) * a.tokens, rows = min(a.tokens, a.T - t0), wrow = 0, expert = 0;
  const CUtensorMap* wmap = &tm_w;
  if (GROUPED) {
    grid_wait();
    if (tile / CT >= p.counters[MOONEP_CNT_MTILES]) return;  // (the same for a whole cluster)
    const MTile mt = p.mtiles[tile / CT];
    t0 = mt.row0;
    rows = max(1, min(mt.rows, a.tokens));  // (a failed plan may hold anything; nothing is stored then)
    if (mt.wsel < 0) wmap = &tm_slots;
    expert = mt.wsel;
    wrow = (mt.wsel >= 0 ? mt.wsel : -1 - mt.wsel) * a.depth;
  }
  const int KB = (a.depth + kDepth - 1) / kDepth;
  const int kb0 = (int)((int64_t)KB * rank / S), kb1 = (int)((int64_t)KB * (rank + 1) / S);
  const int panels = (a.tokens + 63) / 64;  // of x^T
  const uint32_t stage_bytes = 2 * kPanelBytes + (BMN ? panels * kPanelBytes : a.tokens * 128);
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
  if (!GROUPED) grid_wait();  // (what is above runs while the kernel before this one ends)

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
          tma_load_2d(sa, wmap, full(stage), c0, wrow + k0);
          tma_load_2d(sa + kPanelBytes, wmap, full(stage), a.half ? a.half + c0 : c0 + 64, wrow + k0);
        } else {
          tma_load_2d(sa, &tm_w, full(stage), k0, c0);
        }
        if (BMN) {
          for (int j = 0; j < panels; ++j)
            tma_load_2d(sa + (2 + j) * kPanelBytes, &tm_x, full(stage), t0 + 64 * j, k0);
        } else {
          tma_load_2d(sa + 2 * kPanelBytes, &tm_x, full(stage), k0, t0);
        }
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
      const uint32_t idesc = product_idesc(128, a.tokens, AMN, BMN);
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
          umma_bf16(acc, stage_desc(sa, k, AMN), stage_desc(sb, k, BMN), idesc, left != 0 || k != 0);
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

  const int valid = rows;                      // of this tile
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
        const float* from = a.bias + x;
        if (GROUPED) from += (size_t)(expert >= 0 ? expert : p.slot_expert[-1 - expert]) * a.columns;
        bias = *reinterpret_cast<const float2*>(from);
        if (a.half) bias_up = *reinterpret_cast<const float2*>(from + a.half);
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
              if (j < left) res[j] = *reinterpret_cast<const uint32_t*>(r);
          }
          if (a.z != nullptr) put(a.z + at_z, a.columns, v);
          if (a.half) {
            float u[2][4];
            get(u, 64, bias_up);
            if (a.z != nullptr) put(a.z + at_z + a.half, a.columns, u);
            swiglu_each(v[0], u[0]);
            swiglu_each(v[1], u[1]);
          } else if (a.act != kActNone) {
            act_each(a.act, v[0]);
            act_each(a.act, v[1]);
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
            if (j < left) {
              float2 f = make_float2(v[0][j], v[1][j]);
              if (KIND == kWeightGrad && a.add) {
                const float2 was = *reinterpret_cast<const float2*>(o);
                f.x += was.x, f.y += was.y;
              }
              *reinterpret_cast<float2*>(o) = f;
            }
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
static int span_of(int tokens) {  // columns of TMEM that one accumulator takes
  return tokens <= 32 ? 32 : (tokens <= 64 ? 64 : (tokens <= 128 ? 128 : 256));
}

template <int KIND, bool GROUPED>
static cudaError_t opt_in() {
  static PerDevice kept;
  int set = 0;
  return kept(&set, [&](int* done) {
    *done = 1;
    return cudaFuncSetAttribute(k_product_split<KIND, GROUPED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSplitSmem);
  });
}

// The GPU's processing clusters do not all have a multiple of eight multiprocessors.
int at_once(int splits) {
  static PerDevice kept[4];
  const int which = splits == 1 ? 0 : (splits == 2 ? 1 : (splits == 4 ? 2 : 3));
  int n = 0;
  const cudaError_t e = kept[which](&n, [&](int* found) {
    if (splits == 1) return *found = sm_count_gemm(), cudaSuccess;
    const cudaError_t e = opt_in<kForward, false>();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = splits;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits * 64);
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = kSplitSmem;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    int clusters = 0;
    const cudaError_t e2 = cudaOccupancyMaxActiveClusters(&clusters, (void*)k_product_split<kForward, false>, &cfg);
    *found = std::max(1, clusters) * splits;
    return e2;
  });
  return e == cudaSuccess ? n : 0;
}

// How the rows are cut and the depth is split, or splits = 0 where the pair kernel's tiles are the
// better choice.  The two kernels' times in microseconds, fitted to 25 shapes of 1 to 8192 rows (each
// with up to 15 choices; on the average off by 11 %, and the choice 1 % from the best one):
// a block of 64 of the depth costs an instruction's least time or grows with its tokens, 0.16 to 0.33;
// a round of CTAs begins and ends in 3 + 0.02 a token, a cluster's exchange adds 0.9 + 0.005 a token.
// The pair kernel takes 0.27 for a block of a tile, 2 more for a round of tiles and 4.25 once.
SplitPlan plan_split(int T, int columns, int half, int depth, bool f32) {
  const int64_t CT = half ? (half + 63) / 64 : (columns + 127) / 128;
  const int KB = (depth + kDepth - 1) / kDepth;
  const int64_t pairs = std::max(1, at_once(1) / 2);
  const int64_t pair_tiles =
      ((T + 255) / 256) * (int64_t)(half ? (half + 127) / 128 : (columns + 255) / 256);
  const double rounds = (double)((pair_tiles + pairs - 1) / pairs);
  SplitPlan best{0, 0};
  double cost = rounds * (0.2685 * KB + 2.0) + 4.25;
  for (int S = 1; S <= 8 && (S == 1 || KB >= 2 * S); S *= 2) {
    const int room = at_once(S);
    if (room == 0) continue;
    const int blocks = (KB + S - 1) / S;
    for (int waves = 0; waves <= 3; ++waves) {  // 0: as few cuts as there can be
      const int64_t fewest = (T + 255) / 256;
      const int64_t cuts = waves ? waves * room / (CT * S) : fewest;
      if (cuts < fewest) continue;
      const int tokens = (int)(((T + cuts - 1) / cuts + 15) / 16 * 16);
      // fp32 sums in parts: each has its columns of TMEM
      if (f32 && blocks > 512 / span_of(tokens) * kPartBlocks) continue;
      const int64_t ctas = (T + tokens - 1) / tokens * CT * S;
      const double c = (double)((ctas + room - 1) / room) *
                       (blocks * std::max(0.1585, 0.073 + 0.001 * tokens) + 3.02 + 0.0207 * tokens +
                        (S > 1 ? 0.914 + 0.0047 * tokens : 0.0));
      if (c < cost) cost = c, best = {tokens, S};
    }
  }
  return best;
}

// The same for the plan's tiles, where no rank has more than 128 rows: the tiles that so many copies of
// evenly chosen experts make, against the product on tiles of one CTA (0.5 us for a block of 64 by 256
// columns that memory has to bring).  Where reading the weights takes longer than either, the wide tiles
// read them faster as soon as they fill the GPU twice, by 2 to 12 % (16 tokens x 8 of 64 experts, 4096 x
// 2048: 123 us against 138), and slower below that, by 3 to 38 % (1 x 8 of 64, 7168 x 4096: 96 against 72;
// 4 x 8 of 64, 4096 x 2048: 73 against 64), but for many tokens, whose rows the narrow tiles load twice as
// often (128 x 1 of 16, 4096 x 4096: 84 against 95).
SplitPlan plan_split_grouped(const Dims& d, int half) {
  SplitPlan best{0, 0};
  if (d.C > kMmaM) return best;
  const int KB = d.H / kDepth;
  const double met = d.E * (1 - std::pow(1 - 1.0 / d.E, (double)d.N));
  const int64_t tiles = (int64_t)std::ceil(met);
  const int64_t CT = half ? (half + 63) / 64 : (d.Hp + 127) / 128;
  const int64_t wide = half ? (half + 127) / 128 : (d.Hp + 255) / 256;
  const int64_t sms = std::max(1, at_once(1));
  const int tokens = (std::min(d.C, 128) + 15) / 16 * 16;
  const double read = met * d.H * d.Hp * 2 / 6.5e6;  // us
  double cost = (tiles * wide >= 2 * sms ? 0.9 : 1.05) *
                std::max(read, (double)((tiles * wide + sms - 1) / sms) * (0.5 * KB + 1.0) + 4.0);
  for (int S = 1; S <= 8 && (S == 1 || KB >= 2 * S); S *= 2) {
    const int room = at_once(S);
    if (room == 0) continue;
    const double c = std::max(read * (1 + tokens / 1280.0), (double)((tiles * CT * S + room - 1) / room) *
                         ((KB + S - 1) / S * std::max(0.1585, 0.073 + 0.001 * tokens) + 3.02 +
                          0.0207 * tokens + (S > 1 ? 0.914 + 0.0047 * tokens : 0.0)) +
                     1.0);
    if (c < cost) cost = c, best = {tokens, S};
  }
  return best;
}

template <int KIND, bool GROUPED>
static cudaError_t launch_kind(const CUtensorMap& w, const CUtensorMap& slots, const CUtensorMap& x,
                               const SplitArgs& a, const PlanPtrs& p, int64_t ctas, cudaStream_t st) {
  const cudaError_t e = opt_in<KIND, GROUPED>();
  if (e != cudaSuccess) return e;
  return launch_after(k_product_split<KIND, GROUPED>, (unsigned)ctas, kSplitThreads, kSplitSmem, st,
                      a.splits, w, slots, x, a, p);
}

// x and w: the operands as the kernel has them (see there), `out` [T][C]
cudaError_t launch_split(Kind kind, const LinearDims& d, SplitPlan plan, const void* x, const void* w,
                         const float* bias, const void* residual, void* out, void* z, int add,
                         int32_t* status, cudaStream_t st) {
  SplitArgs a = {};
  a.T = kind == kWeightGrad ? d.K : d.T;
  a.tokens = plan.tokens;
  a.splits = plan.splits;
  const int rows_bytes = kind == kWeightGrad ? (plan.tokens + 63) / 64 * kPanelBytes : plan.tokens * 128;
  a.stages = std::min(kSplitStages, kSplitRing / (2 * kPanelBytes + rows_bytes));
  a.out = out;
  a.status = status;
  CUtensorMap tw, tx;
  bool ok;
  if (kind == kForward) {
    a.columns = d.N, a.depth = d.K;
    a.half = d.half, a.act = d.act, a.f32 = d.f32;
    a.bias = bias;
    a.residual = (const uint16_t*)residual;
    a.z = (uint16_t*)z;
    ok = encode_matrix(&tw, w, d.N, d.K, d.N, 64) && encode_matrix(&tx, x, d.K, d.T, d.K, plan.tokens);
  } else if (kind == kInputGrad) {
    a.columns = d.K, a.depth = d.N;
    ok = encode_matrix(&tw, w, d.N, d.K, d.N, 128) && encode_matrix(&tx, x, d.N, d.T, d.N, plan.tokens);
  } else {
    a.columns = d.N, a.depth = d.T;
    a.f32 = 1, a.add = add;
    ok = encode_matrix(&tw, w, d.N, d.T, d.N, 64) && encode_matrix(&tx, x, d.K, d.T, d.K, 64);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int64_t CT = a.half ? (a.half + 63) / 64 : (a.columns + 127) / 128;
  const int64_t ctas = ((a.T + plan.tokens - 1) / plan.tokens) * CT * plan.splits;
  a.parts = 1;
  if (a.f32) {
    const int blocks = ((a.depth + kDepth - 1) / kDepth + plan.splits - 1) / plan.splits;
    while (a.parts * kPartBlocks < blocks && a.parts * span_of(plan.tokens) < 512) a.parts *= 2;
  }
  const PlanPtrs none{};
  if (kind == kForward) return launch_kind<kForward, false>(tw, tw, tx, a, none, ctas, st);
  if (kind == kInputGrad) return launch_kind<kInputGrad, false>(tw, tw, tx, a, none, ctas, st);
  return launch_kind<kWeightGrad, false>(tw, tw, tx, a, none, ctas, st);
}

cudaError_t launch_split_grouped(const Dims& d, const PlanPtrs& p, SplitPlan plan, int act, int half,
                                 const void* recv, const void* w_home, const void* w_slot,
                                 const float* bias, void* y, void* z, cudaStream_t st) {
  SplitArgs a = {};
  a.T = d.N, a.columns = d.Hp, a.depth = d.H;
  a.half = half, a.act = act;
  a.tokens = plan.tokens;
  a.splits = plan.splits;
  a.stages = std::min(kSplitStages, kSplitRing / (2 * kPanelBytes + plan.tokens * 128));
  a.parts = 1;
  a.bias = bias;
  a.out = y;
  a.z = (uint16_t*)z;
  a.status = p.status;
  CUtensorMap tw, ts, tx;
  if (!encode_matrix(&tw, w_home, d.Hp, (int64_t)d.E * d.H, d.Hp, 64) ||
      !encode_matrix(&tx, recv, d.H, d.N, d.H, plan.tokens))
    return cudaErrorInvalidValue;
  ts = tw;
  if (w_slot != nullptr && d.B > 0 &&
      !encode_matrix(&ts, w_slot, d.Hp, (int64_t)d.R * d.B * d.H, d.Hp, 64))
    return cudaErrorInvalidValue;
  const int64_t CT = half ? (half + 63) / 64 : (d.Hp + 127) / 128;
  // work tiles: at most one a copy, and one a group
  const int64_t ctas = std::min<int64_t>(d.max_mtiles, std::min<int64_t>(d.N, d.max_groups)) * CT * plan.splits;
  if (ctas >= int64_t(1) << 31) return cudaErrorInvalidConfiguration;
  return launch_kind<kForward, true>(tw, ts, tx, a, p, ctas, st);
}

}  // namespace moonep
