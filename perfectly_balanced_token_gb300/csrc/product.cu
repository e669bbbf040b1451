// Products with bias, activation and residual in the epilogue, dense and over the plan's groups,
// and the dense product's gradients:
//
//   forward          z = x w + bias,  out = residual + act(z)
//   input gradient   d_x = d_z w^T
//   weight gradient  d_w (+)= x^T d_z
//
// One kernel, C[M x N] = A[M x K] . B[K x N] on 256-row tiles of a CTA pair (cta_group::2) or
// 128-row tiles of one CTA, 256 columns a tile:
//  * warp 0 feeds a ring of 64-deep stages by TMA, warp 1's elected lane issues the MMAs into one of
//    two accumulators in TMEM, warps 2..5 drain the other: bias, z, activation, residual and one
//    rounding happen in registers, so z and the activation never make a trip through memory that
//    the caller did not ask for.
//  * swiglu: a tile takes 128 gate columns and the 128 columns of the same numbers in the up half,
//    so one lane holds both factors of a value.  On a pair, the first CTA brings the gates and the
//    second the up columns of B; the MMA gives either CTA both for its rows.
//  * outputs leave by TMA stores of 32 rows x 128 bytes, staged in shared memory; their maps clip
//    what lies past the last row or column, so sizes need not divide the tile.  Rows of a group that
//    ends inside a tile are stored one by one, as the next group's rows follow.
//  * dense tiles are walked with a fixed stride, the plan's tiles claimed in order (tcgen05.cuh).
// What bounds it: the MMA rate and, at its full rate, the power limit.
#include <algorithm>
#include <type_traits>

#include "activation.cuh"
#include "ffn.h"
#include "tcgen05.cuh"

namespace moonep {

constexpr int kDepth = 64;          // of a stage: 64 bf16 = one 128-byte swizzle row
constexpr int kProductThreads = 192;
constexpr int kPanelBytes = 64 * 128;  // 64 rows of 64 bf16

enum Kind { kForward, kInputGrad, kWeightGrad };

template <bool PAIR>
struct ProductCfg {
  static constexpr int kStages = PAIR ? 6 : 4;
  static constexpr int kTileM = PAIR ? 256 : 128;
  static constexpr int kABytes = 128 * kDepth * 2;
  static constexpr int kBPanels = PAIR ? 2 : 4;  // of 64 columns, in one CTA
  static constexpr int kStageBytes = kABytes + kBPanels * kPanelBytes;
  static constexpr int kOutWarpBytes = 2 * 4096;  // two buffers of 32 rows x 128 bytes
  static constexpr int kOutBytes = 4 * kOutWarpBytes;
  static constexpr int kNumBars = 2 * kStages + 5 + 2 * kQueue;
  static constexpr int kBarBytes = kNumBars * 8 + 16 + 4 * kQueue;
  static constexpr int kSmem = kStages * kStageBytes + kOutBytes + 1024 + kBarBytes;
};
static_assert(ProductCfg<true>::kSmem <= 232448 && ProductCfg<false>::kSmem <= 232448,
              "shared memory of a CTA");

struct ProductArgs {
  int M, N, K;     // C's rows and columns, the depth; grouped: M rows of all groups together
  int wrows;       // grouped: rows of an expert's weight
  int act;         // Act
  int half;        // swiglu: N / 2, otherwise 0
  int f32, add;    // C in fp32; added into (both for outputs without groups)
  const float* bias;  // [N], grouped [E][N]; or null
  const uint16_t* residual;  // [M][out columns] or null
  uint16_t *out, *z;         // for rows stored one by one; z null if not asked for
  int has_z;
  int32_t* status;
};

struct ProductMaps {
  CUtensorMap a, b, b_slots, out, z, z_up;
};

template <bool PAIR>
struct Issue {  // the forms of one CTA and of a pair
  static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x,
                                              int y) {
    if (PAIR) tma_load_2d_pair(dst, m, bar, x, y);
    else tma_load_2d(dst, m, bar, x, y);
  }
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t i, bool acc) {
    if (PAIR) umma_bf16_pair(d, a, b, i, acc);
    else umma_bf16(d, a, b, i, acc);
  }
  static __device__ __forceinline__ void commit(uint32_t bar) {
    if (PAIR) umma_commit_pair_both(bar);
    else umma_commit(bar);
  }
};

// kind::f16: fp32 accumulator, bf16 operands; which of them run along M or N in memory
__host__ __device__ constexpr uint32_t product_idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Descriptor of the k-th 16 of a stage: rows of 128 bytes along the depth, or panels of 64 columns.
__device__ __forceinline__ uint64_t stage_desc(uint32_t at, int k, bool mn) {
  return mn ? sw128_desc(at + k * (16 * 128), kPanelBytes, 1024) : sw128_desc(at + k * 32, 16, 1024);
}

// A warp's two staging buffers of 32 rows x 128 bytes (128-byte swizzle) and the stores from them.
struct OutRing {
  uint8_t* base;
  int n, lane;
  // writes this lane's row (32 words) and stores the box at column x, row y
  __device__ __forceinline__ void put(const uint32_t (&v)[32], const CUtensorMap* m, int x, int y,
                                      bool add) {
    uint8_t* buf = base + (n & 1) * 4096;
    ++n;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    uint4* row = reinterpret_cast<uint4*>(buf + lane * 128);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      row[j ^ (lane & 7)] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      if (add)
        asm volatile(
            "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group"
            " [%0, {%1, %2}], [%3];" ::"l"((uint64_t)m), "r"(x), "r"(y), "r"(smem_u32(buf))
            : "memory");
      else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         (uint64_t)m),
                     "r"(x), "r"(y), "r"(smem_u32(buf))
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
};

// The first `cols` (a multiple of 8) of a row's 64 bf16 values.
__device__ __forceinline__ void put_row(const uint32_t (&v)[32], uint16_t* at, int cols) {
  uint4* p = reinterpret_cast<uint4*>(at);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (8 * j < cols) p[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// v += bias[0 .. 31], of which the first `cols` (a multiple of 8) are there; every lane has the same
__device__ __forceinline__ void add_bias(float (&v)[32], const float* bias, int cols) {
  const float4* b = reinterpret_cast<const float4*>(bias);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (4 * j < cols) {
      const float4 f = __ldg(b + j);
      v[4 * j] += f.x;
      v[4 * j + 1] += f.y;
      v[4 * j + 2] += f.z;
      v[4 * j + 3] += f.w;
    }
  }
}

__device__ __forceinline__ void add_residual(float (&v)[32], const uint16_t* at, int cols) {
  const uint4* p = reinterpret_cast<const uint4*>(at);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (8 * j < cols) {
      const uint4 r = __ldg(p + j);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * j + 2 * i] += __uint_as_float(w[i] << 16);
        v[8 * j + 2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}

// bf16 of v into the h-th half of p
template <int H>
__device__ __forceinline__ void pack32(uint32_t (&p)[32], const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    p[16 * H + i] = pack_bf16x2(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]));
}

__device__ __forceinline__ void load32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld_x32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 columns of a lane's row from TMEM to the output's values: z and, for swiglu, the up half of z
// packed into pz and pu on the way, the result in v.  x: the first column, cols: how many are left.
template <int H>
__device__ __forceinline__ void forward32(const ProductArgs& a, const float* bias,
                                          const uint16_t* residual, uint32_t taddr, int x, int cols,
                                          float (&v)[32], uint32_t (&pz)[32], uint32_t (&pu)[32]) {
  load32(taddr + 32 * H, v);
  x += 32 * H;
  cols -= 32 * H;
  if (bias != nullptr) add_bias(v, bias + x, cols);
  pack32<H>(pz, v);
  if (a.half) {
    float u[32];
    load32(taddr + 128 + 32 * H, u);
    if (bias != nullptr) add_bias(u, bias + a.half + x, cols);
    pack32<H>(pu, u);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = v[j] * sigmoid_f(v[j]) * u[j];
  } else if (a.act == kActRelu) {  // one loop for each, so that the choice is not made 32 times
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = act_value(kActRelu, v[j]);
  } else if (a.act == kActGelu) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = act_value(kActGelu, v[j]);
  } else if (a.act == kActSilu) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = act_value(kActSilu, v[j]);
  }
  if (residual != nullptr) add_residual(v, residual + x, cols);
}

template <bool PAIR, int KIND, bool DENSE>
__global__ void __launch_bounds__(kProductThreads, 1)
k_product(const __grid_constant__ ProductMaps tm, const __grid_constant__ ProductArgs a,
          const __grid_constant__ PlanPtrs p) {
  using Cfg = ProductCfg<PAIR>;
  using Op = Issue<PAIR>;
  constexpr int STAGES = Cfg::kStages;
  constexpr bool AMN = KIND == kWeightGrad;  // A = x^T: runs along M in memory
  constexpr bool BMN = KIND != kInputGrad;   // B = w^T there: runs along the depth
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* out_stage = smem + STAGES * Cfg::kStageBytes;  // 1024-aligned
  uint64_t* bars = (uint64_t*)(out_stage + Cfg::kOutBytes);
  uint32_t* tmem_slot = (uint32_t*)(bars + Cfg::kNumBars);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
  const uint32_t drain = bar0 + 8u * (2 * STAGES + 4);
  const PairQueue q{bar0 + 8u * (2 * STAGES + 5), bar0 + 8u * (2 * STAGES + 5 + kQueue),
                    (int32_t*)(tmem_slot + 2)};
  constexpr uint64_t kDrainNs = 200000000ull;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = PAIR ? pair_rank() : 0u;
  const bool leader = crank == 0;
  const int nwork = PAIR ? gridDim.x >> 1 : gridDim.x;   // pairs or CTAs
  const int work = PAIR ? blockIdx.x >> 1 : blockIdx.x;  // this one
  if (plan_failed(a.status)) return;  // uniform over the pair: before any barrier
  if (!DENSE && p.counters[MOONEP_CNT_TILE_ROWS] != Cfg::kTileM) return;
  const int NT = a.half ? (a.half + 127) / 128 : (a.N + 255) / 256;
  const int MT = DENSE ? (a.M + Cfg::kTileM - 1) / Cfg::kTileM : p.counters[MOONEP_CNT_MTILES];
  const int total = MT * NT;
  const int KB = (a.K + kDepth - 1) / kDepth;
  int32_t* sched = DENSE ? nullptr : p.sched + (PAIR ? 0 : 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), PAIR ? 8 : 4);  // four epilogue warps in each CTA
    }
    mbar_init(drain, 1);
    if (!DENSE) queue_init(q, PAIR ? kQueueConsumers : kQueueConsumersSolo);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm.a);
    prefetch_tmap(&tm.b);
    prefetch_tmap(&tm.out);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (PAIR) pair_sync();  // the peer's barriers are initialised before anything reaches them
  const uint32_t tmem_base = *tmem_slot;

  auto fail = [&]() {
    *abort_flag = 1;
    set_error(a.status, MOONEP_ERR_TIMEOUT);
  };
  // tile t's rows (first, number, weight and rank as the plan lists them) and first column
  auto tile = [&](int t, MTile& mt, int& n0) {
    if (DENSE) {
      mt.row0 = (t / NT) * Cfg::kTileM;
      mt.rows = min(Cfg::kTileM, a.M - mt.row0);
      mt.wsel = 0;
    } else {
      mt = p.mtiles[t / NT];
    }
    n0 = (t % NT) * (a.half ? 128 : 256);
  };

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      int next = 0;
      if (!DENSE && leader) next = atomicAdd(sched, 1);
      for (int i = 0; ok; ++i) {
        int t;
        if (DENSE) {
          t = work + i * nwork;
          if (t >= total) break;
        } else if (leader) {  // hand the claimed tile out, claim the one after it
          t = next >= total ? -1 : next;
          if (!queue_push(q, i, t, abort_flag, PAIR)) { ok = false; break; }
          if (t >= 0) next = atomicAdd(sched, 1);
        } else if (!queue_take(q, i, false, true, t, abort_flag)) {
          ok = false;
          break;
        }
        if (t < 0) break;
        MTile mt;
        int n0;
        tile(t, mt, n0);
        const CUtensorMap* bmap = mt.wsel >= 0 ? &tm.b : &tm.b_slots;
        const int wrow = (mt.wsel >= 0 ? mt.wsel : (-1 - mt.wsel)) * a.wrows;
        const int row0 = mt.row0 + (int)crank * 128;
        // this CTA's columns of B: panel j begins at col0 + 64 j, or col1 + 64 (j - 2)
        const int col0 = PAIR ? (a.half ? (int)crank * a.half + n0 : n0 + (int)crank * 128) : n0;
        const int col1 = a.half ? a.half + n0 : n0 + 128;  // (one CTA only)
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(empty(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t fb = PAIR ? pair_map(full(stage), 0) : full(stage);
          if (leader) mbar_expect_tx(full(stage), (PAIR ? 2 : 1) * Cfg::kStageBytes);
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
          const uint32_t sb = sa + Cfg::kABytes;
          const int k0 = kb * kDepth;
          if (AMN) {
            Op::load(sa, &tm.a, fb, row0, k0);
            Op::load(sa + kPanelBytes, &tm.a, fb, row0 + 64, k0);
          } else {
            Op::load(sa, &tm.a, fb, k0, row0);
          }
          if (BMN) {
            Op::load(sb, bmap, fb, col0, wrow + k0);
            Op::load(sb + kPanelBytes, bmap, fb, col0 + 64, wrow + k0);
            if (!PAIR) {
              Op::load(sb + 2 * kPanelBytes, bmap, fb, col1, wrow + k0);
              Op::load(sb + 3 * kPanelBytes, bmap, fb, col1 + 64, wrow + k0);
            }
          } else {
            Op::load(sb, bmap, fb, k0, wrow + col0);
            if (!PAIR) Op::load(sb + 2 * kPanelBytes, bmap, fb, k0, wrow + col1);
          }
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!DENSE && leader) queue_finish(sched, sched + 1, nwork);
      if (ok) {
        for (int i = 0; i < STAGES; ++i) {  // every fill released: no commit still in flight
          if (!mbar_wait(empty(stage), phase ^ 1u, nullptr)) { ok = false; break; }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) set_error(a.status, MOONEP_ERR_TIMEOUT);
      } else {
        fail();
        if (leader) {  // wait (time-bounded) for the copies in flight
          for (int i = 0; i < min(issued, STAGES); ++i) {
            if (stage == 0) { stage = STAGES - 1; phase ^= 1u; } else { --stage; }
            mbar_wait(full(stage), phase, nullptr, kDrainNs);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (leader only) ----------------
    if (leader && elect_one()) {
      constexpr uint32_t idesc = product_idesc(Cfg::kTileM, 256, AMN, BMN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        int t;
        if (DENSE) {
          if (work + i * nwork >= total) break;
        } else {
          if (!queue_take(q, i, true, true, t, abort_flag)) { ok = false; break; }
          if (t < 0) break;
        }
        if (!mbar_wait(tempty(acc), acc_phase ^ 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t dtm = tmem_base + (uint32_t)(acc * 256);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(full(stage), phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
          const uint32_t sb = sa + Cfg::kABytes;
#pragma unroll
          for (int k = 0; k < kDepth / 16; ++k)
            Op::mma(dtm, stage_desc(sa, k, AMN), stage_desc(sb, k, BMN), idesc, (kb | k) != 0);
          Op::commit(empty(stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        Op::commit(tfull(acc));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (!ok) {
        fail();
        if (PAIR) umma_commit_pair_self(drain);
        else umma_commit(drain);
        mbar_wait(drain, 0, nullptr);
      }
    }
  } else {
    // ---------------- epilogue (warps 2..5, both CTAs) ----------------
    const int qw = warp & 3;  // TMEM lanes 32 qw .. are this warp's rows
    OutRing ring{out_stage + qw * Cfg::kOutWarpBytes, 0, lane};
    const int ocols = a.half ? a.half : a.N;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int i = 0;; ++i) {
      int t;
      if (DENSE) {
        t = work + i * nwork;
        if (t >= total) break;
      } else {
        if (!queue_take_warp(q, i, leader, t, abort_flag)) {
          if (lane == 0) fail();
          break;
        }
        if (t < 0) break;
      }
      MTile mt;
      int n0;
      tile(t, mt, n0);
      const int first = (int)crank * 128 + qw * 32;  // this warp's first row of the tile
      const int row = mt.row0 + first + lane;        // this lane's row of C
      const bool valid = first + lane < mt.rows;
      const bool whole = DENSE || first + 32 <= mt.rows;  // stored as boxes
      const float* bias = a.bias;
      if (!DENSE && bias != nullptr) {
        int e = mt.wsel >= 0 ? mt.wsel : p.slot_expert[-1 - mt.wsel];
        bias += (size_t)e * a.N;
      }
      // (lanes past the last row read that one: the warp stays together)
      const uint16_t* residual =
          a.residual != nullptr ? a.residual + (size_t)min(row, a.M - 1) * ocols : nullptr;
      const bool ok = mbar_wait(tfull(acc), acc_phase, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((uint32_t)(qw * 32) << 16) + (uint32_t)(acc * 256);
      auto put = [&](const uint32_t (&v)[32], const CUtensorMap* m, int x, uint16_t* plain, int pitch,
                     int cols) {
        if (whole) ring.put(v, m, x, mt.row0 + first, false);
        else if (valid) put_row(v, plain + (size_t)row * pitch + x, cols);
      };
      // (a warp all of whose rows lie past the last one has nothing to store)
      const int chunks = first < mt.rows ? (a.half ? 2 : 4) : 0;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int x = n0 + 64 * c;  // first output column
        const int cols = min(64, ocols - x);
        if (cols <= 0) break;
        __syncwarp();
        uint32_t pz[32], pu[32], po[32];
        float v[32];
        auto half = [&](auto h) {
          constexpr int H = decltype(h)::value;
          if (KIND == kForward)
            forward32<H>(a, bias, residual, tbase + 64 * c, x, cols, v, pz, pu);
          else
            load32(tbase + 64 * c + 32 * H, v);
          if (DENSE && a.f32) {  // 32 columns a store
#pragma unroll
            for (int j = 0; j < 32; ++j) po[j] = __float_as_uint(v[j]);
            if (32 * H < cols) ring.put(po, &tm.out, x + 32 * H, mt.row0 + first, a.add);
          } else {
            pack32<H>(po, v);
          }
        };
        half(std::integral_constant<int, 0>());
        half(std::integral_constant<int, 1>());
        if (!(DENSE && a.f32)) put(po, &tm.out, x, a.out, ocols, cols);
        if (KIND == kForward && a.has_z) {
          put(pz, &tm.z, x, a.z, a.N, cols);
          if (a.half) put(pu, &tm.z_up, x, a.z + a.half, a.N, cols);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_remote(pair_map(tempty(acc), 0));
        else mbar_arrive(tempty(acc));
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // this warp's stores
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) pair_sync();  // both CTAs done with TMEM and with each other's barriers
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, 512);
    else tmem_dealloc(tmem_base, 512);
  }
}

// -- host side ------------------------------------------------------------------
// A row-major matrix [rows][cols] with `pitch` elements a row; boxes of 128 bytes x `box` rows,
// 128-byte swizzle.
static bool encode(CUtensorMap* m, const void* base, int cols, int64_t rows, int64_t pitch, int box,
                   bool f32 = false) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const int size = f32 ? 4 : 2;
  cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t stride[1] = {(cuuint64_t)(pitch * size)};
  cuuint32_t b[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box};
  cuuint32_t one[2] = {1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dim, stride, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PAIR, int KIND, bool DENSE>
static cudaError_t launch_one(const ProductMaps& tm, const ProductArgs& a, const PlanPtrs& p,
                              int64_t tiles, cudaStream_t st) {
  using Cfg = ProductCfg<PAIR>;
  constexpr int CG = PAIR ? 2 : 1;
  auto* kernel = k_product<PAIR, KIND, DENSE>;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = CG;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kProductThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = PAIR ? 1 : 0;
  static PerDevice kept;
  int most = 0;  // CTAs (pairs) that run at once
  const cudaError_t e = kept(&most, [&](int* found) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    if (!PAIR) return *found = sm_count_gemm(), cudaSuccess;
    cfg.gridDim = dim3(2 * std::max(1, sm_count_gemm() / 2));
    int n = 0;
    const cudaError_t e2 = cudaOccupancyMaxActiveClusters(&n, (void*)kernel, &cfg);
    *found = std::max(1, n);
    return e2;
  });
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(CG * (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, tiles)));
  void* args[] = {const_cast<ProductMaps*>(&tm), const_cast<ProductArgs*>(&a),
                  const_cast<PlanPtrs*>(&p)};
  return cudaLaunchKernelExC(&cfg, (const void*)kernel, args);
}

static int64_t tiles_of(int64_t M, int N, int half, int rows) {
  return ((M + rows - 1) / rows) * (half ? (half + 127) / 128 : (N + 255) / 256);
}

cudaError_t launch_linear(const LinearDims& d, const void* x, const void* w, const float* bias,
                          const void* residual, void* out, void* z, int32_t* status, cudaStream_t st,
                          int* launches) {
  ProductMaps tm;
  const int ocols = d.half ? d.half : d.N;
  if (!encode(&tm.a, x, d.K, d.T, d.K, 128) || !encode(&tm.b, w, d.N, d.K, d.N, 64) ||
      !encode(&tm.out, out, ocols, d.T, ocols, 32, d.f32))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  tm.z = tm.z_up = tm.out;
  if (z != nullptr) {  // the halves have maps of their own, so that either is clipped at its end
    if (!encode(&tm.z, z, ocols, d.T, d.N, 32)) return cudaErrorInvalidValue;
    if (d.half && !encode(&tm.z_up, (uint16_t*)z + d.half, ocols, d.T, d.N, 32))
      return cudaErrorInvalidValue;
  }
  ProductArgs a = {};
  a.M = d.T, a.N = d.N, a.K = d.K;
  a.act = d.act, a.half = d.half, a.f32 = d.f32;
  a.bias = bias;
  a.residual = (const uint16_t*)residual;
  a.has_z = z != nullptr;
  a.status = status;
  *launches += 1;
  return launch_one<true, kForward, true>(tm, a, PlanPtrs{}, tiles_of(d.T, d.N, d.half, 256), st);
}

cudaError_t launch_linear_dx(const LinearDims& d, const void* d_z, const void* w, void* d_x,
                             int32_t* status, cudaStream_t st, int* launches) {
  ProductMaps tm;
  if (!encode(&tm.a, d_z, d.N, d.T, d.N, 128) || !encode(&tm.b, w, d.N, d.K, d.N, 128) ||
      !encode(&tm.out, d_x, d.K, d.T, d.K, 32))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  tm.z = tm.z_up = tm.out;
  ProductArgs a = {};
  a.M = d.T, a.N = d.K, a.K = d.N;
  a.status = status;
  *launches += 1;
  return launch_one<true, kInputGrad, true>(tm, a, PlanPtrs{}, tiles_of(d.T, d.K, 0, 256), st);
}

cudaError_t launch_linear_dw(const LinearDims& d, const void* x, const void* d_z, float* d_w,
                             int add, int32_t* status, cudaStream_t st, int* launches) {
  ProductMaps tm;
  if (!encode(&tm.a, x, d.K, d.T, d.K, 64) || !encode(&tm.b, d_z, d.N, d.T, d.N, 64) ||
      !encode(&tm.out, d_w, d.N, d.K, d.N, 32, true))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  tm.z = tm.z_up = tm.out;
  ProductArgs a = {};
  a.M = d.K, a.N = d.N, a.K = d.T;
  a.f32 = 1, a.add = add;
  a.status = status;
  *launches += 1;
  return launch_one<true, kWeightGrad, true>(tm, a, PlanPtrs{}, tiles_of(d.K, d.N, 0, 256), st);
}

cudaError_t launch_grouped_gemm_act(const Dims& d, const PlanPtrs& p, int act, const void* recv,
                                    const void* w_home, const void* w_slot, const float* bias, void* y,
                                    void* z, cudaStream_t st, int* launches) {
  ProductMaps tm;
  const int half = act == kActSwiglu ? d.Hp / 2 : 0;
  const int ocols = half ? half : d.Hp;
  const bool slots = w_slot != nullptr && d.B > 0;
  if (!encode(&tm.a, recv, d.H, d.N, d.H, 128) ||
      !encode(&tm.b, w_home, d.Hp, (int64_t)d.E * d.H, d.Hp, 64) ||
      !encode(&tm.out, y, ocols, d.N, ocols, 32))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  if (slots && !encode(&tm.b_slots, w_slot, d.Hp, (int64_t)d.R * d.B * d.H, d.Hp, 64))
    return cudaErrorInvalidValue;
  tm.z = tm.z_up = tm.out;
  if (z != nullptr) {
    if (!encode(&tm.z, z, ocols, d.N, d.Hp, 32)) return cudaErrorInvalidValue;
    if (half && !encode(&tm.z_up, (uint16_t*)z + half, ocols, d.N, d.Hp, 32))
      return cudaErrorInvalidValue;
  }
  ProductArgs a = {};
  a.M = d.N, a.N = d.Hp, a.K = d.H, a.wrows = d.H;
  a.act = act, a.half = half;
  a.bias = bias;
  a.out = (uint16_t*)y;
  a.z = (uint16_t*)z;
  a.has_z = z != nullptr;
  a.status = p.status;
  // with the height left to the plan both are launched; the one it did not choose returns at once
  const int64_t tiles = (int64_t)d.max_mtiles * (half ? (half + 127) / 128 : (d.Hp + 255) / 256);
  if (d.tile_m != 2 * kMmaM) {
    const cudaError_t e = launch_one<false, kForward, false>(tm, a, p, tiles, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  if (d.tile_m != kMmaM) {
    const cudaError_t e = launch_one<true, kForward, false>(tm, a, p, tiles, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  return cudaSuccess;
}

}  // namespace moonep
