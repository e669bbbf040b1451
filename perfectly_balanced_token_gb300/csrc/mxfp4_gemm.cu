// Grouped product on MXFP4 operands with the block-scaled tensor-core instruction.
//
//   y[i][n] = sum_k 2^(sa[i][k/32] - 127) a[i][k] 2^(sb[n][k/32] - 127) b[n][k]
//
// a: the E2M1 codes of recv, b: those of the transposed expert weights, so both
// are K-major, which 4-bit operands have to be.  tcgen05.mma kind::mxf4 multiplies
// 64 codes of K at a time and applies the two scales of each row and column
// inside the instruction; accumulation is fp32 in TMEM.
//
// Shape of the work: the plan's work tiles as in the bf16 product, 256 rows on a
// CTA pair or 128 rows on one CTA, times 256 columns.  A stage holds 256 values
// of K: 128-byte rows, as the bf16 kernels' 64 values are, so the bytes a stage
// brings in are the same and the MMA work is four times as much in the same time.
//
// Scales: the instruction reads them from TMEM, where lane l of column j holds the
// four scale bytes (128 values of K) of row 32 j + l, once for each of the four
// lane groups.  A warp for each 128 rows loads 16 scale bytes a row (512 of K) one
// load ahead, writes them to the stage in that order (one 16-byte store a lane
// and 128 of K) and arrives on the stage's barrier next to the TMA copies; the
// MMA thread moves them to TMEM with tcgen05.cp, which the tensor core runs in
// order with the products.
#include <algorithm>

#include "ops.h"
#include "tcgen05.cuh"

namespace moonep {

constexpr int kMxK = 256;     // K per stage: 128 bytes of codes a row
constexpr int kMxUmmaK = 64;  // K of one MMA
constexpr int kMxBN = 256;    // columns of a work tile

// Per CTA: 128 rows of A, kMxBN / CG of the weights' rows, and the scales of its
// rows and of all kMxBN columns.
template <int CG>
struct MxCfg {
  static constexpr int kABytes = kMmaM * kMxK / 2;
  static constexpr int kBRows = kMxBN / CG;
  static constexpr int kBBytes = kBRows * kMxK / 2;
  static constexpr int kAtoms = 1 + kMxBN / 128;  // 128-row scale blocks: A, then B
  static constexpr int kScaleBytes = (kMxK / 128) * kAtoms * 512;
  static constexpr int kStageBytes = kABytes + kBBytes + kScaleBytes;
  static constexpr int kStages = CG == 2 ? 5 : 4;
  static constexpr int kOutBufs = CG == 2 ? 2 : 1;  // 32 x 64 bf16 staging buffers a warp
  static constexpr int kOutWarpBytes = kOutBufs * 4096;
  static constexpr int kOutBytes = 4 * kOutWarpBytes;
  static constexpr int kThreads = 192 + 32 * kAtoms;
  static constexpr int kConsumers = CG == 2 ? 2 * (5 + kAtoms) : 5 + kAtoms;
  static constexpr int kNumBars = 2 * kStages + 3 + 2 * kQueue;
  static constexpr int kSmem =
      kStages * kStageBytes + kOutBytes + 1024 + kNumBars * 8 + 16 + 4 * kQueue;
};
static_assert(MxCfg<1>::kSmem <= 232448 && MxCfg<2>::kSmem <= 232448, "shared memory of a CTA");
static_assert(MxCfg<1>::kScaleBytes % 1024 == 0, "stages stay 1024-byte aligned");

constexpr uint32_t kMxTmemCols = 512;
constexpr uint32_t kMxScaleCol = kMxBN;  // A: 2 x 4 columns, then B: 2 x 8

// Instruction descriptor, kind::mxf4: A and B E2M1 (bits 7-9 and 10-11 = 1), both
// K-major, N >> 3 in bits 17-22, E8M0 scales (bit 23), M >> 7 in bits 27-28; the
// half of the scale word in use (0 or 2) in bits 4-5 (B) and 29-30 (A).
constexpr uint32_t mx_idesc(int M, int N, int half) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27) | ((uint32_t)half << 4) | ((uint32_t)half << 29);
}

template <int CG>
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (CG == 2) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  }
}

// 512 bytes of scales (32 rows of 16) from shared memory to four TMEM columns,
// repeated for the four lane groups; in both CTAs of a pair, each from its own.
template <int CG>
__device__ __forceinline__ void mx_copy_scales(uint32_t tmem, uint32_t saddr) {
  // no swizzle: 8-row groups of 16-byte rows 128 bytes apart
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
                        ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}

struct MxScales {
  const uint8_t *a, *home, *slot;
  int pitch;                  // bytes a row
  int a_rows, home_rows, slot_rows;
};

template <int CG>
__global__ void __launch_bounds__(MxCfg<CG>::kThreads, 1)
k_mxfp4_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_wh,
             const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_y,
             MxScales sc, int K, int N, PlanPtrs p, uint16_t* __restrict__ y) {
  using Cfg = MxCfg<CG>;
  constexpr int STAGES = Cfg::kStages;
  constexpr bool kPair = CG == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* out_stage = smem + STAGES * Cfg::kStageBytes;
  uint64_t* bars = (uint64_t*)(out_stage + Cfg::kOutBytes);
  uint32_t* tmem_slot = (uint32_t*)(bars + Cfg::kNumBars);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t tfull = bar0 + 8u * (2 * STAGES);
  const uint32_t tempty = tfull + 8u;
  const uint32_t drain = tfull + 16u;
  const PairQueue q{tfull + 24u, tfull + 24u + 8u * kQueue, (int32_t*)(tmem_slot + 2)};
  constexpr uint64_t kDrainNs = 200000000ull;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = kPair ? pair_rank() : 0;
  const bool leader = crank == 0;
  if (plan_failed(p.status)) return;  // uniform over the pair: before any barrier
  if (p.counters[MOONEP_CNT_TILE_ROWS] != CG * kMmaM) return;
  const int NT = (N + kMxBN - 1) / kMxBN;
  const int total = p.counters[MOONEP_CNT_MTILES] * NT;
  const int KB = (K + kMxK - 1) / kMxK;
  int32_t* sched = p.sched + (kPair ? 0 : 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1 + CG * Cfg::kAtoms);  // the TMA bytes and every scale warp
      mbar_init(empty(s), 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 4 * CG);
    mbar_init(drain, 1);
    queue_init(q, Cfg::kConsumers);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_wh);
    prefetch_tmap(&tm_ws);
    prefetch_tmap(&tm_y);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(smem_u32(tmem_slot), kMxTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), kMxTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (kPair) pair_sync();  // the peer's barriers are ready
  const uint32_t tmem_base = *tmem_slot;
  auto fail = [&]() {
    *abort_flag = 1;
    set_error(p.status, MOONEP_ERR_TIMEOUT);
  };

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      int next = leader ? atomicAdd(sched, 1) : 0;  // claimed one item ahead
      for (int i = 0; ok; ++i) {
        int t;
        if (leader) {
          t = next >= total ? -1 : next;
          if (!queue_push(q, i, t, abort_flag, kPair)) { ok = false; break; }
          if (t >= 0) next = atomicAdd(sched, 1);
        } else if (!queue_take(q, i, false, true, t, abort_flag)) {
          ok = false;
          break;
        }
        if (t < 0) break;
        const MTile mt = p.mtiles[t / NT];
        const int n0 = (t % NT) * kMxBN + (int)crank * Cfg::kBRows;
        const CUtensorMap* wmap = mt.wsel >= 0 ? &tm_wh : &tm_ws;
        const int wrow = (mt.wsel >= 0 ? mt.wsel : (-1 - mt.wsel)) * N + n0;
        const int row0 = mt.row0 + (int)crank * kMmaM;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(empty(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
          if (leader) mbar_expect_tx(full(stage), CG * (Cfg::kABytes + Cfg::kBBytes));
          if constexpr (kPair) {
            const uint32_t fb = pair_map(full(stage), 0);
            tma_load_2d_pair(sa, &tm_a, fb, kb * (kMxK / 2), row0);
            tma_load_2d_pair(sa + Cfg::kABytes, wmap, fb, kb * (kMxK / 2), wrow);
          } else {
            tma_load_2d(sa, &tm_a, full(stage), kb * (kMxK / 2), row0);
            tma_load_2d(sa + Cfg::kABytes, wmap, full(stage), kb * (kMxK / 2), wrow);
          }
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (leader) queue_finish(sched, sched + 1, gridDim.x / CG);
      if (ok) {
        for (int i = 0; i < STAGES; ++i) {  // every fill released: no commit still in flight
          if (!mbar_wait(empty(stage), phase ^ 1u, nullptr)) { ok = false; break; }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) set_error(p.status, MOONEP_ERR_TIMEOUT);
      } else {
        fail();
        if (leader) {  // the copies in flight complete on the leader's barriers
          for (int i = 0; i < min(issued, STAGES); ++i) {
            if (stage == 0) { stage = STAGES - 1; phase ^= 1u; } else { --stage; }
            mbar_wait(full(stage), phase, nullptr, kDrainNs);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (leader only) ----------------
    if (leader && lane == 0) {
      constexpr uint32_t idesc[2] = {mx_idesc(CG * kMmaM, kMxBN, 0), mx_idesc(CG * kMmaM, kMxBN, 2)};
      const uint32_t sfa = tmem_base + kMxScaleCol, sfb = sfa + 8;
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        int t;
        if (!queue_take(q, i, true, true, t, abort_flag)) { ok = false; break; }
        if (t < 0) break;
        if (!mbar_wait_cluster(tempty, acc_phase ^ 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_cluster(full(stage), phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
          const uint32_t sb = sa + Cfg::kABytes;
          const uint32_t ss = sb + Cfg::kBBytes;
#pragma unroll
          for (int c = 0; c < kMxK / 128; ++c) {
            const uint32_t src = ss + c * Cfg::kAtoms * 512;
            mx_copy_scales<CG>(sfa + c * 4, src);
            mx_copy_scales<CG>(sfb + c * 8, src + 512);
            mx_copy_scales<CG>(sfb + c * 8 + 4, src + 1024);
          }
          const int steps = min(kMxK, K - kb * kMxK) / kMxUmmaK;
#pragma unroll
          for (int k = 0; k < kMxK / kMxUmmaK; ++k)
            if (k < steps)
              mx_mma<CG>(tmem_base, sw128_desc(sa + k * (kMxUmmaK / 2), 16, 1024),
                         sw128_desc(sb + k * (kMxUmmaK / 2), 16, 1024), idesc[k & 1],
                         sfa + (k >> 1) * 4, sfb + (k >> 1) * 8, (kb | k) != 0);
          if constexpr (kPair) umma_commit_pair_both(empty(stage));
          else umma_commit(empty(stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if constexpr (kPair) umma_commit_pair_both(tfull);
        else umma_commit(tfull);
        acc_phase ^= 1u;
      }
      if (!ok) {
        fail();
        if constexpr (kPair) umma_commit_pair_self(drain);
        else umma_commit(drain);
        mbar_wait(drain, 0, nullptr);
      }
    }
  } else if (warp < 6) {
    // ---------------- epilogue ----------------
    const int qw = warp & 3;
    int nstore = 0;
    uint32_t acc_phase = 0;
    for (int i = 0;; ++i) {
      int t;
      if (!queue_take_warp(q, i, leader, t, abort_flag)) {
        if (lane == 0) fail();
        break;
      }
      if (t < 0) break;
      const MTile mt = p.mtiles[t / NT];
      const int n0 = (t % NT) * kMxBN;
      if (!__all_sync(0xffffffffu, mbar_wait(tfull, acc_phase, abort_flag))) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const int wrow0 = (int)crank * kMmaM + qw * 32;  // this warp's first row of the tile
      const uint32_t tbase = tmem_base + ((uint32_t)(qw * 32) << 16);
      const bool whole = wrow0 + 32 <= mt.rows;  // all 32 rows inside the group
      const bool valid = wrow0 + lane < mt.rows;
      uint16_t* yrow = y + (size_t)(mt.row0 + wrow0 + lane) * N + n0;
#pragma unroll 1
      for (int c = 0; c < kMxBN / 64 && n0 + c * 64 < N; ++c) {  // N is a multiple of 64
        uint32_t lo[32], hi[32];
        tmem_ld_x32(tbase + c * 64, lo);
        tmem_ld_x32(tbase + c * 64 + 32, hi);
        tmem_ld_wait();
        uint4 o[8];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          o[v] = make_uint4(pack_bf16x2(lo[8 * v], lo[8 * v + 1]), pack_bf16x2(lo[8 * v + 2], lo[8 * v + 3]),
                            pack_bf16x2(lo[8 * v + 4], lo[8 * v + 5]), pack_bf16x2(lo[8 * v + 6], lo[8 * v + 7]));
          o[4 + v] = make_uint4(pack_bf16x2(hi[8 * v], hi[8 * v + 1]), pack_bf16x2(hi[8 * v + 2], hi[8 * v + 3]),
                                pack_bf16x2(hi[8 * v + 4], hi[8 * v + 5]), pack_bf16x2(hi[8 * v + 6], hi[8 * v + 7]));
        }
        if (whole) {
          // staged with the 128-byte swizzle, so that the lanes of a store phase hit
          // distinct bank groups, and written by one TMA store
          uint8_t* buf = out_stage + qw * Cfg::kOutWarpBytes + (nstore % Cfg::kOutBufs) * 4096;
          if (lane == 0)
            asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(Cfg::kOutBufs - 1) : "memory");
          __syncwarp();
          uint4* rowp = reinterpret_cast<uint4*>(buf + lane * 128);
#pragma unroll
          for (int v = 0; v < 8; ++v) rowp[v ^ (lane & 7)] = o[v];
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                    (uint64_t)&tm_y),
                "r"(n0 + c * 64), "r"(mt.row0 + wrow0), "r"(smem_u32(buf))
                : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          ++nstore;
        } else if (valid) {  // rows past the group's end are the next group's
#pragma unroll
          for (int v = 0; v < 8; ++v) reinterpret_cast<uint4*>(yrow + c * 64)[v] = o[v];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_remote(pair_map(tempty, 0));
        else mbar_arrive(tempty);
      }
      acc_phase ^= 1u;
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  } else {
    // ---------------- scales: 128 rows of A or 128 columns of B each ----------------
    const int atom = warp - 6;
    const int KG = sc.pitch / 16;  // loads a row: 16 scale bytes, two stages
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      int t;
      if (!queue_take_warp(q, i, leader, t, abort_flag)) { ok = false; break; }
      if (t < 0) break;
      const MTile mt = p.mtiles[t / NT];
      const uint8_t* src;
      int first, rows;
      if (atom == 0) {
        src = sc.a, rows = sc.a_rows;
        first = mt.row0 + (int)crank * kMmaM;
      } else {
        const bool home = mt.wsel >= 0;
        src = home ? sc.home : sc.slot, rows = home ? sc.home_rows : sc.slot_rows;
        first = (home ? mt.wsel : -1 - mt.wsel) * N + (t % NT) * kMxBN + (atom - 1) * 128;
      }
      // rows past the group, the matrix or the tensor feed results that are not
      // stored: any scale in range will do
      const uint4* row[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        row[j] = reinterpret_cast<const uint4*>(
            src + (size_t)min(first + 32 * j + lane, rows - 1) * sc.pitch);
      uint4 now[4], then[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) now[j] = __ldg(row[j]);
      for (int g = 0; ok && g < KG; ++g) {
        if (g + 1 < KG) {
#pragma unroll
          for (int j = 0; j < 4; ++j) then[j] = __ldg(row[j] + g + 1);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (2 * g + h >= KB) break;
          if (!__all_sync(0xffffffffu, mbar_wait(empty(stage), phase ^ 1u, abort_flag))) {
            ok = false;
            break;
          }
          uint4* dst = reinterpret_cast<uint4*>(smem + stage * Cfg::kStageBytes + Cfg::kABytes +
                                                Cfg::kBBytes + atom * 512) + lane;
          if (h == 0) {
            dst[0] = make_uint4(now[0].x, now[1].x, now[2].x, now[3].x);
            dst[Cfg::kAtoms * 32] = make_uint4(now[0].y, now[1].y, now[2].y, now[3].y);
          } else {
            dst[0] = make_uint4(now[0].z, now[1].z, now[2].z, now[3].z);
            dst[Cfg::kAtoms * 32] = make_uint4(now[0].w, now[1].w, now[2].w, now[3].w);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair) mbar_arrive_remote(pair_map(full(stage), 0));
            else mbar_arrive(full(stage));
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) now[j] = then[j];
      }
    }
    if (!ok && lane == 0) fail();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) pair_sync();  // both CTAs done with TMEM and each other's barriers
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, kMxTmemCols);
    else tmem_dealloc(tmem_base, kMxTmemCols);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Codes [rows][bytes], box of box_rows rows of 128 bytes, 128-byte swizzle; what
// lies past a row's or the tensor's end reads as zeros.
static bool encode_codes(CUtensorMap* m, const void* base, uint64_t bytes, uint64_t rows,
                         uint32_t box_rows) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t gdim[2] = {bytes, rows};
  cuuint64_t gstride[1] = {bytes};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y bf16 [rows][N], store boxes of 32 rows by 64 columns.
static bool encode_out(CUtensorMap* m, const void* base, uint64_t N, uint64_t rows) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t gdim[2] = {N, rows};
  cuuint64_t gstride[1] = {N * 2};
  cuuint32_t box[2] = {64, 32};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG>
static cudaError_t launch_mx(const Dims& d, const PlanPtrs& p, const CUtensorMap& ta,
                             const uint8_t* home, const uint8_t* slot, const CUtensorMap& ty,
                             const MxScales& sc, uint16_t* y, cudaStream_t st) {
  using Cfg = MxCfg<CG>;
  CUtensorMap twh, tws;
  if (!encode_codes(&twh, home, d.H / 2, (uint64_t)sc.home_rows, Cfg::kBRows) ||
      !encode_codes(&tws, slot, d.H / 2, (uint64_t)sc.slot_rows, Cfg::kBRows))
    return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static int grid = 0;
  if (grid == 0) {
    cudaError_t e = cudaFuncSetAttribute(k_mxfp4_gemm<CG>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    int n = sm_count_gemm();
    if (CG == 2) {  // one CTA pair per co-resident cluster
      cfg.gridDim = dim3(2 * std::max(1, n / 2));
      e = cudaOccupancyMaxActiveClusters(&n, (void*)k_mxfp4_gemm<CG>, &cfg);
      if (e != cudaSuccess) return e;
    }
    grid = CG * std::max(1, n);
  }
  const long long items = (long long)d.max_mtiles * ((d.Hp + kMxBN - 1) / kMxBN);
  cfg.gridDim = dim3((unsigned)std::min<long long>(grid, CG * items));
  return cudaLaunchKernelEx(&cfg, k_mxfp4_gemm<CG>, ta, twh, tws, ty, sc, d.H, d.Hp, p, y);
}

cudaError_t launch_mxfp4_grouped_gemm(const Dims& d, const PlanPtrs& p, const uint8_t* a,
                                      const uint8_t* a_scales, const uint8_t* home,
                                      const uint8_t* home_scales, const uint8_t* slot,
                                      const uint8_t* slot_scales, void* y, cudaStream_t st,
                                      int* launches) {
  const bool slots = slot != nullptr && d.B > 0;
  const MxScales sc{a_scales, home_scales, slots ? slot_scales : home_scales,
                    MOONEP_MXFP4_SCALE_PITCH(d.H), d.R * d.C, d.E * d.Hp,
                    slots ? d.R * d.B * d.Hp : d.E * d.Hp};
  const uint8_t* sl = slots ? slot : home;
  CUtensorMap ta, ty;
  if (!encode_codes(&ta, a, d.H / 2, (uint64_t)d.R * d.C, kMmaM) ||
      !encode_out(&ty, y, (uint64_t)d.Hp, (uint64_t)d.R * d.C))
    return cudaErrorInvalidValue;
  // the plan's tile height is on the device: the variant it did not choose
  // returns at once (as in the bf16 product)
  if (d.tile_m != 2 * kMmaM) {
    const cudaError_t e = launch_mx<1>(d, p, ta, home, sl, ty, sc, (uint16_t*)y, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  if (d.tile_m != kMmaM) {
    const cudaError_t e = launch_mx<2>(d, p, ta, home, sl, ty, sc, (uint16_t*)y, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  return cudaSuccess;
}

}  // namespace moonep
