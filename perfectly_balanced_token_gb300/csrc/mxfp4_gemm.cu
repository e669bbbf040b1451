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
// four scale bytes (128 values of K) of row 32 j + l, repeated for the four lane
// groups.  One thread has TMA bring 16 scale bytes (512 of K) of every row into a
// ring of its own; four warps, one for each lane group, read them as 16 bytes a
// row, which the order of registers turns around, and store them to TMEM.  (The
// other way into TMEM, tcgen05.cp, measured 100 clocks for each 512 bytes, 600 for
// a stage's six, where the stage's products take 512.)
//
// TMEM: two accumulators of 256 columns that share 128, and 5 x 24 columns of
// scales.  The epilogue takes the shared columns first, so the next tile's
// products start when half of a tile is in registers.
#include <algorithm>

#include "ops.h"
#include "tcgen05.cuh"

namespace moonep {

constexpr int kMxK = 256;     // K per stage: 128 bytes of codes a row
constexpr int kMxUmmaK = 64;  // K of one MMA
constexpr int kMxBN = 256;    // columns of a work tile
constexpr int kMxGroup = 2;   // stages that one load of scales lasts: 512 values of K

constexpr int kMxQueue = 3;   // work items handed out ahead of the epilogue

constexpr uint32_t kMxTmemCols = 512;
constexpr uint32_t kMxAccStep = 128;   // the second accumulator starts here: 128 columns shared
constexpr uint32_t kMxScaleCol = 384;  // a slot for a stage's scales: A 2 x 4 columns, B 2 x 8
constexpr int kMxSlotCols = 24, kMxTmemSlots = 5;
static_assert(kMxAccStep + kMxBN <= kMxScaleCol &&
              kMxScaleCol + kMxTmemSlots * kMxSlotCols <= kMxTmemCols, "TMEM columns");

// Per CTA: 128 rows of A, kMxBN / CG of the weights' rows, and the scales of its
// rows and of all kMxBN columns.
template <int CG>
struct MxCfg {
  static constexpr int kABytes = kMmaM * kMxK / 2;
  static constexpr int kBRows = kMxBN / CG;
  static constexpr int kBBytes = kBRows * kMxK / 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = CG == 2 ? 6 : 4;
  static constexpr int kScaleBytes = (kMmaM + kMxBN) * 16;  // a slot: A's rows, then B's
  static constexpr int kScaleSlots = 2;
  static constexpr int kTmemSlots = kMxTmemSlots < kStages ? kMxTmemSlots : kStages;
  static constexpr int kOutBytes = 4 * 4096;  // a 32 x 64 bf16 staging buffer a warp
  static constexpr int kThreads = 32 * 12;
  static constexpr int kConsumers = CG * 10 + 1;  // two producers, 4 + 4 warps a CTA; the MMAs
  static constexpr int kNumBars = 2 * kStages + 2 * kScaleSlots + 4 + 2 * kMxQueue;
  static constexpr int kSmem = kStages * kStageBytes + kOutBytes + kScaleSlots * kScaleBytes + 1024 +
                               16 * kMxQueue + kNumBars * 8 + 16;
};
static_assert(MxCfg<1>::kSmem <= 232448 && MxCfg<2>::kSmem <= 232448, "shared memory of a CTA");
// (an item takes a copy at most and a stage at least, and a stage is filled again only when
// its last loads have been used)
static_assert(kTmapSlots > MxCfg<1>::kStages && kTmapSlots > MxCfg<2>::kStages,
              "a tensor-map copy must outlive the loads in flight");

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

// 8 or 16 columns of this warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

// A work item as every role needs it, handed out through a ring in shared memory by
// a thread that does nothing else.  With the claims and the tile list read by the TMA
// producer, between one item's loads and the next's, the first two stages of an item
// came some 2500 clocks late: 1193 -> 1117 us at 262144 rows x 7168 x 2048, 459 -> 379 us
// at 262144 rows x 4096 x 1024 in 224 groups (short runs; call after call the power limit
// sets the time, 1311 us at 1450 MHz).  A slot is filled when it is free and not
// before: an item claimed earlier is one that no idle CTA can take (decoding 16
// tokens: 125 us with the next item claimed ahead, 117 without).
struct __align__(16) MxItem {
  int32_t row0;   // first row of the tile in recv and y
  int32_t rows;   // rows inside the group
  int32_t wrow;   // row of the weights of column n0; slots: -1 - that row
  int32_t n0;     // first column; -1 ends the sequence
};

template <int CG>
struct MxQueue {
  uint32_t full0, empty0;  // this CTA's barriers of slot 0
  MxItem* items;
  __device__ uint32_t full(int s) const { return full0 + 8u * s; }
  __device__ uint32_t empty(int s) const { return empty0 + 8u * s; }
  // The i-th item, by every lane of a warp or by one thread
  __device__ __forceinline__ bool wait(int i, bool leader, MxItem& item, volatile int* abort_flag) const {
    const int s = i % kMxQueue;
    const uint32_t parity = (i / kMxQueue) & 1;
    // the leader's items come from its own CTA
    if (!(leader ? mbar_wait(full(s), parity, abort_flag)
                 : mbar_wait_cluster(full(s), parity, abort_flag)))
      return false;
    const int4 v = *reinterpret_cast<const int4*>(items + s);
    item = MxItem{v.x, v.y, v.z, v.w};
    return true;
  }
  // Once a role, after its lanes have read the item.  `read` comes out of the item and
  // is 0: with it in the address the arrival cannot be issued before the load has
  // landed, which nothing else makes an mbarrier operation wait for.
  __device__ __forceinline__ void announce(int i, bool leader, uint32_t read) const {
    const uint32_t bar = empty(i % kMxQueue) + 8u * read;
    if (leader) mbar_arrive(bar);
    else mbar_arrive_remote_relaxed(pair_map(bar, 0));
  }
  __device__ __forceinline__ bool take(int i, bool leader, MxItem& item, volatile int* abort_flag) const {
    if (!wait(i, leader, item, abort_flag)) return false;
    announce(i, leader, item.n0 < -1 ? 1u : 0u);
    return true;
  }
  __device__ __forceinline__ bool take_warp(int i, bool leader, MxItem& item,
                                            volatile int* abort_flag) const {
    if (!__all_sync(0xffffffffu, wait(i, leader, item, abort_flag))) return false;
    const uint32_t read = __any_sync(0xffffffffu, item.n0 < -1) ? 1u : 0u;
    if ((threadIdx.x & 31) == 0) announce(i, leader, read);
    __syncwarp();
    return true;
  }
  // For the thread that hands items out: the i-th slot is free; the i-th item
  __device__ __forceinline__ bool wait_free(int i, volatile int* abort_flag) const {
    return mbar_wait_cluster(empty(i % kMxQueue), ((i / kMxQueue) & 1) ^ 1u, abort_flag);
  }
  __device__ __forceinline__ void push(int i, const MxItem& item) const {
    const int s = i % kMxQueue;
    *reinterpret_cast<int4*>(items + s) = make_int4(item.row0, item.rows, item.wrow, item.n0);
    if constexpr (CG == 2)
      asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                       pair_map(smem_u32(items + s), 1)),
                   "r"(item.row0), "r"(item.rows), "r"(item.wrow), "r"(item.n0)
                   : "memory");
    mbar_arrive(full(s));
    if constexpr (CG == 2) mbar_arrive_remote(pair_map(full(s), 1));
  }
};

template <int CG>
__global__ void __launch_bounds__(MxCfg<CG>::kThreads, 1)
k_mxfp4_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_wh,
             const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_sa,
             const __grid_constant__ CUtensorMap tm_sh, const __grid_constant__ CUtensorMap tm_ss,
             const __grid_constant__ CUtensorMap tm_y, int K, int N, int rank_rows, PlanPtrs p,
             uint16_t* __restrict__ y) {
  using Cfg = MxCfg<CG>;
  constexpr int STAGES = Cfg::kStages, SLOTS = Cfg::kScaleSlots;
  constexpr bool kPair = CG == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* out_stage = smem + STAGES * Cfg::kStageBytes;
  uint8_t* scale_ring = out_stage + Cfg::kOutBytes;
  MxItem* items = (MxItem*)(scale_ring + SLOTS * Cfg::kScaleBytes);
  uint64_t* bars = (uint64_t*)(items + kMxQueue);
  uint32_t* tmem_slot = (uint32_t*)(bars + Cfg::kNumBars);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t bar1 = bar0 + 16u * STAGES;
  auto raw_full = [&](int s) { return bar1 + 8u * s; };  // a ring slot holds its scales
  auto raw_empty = [&](int s) { return bar1 + 8u * (SLOTS + s); };
  const uint32_t bar2 = bar1 + 16u * SLOTS;
  auto tfull = [&](int b) { return bar2 + 8u * b; };
  const uint32_t tempty = bar2 + 16u, drain = bar2 + 24u;
  const MxQueue<CG> q{bar2 + 32u, bar2 + 32u + 8u * kMxQueue, items};
  constexpr uint64_t kDrainNs = 200000000ull;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = kPair ? pair_rank() : 0;
  const bool leader = crank == 0;
  // The pair kernel is launched while the 128-row one runs (only one of them has
  // tiles), and does not end before it.
  if constexpr (!kPair) cudaTriggerProgrammaticLaunchCompletion();
  if (plan_failed(p.status) ||  // uniform over the pair: before any barrier
      // the other kernel's tiles; where a rank has at most 128 rows this one takes all
      (p.counters[MOONEP_CNT_TILE_ROWS] != CG * kMmaM && rank_rows > kMmaM)) {
    if constexpr (kPair) cudaGridDependencySynchronize();
    return;
  }
  const int NT = (N + kMxBN - 1) / kMxBN;
  const int total = p.counters[MOONEP_CNT_MTILES] * NT;
  const int KB = (K + kMxK - 1) / kMxK;
  const int KG = (KB + kMxGroup - 1) / kMxGroup;
  int32_t* sched = p.sched + (kPair ? 0 : 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1 + 4 * CG);  // the codes' bytes and the scale warps (leader's)
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), 4);  // the four scale warps
    }
    for (int b = 0; b < 2; ++b) mbar_init(tfull(b), 1);
    mbar_init(tempty, 4 * CG);
    mbar_init(drain, 1);
    for (int s = 0; s < kMxQueue; ++s) {
      mbar_init(q.full(s), 1);
      mbar_init(q.empty(s), Cfg::kConsumers);
    }
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
  __syncwarp();
  tc_fence_after();
  if constexpr (kPair) pair_sync();  // the peer's barriers are ready
  const uint32_t tmem_base = *tmem_slot;
  auto fail = [&]() {
    *abort_flag = 1;
    set_error(p.status, MOONEP_ERR_TIMEOUT);
  };
  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (elect_one()) {
      // this CTA's ring of copies of A's tensor map (the first map of each slot)
      uint4* maps = reinterpret_cast<uint4*>(p.tmaps) + (size_t)blockIdx.x * kTmapSlots * 16;
      for (int i = 0; i < kTmapSlots; ++i)
        for (int j = 0; j < 8; ++j) maps[i * 16 + j] = reinterpret_cast<const uint4*>(&tm_a)[j];
      int stage = 0, issued = 0, slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        MxItem it;
        if (!q.take(i, leader, it, abort_flag)) { ok = false; break; }
        if (it.n0 < 0) break;
        const CUtensorMap* wmap = it.wrow >= 0 ? &tm_wh : &tm_ws;
        const int wrow = (it.wrow >= 0 ? it.wrow : -1 - it.wrow) + (int)crank * Cfg::kBRows;
        const int row0 = it.row0 + (int)crank * kMmaM;
        // Rows past the group's end are loaded as zeros, through a copy of the map that
        // ends there: their products are not stored, and on zeros they take less power
        const CUtensorMap* amap = &tm_a;
        if (it.rows < (int)(crank + 1) * kMmaM) {
          uint4* m = maps + slot * 16;
          tmap_set_dim1(m, it.row0 + it.rows);
          tmap_publish(m);
          amap = reinterpret_cast<const CUtensorMap*>(m);
          if (++slot == kTmapSlots) slot = 0;
        }
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(empty(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
          if (leader) mbar_expect_tx(full(stage), CG * Cfg::kStageBytes);
          if constexpr (kPair) {
            const uint32_t fb = pair_map(full(stage), 0);
            tma_load_2d_pair(sa, amap, fb, kb * (kMxK / 2), row0);
            tma_load_2d_pair(sa + Cfg::kABytes, wmap, fb, kb * (kMxK / 2), wrow);
          } else {
            tma_load_2d(sa, amap, full(stage), kb * (kMxK / 2), row0);
            for (int h = 0; h < 2; ++h)
              tma_load_2d(sa + Cfg::kABytes + h * 128 * 128, wmap, full(stage), kb * (kMxK / 2),
                          wrow + h * 128);
          }
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
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
    // (elect_one instead of lane 0: 1355 -> 1229 us at 262144 rows x 7168 x 2048, short runs)
    if (leader && elect_one()) {
      constexpr uint32_t idesc[2] = {mx_idesc(CG * kMmaM, kMxBN, 0), mx_idesc(CG * kMmaM, kMxBN, 2)};
      int stage = 0, slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        MxItem it;
        if (!q.take(i, true, it, abort_flag)) { ok = false; break; }
        if (it.n0 < 0) break;
        // the shared columns of the tile before are drained
        if (!mbar_wait(tempty, (i & 1) ^ 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t dtm = tmem_base + (uint32_t)(i & 1) * kMxAccStep;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(full(stage), phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
          const uint32_t sb = sa + Cfg::kABytes;
          const uint32_t sfa = tmem_base + kMxScaleCol + (uint32_t)slot * kMxSlotCols, sfb = sfa + 8;
          const int steps = min(kMxK, K - kb * kMxK) / kMxUmmaK;
#pragma unroll
          for (int k = 0; k < kMxK / kMxUmmaK; ++k)
            if (k < steps)
              mx_mma<CG>(dtm, sw128_desc(sa + k * (kMxUmmaK / 2), 16, 1024),
                         sw128_desc(sb + k * (kMxUmmaK / 2), 16, 1024), idesc[k & 1],
                         sfa + (k >> 1) * 4, sfb + (k >> 1) * 8, (kb | k) != 0);
          if constexpr (kPair) umma_commit_pair_both(empty(stage));
          else umma_commit(empty(stage));
          if (++slot == Cfg::kTmemSlots) slot = 0;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if constexpr (kPair) umma_commit_pair_both(tfull(i & 1));
        else umma_commit(tfull(i & 1));
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
    uint8_t* buf = out_stage + qw * 4096;
    for (int i = 0;; ++i) {
      MxItem it;
      if (!q.take_warp(i, leader, it, abort_flag)) {
        if (lane == 0) fail();
        break;
      }
      if (it.n0 < 0) break;
      const int n0 = it.n0;
      const int acc = i & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(tfull(acc), (i >> 1) & 1, abort_flag))) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const int wrow0 = (int)crank * kMmaM + qw * 32;  // this warp's first row of the tile
      const uint32_t tbase = tmem_base + ((uint32_t)(qw * 32) << 16) + (uint32_t)acc * kMxAccStep;
      const bool whole = wrow0 + 32 <= it.rows;  // all 32 rows inside the group
      const bool valid = wrow0 + lane < it.rows;
      uint16_t* yrow = y + (size_t)(it.row0 + wrow0 + lane) * N + n0;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        // the columns that both accumulators use come first: the last 128 of the
        // first accumulator, the first 128 of the second
        const int c0 = (half ^ acc ^ 1) * 128;
        uint32_t r[4][32];
        __syncwarp();  // one lane issued the stores before: tcgen05.ld wants the warp together
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_x32(tbase + c0 + c * 32, r[c]);
        tmem_ld_wait();
        if (half == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair) mbar_arrive_remote_relaxed(pair_map(tempty, 0));
            else mbar_arrive(tempty);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int n = c0 + c * 64;
          if (n0 + n >= N) break;  // N is a multiple of 64
          // The one rounding of the fp32 sums: bf16 is the type that moonep_combine reads,
          // as in the bf16 product (layer of 8192 tokens x 1024 x 512, K 4: 2.35e-3 from 64
          // bits; with fp32 kept up to the combined output 1.66e-3)
          uint4 o[8];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const uint32_t* f = &r[2 * c + v / 4][8 * (v % 4)];
            o[v] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
          }
          if (whole) {
            // staged with the 128-byte swizzle, so that the lanes of a store phase hit
            // distinct bank groups, and written by one TMA store
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
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
                  "r"(n0 + n), "r"(it.row0 + wrow0), "r"(smem_u32(buf))
                  : "memory");
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          } else if (valid) {  // rows past the group's end are the next group's
#pragma unroll
            for (int v = 0; v < 8; ++v) reinterpret_cast<uint4*>(yrow + n)[v] = o[v];
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  } else if (warp < 10) {
    // ---------------- scales to TMEM: one warp for each lane group ----------------
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // Stage n's scales take TMEM slot n % kTmemSlots, free once the products of stage
    // n - kTmemSlots are done: the `empty` barrier of that stage (which cannot be a
    // phase further, as the stage STAGES later waits for these scales).
    int slot = 0, tslot = 0, stage = 0, old = 0;
    uint32_t phase = 0, old_phase = 0;
    int before = Cfg::kTmemSlots;  // stages still without an earlier one
    bool ok = true;
    for (int i = 0; ok; ++i) {
      MxItem it;
      if (!q.take_warp(i, leader, it, abort_flag)) { ok = false; break; }
      if (it.n0 < 0) break;
      for (int kb = 0; ok && kb < KB;) {
        if (!__all_sync(0xffffffffu, mbar_wait(raw_full(slot), phase, abort_flag))) {
          ok = false;
          break;
        }
        const uint4* rows = reinterpret_cast<const uint4*>(scale_ring + slot * Cfg::kScaleBytes);
        uint4 v[3][4];
#pragma unroll
        for (int a = 0; a < 3; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[a][j] = rows[a * 128 + 32 * j + lane];
#pragma unroll
        for (int h = 0; h < kMxGroup; ++h) {
          if (kb == KB) break;
          if (before > 0) {
            --before;
          } else {
            if (!__all_sync(0xffffffffu, mbar_wait(empty(old), old_phase, abort_flag))) {
              ok = false;
              break;
            }
            if (++old == STAGES) { old = 0; old_phase ^= 1u; }
            tc_fence_after();
          }
          const uint32_t dst = tmem_base + lanes + kMxScaleCol + (uint32_t)tslot * kMxSlotCols;
          // columns 4 w + j of A, then 8 w + 4 a + j of B: word w of row 32 j + lane
          uint32_t ra[8], rb[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ra[j] = h == 0 ? v[0][j].x : v[0][j].z;
            ra[4 + j] = h == 0 ? v[0][j].y : v[0][j].w;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              rb[4 * a + j] = h == 0 ? v[1 + a][j].x : v[1 + a][j].z;
              rb[8 + 4 * a + j] = h == 0 ? v[1 + a][j].y : v[1 + a][j].w;
            }
          }
          __syncwarp();  // one lane announced the stage before
          tmem_st_x8(dst, ra);
          tmem_st_x16(dst + 8, rb);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (h == 0) {
            // The ring slot is free only now: the stores took every loaded vector.  An
            // arrival right after the loads overtook some of them (an mbarrier
            // operation does not wait for loads in flight): the next scales in the
            // slot were read instead, once in about 10^5 to 10^7 stages.
            if (lane == 0) mbar_arrive(raw_empty(slot));
            if (++slot == SLOTS) { slot = 0; phase ^= 1u; }
          }
          if (lane == 0) {
            if constexpr (kPair) mbar_arrive_remote_relaxed(pair_map(full(stage), 0));
            else mbar_arrive(full(stage));
          }
          ++kb;
          if (++tslot == Cfg::kTmemSlots) tslot = 0;
          if (++stage == STAGES) stage = 0;
        }
      }
    }
    if (!ok && lane == 0) fail();
    __syncwarp();
  } else if (warp == 10) {
    // ---------------- scales to shared memory ----------------
    if (elect_one()) {
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        MxItem it;
        if (!q.take(i, leader, it, abort_flag)) { ok = false; break; }
        if (it.n0 < 0) break;
        const CUtensorMap* smap = it.wrow >= 0 ? &tm_sh : &tm_ss;
        const int wrow = it.wrow >= 0 ? it.wrow : -1 - it.wrow, row0 = it.row0 + (int)crank * kMmaM;
        for (int g = 0; g < KG; ++g) {
          if (!mbar_wait(raw_empty(slot), phase ^ 1u, abort_flag)) { ok = false; break; }
          mbar_expect_tx(raw_full(slot), Cfg::kScaleBytes);
          const uint32_t dst = smem_u32(scale_ring + slot * Cfg::kScaleBytes);
          tma_load_2d(dst, &tm_sa, raw_full(slot), g * 16, row0);
          tma_load_2d(dst + kMmaM * 16, smap, raw_full(slot), g * 16, wrow);
          ++issued;
          if (++slot == SLOTS) { slot = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        fail();
        for (int i = 0; i < min(issued, SLOTS); ++i) {  // the copies this thread started
          if (slot == 0) { slot = SLOTS - 1; phase ^= 1u; } else { --slot; }
          mbar_wait(raw_full(slot), phase, nullptr, kDrainNs);
        }
      }
    }
  } else if (leader && lane == 0) {
    // ---------------- work items ----------------
    bool ok = true;
    for (int i = 0; (ok = q.wait_free(i, abort_flag)); ++i) {
      const int t = atomicAdd(sched, 1);
      if (t >= total) {
        q.push(i, MxItem{0, 0, 0, -1});
        break;
      }
      const MTile mt = p.mtiles[t / NT];
      const int n0 = (t % NT) * kMxBN;
      const int wrow = (mt.wsel >= 0 ? mt.wsel : -1 - mt.wsel) * N + n0;
      q.push(i, MxItem{mt.row0, mt.rows, mt.wsel >= 0 ? wrow : -1 - wrow, n0});
    }
    queue_finish(sched, sched + 1, gridDim.x / CG);
    if (!ok) fail();
  }

  // roles of one thread end here one by one: the warps' other lanes wait, and the
  // instructions that take whole warps come after they are together again
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if constexpr (kPair) pair_sync();  // both CTAs done with TMEM and each other's barriers
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, kMxTmemCols);
    else tmem_dealloc(tmem_base, kMxTmemCols);
  }
  if constexpr (kPair) cudaGridDependencySynchronize();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// A byte matrix [rows][bytes], box of box_rows rows of box_bytes (128: swizzled over
// 128 bytes); what lies past a row's or the tensor's end reads as zeros.
static bool encode_bytes(CUtensorMap* m, const void* base, uint64_t bytes, uint64_t rows,
                         uint32_t box_bytes, uint32_t box_rows) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t gdim[2] = {bytes, rows};
  cuuint64_t gstride[1] = {bytes};
  cuuint32_t box[2] = {box_bytes, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
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

struct MxMaps {
  CUtensorMap a, a_scales, home, home_scales, slot, slot_scales, y;
};

template <int CG>
static cudaError_t launch_mx(const Dims& d, const PlanPtrs& p, const MxMaps& m,
                             uint16_t* y, bool after_other, cudaStream_t st) {
  using Cfg = MxCfg<CG>;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static PerDevice kept;
  int grid = 0;
  const cudaError_t e = kept(&grid, [&](int* found) {
    cudaError_t e = cudaFuncSetAttribute(k_mxfp4_gemm<CG>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    int n = sm_count_gemm();
    if (CG == 2) {  // one CTA pair per co-resident cluster
      cfg.gridDim = dim3(2 * std::max(1, n / 2));
      e = cudaOccupancyMaxActiveClusters(&n, (void*)k_mxfp4_gemm<CG>, &cfg);
    }
    *found = CG * std::max(1, n);
    return e;
  });
  if (e != cudaSuccess) return e;
  const long long items = (long long)d.max_mtiles * ((d.Hp + kMxBN - 1) / kMxBN);
  if (grid > kMaxGemmCtas) return cudaErrorInvalidConfiguration;  // tensor-map scratch per CTA
  cfg.gridDim = dim3((unsigned)std::min<long long>(grid, CG * items));
  if (after_other) cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_mxfp4_gemm<CG>, m.a, m.home, m.slot, m.a_scales,
                            m.home_scales, m.slot_scales, m.y, d.H, d.Hp, d.C, p, y);
}

cudaError_t launch_mxfp4_grouped_gemm(const Dims& d, const PlanPtrs& p, const uint8_t* a,
                                      const uint8_t* a_scales, const uint8_t* home,
                                      const uint8_t* home_scales, const uint8_t* slot,
                                      const uint8_t* slot_scales, void* y, cudaStream_t st,
                                      int* launches) {
  const bool slots = slot != nullptr && d.B > 0;
  const uint64_t bytes = d.H / 2, pitch = MOONEP_MXFP4_SCALE_PITCH(d.H);
  const uint64_t rows = (uint64_t)d.R * d.C, home_rows = (uint64_t)d.E * d.Hp;
  const uint64_t slot_rows = (uint64_t)d.R * d.B * d.Hp;
  MxMaps m;
  if (!encode_bytes(&m.a, a, bytes, rows, 128, kMmaM) ||
      !encode_bytes(&m.a_scales, a_scales, pitch, rows, 16, kMmaM) ||
      !encode_bytes(&m.home, home, bytes, home_rows, 128, 128) ||
      !encode_bytes(&m.home_scales, home_scales, pitch, home_rows, 16, kMxBN) ||
      !encode_out(&m.y, y, (uint64_t)d.Hp, rows))
    return cudaErrorInvalidValue;
  m.slot = m.home;
  m.slot_scales = m.home_scales;
  if (slots && (!encode_bytes(&m.slot, slot, bytes, slot_rows, 128, 128) ||
                !encode_bytes(&m.slot_scales, slot_scales, pitch, slot_rows, 16, kMxBN)))
    return cudaErrorInvalidValue;
  // The plan's tile height is on the device: the variant it did not choose returns at
  // once (as in the bf16 product).  Where no rank has more than 128 rows, no tile has,
  // whatever its height, and the 128-row kernel takes both.
  const bool pair = d.tile_m != kMmaM && d.C > kMmaM;
  const bool solo = d.tile_m != 2 * kMmaM || !pair;
  if (solo) {
    const cudaError_t e = launch_mx<1>(d, p, m, (uint16_t*)y, false, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  if (pair) {
    const cudaError_t e = launch_mx<2>(d, p, m, (uint16_t*)y, solo, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  return cudaSuccess;
}

}  // namespace moonep
