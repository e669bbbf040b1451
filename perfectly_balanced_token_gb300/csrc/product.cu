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
//    two accumulators in TMEM, warps 2..9 drain the other: bias, z, activation, residual and one
//    rounding happen in registers, so z and the activation never make a trip through memory that
//    the caller did not ask for.
//  * swiglu: a tile takes 128 gate columns and the 128 columns of the same numbers in the up half,
//    so one lane holds both factors of a value.  On a pair, the first CTA brings the gates and the
//    second the up columns of B; the MMA gives either CTA both for its rows.
//  * outputs leave by TMA stores of 32 rows x 32 columns, staged in shared memory; their maps clip
//    what lies past the last row or column, so sizes need not divide the tile.  Rows of a group that
//    ends inside a tile are stored one by one, as the next group's rows follow.
//  * dense tiles are walked with a fixed stride, the plan's tiles claimed in order (tcgen05.cuh).
// What bounds it: L2's feed of the stages (32 KB a CTA for 64 of the depth, 15 TB/s over the GPU) while the
// clock is high, power in long products.  Measured: 65536 x 7168 x 4096 of swiglu with bias and z 2231 to
// 2314 us (1.72 to 1.66 PFLOP/s), 8192 rows 257 us with pauses between the calls and 292 without (1.87 and
// 1.65), the gradients at 32768 rows 2282 to 2348 us together.
#include <algorithm>
#include <type_traits>

#include "product.cuh"

namespace moonep {

constexpr int kEpilogueWarps = 8;  // two for each 32 lanes of TMEM, half of a tile's columns each
constexpr int kProductThreads = 64 + 32 * kEpilogueWarps;

template <bool PAIR, bool F32>
struct ProductCfg {
  static constexpr int kStages = PAIR ? 6 : 4;
  static constexpr int kTileM = PAIR ? 256 : 128;
  static constexpr int kABytes = 128 * kDepth * 2;
  static constexpr int kBPanels = PAIR ? 2 : 4;  // of 64 columns, in one CTA
  static constexpr int kStageBytes = kABytes + kBPanels * kPanelBytes;
  static constexpr int kOutWarpBytes = 4096;  // staging of a warp's stores
  static constexpr int kOutBytes = kEpilogueWarps * kOutWarpBytes;
  static constexpr int kNumBars = 2 * kStages + 5 + 2 * kQueue;
  static constexpr int kBarBytes = kNumBars * 8 + 16 + 4 * kQueue;
  static constexpr int kSmem = kStages * kStageBytes + kOutBytes + 1024 + kBarBytes;
  // With z kept, 32 columns have two or three stores where they had one, and waiting until TMA has
  // read the buffer of the one before the last costs more than a stage is worth: the last stage's
  // memory becomes two more buffers a warp (12000 rows x 1024 x 576, gelu and z: 69 -> 61 us).
  static constexpr bool kCanDeepen = PAIR && !F32;
};
static_assert(kTmapSlots > ProductCfg<true, false>::kStages, "a map's copy outlives the loads in flight");
static_assert(ProductCfg<true, false>::kSmem <= 232448 && ProductCfg<true, true>::kSmem <= 232448 &&
                  ProductCfg<false, false>::kSmem <= 232448,
              "shared memory of a CTA");

struct ProductArgs {
  int M, N, K;     // C's rows and columns, the depth; grouped: M rows of all groups together
  int wrows;       // grouped: rows of an expert's weight
  int act;         // Act
  int half;        // swiglu: N / 2, otherwise 0
  int add;         // fp32 C: added into
  int bn;          // columns of a tile: 256, 192 or 128 (swiglu: half of them gates)
                   // (the eighth word: the host tests read it in a launch's arguments)
  const float* bias;  // [N], grouped [E][N]; or null
  const uint16_t* residual;  // [M][out columns] or null
  uint16_t *out, *z;         // for rows stored one by one; z null if not asked for
  int has_z;
  int all;  // grouped, one CTA: takes the plan's tiles whatever height it chose
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

// A warp's staging buffers and the stores from them: boxes of 32 rows x 32 columns, bf16 (2 KB, 64-byte
// swizzle; two or four buffers) or fp32 (4 KB, 128-byte swizzle; one).
struct OutRing {
  uint8_t* base;
  int buffers;
  int n, lane;

  __device__ __forceinline__ uint8_t* begin(int bytes) {
    uint8_t* buf = base + (n & (buffers - 1)) * bytes;
    ++n;
    if (lane == 0) {  // until the store that had this buffer has read it
      if (buffers == 1) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      else if (buffers == 2) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      else asm volatile("cp.async.bulk.wait_group.read 3;" ::: "memory");
    }
    __syncwarp();
    return buf;
  }
  __device__ __forceinline__ void end(const uint8_t* buf, const CUtensorMap* m, int x, int y, bool add) {
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
  __device__ __forceinline__ void put(const uint32_t (&v)[16], const CUtensorMap* m, int x, int y) {
    uint8_t* buf = begin(2048);
    uint4* row = reinterpret_cast<uint4*>(buf + lane * 64);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      row[j ^ ((lane >> 1) & 3)] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    end(buf, m, x, y, false);
  }
  __device__ __forceinline__ void put(const float (&v)[32], const CUtensorMap* m, int x, int y, bool add) {
    uint8_t* buf = begin(4096);
    float4* row = reinterpret_cast<float4*>(buf + lane * 128);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      row[j ^ (lane & 7)] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    end(buf, m, x, y, add);
  }
};

// The first `cols` (a multiple of 8) of a row's 32 bf16 values.
__device__ __forceinline__ void put_row(const uint32_t (&v)[16], uint16_t* at, int cols) {
  uint4* p = reinterpret_cast<uint4*>(at);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (8 * j < cols) p[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// v += bias[0 .. 31], of which the first `cols` (a multiple of 8) are there; every lane has the same
__device__ __forceinline__ void add_bias(float (&v)[32], const float* bias, int cols) {
  const float4* b = reinterpret_cast<const float4*>(bias);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (4 * j < cols) {
      const float4 f = b[j];
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
      const uint4 r = p[j];
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * j + 2 * i] += __uint_as_float(w[i] << 16);
        v[8 * j + 2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ void pack32(uint32_t (&p)[16], const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    p[i] = pack_bf16x2(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]));
}

__device__ __forceinline__ void load32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld_x32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 columns of a lane's row from the sums (v and, for swiglu, u of the up half) to the output's
// values in v; keep_z(v, false) and keep_z(u, true) see z on the way.  x: the first column, cols: how
// many are left.
template <typename Z>
__device__ __forceinline__ void forward32(const ProductArgs& a, const float* bias,
                                          const uint16_t* residual, int x, int cols, float (&v)[32],
                                          float (&u)[32], Z&& keep_z) {
  if (bias != nullptr) add_bias(v, bias + x, cols);
  keep_z(v, false);
  if (a.half) {
    if (bias != nullptr) add_bias(u, bias + a.half + x, cols);
    keep_z(u, true);
    swiglu_each(v, u);
  } else {
    act_each(a.act, v);
  }
  if (residual != nullptr) add_residual(v, residual + x, cols);
}

template <bool PAIR, int KIND, bool DENSE, bool F32>
__global__ void __launch_bounds__(kProductThreads, 1)
k_product(const __grid_constant__ ProductMaps tm, const __grid_constant__ ProductArgs a,
          const __grid_constant__ PlanPtrs p) {
  static_assert(DENSE || !F32, "the grouped output is bf16");
  static_assert(PAIR || KIND == kForward, "one CTA has no loads of w^T or x^T");
  static_assert(DENSE || KIND == kForward, "the plan's gradients are moonep.h's");
  using Cfg = ProductCfg<PAIR, F32>;
  using Op = Issue<PAIR>;
  const bool deep = Cfg::kCanDeepen && a.has_z;
  const int STAGES = Cfg::kStages - (deep ? 1 : 0);
  constexpr bool AMN = KIND == kWeightGrad;  // A = x^T: runs along M in memory
  constexpr bool BMN = KIND != kInputGrad;   // B = w^T there: runs along the depth
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* out_stage = smem + STAGES * Cfg::kStageBytes;  // 1024-aligned
  uint64_t* bars = (uint64_t*)(smem + Cfg::kStages * Cfg::kStageBytes + Cfg::kOutBytes);
  uint32_t* tmem_slot = (uint32_t*)(bars + Cfg::kNumBars);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* dead = (volatile int*)(tmem_slot + 2 + kQueue);  // the status was set
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
  if (!DENSE) {
    grid_wait();
    if (p.counters[MOONEP_CNT_TILE_ROWS] != Cfg::kTileM && (PAIR || !a.all)) return;
  }
  const int step = a.half ? a.bn / 2 : a.bn;  // output columns of a tile
  const int NT = ((a.half ? a.half : a.N) + step - 1) / step;
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
      mbar_init(tempty(b), (PAIR ? 2 : 1) * kEpilogueWarps);
    }
    mbar_init(drain, 1);
    // who takes a tile: the issuer and the epilogue's warps, in a pair also the other CTA's feeder
    if (!DENSE) queue_init(q, (PAIR ? 2 : 1) * (1 + kEpilogueWarps));
    *abort_flag = 0;
    fence_barrier_init();
    if (DENSE) grid_wait();
    *dead = plan_failed(a.status);
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
  if (DENSE) grid_wait();  // (what is above runs while the kernel before this one ends)
  grid_trigger();
  // both CTAs go by what either found in the status word: another pair may set it meanwhile
  int skip = *dead;
  if (PAIR) {
    int other;
    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                 : "=r"(other)
                 : "r"(pair_map(smem_u32((const void*)dead), crank ^ 1u)));
    skip |= other;
  }

  auto fail = [&]() {
    *abort_flag = 1;
    set_error(a.status, MOONEP_ERR_TIMEOUT);
  };
  // Tile t's rows (first, number, weight and rank as the plan lists them) and first column.  The tiles
  // that run together are to be near a square of rows and columns, which needs the fewest panels: strips
  // of 8 column tiles, in a strip one row tile after the other (65536 x 7168 x 4096: 2309 us with rows
  // across all 16 columns, 2231 so); of the plan's tiles, whose weights differ from group to group,
  // blocks of 18 row tiles are taken strip by strip (131072 rows: 5117 and 5078 us).
  constexpr int kStrip = 8, kBlockRows = 18;
  auto tile = [&](int t, MTile& mt, int& n0) {
    const int rows = DENSE ? MT : kBlockRows;
    const int block = DENSE ? 0 : t / (rows * NT);
    t -= block * rows * NT;
    const int here = DENSE ? MT : min(rows, MT - block * rows);
    const int strip = t / (here * kStrip);
    t -= strip * here * kStrip;
    const int wide = min(kStrip, NT - strip * kStrip);
    const int r = t / wide;
    n0 = (strip * kStrip + t - r * wide) * step;
    if (DENSE) {
      mt.row0 = r * Cfg::kTileM;
      mt.rows = min(Cfg::kTileM, a.M - mt.row0);
      mt.wsel = 0;
    } else {
      mt = p.mtiles[block * rows + r];
    }
  };

  if (skip) {
    // (on to the end, where the pair meets)
  } else if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    if (elect_one()) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      int next = 0;
      if (!DENSE && leader) next = atomicAdd(sched, 1);
      // Rows past a group's end are loaded as zeros, through copies of A's map that end there: they
      // are never stored, but products of zeros take less of the power that limits long products.
      // A copy is rewritten eight such tiles later, when the loads through it are over.
      constexpr bool kCut = PAIR && !DENSE;
      uint4* maps = kCut ? reinterpret_cast<uint4*>(p.tmaps) + (size_t)blockIdx.x * kTmapSlots * 16 : nullptr;
      int slot = 0;
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
        int row0 = mt.row0 + (int)crank * 128;
        const CUtensorMap* amap = &tm.a;
        if (kCut && mt.rows < ((int)crank + 1) * 128) {
          if (mt.rows <= (int)crank * 128) {
            row0 = a.M;  // no row of this CTA's: a box past the last one, all zeros
          } else {
            uint4* m = maps + slot * 16;
            const uint4* from = reinterpret_cast<const uint4*>(&tm.a);
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = from[j];
            tmap_set_dim1(m, mt.row0 + mt.rows);
            tmap_publish(m);
            amap = reinterpret_cast<const CUtensorMap*>(m);
            if (++slot == kTmapSlots) slot = 0;
          }
        }
        // this CTA's columns of B, in panels of 64
        const int mine = PAIR ? (a.half ? (int)crank * a.half + n0 : n0 + (int)crank * (a.bn / 2)) : n0;
        const int panels = PAIR ? (a.bn / 2 + 63) / 64 : a.bn / 64;
        auto column = [&](int j) {
          return !PAIR && a.half && j >= panels / 2 ? a.half + n0 + 64 * (j - panels / 2) : mine + 64 * j;
        };
        const uint32_t bytes = Cfg::kABytes + (BMN ? panels : Cfg::kBPanels) * kPanelBytes;
        // Input gradient: row tiles begin at other blocks of the depth, so that the pairs that read one
        // panel of w, whose rows lie 2 N bytes apart, do not do so at the same moment (8192 x 7168 x
        // 4096: 284 -> 270 us).  The products along N-major panels are faster in step (271 and 280).
        const int turn = KIND == kInputGrad ? (int)((unsigned)(mt.row0 / Cfg::kTileM) * 7u % (unsigned)KB) : 0;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(empty(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t fb = PAIR ? pair_map(full(stage), 0) : full(stage);
          if (leader) mbar_expect_tx(full(stage), (PAIR ? 2 : 1) * bytes);
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
          const uint32_t sb = sa + Cfg::kABytes;
          const int k0 = (kb + turn < KB ? kb + turn : kb + turn - KB) * kDepth;
          if (AMN) {
            Op::load(sa, &tm.a, fb, row0, k0);
            Op::load(sa + kPanelBytes, &tm.a, fb, row0 + 64, k0);
          } else {
            Op::load(sa, amap, fb, k0, row0);
          }
          if (BMN) {
#pragma unroll
            for (int j = 0; j < Cfg::kBPanels; ++j)
              if (j < panels) Op::load(sb + j * kPanelBytes, bmap, fb, column(j), wrow + k0);
          } else {  // 128 rows of w, of which the tile's width is used
            Op::load(sb, bmap, fb, k0, mine);
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
      const uint32_t idesc = product_idesc(Cfg::kTileM, a.bn, AMN, BMN);
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
        const int part = F32 ? kPartBlocks : KB;  // what one accumulator sums
        for (int kp = 0; kp < KB && ok; kp += part) {
          if (!mbar_wait(tempty(acc), acc_phase ^ 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t dtm = tmem_base + (uint32_t)(acc * 256);
          const int end = F32 ? min(kp + part, KB) : KB;
          for (int kb = kp; kb < end; ++kb) {
            if (!mbar_wait(full(stage), phase, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
            const uint32_t sb = sa + Cfg::kABytes;
#pragma unroll
            for (int k = 0; k < kDepth / 16; ++k)
              Op::mma(dtm, stage_desc(sa, k, AMN), stage_desc(sb, k, BMN), idesc, kb != kp || k != 0);
            Op::commit(empty(stage));
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          Op::commit(tfull(acc));
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (!ok) {
        fail();
        if (PAIR) umma_commit_pair_self(drain);
        else umma_commit(drain);
        mbar_wait(drain, 0, nullptr);
      }
    }
  } else {
    // ---------------- epilogue (warps 2.., both CTAs) ----------------
    const int qw = warp & 3;         // TMEM lanes 32 qw .. are this warp's rows
    const int hs = (warp - 2) >> 2;  // which half of the columns is this warp's
    OutRing ring{out_stage + (warp - 2) * Cfg::kOutWarpBytes * (deep ? 2 : 1),
                 F32 ? 1 : (deep ? 4 : 2), 0, lane};
    // its columns of a tile: `own` from the accumulator's column hs own on (swiglu: gates, with the up
    // columns of the same numbers bn / 2 further)
    const int own = step / 2;
    const int ocols = a.half ? a.half : a.N;
    const int parts = F32 ? (KB + kPartBlocks - 1) / kPartBlocks : 1;
    int acc = 0;
    uint32_t acc_phase = 0;
    auto take = [&]() {  // the next accumulator, once its sums are complete
      const bool ok = mbar_wait(tfull(acc), acc_phase, abort_flag);
      tc_fence_after();
      return __all_sync(0xffffffffu, ok) != 0;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_remote(pair_map(tempty(acc), 0));
        else mbar_arrive(tempty(acc));
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    };
    auto lanes_at = [&]() {
      return tmem_base + ((uint32_t)(qw * 32) << 16) + (uint32_t)(acc * 256);
    };
    bool ok = true;
    for (int i = 0; ok; ++i) {
      int t;
      if (DENSE) {
        t = work + i * nwork;
        if (t >= total) break;
      } else {
        if (!queue_take_warp(q, i, leader, t, abort_flag)) { ok = false; break; }
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
      if (!DENSE && bias != nullptr)
        bias += (size_t)(mt.wsel >= 0 ? mt.wsel : p.slot_expert[-1 - mt.wsel]) * a.N;
      // (lanes past the last row read that one: the warp stays together)
      const uint16_t* residual =
          a.residual != nullptr ? a.residual + (size_t)min(row, a.M - 1) * ocols : nullptr;
      const bool any = first < mt.rows;  // otherwise none of this warp's rows is stored
      auto put = [&](const float (&v)[32], const CUtensorMap* m, int x, uint16_t* plain, int pitch,
                     int cols) {
        uint32_t packed[16];
        pack32(packed, v);
        if (whole) ring.put(packed, m, x, mt.row0 + first);
        else if (valid) put_row(packed, plain + (size_t)row * pitch + x, cols);
        __syncwarp();
      };
      if constexpr (F32) {
        // up to 128 columns: for swiglu 64 gates and the 64 up columns of the same numbers, otherwise
        // half of the tile's
        float sum[4][32];
        const int width = a.bn / 2;
        for (int k = 0; k < parts && ok; ++k) {
          ok = take();
          if (!ok) break;
          // (16 columns at a time: the sums leave few registers)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (16 * j < width) {
              const int at = a.half ? 128 * (j >> 2) + 64 * hs + 16 * (j & 3) : width * hs + 16 * j;
              uint32_t v[16];
              tmem_ld_x16(lanes_at() + at, v);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                float& to = sum[j >> 1][16 * (j & 1) + c];
                to = __uint_as_float(v[c]) + (k == 0 ? 0.f : to);
              }
            }
          }
          release();
        }
        if (!ok || !any) continue;
        auto quarter = [&](auto number) {  // 32 output columns
          constexpr int Q = decltype(number)::value;
          const int x = n0 + own * hs + 32 * Q;
          const int cols = min(32, ocols - x);
          if (32 * Q >= own || cols <= 0) return;
          if (KIND == kForward)
            forward32(a, bias, residual, x, cols, sum[Q], sum[(2 + Q) & 3],
                      [&](const float(&z)[32], bool up) {
                        // (bf16, and no buffer of its own: row by row)
                        uint32_t packed[16];
                        pack32(packed, z);
                        if (a.has_z && valid)
                          put_row(packed, a.z + (size_t)row * a.N + (up ? a.half : 0) + x, cols);
                        __syncwarp();
                      });
          ring.put(sum[Q], &tm.out, x, mt.row0 + first, a.add);
        };
        quarter(std::integral_constant<int, 0>());
        quarter(std::integral_constant<int, 1>());
        if (!a.half) {
          quarter(std::integral_constant<int, 2>());
          quarter(std::integral_constant<int, 3>());
        }
      } else {
        ok = take();
        if (!ok) break;
#pragma unroll 1
        for (int c = own * hs; any && c < own * (hs + 1); c += 32) {
          const int x = n0 + c;  // first output column
          const int cols = min(32, ocols - x);
          if (cols <= 0) break;
          float v[32], u[32];
          load32(lanes_at() + c, v);
          if (KIND == kForward) {
            if (a.half) load32(lanes_at() + a.bn / 2 + c, u);
            forward32(a, bias, residual, x, cols, v, u, [&](const float(&z)[32], bool up) {
              if (!a.has_z) return;
              if (up) put(z, &tm.z_up, x, a.z + a.half, a.N, cols);
              else put(z, &tm.z, x, a.z, a.N, cols);
            });
          }
          put(v, &tm.out, x, a.out, ocols, cols);
        }
        release();
      }
    }
    if (!ok && lane == 0) fail();
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
template <bool PAIR, int KIND, bool DENSE, bool F32>
static cudaError_t launch_one(const ProductMaps& tm, const ProductArgs& a, const PlanPtrs& p,
                              int64_t tiles, cudaStream_t st) {
  using Cfg = ProductCfg<PAIR, F32>;
  constexpr int CG = PAIR ? 2 : 1;
  auto* kernel = k_product<PAIR, KIND, DENSE, F32>;
  static PerDevice kept;
  int most = 0;  // CTAs (pairs) that run at once
  const cudaError_t e = kept(&most, [&](int* found) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    if (!PAIR) return *found = sm_count_gemm(), cudaSuccess;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = CG;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * std::max(1, sm_count_gemm() / 2));
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    int n = 0;
    const cudaError_t e2 = cudaOccupancyMaxActiveClusters(&n, (void*)kernel, &cfg);
    *found = std::max(1, n);
    return e2;
  });
  if (e != cudaSuccess) return e;
  const unsigned grid = CG * (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, tiles));
  if (!DENSE && grid > (unsigned)kMaxGemmCtas) return cudaErrorInvalidConfiguration;  // maps' copies
  return launch_after(kernel, grid, kProductThreads, Cfg::kSmem, st, CG, tm, a, p);
}

static int64_t tiles_of(int64_t M, const ProductArgs& a, int rows) {
  const int step = a.half ? a.bn / 2 : a.bn;
  return ((M + rows - 1) / rows) * (((a.half ? a.half : a.N) + step - 1) / step);
}

// Columns of a tile: 256, or 192 or 128 where that makes up for what a narrower tile loses.  It does
// not take that much less time, as its rows are loaded all the same and L2's feed is what bounds the
// wide tile already: 0.88 and 0.75 of a wide one's (8192 x 7168 x 384: 39.5 us with 256, 35.2 with 192;
// 4096 x 7168 x 4096 of swiglu: 204 us with 128, 150 with 256).  `rounds` counts what a choice makes the
// fullest pair do; the plan's tiles are not known here, and their number of column tiles stands for it.
template <typename F>
static int pick_bn(int half, bool f32, F&& rounds) {
  int best = 256;
  double least = rounds(256);
  // (halves of 64 columns; fp32 sums of 192 or 256)
  if (!half && 0.88 * rounds(192) < least) least = 0.88 * rounds(192), best = 192;
  if (!f32 && 0.75 * rounds(128) < least) best = 128;
  return best;
}
static int pick_bn_dense(int M, int N, int half, bool f32) {
  const int64_t pairs = std::max(1, at_once(2) / 2);
  return pick_bn(half, f32, [&](int bn) {
    const int step = half ? bn / 2 : bn;
    const int64_t tiles = (int64_t)((M + 255) / 256) * (((half ? half : N) + step - 1) / step);
    return (double)((tiles + pairs - 1) / pairs);
  });
}
static int pick_bn_grouped(int N, int half) {
  return pick_bn(half, false, [&](int bn) {
    const int step = half ? bn / 2 : bn;
    return (double)(((half ? half : N) + step - 1) / step);
  });
}

cudaError_t launch_linear(const LinearDims& d, const void* x, const void* w, const float* bias,
                          const void* residual, void* out, void* z, int32_t* status, cudaStream_t st,
                          int* launches) {
  const SplitPlan split = plan_split(d.T, d.N, d.half, d.K, d.f32);
  if (split.splits) {
    *launches += 1;
    return launch_split(kForward, d, split, x, w, bias, residual, out, z, 0, status, st);
  }
  ProductMaps tm;
  const int ocols = d.half ? d.half : d.N;
  if (!encode_matrix(&tm.a, x, d.K, d.T, d.K, 128) || !encode_matrix(&tm.b, w, d.N, d.K, d.N, 64) ||
      !encode_out(&tm.out, out, ocols, d.T, ocols, d.f32))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  tm.z = tm.z_up = tm.out;
  if (z != nullptr) {  // the halves have maps of their own, so that either is clipped at its end
    if (!encode_out(&tm.z, z, ocols, d.T, d.N)) return cudaErrorInvalidValue;
    if (d.half && !encode_out(&tm.z_up, (uint16_t*)z + d.half, ocols, d.T, d.N))
      return cudaErrorInvalidValue;
  }
  ProductArgs a = {};
  a.M = d.T, a.N = d.N, a.K = d.K;
  a.act = d.act, a.half = d.half;
  a.bias = bias;
  a.residual = (const uint16_t*)residual;
  a.z = (uint16_t*)z;
  a.has_z = z != nullptr;
  a.status = status;
  a.bn = pick_bn_dense(d.T, d.N, d.half, d.f32);
  *launches += 1;
  const int64_t tiles = tiles_of(d.T, a, 256);
  return d.f32 ? launch_one<true, kForward, true, true>(tm, a, PlanPtrs{}, tiles, st)
               : launch_one<true, kForward, true, false>(tm, a, PlanPtrs{}, tiles, st);
}

cudaError_t launch_linear_dx(const LinearDims& d, const void* d_z, const void* w, void* d_x,
                             int32_t* status, cudaStream_t st, int* launches) {
  const SplitPlan split = plan_split(d.T, d.K, 0, d.N, false);
  if (split.splits) {
    *launches += 1;
    return launch_split(kInputGrad, d, split, d_z, w, nullptr, nullptr, d_x, nullptr, 0, status, st);
  }
  ProductMaps tm;
  if (!encode_matrix(&tm.a, d_z, d.N, d.T, d.N, 128) || !encode_matrix(&tm.b, w, d.N, d.K, d.N, 128) ||
      !encode_out(&tm.out, d_x, d.K, d.T, d.K))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  tm.z = tm.z_up = tm.out;
  ProductArgs a = {};
  a.M = d.T, a.N = d.K, a.K = d.N;
  a.status = status;
  a.bn = pick_bn_dense(d.T, d.K, 0, false);
  *launches += 1;
  return launch_one<true, kInputGrad, true, false>(tm, a, PlanPtrs{}, tiles_of(d.T, a, 256), st);
}

cudaError_t launch_linear_dw(const LinearDims& d, const void* x, const void* d_z, float* d_w,
                             int add, int32_t* status, cudaStream_t st, int* launches) {
  const SplitPlan split = plan_split(d.K, d.N, 0, d.T, true);
  if (split.splits) {
    *launches += 1;
    return launch_split(kWeightGrad, d, split, x, d_z, nullptr, nullptr, d_w, nullptr, add, status, st);
  }
  ProductMaps tm;
  if (!encode_matrix(&tm.a, x, d.K, d.T, d.K, 64) || !encode_matrix(&tm.b, d_z, d.N, d.T, d.N, 64) ||
      !encode_out(&tm.out, d_w, d.N, d.K, d.N, true))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  tm.z = tm.z_up = tm.out;
  ProductArgs a = {};
  a.M = d.K, a.N = d.N, a.K = d.T;
  a.add = add;
  a.status = status;
  a.bn = pick_bn_dense(d.K, d.N, 0, true);
  *launches += 1;
  return launch_one<true, kWeightGrad, true, true>(tm, a, PlanPtrs{}, tiles_of(d.K, a, 256), st);
}

cudaError_t launch_grouped_gemm_act(const Dims& d, const PlanPtrs& p, int act, const void* recv,
                                    const void* w_home, const void* w_slot, const float* bias, void* y,
                                    void* z, cudaStream_t st, int* launches) {
  const int half = act == kActSwiglu ? d.Hp / 2 : 0;
  const SplitPlan split = plan_split_grouped(d, half);
  if (split.splits) {
    *launches += 1;
    return launch_split_grouped(d, p, split, act, half, recv, w_home, w_slot, bias, y, z, st);
  }
  ProductMaps tm;
  const int ocols = half ? half : d.Hp;
  const bool slots = w_slot != nullptr && d.B > 0;
  if (!encode_matrix(&tm.a, recv, d.H, d.N, d.H, 128) ||
      !encode_matrix(&tm.b, w_home, d.Hp, (int64_t)d.E * d.H, d.Hp, 64) ||
      !encode_out(&tm.out, y, ocols, d.N, ocols))
    return cudaErrorInvalidValue;
  tm.b_slots = tm.b;
  if (slots && !encode_matrix(&tm.b_slots, w_slot, d.Hp, (int64_t)d.R * d.B * d.H, d.Hp, 64))
    return cudaErrorInvalidValue;
  tm.z = tm.z_up = tm.out;
  if (z != nullptr) {
    if (!encode_out(&tm.z, z, ocols, d.N, d.Hp)) return cudaErrorInvalidValue;
    if (half && !encode_out(&tm.z_up, (uint16_t*)z + half, ocols, d.N, d.Hp))
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
  // With the height left to the plan both are launched; the one it did not choose returns at once.  Where
  // no rank has more than 128 rows, no tile has, and one CTA takes them all.
  const bool pair = d.tile_m != kMmaM && d.C > kMmaM;
  const bool solo = d.tile_m != 2 * kMmaM || !pair;
  a.all = !pair;
  a.bn = pick_bn_grouped(d.Hp, half);
  const int64_t tiles = (int64_t)d.max_mtiles * tiles_of(1, a, 256);
  if (solo) {
    const cudaError_t e = launch_one<false, kForward, false, false>(tm, a, p, tiles, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  if (pair) {
    const cudaError_t e = launch_one<true, kForward, false, false>(tm, a, p, tiles, st);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  return cudaSuccess;
}

}  // namespace moonep
