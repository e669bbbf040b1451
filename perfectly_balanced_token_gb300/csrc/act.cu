// Gradient of the feed-forward network's activation, with that of the bias.  Bound by memory:
// 16-byte accesses, each value read and written once, four rows of loads in flight in every thread.
#include <algorithm>

#include "activation.cuh"
#include "ffn.h"
#include "pdl.cuh"
#include "vec.cuh"

namespace moonep {

// ---------------------------------------------------------------------------
// d_z = act'(z) d_out, with column sums of d_z (in fp32, before d_z is rounded).
//
// An item is a chunk of rows (64, or a work tile of the plan: rows of one expert) by 256 columns;
// a warp's lanes cover the columns and its rows are every eighth of the chunk.  The chunk's sums go
// to scratch, one row a chunk, and a second kernel adds them in ascending order: the same bits in
// every run, whatever runs when.
// ---------------------------------------------------------------------------
constexpr int kActThreads = 256;
constexpr int kActWarps = kActThreads / 32;
constexpr int kActRows = 64;
constexpr int kActCols = 256;

struct ActArgs {
  int64_t rows;
  int cols;  // of z
  const uint16_t *z, *d_out;
  uint16_t* d_z;
  float* sums;  // [chunks][cols] or null
};

template <int ACT>
__global__ void __launch_bounds__(kActThreads, 3) k_act_backward(ActArgs a, PlanPtrs p, int plan) {
  constexpr bool GATED = ACT == kActSwiglu;
  __shared__ float part[GATED ? 2 : 1][kActWarps][kActCols];
  grid_wait();
  grid_trigger();
  // plan: 0 = none, 1 = chunks are its work tiles, 2 = only its status counts
  if (plan && plan_failed(p.status)) return;
  const bool grouped = plan == 1;
  const int ocols = GATED ? a.cols / 2 : a.cols;
  const int nct = (ocols + kActCols - 1) / kActCols;
  const int64_t chunks = grouped ? p.counters[MOONEP_CNT_MTILES] : (a.rows + kActRows - 1) / kActRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t item = blockIdx.x; item < chunks * nct; item += gridDim.x) {
    const int64_t chunk = item / nct;
    const int col = (int)(item % nct) * kActCols + lane * 8;
    int64_t row0;
    int rows;
    if (grouped) {
      const MTile mt = p.mtiles[chunk];
      row0 = mt.row0;
      rows = mt.rows;
    } else {
      row0 = chunk * kActRows;
      rows = (int)min((int64_t)kActRows, a.rows - row0);
    }
    float sum[8] = {}, sum_up[8] = {};
    if (col < ocols) {
      constexpr int U = 2;  // rows in flight
      for (int r0 = warp; r0 < rows; r0 += U * kActWarps) {
        uint4 vz[U], vu[U], vd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * kActWarps;
          if (r < rows) {
            const int64_t row = row0 + r;
            vd[u] = __ldcs(reinterpret_cast<const uint4*>(a.d_out + row * ocols + col));
            if (ACT != kActNone)
              vz[u] = __ldcs(reinterpret_cast<const uint4*>(a.z + row * a.cols + col));
            if (GATED)
              vu[u] = __ldcs(reinterpret_cast<const uint4*>(a.z + row * a.cols + ocols + col));
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * kActWarps;
          if (r < rows) {
            const int64_t row = row0 + r;
            float d[8], z[8], up[8];
            unpack8(d, vd[u]);
            if (ACT != kActNone) unpack8(z, vz[u]);
            if (GATED) {
              unpack8(up, vu[u]);
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                // one sigmoid serves both: a = z s(z), a' = s (1 + z (1 - s))
                const F2 zz(z[i], z[i + 1]), dd(d[i], d[i + 1]), uu(up[i], up[i + 1]);
                const F2 s = sigmoid2(zz);
                const F2 du = dd * (zz * s);
                const F2 dz = dd * uu * (s * fma2(zz, fma2(s, F2(-1.f), F2(1.f)), F2(1.f)));
                dz.get(z[i], z[i + 1]);
                du.get(up[i], up[i + 1]);
                (F2(sum_up[i], sum_up[i + 1]) + du).get(sum_up[i], sum_up[i + 1]);
              }
              __stcs(reinterpret_cast<uint4*>(a.d_z + row * a.cols + ocols + col), pack8(up));
            } else {
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                const F2 dd(d[i], d[i + 1]);
                (ACT == kActNone ? dd : dd * act_slope2<ACT>(F2(z[i], z[i + 1]))).get(z[i], z[i + 1]);
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += z[i];
            if (a.d_z != nullptr) __stcs(reinterpret_cast<uint4*>(a.d_z + row * a.cols + col), pack8(z));
          }
        }
      }
    }
    if (a.sums == nullptr) continue;
    __syncthreads();  // the previous item's sums are read
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      part[0][warp][lane * 8 + i] = sum[i];
      if (GATED) part[GATED ? 1 : 0][warp][lane * 8 + i] = sum_up[i];
    }
    __syncthreads();
    const int c = (int)(item % nct) * kActCols + threadIdx.x;
    if (c < ocols) {
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kActWarps; ++w) s += part[h][w][threadIdx.x];
        a.sums[chunk * a.cols + h * ocols + c] = s;
      }
    }
  }
}

// d_bias[c] (+)= sum over chunks of sums[chunk][c]: 32 columns a block, 32 threads a column
__global__ void __launch_bounds__(1024) k_sum_chunks(const float* __restrict__ sums, int64_t chunks,
                                                     int cols, float* __restrict__ d_bias, int add) {
  __shared__ float part[32][33];
  grid_wait();
  grid_trigger();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float s = 0.f;
  if (c < cols)
    for (int64_t k = y; k < chunks; k += 32) s += sums[k * cols + c];
  part[y][x] = s;
  __syncthreads();
  if (y == 0 && c < cols) {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) total += part[i][x];
    d_bias[c] = add ? d_bias[c] + total : total;
  }
}

// The same for each expert over its work tiles: a block an expert and 1024 columns, which picks the
// expert's tiles out of the plan's list, 1024 at a time and in order, and adds their rows of sums.
constexpr int kPickThreads = 1024;
__global__ void __launch_bounds__(kPickThreads)
k_sum_tiles(PlanPtrs p, const float* __restrict__ sums, int cols, float* __restrict__ d_bias, int add) {
  __shared__ int picked[kPickThreads];
  __shared__ int count[kPickThreads / 32];
  grid_wait();
  grid_trigger();
  if (plan_failed(p.status)) return;
  const int e = blockIdx.x, c = blockIdx.y * kPickThreads + threadIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = p.counters[MOONEP_CNT_MTILES];
  float s = 0.f;
  for (int t0 = 0; t0 < tiles; t0 += kPickThreads) {
    const int t = t0 + threadIdx.x;
    bool mine = false;
    if (t < tiles) {
      const int w = p.mtiles[t].wsel;
      mine = (w >= 0 ? w : p.slot_expert[-1 - w]) == e;
    }
    const uint32_t b = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) count[warp] = __popc(b);
    __syncthreads();
    int before = 0, n = 0;
#pragma unroll
    for (int w = 0; w < kPickThreads / 32; ++w) {
      if (w < warp) before += count[w];
      n += count[w];
    }
    if (mine) picked[before + __popc(b & ((1u << lane) - 1))] = t;
    __syncthreads();
    if (c < cols) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) s += sums[(size_t)picked[i] * cols + c];
    }
    __syncthreads();
  }
  if (c < cols) {
    float* to = d_bias + (size_t)e * cols + c;
    *to = add ? *to + s : s;
  }
}

// -- host side ------------------------------------------------------------------
int64_t act_chunks(int64_t rows) { return (rows + kActRows - 1) / kActRows; }

static cudaError_t launch_act(int act, const ActArgs& a, const PlanPtrs& p, int plan,
                              int64_t chunks, cudaStream_t st) {
  const int ocols = act == kActSwiglu ? a.cols / 2 : a.cols;
  const int64_t items = chunks * ((ocols + kActCols - 1) / kActCols);
  const int grid = (int)std::min<int64_t>(items, (int64_t)sm_count_gemm() * 16);
  auto go = [&](auto kernel) { return launch_after(kernel, grid, kActThreads, 0, st, 1, a, p, plan); };
  if (act == kActNone) return go(k_act_backward<kActNone>);
  if (act == kActRelu) return go(k_act_backward<kActRelu>);
  if (act == kActGelu) return go(k_act_backward<kActGelu>);
  if (act == kActSilu) return go(k_act_backward<kActSilu>);
  return go(k_act_backward<kActSwiglu>);
}

cudaError_t launch_act_backward(int64_t rows, int cols, int act, const void* z, const void* d_out,
                                void* d_z, float* d_bias, int add, float* scratch, cudaStream_t st,
                                int* launches) {
  const ActArgs a{rows, cols, (const uint16_t*)z, (const uint16_t*)d_out, (uint16_t*)d_z,
                  d_bias ? scratch : nullptr};
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    e = launch_act(act, a, PlanPtrs{}, 0, act_chunks(rows), st);
    *launches += 1;
  }
  if (e != cudaSuccess || d_bias == nullptr) return e;
  *launches += 1;
  return launch_after(k_sum_chunks, (cols + 31) / 32, 1024, 0, st, 1, scratch, act_chunks(rows), cols,
                      d_bias, add);
}

cudaError_t launch_grouped_act_backward(const Dims& d, const PlanPtrs& p, int act, const void* z,
                                        const void* d_y, void* d_z, float* d_bias, int add,
                                        float* scratch, cudaStream_t st, int* launches) {
  const ActArgs a{d.N, d.Hp, (const uint16_t*)z, (const uint16_t*)d_y, (uint16_t*)d_z,
                  d_bias ? scratch : nullptr};
  // rows of one expert matter to the sums alone
  const cudaError_t e = launch_act(act, a, p, d_bias ? 1 : 2, d_bias ? d.max_mtiles : act_chunks(d.N), st);
  *launches += 1;
  if (e != cudaSuccess || d_bias == nullptr) return e;
  *launches += 1;
  return launch_after(k_sum_tiles, dim3(d.E, (d.Hp + kPickThreads - 1) / kPickThreads), kPickThreads, 0,
                      st, 1, p, scratch, d.Hp, d_bias, add);
}

}  // namespace moonep
