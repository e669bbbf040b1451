// Gradient of the feed-forward network's activation, with that of the bias.  Bound by memory:
// 16-byte accesses, each value read and written once, two rows of loads in flight in every thread
// (6.4 to 6.55 TB/s at 32768 x 4096).
#include <algorithm>

#include "activation.cuh"
#include "ffn.h"
#include "pdl.cuh"
#include "vec.cuh"

namespace moonep {

// ---------------------------------------------------------------------------
// d_z = act'(z) d_out, with column sums of d_z (in fp32, before d_z is rounded).
//
// A block takes a chunk of rows by a strip of 8 to 256 columns: 1 to 32 lanes of a warp, eight columns
// each, cover the strip, the other lanes and warps further rows.  Dense chunks are cut so that the
// strips' blocks make two rounds of what the GPU holds at once (a chunk of 64 rows a block, with its sums and
// barriers, took 152 us for 32768 x 4096 of swiglu where long chunks took 107); with a plan and sums
// a chunk is a work tile, whose rows are of one expert.  A chunk's sums go to scratch, one row a
// chunk, and a second kernel adds them in ascending order: the same bits in every run.
// ---------------------------------------------------------------------------
constexpr int kActThreads = 256;
constexpr int kActWarps = kActThreads / 32;
// Where the gradient takes long to compute the next rows are loaded before these are computed, with as many
// blocks a multiprocessor as registers allow: 32768 x 4096 with bias, gelu 142 -> 126 us (three blocks for
// four), swiglu 107 -> 102.5 (two for three; three and ahead 109, two and not ahead 104); 32768 x 576 of silu
// 26.4 -> 23.5.  Relu has nothing to hide: 124 so, 126 with three and ahead.
constexpr bool act_ahead(int act) { return act != kActNone && act != kActRelu; }
constexpr int act_blocks(int act) { return act == kActSwiglu ? 2 : (act_ahead(act) ? 3 : 4); }
constexpr int kActMostChunks = 512;  // dense: rows of scratch

struct ActArgs {
  int64_t rows, chunk;  // of all, of a dense chunk
  int cols;             // of z
  int lanes, strips;    // lanes across a strip, strips across the output's columns
  const uint16_t *z, *d_out;
  uint16_t* d_z;
  float* sums;  // [chunks][cols] or null
};

template <int ACT>
__device__ __forceinline__ void act_chunk(const ActArgs& a, float (*part)[kActWarps][256], int64_t row0,
                                          int64_t rows, int64_t chunk, int strip) {
  constexpr bool GATED = ACT == kActSwiglu, AHEAD = act_ahead(ACT);
  const int ocols = GATED ? a.cols / 2 : a.cols;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int across = lane & (a.lanes - 1), sub = lane / a.lanes, step = kActWarps * (32 / a.lanes);
  const int col = (strip * a.lanes + across) * 8;
  float sum[8] = {}, sum_up[8] = {};
  if (col < ocols) {
    constexpr int U = 2;  // rows in flight
    const int64_t first = row0 + warp * (32 / a.lanes) + sub;
    const int64_t pitch = (int64_t)step * ocols, pitch_z = (int64_t)step * a.cols;
    const uint16_t* pd = a.d_out + first * ocols + col;
    const uint16_t* pz = a.z + first * a.cols + col;
    uint16_t* po = a.d_z == nullptr ? nullptr : a.d_z + first * a.cols + col;
    uint4 nz[U], nu[U], nd[U];
    auto load = [&](int64_t left) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * step < left) {
          nd[u] = __ldcs(reinterpret_cast<const uint4*>(pd + u * pitch));
          if (ACT != kActNone) nz[u] = __ldcs(reinterpret_cast<const uint4*>(pz + u * pitch_z));
          if (GATED) nu[u] = __ldcs(reinterpret_cast<const uint4*>(pz + u * pitch_z + ocols));
        }
      }
      pd += U * pitch;
      pz += U * pitch_z;
    };
    int64_t left = row0 + rows - first;
    if (AHEAD) load(left);
    for (; left > 0; left -= U * step) {
      if (!AHEAD) load(left);
      uint4 vz[U], vu[U], vd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) vz[u] = nz[u], vu[u] = nu[u], vd[u] = nd[u];
      if (AHEAD && left > U * step) load(left - U * step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * step < left) {
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
            __stcs(reinterpret_cast<uint4*>(po + u * pitch_z + ocols), pack8(up));
          } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const F2 dd(d[i], d[i + 1]);
              (ACT == kActNone ? dd : dd * act_slope2<ACT>(F2(z[i], z[i + 1]))).get(z[i], z[i + 1]);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            (F2(sum[i], sum[i + 1]) + F2(z[i], z[i + 1])).get(sum[i], sum[i + 1]);
          if (po != nullptr) __stcs(reinterpret_cast<uint4*>(po + u * pitch_z), pack8(z));
        }
      }
      if (po != nullptr) po += U * pitch_z;
    }
  }
  if (a.sums == nullptr) return;
  __syncwarp();
  for (int off = a.lanes; off < 32; off *= 2) {  // the lanes that share columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
      if (GATED) sum_up[i] += __shfl_xor_sync(0xffffffffu, sum_up[i], off);
    }
  }
  __syncthreads();  // the sums of the block's previous chunk are read
  if (sub == 0) {
    float4* to = reinterpret_cast<float4*>(&part[0][warp][across * 8]);
    to[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    to[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    if (GATED) {
      to = reinterpret_cast<float4*>(&part[GATED ? 1 : 0][warp][across * 8]);
      to[0] = make_float4(sum_up[0], sum_up[1], sum_up[2], sum_up[3]);
      to[1] = make_float4(sum_up[4], sum_up[5], sum_up[6], sum_up[7]);
    }
  }
  __syncthreads();
  const int c = strip * a.lanes * 8 + threadIdx.x;
  if (threadIdx.x < a.lanes * 8 && c < ocols) {
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kActWarps; ++w) s += part[h][w][threadIdx.x];
      a.sums[chunk * a.cols + h * ocols + c] = s;
    }
  }
}

// plan: 0 = none, 1 = chunks are its work tiles, 2 = only its status counts
template <int ACT>
__global__ void __launch_bounds__(kActThreads, act_blocks(ACT))
k_act_backward(ActArgs a, PlanPtrs p, int plan) {
  __shared__ float part[ACT == kActSwiglu ? 2 : 1][kActWarps][256];
  grid_wait();
  grid_trigger();
  if (plan && plan_failed(p.status)) return;
  if (plan != 1) {
    const int64_t chunk = blockIdx.x / a.strips;
    const int64_t row0 = chunk * a.chunk;
    act_chunk<ACT>(a, part, row0, min(a.chunk, a.rows - row0), chunk, blockIdx.x % a.strips);
    return;
  }
  const int64_t items = (int64_t)p.counters[MOONEP_CNT_MTILES] * a.strips;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const MTile mt = p.mtiles[item / a.strips];
    act_chunk<ACT>(a, part, mt.row0, mt.rows, item / a.strips, (int)(item % a.strips));
  }
}

// d_bias[c] (+)= sum over chunks of sums[chunk][c]: 32 columns a block, 32 threads a column
__global__ void __launch_bounds__(1024) k_sum_chunks(const float* sums, int64_t chunks,
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
k_sum_tiles(PlanPtrs p, const float* sums, int cols, float* __restrict__ d_bias, int add) {
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
// Rows of scratch that the dense gradient may need, on whatever GPU.
int64_t act_chunks(int64_t rows) { return std::min<int64_t>((rows + 63) / 64, kActMostChunks); }

// Lanes across a strip: the most that are asked for, fewer where a last strip would leave them
// without columns.
static void cut_columns(ActArgs* a, int act, int most) {
  const int vectors = (act == kActSwiglu ? a->cols / 2 : a->cols) / 8;
  a->lanes = most;
  for (int lanes = most / 2; lanes >= 4; lanes /= 2) {
    const int had = (vectors + a->lanes - 1) / a->lanes * a->lanes;
    const int has = (vectors + lanes - 1) / lanes * lanes;
    if (has * 8 <= had * 7) a->lanes = lanes;
  }
  a->strips = (vectors + a->lanes - 1) / a->lanes;
}

static cudaError_t launch_act(int act, const ActArgs& a, const PlanPtrs& p, int plan, int64_t chunks,
                              cudaStream_t st) {
  const int64_t items = chunks * a.strips;
  // (of a plan's items there are at most as many as the host can know of; blocks without one end at once)
  const unsigned grid = (unsigned)(plan == 1 ? std::min<int64_t>(items, 1 << 16) : items);
  auto go = [&](auto kernel) { return launch_after(kernel, grid, kActThreads, 0, st, 1, a, p, plan); };
  if (act == kActNone) return go(k_act_backward<kActNone>);
  if (act == kActRelu) return go(k_act_backward<kActRelu>);
  if (act == kActGelu) return go(k_act_backward<kActGelu>);
  if (act == kActSilu) return go(k_act_backward<kActSilu>);
  return go(k_act_backward<kActSwiglu>);
}

// Dense chunks: two rounds of blocks (one leaves the slowest multiprocessor alone at the end).
static int64_t cut_rows(ActArgs* a, int act) {
  const int64_t blocks = (int64_t)sm_count_gemm() * act_blocks(act) * 2;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(act_chunks(a->rows), blocks / a->strips));
  a->chunk = (a->rows + most - 1) / most;
  return (a->rows + a->chunk - 1) / a->chunk;
}

cudaError_t launch_act_backward(int64_t rows, int cols, int act, const void* z, const void* d_out,
                                void* d_z, float* d_bias, int add, float* scratch, cudaStream_t st,
                                int* launches) {
  ActArgs a{rows, 0, cols, 0, 0, (const uint16_t*)z, (const uint16_t*)d_out, (uint16_t*)d_z,
            d_bias ? scratch : nullptr};
  cut_columns(&a, act, 32);
  const int64_t chunks = cut_rows(&a, act);
  cudaError_t e = launch_act(act, a, PlanPtrs{}, 0, chunks, st);
  *launches += 1;
  if (e != cudaSuccess || d_bias == nullptr) return e;
  *launches += 1;
  return launch_after(k_sum_chunks, (cols + 31) / 32, 1024, 0, st, 1, scratch, chunks, cols, d_bias,
                      add);
}

cudaError_t launch_grouped_act_backward(const Dims& d, const PlanPtrs& p, int act, const void* z,
                                        const void* d_y, void* d_z, float* d_bias, int add,
                                        float* scratch, cudaStream_t st, int* launches) {
  ActArgs a{d.N, 0, d.Hp, 0, 0, (const uint16_t*)z, (const uint16_t*)d_y, (uint16_t*)d_z,
            d_bias ? scratch : nullptr};
  // (rows of one expert matter to the sums alone; work tiles are few, so narrower strips of them even
  // out the multiprocessors' shares)
  cut_columns(&a, act, d_bias ? 16 : 32);
  const int64_t chunks = d_bias ? d.max_mtiles : cut_rows(&a, act);
  const cudaError_t e = launch_act(act, a, p, d_bias ? 1 : 2, chunks, st);
  *launches += 1;
  if (e != cudaSuccess || d_bias == nullptr) return e;
  *launches += 1;
  return launch_after(k_sum_tiles, dim3(d.E, (d.Hp + kPickThreads - 1) / kPickThreads), kPickThreads, 0,
                      st, 1, p, scratch, d.Hp, d_bias, add);
}

}  // namespace moonep
