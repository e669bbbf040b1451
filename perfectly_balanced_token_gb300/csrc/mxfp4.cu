// MXFP4 quantisation: rows, expert weights (transposing), the dispatch that
// quantises on the way, and the way back to bf16.
//
// A block of 32 values with largest magnitude m = f 2^e, 1 <= f < 2, has the
// scale 2^(e - 2) (6 = 1.5 2^2 is the largest code), clamped to 2^-127.  The
// exponent is read off the bf16 pattern and the division by the scale is a
// multiplication by a power of two, so the only rounding is the conversion to
// E2M1 (nearest, ties to even, at most 6).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ops.h"

namespace moonep {

// Scale byte of a block from its largest bf16 magnitude pattern; 255 for a
// block that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t magnitude) {
  const uint32_t e = magnitude >> 7;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - b) of a scale byte b <= 253; 0 for 255 (its codes are cleared)
__device__ __forceinline__ float inverse_scale(uint32_t b) {
  return b == 255u ? 0.f : __uint_as_float((254u - b) << 23);
}
// 2^(b - 127), NaN for 255
__device__ __forceinline__ float scale_value(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(b == 0u ? 1u << 22 : b << 23);
}
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t m, uint32_t bf16x2) {
  return __vmaxu2(m, bf16x2 & 0x7fff7fffu);
}
__device__ __forceinline__ float lo_f32(uint32_t bf16x2) { return __uint_as_float(bf16x2 << 16); }
__device__ __forceinline__ float hi_f32(uint32_t bf16x2) {
  return __uint_as_float(bf16x2 & 0xffff0000u);
}

// Eight scaled values to eight codes, the first in the low four bits.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ uint32_t encode8(const uint4& x, uint32_t b) {
  const float f = inverse_scale(b);
  const float v[8] = {lo_f32(x.x) * f, hi_f32(x.x) * f, lo_f32(x.y) * f, hi_f32(x.y) * f,
                      lo_f32(x.z) * f, hi_f32(x.z) * f, lo_f32(x.w) * f, hi_f32(x.w) * f};
  return b == 255u ? 0u : encode8(v);
}

// A warp's unit of a row is 16 blocks (512 values, 256 bytes of codes, 16 scale
// bytes): lane i holds eight values of block i / 4 and eight of block 8 + i / 4,
// so loads and code stores are coalesced and a block's maximum takes two
// shuffles.  Past the row's end the scale bytes are 0.
constexpr int kUnit = 512;

struct UnitCodes {
  uint32_t code[2];
  uint4 scales;  // all 16, in every lane
};

__device__ __forceinline__ void load_unit(const uint16_t* row, int cols, int unit, int lane,
                                          uint4 (&x)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = unit * kUnit + h * 256 + lane * 8;
    x[h] = make_uint4(0, 0, 0, 0);
    if (at < cols) x[h] = __ldcs(reinterpret_cast<const uint4*>(row + at));
  }
}

__device__ __forceinline__ UnitCodes encode_unit(const uint4 (&x)[2], int lane, uint8_t* s_bytes) {
  UnitCodes r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t m = max_magnitude2(max_magnitude2(0u, x[h].x), x[h].y);
    m = max_magnitude2(max_magnitude2(m, x[h].z), x[h].w);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t b = scale_byte(max(m & 0xffffu, m >> 16));
    r.code[h] = encode8(x[h], b);
    if ((lane & 3) == 0) s_bytes[h * 8 + (lane >> 2)] = (uint8_t)b;
  }
  __syncwarp();
  r.scales = *reinterpret_cast<const uint4*>(s_bytes);
  __syncwarp();
  return r;
}

constexpr int kQuantThreads = 128;
constexpr int kQuantWarps = kQuantThreads / 32;

// The units of all rows, warp by warp over the whole grid: neighbouring warps take
// neighbouring units, and all take equally many (a block per row would leave two of
// its four warps idle for a seventh of the time at 14 units).  The row advances
// without a division.
struct UnitWalk {
  int64_t row, rows_ahead;
  int unit, units_ahead, per_row;
  __device__ __forceinline__ UnitWalk(int per_row_) : per_row(per_row_) {
    const int64_t first = (int64_t)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
    const int64_t stride = (int64_t)gridDim.x * kQuantWarps;
    row = first / per_row, unit = (int)(first % per_row);
    rows_ahead = stride / per_row, units_ahead = (int)(stride % per_row);
  }
  __device__ __forceinline__ void advance() {
    row += rows_ahead, unit += units_ahead;
    if (unit >= per_row) unit -= per_row, ++row;
  }
};

// (Loading a warp's next unit before it works on this one costs more warps than it
// saves waiting here: 103 -> 110 us at 32768 x 7168, and 107 -> 120 us on the way back.)
__global__ void __launch_bounds__(kQuantThreads)
k_mxfp4_quantize(int64_t rows, int per_row, int cols, const uint16_t* __restrict__ src,
                 uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t s_bytes[kQuantWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (UnitWalk w(per_row); w.row < rows; w.advance()) {
    uint4 x[2];
    load_unit(src + w.row * cols, cols, w.unit, lane, x);
    const UnitCodes r = encode_unit(x, lane, s_bytes[warp]);
    uint8_t* out = codes + w.row * (cols / 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = w.unit * kUnit + h * 256 + lane * 8;
      if (at < cols) *reinterpret_cast<uint32_t*>(out + at / 2) = r.code[h];
    }
    if (lane == 0) *reinterpret_cast<uint4*>(scales + (w.row * per_row + w.unit) * 16) = r.scales;
  }
}

// Eight codes to eight bf16 values times f (exact but for scales past bf16's range)
__device__ __forceinline__ uint4 decode8(uint32_t codes, float f) {
  uint32_t half2[4], o[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(half2[0]), "=r"(half2[1]), "=r"(half2[2]), "=r"(half2[3])
      : "r"(codes));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&half2[k]));
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);
    o[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kQuantThreads)
k_mxfp4_dequantize(int64_t rows, int per_row, int cols, const uint8_t* __restrict__ codes,
                   const uint8_t* __restrict__ scales, uint16_t* __restrict__ dst) {
  const int lane = threadIdx.x & 31;
  for (UnitWalk w(per_row); w.row < rows; w.advance()) {
    const uint8_t* in = codes + w.row * (cols / 2);
    const int first = w.unit * kUnit + lane * 8;
    uint32_t c[2], b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (first + h * 256 < cols) {
        c[h] = __ldcs(reinterpret_cast<const uint32_t*>(in + (first + h * 256) / 2));
        b[h] = __ldg(scales + (w.row * per_row + w.unit) * 16 + h * 8 + (lane >> 2));
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (first + h * 256 < cols)
        __stcs(reinterpret_cast<uint4*>(dst + w.row * cols + first + h * 256),
               decode8(c[h], scale_value(b[h])));
  }
}

// Weights [H][Hp] to the rows of their transpose: a block of threads takes 256
// values of H by 64 columns; a thread reads two columns of one MXFP4 block (the
// warp 128 contiguous bytes of each of the 32 rows), so the maximum needs no
// other thread, and the codes pass through shared memory to leave as 128
// contiguous bytes a column.
constexpr int kWTileH = 256, kWTileN = 64;

__global__ void __launch_bounds__(256)
k_mxfp4_quantize_weights(int h_tiles, int H, int Hp, int pitch, const uint16_t* __restrict__ w,
                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint4 s_code[kWTileN][9];  // 8 of 9: 144-byte rows spread the banks
  __shared__ __align__(8) uint8_t s_scale[kWTileN][8];
  const int block = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = blockIdx.x / h_tiles, h0 = (blockIdx.x % h_tiles) * kWTileH;
  const int n0 = blockIdx.y * kWTileN;
  const int h = h0 + block * 32;
  if (h < H) {  // H is a multiple of 64: a block of 32 is inside or outside as a whole
    const uint16_t* src = w + ((size_t)e * H + h) * Hp + n0 + lane * 2;
    uint32_t x[32];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      x[i] = __ldcs(reinterpret_cast<const uint32_t*>(src + (size_t)i * Hp));
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max_magnitude2(m, x[i]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t b = scale_byte(c == 0 ? m & 0xffffu : m >> 16);
      const float f = inverse_scale(b);
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = (c == 0 ? lo_f32(x[q * 8 + i]) : hi_f32(x[q * 8 + i])) * f;
        o[q] = b == 255u ? 0u : encode8(v);
      }
      s_code[lane * 2 + c][block] = make_uint4(o[0], o[1], o[2], o[3]);
      s_scale[lane * 2 + c][block] = (uint8_t)b;
    }
  } else {
    s_scale[lane * 2][block] = s_scale[lane * 2 + 1][block] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kWTileN * 8; i += 256) {
    const int n = i >> 3, b = i & 7;
    if (h0 + b * 32 < H)
      *reinterpret_cast<uint4*>(codes + ((size_t)e * Hp + n0 + n) * (H / 2) + h0 / 2 + b * 16) =
          s_code[n][b];
  }
  if (threadIdx.x < kWTileN)
    *reinterpret_cast<uint2*>(scales + ((size_t)e * Hp + n0 + threadIdx.x) * pitch + h0 / 32) =
        *reinterpret_cast<const uint2*>(s_scale[threadIdx.x]);
}

// Dispatch: a warp quantises a unit of a token's row once and stores it to the
// token's K rows; the next unit is loaded meanwhile (16384 tokens x 7168, K = 8:
// 145 -> 130 us, 734 MB that it has to move).
__global__ void __launch_bounds__(kQuantThreads)
k_mxfp4_dispatch(Dims d, PlanPtrs p, int pitch, const uint16_t* __restrict__ x,
                 uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  if (plan_failed(p.status)) return;
  __shared__ __align__(16) uint8_t s_bytes[kQuantWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntok = d.R * d.S;
  UnitWalk w(pitch / 16);
  uint4 next[2];
  int next_row = 0;  // lane k: the unit's k-th destination row, of the first 32
  auto load = [&]() {
    load_unit(x + w.row * d.H, d.H, w.unit, lane, next);
    if (lane < d.K) next_row = __ldg(p.dst + w.row * d.K + lane);
  };
  if (w.row < ntok) load();
  while (w.row < ntok) {
    const int64_t token = w.row;
    const int unit = w.unit, row = next_row;
    const uint4 v[2] = {next[0], next[1]};
    w.advance();
    if (w.row < ntok) load();
    const UnitCodes r = encode_unit(v, lane, s_bytes[warp]);
    const int at = unit * kUnit + lane * 8;
    auto store = [&](int to) {
      uint8_t* out = codes + (size_t)to * (d.H / 2) + at / 2;
      if (at < d.H) *reinterpret_cast<uint32_t*>(out) = r.code[0];
      if (at + 256 < d.H) *reinterpret_cast<uint32_t*>(out + 128) = r.code[1];
    };
    auto store_scales = [&](int to) {
      *reinterpret_cast<uint4*>(scales + (size_t)to * pitch + unit * 16) = r.scales;
    };
    const int k32 = min(d.K, 32);
#pragma unroll 4
    for (int k = 0; k < k32; ++k) store(__shfl_sync(0xffffffffu, row, k));
    if (lane < d.K) store_scales(row);
    for (int k = 32; k < d.K; ++k) {
      const int to = __ldg(p.dst + token * d.K + k);
      store(to);
      if (lane == 0) store_scales(to);
    }
  }
}

// Prefetch: the occupied slots' codes and scales in one launch, 16 KiB at a time,
// the next piece loaded before this one is stored.
constexpr int kPieceVec = 4;
constexpr int kPieceThreads = 256;
constexpr int kPiece = kPieceThreads * kPieceVec;  // 16-byte vectors

__global__ void __launch_bounds__(kPieceThreads)
k_mxfp4_prefetch(PlanPtrs p, int code_vecs, int scale_vecs, const uint4* __restrict__ home_codes,
                 const uint4* __restrict__ home_scales, uint4* __restrict__ slot_codes,
                 uint4* __restrict__ slot_scales) {
  if (plan_failed(p.status)) return;
  const int code_pieces = (code_vecs + kPiece - 1) / kPiece;
  const int pieces = code_pieces + (scale_vecs + kPiece - 1) / kPiece;
  const int64_t items = (int64_t)p.counters[MOONEP_CNT_OCCUPIED] * pieces;
  uint4 v[kPieceVec], next[kPieceVec];
  auto visit = [&](int64_t it, auto&& f) {  // f(home, slot, vectors) of each vector held here
    const int s = p.occupied[it / pieces], piece = (int)(it % pieces);
    const int e = p.slot_expert[s];
    const bool code = piece < code_pieces;
    const int n = code ? code_vecs : scale_vecs;
    const uint4* home = (code ? home_codes : home_scales) + (size_t)e * n;
    uint4* slot = (code ? slot_codes : slot_scales) + (size_t)s * n;
    const int at = (code ? piece : piece - code_pieces) * kPiece + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kPieceVec; ++i)
      if (at + i * kPieceThreads < n) f(i, home + at + i * kPieceThreads, slot + at + i * kPieceThreads);
  };
  int64_t it = blockIdx.x;
  if (it < items) visit(it, [&](int i, const uint4* home, uint4*) { v[i] = __ldcs(home); });
  for (; it < items; it += gridDim.x) {
    if (it + gridDim.x < items)
      visit(it + gridDim.x, [&](int i, const uint4* home, uint4*) { next[i] = __ldcs(home); });
    visit(it, [&](int i, const uint4*, uint4* slot) { __stcs(slot, v[i]); });
#pragma unroll
    for (int i = 0; i < kPieceVec; ++i) v[i] = next[i];
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
static int multiprocessors() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

static int blocks_for(int64_t units, int per_multiprocessor) {
  const int64_t want = (units + kQuantWarps - 1) / kQuantWarps;
  const int64_t most = (int64_t)multiprocessors() * per_multiprocessor;
  return (int)(want < most ? want : most);
}
// Streams in and out: four rounds of 16 blocks, so that a block that is late leaves
// no multiprocessor idle at the end (32768 x 7168: 98 and 97 us against 103 and 107
// with one round; one unit a warp and no loop, 121 and 99).
constexpr int kStreamBlocks = 64;
// The dispatch overlaps its loads across units instead, and runs in one round.
constexpr int kDispatchBlocks = 16;

cudaError_t launch_mxfp4_quantize(int64_t rows, int cols, const void* src, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st, int* launches) {
  const int per_row = MOONEP_MXFP4_SCALE_PITCH(cols) / 16;
  if (rows == 0) return cudaSuccess;
  k_mxfp4_quantize<<<blocks_for(rows * per_row, kStreamBlocks), kQuantThreads, 0, st>>>(
      rows, per_row, cols, (const uint16_t*)src, codes, scales);
  *launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(int64_t rows, int cols, const uint8_t* codes,
                                    const uint8_t* scales, void* dst, cudaStream_t st,
                                    int* launches) {
  const int per_row = MOONEP_MXFP4_SCALE_PITCH(cols) / 16;
  if (rows == 0) return cudaSuccess;
  k_mxfp4_dequantize<<<blocks_for(rows * per_row, kStreamBlocks), kQuantThreads, 0, st>>>(
      rows, per_row, cols, codes, scales, (uint16_t*)dst);
  *launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_quantize_weights(int n, int H, int Hp, const void* w, uint8_t* codes,
                                          uint8_t* scales, cudaStream_t st, int* launches) {
  if (n == 0) return cudaSuccess;
  const int pitch = MOONEP_MXFP4_SCALE_PITCH(H);
  const int h_tiles = pitch / (kWTileH / 32);  // covers the scale row's padding too
  const dim3 grid((unsigned)n * h_tiles, Hp / kWTileN);
  k_mxfp4_quantize_weights<<<grid, 256, 0, st>>>(h_tiles, H, Hp, pitch, (const uint16_t*)w, codes,
                                                 scales);
  *launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dispatch(const Dims& d, const PlanPtrs& p, const void* x, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st, int* launches) {
  const int pitch = MOONEP_MXFP4_SCALE_PITCH(d.H);
  const int grid = blocks_for((int64_t)d.R * d.S * (pitch / 16), kDispatchBlocks);
  k_mxfp4_dispatch<<<grid, kQuantThreads, 0, st>>>(d, p, pitch, (const uint16_t*)x, codes, scales);
  *launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_prefetch(const Dims& d, const PlanPtrs& p, const uint8_t* home_codes,
                                  const uint8_t* home_scales, uint8_t* slot_codes,
                                  uint8_t* slot_scales, cudaStream_t st, int* launches) {
  if (d.B == 0) return cudaSuccess;
  const int64_t code = (int64_t)d.Hp * (d.H / 2) / 16;
  const int64_t scale = (int64_t)d.Hp * MOONEP_MXFP4_SCALE_PITCH(d.H) / 16;
  if (code >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
  // eight blocks a multiprocessor: with sixteen a prefetch of two slots takes longer
  // to start its blocks than to copy
  k_mxfp4_prefetch<<<multiprocessors() * 8, kPieceThreads, 0, st>>>(
      p, (int)code, (int)scale, (const uint4*)home_codes, (const uint4*)home_scales,
      (uint4*)slot_codes, (uint4*)slot_scales);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace moonep
