// What the kernels of the dense and grouped products share.
#pragma once

#include "activation.cuh"
#include "ffn.h"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace moonep {

constexpr int kDepth = 64;             // of a stage: 64 bf16 = one 128-byte swizzle row
constexpr int kPanelBytes = 64 * 128;  // 64 rows of 64 bf16

// Blocks of the depth that one accumulator sums where C is fp32.  The instruction cuts off what its
// fp32 sums do not hold, always towards zero, so a long sum drifts: against 64 bits, with the whole
// depth in one accumulator, 7e-6 of C at a depth of 7168 and past 2e-5 at 32768.  The epilogues add
// the parts in registers, rounding to nearest.  (A bf16 C's own rounding is 250 times larger, and it keeps one
// accumulator: at a depth of 7168 0.44 % of its values are the neighbour of the one nearest to the 64-bit
// sum, 0.06 % with sums rounded to nearest, and its distance from 64 bits is 0.165854 % and 0.165852 %.)
constexpr int kPartBlocks = 12;

enum Kind { kForward, kInputGrad, kWeightGrad };

// kind::f16: fp32 accumulator, bf16 operands; which of them run along M or N in memory
__host__ __device__ constexpr uint32_t product_idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Descriptor of the k-th 16 of a stage: rows of 128 bytes along the depth, or panels of 64 columns.
__device__ __forceinline__ uint64_t stage_desc(uint32_t at, int k, bool mn) {
  return mn ? sw128_desc(at + k * (16 * 128), kPanelBytes, 1024) : sw128_desc(at + k * 32, 16, 1024);
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// A row-major matrix [rows][cols] with `pitch` elements a row.
inline bool encode_boxes(CUtensorMap* m, const void* base, int cols, int64_t rows, int64_t pitch,
                         int box_cols, int box_rows, bool f32) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const int size = f32 ? 4 : 2;
  cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t stride[1] = {(cuuint64_t)(pitch * size)};
  cuuint32_t b[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t one[2] = {1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dim, stride, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// An operand: boxes of 64 bf16 (128 bytes, 128-byte swizzle) x `box` rows.
inline bool encode_matrix(CUtensorMap* m, const void* base, int cols, int64_t rows, int64_t pitch,
                          int box) {
  return encode_boxes(m, base, cols, rows, pitch, 64, box, false);
}
// An output: boxes of 32 columns x 32 rows.
inline bool encode_out(CUtensorMap* m, const void* base, int cols, int64_t rows, int64_t pitch,
                       bool f32 = false) {
  return encode_boxes(m, base, cols, rows, pitch, 32, 32, f32);
}

// product_split.cu: products of few tiles, split along the depth.
struct SplitPlan {
  int tokens, splits;  // rows of a tile, CTAs that share its depth; splits = 0: not for these sizes
};
// CTAs, one a multiprocessor, that run at once in clusters of `splits` (1, 2, 4 or 8); 0 if the runtime
// will not say.
int at_once(int splits);
SplitPlan plan_split(int T, int columns, int half, int depth, bool f32);
cudaError_t launch_split(Kind kind, const LinearDims& d, SplitPlan plan, const void* x, const void* w,
                         const float* bias, const void* residual, void* out, void* z, int add,
                         int32_t* status, cudaStream_t st);

SplitPlan plan_split_grouped(const Dims& d, int half);
cudaError_t launch_split_grouped(const Dims& d, const PlanPtrs& p, SplitPlan plan, int act, int half,
                                 const void* recv, const void* w_home, const void* w_slot,
                                 const float* bias, void* y, void* z, cudaStream_t st);

}  // namespace moonep
